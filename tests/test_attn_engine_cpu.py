"""Host logic of the paged cache of the softmax-attention layers
(attn_engine.JetAttnEngine) and of JetEngine.fork, on the CPU with stand-ins
for the library's calls: pages handed out, shared, copied, given up and
compacted. The stand-ins act on the pools as the kernels do."""
import random

import pytest
import torch

from linear_attention_lm_gen_b200 import attn_engine as ae
from linear_attention_lm_gen_b200 import engine as eng

PAGE = 16


def fake_copy(pools, src, dst):
    assert len(set(dst)) == len(dst) and not set(src) & set(dst)
    for p in pools:
        p[dst] = p[src].clone()


def fake_append(q, k, v, gq, gk, inv_freq, cu, lens, table, kp, vp, q_out, *, eps, interleaved):
    """Writes the tokens' values at their positions (no norm, no rotation)."""
    for s in range(len(lens)):
        n = int(cu[s + 1] - cu[s])
        for i in range(n):
            p = int(lens[s]) - n + i
            page = int(table[s, p // PAGE])
            assert page >= 0
            kp[page, :, p % PAGE], vp[page, :, p % PAGE] = k[int(cu[s]) + i], v[int(cu[s]) + i]
    return q


def fake_paged(q, kp, vp, cu, lens, table, max_new, o, ws, *, window, scale):
    """The first element of every position that each sequence's last token sees, in order."""
    assert max_new == int((cu[1:] - cu[:-1]).max())
    out = []
    for s in range(len(lens)):
        L = int(lens[s])
        lo = max(0, L - window) if window else 0
        seen = []
        for p in range(lo, L):
            page = int(table[s, p // PAGE])
            assert page >= 0
            assert float(kp[page, 0, p % PAGE, 0]) == float(vp[page, 0, p % PAGE, 0])
            seen.append(float(vp[page, 0, p % PAGE, 0]))
        out.append(seen)
    return out


def fake_compact(pools, table, lens, page):
    P = pools[0].shape[0]
    held = set()
    for s in range(len(lens)):
        held |= {int(x) for x in table[s, :-(-int(lens[s]) // page)] if x >= 0}
    holes = [i for i in range(len(held)) if i not in held]
    to = {i: i for i in held if i < len(held)}
    to.update(zip(sorted(i for i in held if i >= len(held)), holes))
    for p in pools:
        old = p.clone()
        for a, b in to.items():
            p[b] = old[a]
        p[len(held):P] = float("nan")
    out = torch.full_like(table, -1)
    for s in range(len(lens)):
        for i in range(-(-int(lens[s]) // page)):
            if table[s, i] >= 0:
                out[s, i] = to[int(table[s, i])]
    return out, torch.tensor([len(held)], dtype=torch.int32)


@pytest.fixture
def make(monkeypatch):
    monkeypatch.setattr(ae, "jet_cache_copy", fake_copy)
    monkeypatch.setattr(ae, "jet_attn_rope_append", fake_append)
    monkeypatch.setattr(ae, "jet_attn_paged", fake_paged)
    monkeypatch.setattr(ae, "jet_cache_compact", fake_compact)
    monkeypatch.setattr(ae, "jet_attn_paged_workspace_size", lambda *a: 16)
    return lambda n_pages=20, **kw: ae.JetAttnEngine(2, 2, 1, 8, n_pages, PAGE, 6, 200, dtype=torch.float32,
                                                     device="cpu", **kw)


class Texts:
    """What each sequence holds, position by position, and a step through the engine."""

    def __init__(self, e):
        self.e, self.text, self.next = e, {}, 1.0

    def step(self, new):
        b = self.e.begin(new)
        vals = []
        for s, n in new.items():
            mine = [self.next + i for i in range(n)]
            self.next += n
            self.text[s] = self.text.get(s, []) + mine
            vals += mine
        x = torch.tensor(vals).view(-1, 1, 1).expand(-1, 1, 8)
        q = torch.zeros(len(vals), 2, 8)
        for layer in range(2):
            seen = self.e.attend(layer, b, q, x, x)
            w = self.e.windows[layer]
            for s, got in zip(new, seen):
                assert got == (self.text[s][-w:] if w else self.text[s]), s

    def fork(self, parent, children):
        self.e.fork(parent, children)
        for c in children:
            self.text[c] = list(self.text[parent])

    def release(self, s):
        self.e.release(s)
        del self.text[s]


def consistent(e):
    held = {}
    for s, r in e.row.items():
        for p in e._table[r][e._table[r] >= 0]:
            held[int(p)] = held.get(int(p), 0) + 1
    assert all(e._ref[p] == n for p, n in held.items()) and int((e._ref > 0).sum()) == len(held)
    assert sorted(e._free) == [p for p in range(e.n_pages) if p not in held]


def test_prompts_decode_and_release(make):
    e = make()
    t = Texts(e)
    for s in "ab":
        e.admit(s)
    t.step({"a": 30, "b": 1})
    t.step({"b": 17, "a": 1})
    t.step({"a": 1, "b": 1})
    consistent(e)
    assert e.free_pages == 20 - 2 - 2
    t.release("a")
    assert e.free_pages == 18
    consistent(e)
    with pytest.raises(KeyError):
        e.begin({"a": 1})


def test_forks_share_whole_pages_and_copy_the_last(make):
    e = make()
    t = Texts(e)
    e.admit("a")
    t.step({"a": 40})                              # two whole pages and half a page
    t.fork("a", ["b", "c"])
    assert e.free_pages == 20 - 3 - 2
    t.step({"a": 1, "b": 20, "c": 1})
    t.fork("b", ["d"])
    t.step({"d": 5, "b": 3})
    consistent(e)
    t.release("a")
    t.step({"c": 30, "b": 1, "d": 1})
    consistent(e)
    t.release("c"), t.release("b")
    consistent(e)
    t.step({"d": 1})
    e.admit("x")
    t.step({"x": 32})
    t.fork("x", ["y"])                             # nothing to copy at a page's end
    consistent(e)
    t.step({"x": 1, "y": 1})


def test_windows_give_pages_up(make):
    e = make(windows=[20, 33])
    t = Texts(e)
    e.admit("a")
    for n in (50, 30, 1, 1, 40, 1, 16, 16):
        t.step({"a": n})
        consistent(e)
    held = 20 - e.free_pages
    assert held <= -(-(33 + 16) // PAGE) + 1
    t.fork("a", ["b"])
    t.step({"a": 40, "b": 2})
    consistent(e)
    e2 = make(windows=[20, 0])                     # one layer sees everything: all pages stay
    t2 = Texts(e2)
    e2.admit("a")
    for _ in range(5):
        t2.step({"a": 30})
    assert e2.free_pages == 20 - 10


def test_a_full_cache_takes_pages_that_the_step_gives_up(make):
    e = make(n_pages=4, windows=[16, 16])
    t = Texts(e)
    e.admit("a")
    t.step({"a": 60})
    t.step({"a": 30})                              # needs two pages, gives two up
    consistent(e)
    with pytest.raises(RuntimeError):
        e.begin({"a": 70})
    consistent(e)


def test_compaction_keeps_every_text(make):
    for seed in range(6):
        r = random.Random(seed)
        e = make(n_pages=40, windows=[30, 40] if seed % 2 else None)
        t = Texts(e)
        names = iter("abcdefghijklmnopqrstuvwxyz")
        for _ in range(25):
            live = list(t.text)
            act = r.random()
            if act < 0.3 and len(live) < 5:
                s = next(names, None)
                if s:
                    e.admit(s)
                    t.step({s: r.randint(1, 50)})
            elif act < 0.4 and live and len(live) < 5:
                s = next(names, None)
                if s:
                    t.fork(r.choice(live), [s])
            elif act < 0.55 and live:
                t.release(r.choice(live))
            elif act < 0.7 and live:
                n = e.compact()
                assert sorted(e._free) == list(range(n, 40))
            elif live:
                for s in live:
                    if e.len[s] < 150:
                        t.step({s: r.randint(1, 20)})
            consistent(e)


def test_checks_come_before_changes(make):
    e = make(n_pages=3)
    t = Texts(e)
    e.admit("a")
    t.step({"a": 20})
    with pytest.raises(KeyError):
        e.admit("a")
    with pytest.raises(KeyError):
        e.begin({"a": 1, "z": 1})
    with pytest.raises(ValueError):
        e.begin({})
    with pytest.raises(ValueError):
        e.begin({"a": 0})
    with pytest.raises(ValueError):
        e.begin({"a": 300})                        # longer than the longest sequence
    with pytest.raises(RuntimeError):
        e.begin({"a": 40})
    with pytest.raises(KeyError):
        e.fork("a", ["b", "b"])
    with pytest.raises(KeyError):
        e.fork("z", ["b"])
    with pytest.raises(RuntimeError):
        e.fork("a", ["b", "c"])                    # two copies of the last page, one page free
    with pytest.raises(RuntimeError):
        e.fork("a", [str(i) for i in range(9)])
    consistent(e)
    assert e.len["a"] == 20 and list(e.row) == ["a"]
    b = e.begin({"a": 2})
    with pytest.raises(ValueError):
        e.attend(0, b, torch.zeros(3, 2, 8), torch.zeros(3, 1, 8), torch.zeros(3, 1, 8))
    with pytest.raises(ValueError):
        ae.JetAttnEngine(2, 2, 1, 8, 0, device="cpu")
    with pytest.raises(ValueError):
        ae.JetAttnEngine(2, 2, 1, 8, 4, windows=[1], device="cpu")


def test_a_batch_from_before_a_compaction_is_refused(make):
    """Its table names pages that have moved."""
    e = make()
    t = Texts(e)
    for s in "ab":
        e.admit(s)
        t.step({s: 20})
    t.release("a")
    b = e.begin({"b": 1})
    e.compact()
    x = torch.zeros(1, 1, 8)
    with pytest.raises(ValueError, match="compaction"):
        e.attend(0, b, torch.zeros(1, 2, 8), x, x)


def test_batches_do_not_share_a_workspace(make, monkeypatch):
    """Two steps may be on different streams, or in two captured graphs."""
    held = []
    monkeypatch.setattr(ae, "jet_attn_paged", lambda *a, **kw: held.append(a[8]))
    e = make()
    x = torch.zeros(1, 1, 8)
    for s in "ab":
        e.admit(s)
        e.attend(0, e.begin({s: 1}), torch.zeros(1, 2, 8), x, x)
    assert held[0].data_ptr() != held[1].data_ptr()


def test_state_engine_forks(monkeypatch):
    monkeypatch.setattr(eng, "jet_cache_copy", fake_copy)
    e = eng.JetEngine(torch.zeros(64, 32), torch.zeros(32, 8), 2, 16, 32, max_seqs=4, chunk_tokens=16)
    e.admit("a")
    e.S[e.slot["a"]] = 3.0
    e.hist[e.slot["a"]] = 5.0
    e.pos["a"] = 17
    e.fork("a", ["b", "c"])
    for s in "bc":
        assert (e.S[e.slot[s]] == 3).all() and (e.hist[e.slot[s]] == 5).all() and e.pos[s] == 17
    assert e.free_slots == 1 and len({e.slot[s] for s in "abc"}) == 3
    with pytest.raises(KeyError):
        e.fork("a", ["b"])
    with pytest.raises(KeyError):
        e.fork("z", ["d"])
    with pytest.raises(RuntimeError):
        e.fork("a", ["d", "e"])
    e.submit("q", tuple(torch.zeros(3, 1) for _ in range(6)))
    with pytest.raises(ValueError):
        e.fork("q", ["d"])
    e.fork("a", [])
    assert e.free_slots == 0
