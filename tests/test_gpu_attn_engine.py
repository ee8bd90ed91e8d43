"""The paged cache of the softmax-attention layers and the forks of the state
cache on the GPU: prompts in pieces, decode, forks, compaction and windows run
together through the engines, every output against the formula in 64 bits."""
import random

import pytest
import torch

import synth
from attn_testlib import BF, F32, attention_bound
from jet_testlib import gpu_inputs
from test_gpu_attn_append import close, freqs, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


class Run:
    """A JetAttnEngine with what its sequences' layers have been given, and checks of every step."""

    def __init__(self, monkeypatch, Hq, Hk, d, page, n_pages, windows, dtype, seed):
        from linear_attention_lm_gen_b200 import attn_engine as ae
        self.Hq, self.Hk, self.d, self.dtype = Hq, Hk, d, dtype
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g = g
        gam = [tuple(1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2)) for _ in windows]
        self.e = ae.JetAttnEngine(len(windows), Hq, Hk, d, n_pages, page, 8, 4096, windows=windows, inv_freq=freqs(d),
                                  gammas=gam, dtype=dtype)
        self.gam = gam
        self.kv = {}           # sequence -> per layer (raw k, v), [T, Hk, d]
        self.turned = []
        real = ae.jet_attn_rope_append

        def spy(*a, **k):
            y = real(*a, **k)
            self.turned.append(y.clone())
            return y
        monkeypatch.setattr(ae, "jet_attn_rope_append", spy)

    def step(self, new):
        b = self.e.begin(new)
        N = b.tokens
        at = [0]
        for n in new.values():
            at.append(at[-1] + n)
        for layer, W in enumerate(self.e.windows):
            x = (torch.randn((N, self.Hq + 2 * self.Hk, self.d), generator=self.g, device="cuda") * 2).to(self.dtype)
            q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hk], x[:, self.Hq + self.Hk:]
            o = self.e.attend(layer, b, q, k, v)
            y = self.turned.pop()
            for s, (seq, n) in enumerate(new.items()):
                old = self.kv.setdefault(seq, {}).get(layer)
                ks, vs = k[at[s]:at[s + 1]], v[at[s]:at[s + 1]]
                self.kv[seq][layer] = (ks.clone(), vs.clone()) if old is None else (torch.cat([old[0], ks]),
                                                                                    torch.cat([old[1], vs]))
                self.check(layer, W, seq, n, y[at[s]:at[s + 1]], o[at[s]:at[s + 1]])

    def check(self, layer, W, seq, n, y, o):
        """The cache holds the sequence's keys and values, and o is the attention of y over them."""
        k, v = self.kv[seq][layer]
        L = k.shape[0]
        assert self.e.len[seq] == L
        lo = max(0, L - n - W + 1) if W else 0
        p = torch.arange(lo, L)
        t = torch.from_numpy(self.e._table[self.e.row[seq]].copy())
        pg, r = t[p // self.e.page].long().cuda(), (p % self.e.page).cuda()
        K, V = self.e.k[layer][pg, :, r], self.e.v[layer][pg, :, r]
        want, mag = reference(k[lo:], self.gam[layer][1], 1e-6, p.cuda(), self.e.inv_freq, False)
        close(K, want, mag, self.dtype)
        assert torch.equal(V, v[lo:])
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        j = p.cuda()[None]
        seen = j <= pos
        if W:
            seen &= j > pos - W
        G = self.Hq // self.Hk
        for h in range(self.Hq):
            x = (y[:, h].double() @ K[:, h // G].double().T) * self.d ** -0.5
            w = torch.softmax(torch.where(seen, x, torch.full_like(x, -torch.inf)), dim=1)
            ref, a = w @ V[:, h // G].double(), w @ V[:, h // G].double().abs()
            bad = ((o[:, h].double() - ref).abs() - attention_bound(ref, a, self.dtype)).amax().item()
            assert bad <= 0, (seq, layer, h, bad)

    def fork(self, parent, children):
        self.e.fork(parent, children)
        for c in children:
            self.kv[c] = dict(self.kv[parent])

    def release(self, seq):
        self.e.release(seq)
        del self.kv[seq]


@pytest.mark.parametrize("dtype,Hq,Hk,d,page,windows", [
    (BF, 12, 2, 128, 64, [0, 0, 100]), (BF, 16, 2, 128, 16, [90, 200]), (F32, 6, 3, 64, 32, [0, 50]),
    (BF, 5, 1, 80, 16, [0])])
def test_serving_steps_with_forks_and_compaction(jet, monkeypatch, dtype, Hq, Hk, d, page, windows):
    r = random.Random(7)
    run = Run(monkeypatch, Hq, Hk, d, page, 4000 // page, windows, dtype, 3)
    e = run.e
    for s in "abc":
        e.admit(s)
    run.step({"a": 300, "b": 1, "c": 70})
    run.step({"b": 130, "a": 1, "c": 1})
    run.fork("a", ["a1", "a2"])
    run.fork("c", ["c1"])
    run.step({s: 1 for s in e.row})
    run.release("a")
    run.step({"a1": 33, "b": 1, "c1": 2})
    before = e.free_pages
    n = e.compact()
    assert e.free_pages == before == e.n_pages - n and sorted(e._free) == list(range(n, e.n_pages))
    for k in e.pools:                       # what lies behind the live pages is not read
        k[n:] = float("nan")
    for _ in range(4):
        run.step({s: r.choice([1, 1, 1, 17]) for s in e.row})
    run.release("b")
    run.fork("a2", ["z"])
    e.compact()
    run.step({s: 1 for s in e.row})
    assert jet.jet_device_error() == 0


def test_state_engine_forks_continue_the_parent(jet):
    """Sequences forked from a prompt decode as if each had run it."""
    s = synth.JetShape("fork", B=1, T=90, H=2, dk=64, dv=128, D=64)
    d = gpu_inputs(synth.prefill_inputs(s, seed=5, T=96))
    from linear_attention_lm_gen_b200.engine import JetEngine
    names = ("x", "q", "k", "v", "g", "beta")
    prompt = lambda a, b: tuple(d[n][0, a:b].contiguous() for n in names)
    tok = lambda i: tuple(d[n][0, 90 + i].contiguous() for n in names)

    def engine():
        return JetEngine(d["W1"], d["W2"], s.H, s.dk, s.dv, max_seqs=6, chunk_tokens=64)
    e = engine()
    e.admit("p")
    e.prefill("p", *prompt(0, 90))
    e.step({"p": tok(0)})
    e.fork("p", ["c0", "c1", "c2"])
    got = {}
    for i in range(2):
        out = e.step({f"c{j}": tok(1 + (i + j) % 5) for j in range(3)})
        for j in range(3):
            got.setdefault(j, []).append(out[f"c{j}"])
    for j in range(3):
        f = engine()
        f.admit("p")
        f.prefill("p", *prompt(0, 90))
        f.step({"p": tok(0)})
        for i in range(2):
            assert torch.equal(f.step({"p": tok(1 + (i + j) % 5)})["p"], got[j][i])
        assert torch.equal(f.S[f.slot["p"]], e.S[e.slot[f"c{j}"]])
        assert torch.equal(f.hist[f.slot["p"]], e.hist[e.slot[f"c{j}"]])
    assert jet.jet_device_error() == 0
