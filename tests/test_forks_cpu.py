"""Forks whose copy fails leave the engines as they were (on the CPU, with
stand-ins for the library's calls)."""
import copy

import pytest
import torch

from linear_attention_lm_gen_b200 import attn_engine as ae
from linear_attention_lm_gen_b200 import engine as eng
from test_attn_engine_cpu import Texts, consistent, fake_copy, make  # noqa: F401


def failing(times):
    """A copy that fails after `times` calls."""
    left = [times]

    def copy_(pools, src, dst):
        if left[0] == 0:
            raise RuntimeError("jet_cache_copy failed")
        left[0] -= 1
        fake_copy(pools, src, dst)
    return copy_


def host_state(e):
    return copy.deepcopy((e.row, e.len, e._first, sorted(e._free), e._rows, e._ref.tolist(), e._table.tolist()))


def test_attention_engine(make, monkeypatch):  # noqa: F811
    e = make()
    t = Texts(e)
    e.admit("a")
    t.step({"a": 40})
    before = host_state(e)
    with monkeypatch.context() as m:
        m.setattr(ae, "jet_cache_copy", failing(0))
        with pytest.raises(RuntimeError, match="jet_cache_copy"):
            e.fork("a", ["b", "c"])
    assert host_state(e) == before
    consistent(e)
    t.fork("a", ["b", "c"])
    t.step({"a": 1, "b": 20, "c": 1})
    consistent(e)


def test_attention_engine_with_more_pools_than_a_call_takes(monkeypatch):
    monkeypatch.setattr(ae, "jet_cache_copy", fake_copy)
    e = ae.JetAttnEngine(40, 2, 1, 8, 8, 16, 4, 64, dtype=torch.float32, device="cpu")
    e.admit("a")
    e.begin({"a": 20})
    before = host_state(e)
    with monkeypatch.context() as m:
        m.setattr(ae, "jet_cache_copy", failing(1))      # the second call of two
        with pytest.raises(RuntimeError, match="jet_cache_copy"):
            e.fork("a", ["b"])
    assert host_state(e) == before
    for p in e.pools:
        p[int(e._table[e.row["a"], 1])] = 3.0
    e.fork("a", ["b"])
    assert all((p[int(e._table[e.row["b"], 1])] == 3).all() for p in e.pools)
    consistent(e)


def test_state_engine(monkeypatch):
    monkeypatch.setattr(eng, "jet_cache_copy", failing(0))
    e = eng.JetEngine(torch.zeros(64, 32), torch.zeros(32, 8), 2, 16, 32, max_seqs=4, chunk_tokens=16)
    e.admit("a")
    e.S[e.slot["a"]] = 3.0
    free = list(e._free)
    with pytest.raises(RuntimeError, match="jet_cache_copy"):
        e.fork("a", ["b", "c"])
    assert e._free == free and list(e.slot) == ["a"] and list(e.pos) == ["a"]
    monkeypatch.setattr(eng, "jet_cache_copy", fake_copy)
    e.fork("a", ["b", "c"])
    assert e.free_slots == 1 and all((e.S[e.slot[s]] == 3).all() for s in "bc")
