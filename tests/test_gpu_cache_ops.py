"""jet_cache_copy and jet_cache_compact against indexing."""
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


def rand(*shape, dtype=BF):
    return torch.randn(shape, device="cuda").to(dtype)


@pytest.mark.parametrize("n", [1, 2, 7, 255, 256, 257, 3584, 3585, 5000])
def test_copies_of_many_entries(jet, n):
    E = 2 * n + 3
    pools = [rand(E, 1, 16, 16), rand(E, 4, dtype=F32)]
    ids = list(range(E))
    random.Random(n).shuffle(ids)
    dst = ids[:n]
    src = [ids[n + (i // 2) % (E - n)] for i in range(n)]
    want = [p.clone() for p in pools]
    for w, p in zip(want, pools):
        w[dst] = p[src]
    jet.jet_cache_copy(pools, src, dst)
    for w, p in zip(want, pools):
        assert torch.equal(w, p)


@pytest.mark.parametrize("shape,dtype", [((1, 16, 16), BF), ((2, 64, 128), BF), ((3, 5, 32), BF), ((12, 256, 96), F32),
                                         ((8,), BF), ((5, 1000, 8), F32), ((2, 32, 80), BF)])
def test_entry_sizes_and_strided_pools(jet, shape, dtype):
    pools = [rand(9, *shape, dtype=dtype), rand(9, 2, *shape, dtype=dtype)[:, 1]]
    if len(shape) == 3:
        pools.append(rand(9, shape[1], shape[0], shape[2], dtype=dtype).transpose(1, 2))
    whole = [p._base if p._base is not None else p for p in pools]
    want = [p.clone() for p in whole]
    for w, p in zip(want, pools):
        view = w if p._base is None else (w[:, 1] if p.stride() != w.transpose(1, 2).stride() or w.dim() == 5
                                          else w.transpose(1, 2))
        view[[3, 0, 8]] = p[[5, 5, 1]]
    jet.jet_cache_copy(pools, [5, 5, 1], torch.tensor([3, 0, 8]))
    for w, p in zip(want, whole):
        assert torch.equal(w, p)


def test_nothing_to_copy(jet):
    before = jet.jet_launch_count()
    jet.jet_cache_copy([rand(4, 8)], [], [])
    assert jet.jet_launch_count() == before


def test_copy_refuses(jet):
    p = rand(6, 2, 16, 16)
    old = p.clone()
    for src, dst in (([0], [6]), ([-1], [2]), ([0, 1], [2, 2]), ([0, 1], [1, 2]), ([3], [3])):
        with pytest.raises(jet.JetError):
            jet.jet_cache_copy([p], src, dst)
    with pytest.raises(ValueError):
        jet.jet_cache_copy([p], [0, 1], [2])
    with pytest.raises(ValueError):
        jet.jet_cache_copy([p, rand(5, 8)], [0], [1])
    with pytest.raises(ValueError):
        jet.jet_cache_copy([p[:, :, :8]], [0], [1])
    with pytest.raises(TypeError):
        jet.jet_cache_copy([p], torch.tensor([0]).cuda(), [1])
    with pytest.raises(TypeError):
        jet.jet_cache_copy([p.cpu()], [0], [1])
    with pytest.raises(jet.JetError):
        jet.jet_cache_copy([rand(6, 3)], [0], [1])          # 6 bytes an entry
    with pytest.raises(jet.JetError):
        jet.jet_cache_copy([p] * 65, [0], [1])
    torch.cuda.synchronize()
    assert torch.equal(p, old)


def test_copy_in_a_graph_and_on_a_stream(jet):
    p = rand(8, 2, 16, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = p.clone()
    want[3] = want[1]
    jet.jet_cache_copy([p], [1], [3], stream=s)
    s.synchronize()
    assert torch.equal(p, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        jet.jet_cache_copy([p], [0, 0], [5, 6])
    p[0] = 1.0
    g.replay()
    assert (p[5] == 1).all() and (p[6] == 1).all()


# ---------------------------------------------------------------- compaction
def expect(table, kv, page, P):
    out, n, to = expect_np(table.numpy(), kv, page, P)
    return torch.from_numpy(out), n, to


def expect_np(table, kv, page, P):
    held = sorted({int(table[s, i]) for s in range(len(kv)) for i in range(-(-kv[s] // page)) if table[s, i] >= 0})
    n = len(held)
    kept = set(held)
    holes = [i for i in range(n) if i not in kept]
    to = {i: i for i in held if i < n}
    to.update(zip([i for i in held if i >= n], holes))
    out = np.full_like(table, -1)
    for s in range(len(kv)):
        for i in range(-(-kv[s] // page)):
            if table[s, i] >= 0:
                out[s, i] = to[int(table[s, i])]
    return out, n, to


def tables(P, kv, page, seed, shared=0, width=None):
    r = random.Random(seed)
    ids = list(range(P))
    r.shuffle(ids)
    need = [-(-x // page) for x in kv]
    table = torch.full((len(kv), width or max(max(need), 1)), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        first = 0
        if shared and s:
            first = min(n, need[s - 1], shared)
            table[s, :first] = table[s - 1, :first]
        for i in range(first, n):
            table[s, i] = ids.pop()
    return table


@pytest.mark.parametrize("P,kv,page,shared", [
    (10, [3], 16, 0), (1, [5], 16, 0), (40, [0, 0], 16, 0), (33, [100, 0, 31, 32], 16, 0), (64, [1024], 16, 0),
    (31, [200, 90], 16, 4), (300, [100, 700, 1, 900, 64], 32, 3), (5000, [40000, 30000, 1], 16, 100),
    (100000, [300000, 200001], 16, 0), (70, [16] * 60, 16, 1)])
def test_compaction(jet, P, kv, page, shared):
    table = tables(P, kv, page, P, shared)
    pools = [rand(P, 1, page, 16), rand(P, 2, 8, dtype=F32)]
    before = [p.clone() for p in pools]
    want, n, to = expect(table, kv, page, P)
    dt, dk = table.cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda")
    out, live = jet.jet_cache_compact(pools, dt, dk, page)
    assert int(live) == n
    assert torch.equal(out.cpu(), want)
    assert torch.equal(dt.cpu(), table)
    if to:
        a, b = torch.tensor(list(to)), torch.tensor(list(to.values()))
        for p, o in zip(pools, before):
            assert torch.equal(p[b], o[a])
    # a second time: nothing moves
    out2, live2 = jet.jet_cache_compact(pools, out, dk, page)
    assert int(live2) == n and torch.equal(out2, out)
    assert jet.jet_device_error() == 0


def test_compaction_in_place_with_given_up_pages_and_stale_entries(jet):
    P, page, kv = 50, 16, [100, 33, 160]
    table = tables(P, kv, page, 1, width=20)
    table[2, 0] = -1                       # before the window
    table[1, 10] = 49                      # behind the sequence's length
    want, n, to = expect(table, kv, page, P)
    pool = rand(P, 2, page, 32)
    old = pool.clone()
    dt = table.cuda()
    out, live = jet.jet_cache_compact([pool], dt, torch.tensor(kv, dtype=torch.int32, device="cuda"), page, dt)
    assert out is dt and torch.equal(dt.cpu(), want) and int(live) == n
    for a, b in to.items():
        assert torch.equal(pool[b], old[a])
    assert jet.jet_device_error() == 0


def test_compaction_flags_bad_tables(jet):
    assert jet.jet_device_error() == 0
    P, page, kv = 20, 16, [64, 64]
    table = tables(P, kv, page, 2)
    table[0, 1] = P
    table[1, 2] = -7
    fixed = table.clone()
    fixed[0, 1] = fixed[1, 2] = -1
    want, n, _ = expect(fixed, kv, page, P)
    out, live = jet.jet_cache_compact([rand(P, 8)], table.cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda"),
                                      page)
    assert torch.equal(out.cpu(), want) and int(live) == n
    assert jet.jet_device_error() == 6
    table = tables(P, kv, page, 3)
    out, live = jet.jet_cache_compact([rand(P, 8)], table.cuda(),
                                      torch.tensor([-5, 1000], dtype=torch.int32, device="cuda"), page)
    want, n, _ = expect(table, [0, 64], page, P)
    assert torch.equal(out.cpu(), want) and int(live) == n
    assert jet.jet_device_error() == 6


def test_compaction_in_a_graph(jet):
    P, page, kv = 60, 16, [200, 300]
    table = tables(P, kv, page, 4)
    pool = rand(P, 2, page, 16)
    dt, dk = table.cuda(), torch.tensor(kv, dtype=torch.int32, device="cuda")
    ws = torch.empty(jet.jet_cache_compact_workspace_size(P), device="cuda", dtype=torch.uint8)
    live = torch.empty(1, device="cuda", dtype=torch.int32)
    out = torch.empty_like(dt)
    jet.jet_cache_compact([pool], dt, dk, page, out, live, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        jet.jet_cache_compact([pool], dt, dk, page, out, live, ws)
    table = tables(P, kv, page, 5)
    kv2 = [90, 10]
    old = pool.clone()
    dt.copy_(table)
    dk.copy_(torch.tensor(kv2, dtype=torch.int32))
    g.replay()
    want, n, to = expect(table, kv2, page, P)
    assert torch.equal(out.cpu(), want) and int(live) == n
    for a, b in to.items():
        assert torch.equal(pool[b], old[a])


def test_compaction_refuses(jet):
    p = rand(10, 8)
    t = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    kv = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(jet.JetError):
        jet.jet_cache_compact([p], t, kv, 24)
    with pytest.raises(jet.JetError):
        jet.jet_cache_compact([p], t, kv, 16, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))
    with pytest.raises(jet.JetError):
        jet.jet_cache_compact([p], t, kv, 16, n_live=t[0, :1])
    with pytest.raises(TypeError):
        jet.jet_cache_compact([p], t.long(), kv, 16)
    with pytest.raises(ValueError):
        jet.jet_cache_compact([p], t, kv[:0], 16)
