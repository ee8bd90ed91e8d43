"""Argument checks of the softmax-attention and cache entry points, without a
GPU: every call here passes an argument that the host rejects before any
launch."""
import ctypes

import pytest
import torch

import linear_attention_lm_gen_b200 as jet
from linear_attention_lm_gen_b200 import build as jbuild

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 7
A = 1 << 40                    # aligned, never-dereferenced addresses, far apart
STEP = 1 << 36
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    jbuild.build()
    return jet.load_library()


def P(x):
    return ctypes.c_void_p(x)


def append(lib, q=A, qs=512, k=A + STEP, ks=128, v=A + 2 * STEP, vs=128, gq=A, gk=A, eps=1e-6, fr=A, rot=64, inter=0,
           qo=A + 3 * STEP, qos=256, kp=A + 4 * STEP, vp=A + 5 * STEP, ps=2 * 16 * 64, hs=16 * 64, rs=64, cu=A, kv=A,
           pt=A, nseq=2, N=5, mp=4, np=9, page=16, Hq=4, Hk=2, d=64, dt=BF16):
    return lib.jet_attn_rope_append(P(q), qs, P(k), ks, P(v), vs, P(gq), P(gk), eps, P(fr), rot, inter, P(qo), qos,
                                    P(kp), P(vp), ps, hs, rs, P(cu), P(kv), P(pt), nseq, N, mp, np, page, Hq, Hk, d,
                                    dt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(cu=None), INVALID), (dict(gk=None), INVALID),
    (dict(fr=None), INVALID), (dict(rot=72), INVALID), (dict(rot=-8), INVALID), (dict(rot=12), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(N=0), INVALID), (dict(nseq=0), INVALID), (dict(mp=0), INVALID), (dict(np=0), INVALID),
    (dict(Hq=5), INVALID), (dict(Hk=0), INVALID), (dict(dt=2), INVALID),
    (dict(d=72, qs=512), UNSUPPORTED), (dict(d=144, qs=1024, ks=512, vs=512, qos=1024, ps=1 << 14, hs=1 << 13, rs=256),
                                        UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(page=24), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
    (dict(nseq=70000), UNSUPPORTED), (dict(mp=1 << 30), UNSUPPORTED),
    (dict(qs=255), INVALID), (dict(ks=127), INVALID), (dict(qs=260), MISALIGNED), (dict(qos=0), INVALID),
    (dict(vs=-128), INVALID), (dict(ps=63), INVALID), (dict(hs=0), INVALID), (dict(rs=68), MISALIGNED),
    (dict(rs=66), MISALIGNED), (dict(q=A + 8), MISALIGNED), (dict(kp=A + 4 * STEP + 8), MISALIGNED),
    (dict(gq=A + 2), MISALIGNED), (dict(pt=A + 1), MISALIGNED),
    (dict(qo=A), INVALID),                       # in place with another stride
    (dict(qo=A + 16), INVALID), (dict(qo=A + STEP), INVALID), (dict(qo=A + 4 * STEP), INVALID),
    (dict(vp=A + 4 * STEP), INVALID), (dict(k=A + 4 * STEP), INVALID),
])
def test_append_rejects(lib, kw, expect):
    assert append(lib, **kw) == expect


def paged(lib, q=A, qs=256, kp=A + STEP, vp=A + 2 * STEP, ps=2 * 16 * 64, hs=16 * 64, rs=64, cu=A, kv=A, pt=A,
          o=A + 3 * STEP, ws=A + 4 * STEP, wsb=1 << 34, nseq=2, N=5, mx=3, mp=4, np=9, page=16, Hq=4, Hk=2, d=64,
          window=0, scale=0.125, dt=BF16):
    return lib.jet_attn_paged(P(q), qs, P(kp), P(vp), ps, hs, rs, P(cu), P(kv), P(pt), P(o), P(ws), wsb, nseq, N, mx,
                              mp, np, page, Hq, Hk, d, window, scale, dt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(vp=None), INVALID), (dict(o=None), INVALID), (dict(pt=None), INVALID),
    (dict(N=0), INVALID), (dict(nseq=-1), INVALID), (dict(Hq=3), INVALID), (dict(dt=-1), INVALID),
    (dict(window=-1), INVALID), (dict(mx=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(d=24), UNSUPPORTED), (dict(page=12), UNSUPPORTED), (dict(Hq=512, Hk=2, qs=1 << 16), UNSUPPORTED),
    (dict(Hq=130, Hk=2, qs=1 << 16), UNSUPPORTED), (dict(mp=1 << 27), UNSUPPORTED),
    (dict(qs=128), INVALID), (dict(qs=260), MISALIGNED), (dict(ps=8), INVALID), (dict(rs=65), MISALIGNED),
    (dict(q=A + 4), MISALIGNED), (dict(o=A + 3 * STEP + 2), MISALIGNED), (dict(ws=A + 4 * STEP + 4), MISALIGNED),
    (dict(cu=A + 2), MISALIGNED),
    (dict(o=A), INVALID), (dict(o=A + STEP), INVALID), (dict(o=A + 2 * STEP + 1024), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=0), WORKSPACE),
])
def test_paged_rejects(lib, kw, expect):
    assert paged(lib, **kw) == expect


def test_paged_workspace_is_host_only_and_bounded(lib):
    assert jet.jet_attn_paged_workspace_size(0, 1, 4, 2, 64) == 0
    assert jet.jet_attn_paged_workspace_size(1, 1, 4, 3, 64) == 0
    small, large = (jet.jet_attn_paged_workspace_size(b, n, 12, 2, 128) for b, n in ((1, 1), (256, 1 << 18)))
    assert 0 < small <= large <= 128 << 20
    n = jet.jet_attn_paged_workspace_size(2, 5, 4, 2, 64)
    assert paged(lib, wsb=n - 1) == WORKSPACE


def arrays(*xs, t=ctypes.c_int64):
    return (t * len(xs))(*xs)


def copy(lib, pools=(A, A + STEP), size=(256, 512), step=(256, 1024), n_pools=2, entries=10, src=(1, 2), dst=(3, 4),
         n=2):
    return lib.jet_cache_copy(arrays(*pools, t=ctypes.c_void_p), arrays(*size), arrays(*step), n_pools, entries,
                              arrays(*src, t=ctypes.c_int), arrays(*dst, t=ctypes.c_int), n, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(pools=(A, None)), INVALID), (dict(n_pools=0), INVALID), (dict(entries=0), INVALID), (dict(n=-1), INVALID),
    (dict(pools=(A,) * 65, size=(16,) * 65, step=(16,) * 65, n_pools=65), UNSUPPORTED),
    (dict(size=(0, 512)), INVALID), (dict(step=(128, 1024)), INVALID), (dict(size=(250, 512)), MISALIGNED),
    (dict(step=(264, 1024)), MISALIGNED), (dict(pools=(A, A + STEP + 8)), MISALIGNED),
    (dict(src=(1, 10)), INVALID), (dict(src=(1, -1)), INVALID), (dict(dst=(3, 10)), INVALID),
    (dict(dst=(3, -1)), INVALID), (dict(dst=(3, 3)), INVALID), (dict(dst=(3, 1)), INVALID),
    (dict(src=(1, 4), dst=(4, 5)), INVALID), (dict(src=(3, 2)), INVALID),
    (dict(entries=1 << 30, src=(1 << 29, 2), dst=(1, 1 << 29)), INVALID),
    (dict(n=0), OK),
])
def test_copy_rejects(lib, kw, expect):
    before = jet.jet_launch_count()
    assert copy(lib, **kw) == expect
    assert jet.jet_launch_count() == before


def test_copy_rejects_null_lists(lib):
    f = lambda *a: lib.jet_cache_copy(*a, None)
    p, z, t = arrays(A, t=ctypes.c_void_p), arrays(256), arrays(256)
    i = arrays(1, t=ctypes.c_int)
    assert f(None, z, t, 1, 4, i, i, 1) == INVALID
    assert f(p, None, t, 1, 4, i, i, 1) == INVALID
    assert f(p, z, None, 1, 4, i, i, 1) == INVALID
    assert f(p, z, t, 1, 4, None, i, 1) == INVALID
    assert f(p, z, t, 1, 4, i, None, 1) == INVALID
    assert f(p, z, t, 1, 4, None, None, 0) == OK


def compact(lib, pool=A, size=256, step=256, pages=10, page=16, pt=A + STEP, kv=A + 2 * STEP, nseq=2, mp=4,
            out=A + 3 * STEP, live=A + 4 * STEP, ws=A + 5 * STEP, wsb=1 << 30):
    return lib.jet_cache_compact(arrays(pool, t=ctypes.c_void_p), arrays(size), arrays(step), 1, pages, page, P(pt),
                                 P(kv), nseq, mp, P(out), P(live), P(ws), wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(pool=None), INVALID), (dict(pt=None), INVALID), (dict(kv=None), INVALID), (dict(out=None), INVALID),
    (dict(live=None), INVALID), (dict(nseq=0), INVALID), (dict(mp=0), INVALID), (dict(page=0), INVALID),
    (dict(pages=0), INVALID), (dict(page=20), UNSUPPORTED), (dict(pages=(1 << 20) + 1), UNSUPPORTED),
    (dict(mp=1 << 28), UNSUPPORTED), (dict(size=200), MISALIGNED), (dict(pt=A + STEP + 2), MISALIGNED),
    (dict(live=A + 2), MISALIGNED), (dict(ws=A + 5 * STEP + 4), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE),
    (dict(out=A + STEP + 4), INVALID), (dict(live=A + STEP), INVALID), (dict(live=A + 3 * STEP + 8), INVALID),
    (dict(live=A + 2 * STEP), INVALID), (dict(out=A + 2 * STEP), INVALID),
])
def test_compact_rejects(lib, kw, expect):
    assert compact(lib, **kw) == expect


def test_compact_workspace(lib):
    assert jet.jet_cache_compact_workspace_size(0) == 0
    assert jet.jet_cache_compact_workspace_size((1 << 20) + 1) == 0
    for n in (1, 2, 31, 33, 8192, 1 << 20):
        need = jet.jet_cache_compact_workspace_size(n)
        assert need >= 4 + 8 * (n // 2) + 4 * n       # count, moves, new indices
        assert compact(lib, pages=n, wsb=need - 1) == WORKSPACE


def test_python_bindings_refuse_cpu_tensors():
    t = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        jet.jet_attn_paged(t, pool, pool, i, i, i.view(1, 3))
    with pytest.raises(TypeError):
        jet.jet_attn_rope_append(t, t, t, None, None, None, i, i, i.view(1, 3), pool, pool)
    with pytest.raises(TypeError):
        jet.jet_cache_copy([pool], [0], [1])
    with pytest.raises(TypeError):
        jet.jet_cache_copy(pool, [0], [1])
    with pytest.raises(TypeError):
        jet.jet_cache_compact([pool], i.view(1, 3), i[:1], 16)
