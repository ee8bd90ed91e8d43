"""jet_attn_rope_append in place, with keys and values beside the queries in
memory: what shares no element is accepted and right, what does is refused."""
import pytest
import torch

from attn_testlib import BF, Batch
from test_gpu_attn_append import freqs

pytestmark = pytest.mark.gpu
Hq, Hk, d = 4, 2, 64


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


def rows(mem, at, stride, heads, N):
    return torch.as_strided(mem, (N, heads, d), (stride, d, 1), at)


# (first element and stride of q, k, v) in one piece of memory
LAYOUTS = {
    "fused": ((0, 512), (256, 512), (384, 512)),
    "fused, keys first": ((256, 512), (0, 512), (128, 512)),
    "a gap behind each row": ((0, 576), (256, 576), (448, 576)),
    "values elsewhere": ((0, 384), (256, 384), (40000, 128)),
    "behind the last row": ((0, 256), (38 * 256, 256), (20000, 256)),
    "behind the last, shorter row": ((0, 512), (37 * 512 + 256, 512), (40000, 512)),
}


@pytest.mark.parametrize("name", list(LAYOUTS))
def test_in_place_beside_keys_and_values(jet, name):
    b = Batch([3, 30, 5], [5, 40, 0], Hq, Hk, d, 16, seed=1)
    assert b.N == 38
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    mem = torch.randn(80000, generator=g, device="cuda").to(BF)
    q, k, v = (rows(mem, *LAYOUTS[name][i], h, b.N) for i, h in enumerate((Hq, Hk, Hk)))
    gam = torch.rand(d, generator=g, device="cuda") + 0.5
    args = (gam, gam, freqs(d), b.cu, b.kv_lens, b.table)
    kp, vp = b.k_pool.clone(), b.v_pool.clone()
    want = jet.jet_attn_rope_append(q.clone(), k.clone(), v.clone(), *args, kp, vp)
    before = mem.clone()
    got = jet.jet_attn_rope_append(q, k, v, *args, b.k_pool, b.v_pool, q)
    assert got is q and torch.equal(q, want)
    same = lambda x, y: torch.equal(x.nan_to_num(99.0), y.nan_to_num(99.0))
    assert same(b.k_pool, kp) and same(b.v_pool, vp)
    rows(before, *LAYOUTS[name][0], Hq, b.N).copy_(q)
    assert torch.equal(mem, before)              # nothing but the queries was written


def test_in_place_over_keys_or_values_is_refused(jet):
    b = Batch([3], [5], Hq, Hq, d, 16, seed=2)
    x = torch.randn((3, Hq, d), device="cuda").to(BF)
    y = torch.randn((3, Hq, d), device="cuda").to(BF)
    args = (None, None, freqs(d), b.cu, b.kv_lens, b.table, b.k_pool, b.v_pool)
    for k, v in ((x, y), (y, x), (x, x)):
        with pytest.raises(jet.JetError):
            jet.jet_attn_rope_append(x, k, v, *args, x)
    for k, v in ((x, y), (x, x)):                # not in place, the same tensor may be all three
        jet.jet_attn_rope_append(x, k, v, *args)
    torch.cuda.synchronize()
    assert jet.jet_device_error() == 0


def test_pools_side_by_side_row_by_row(jet):
    b = Batch([3, 20], [5, 40], Hq, Hk, d, 16, seed=4)
    kv = torch.zeros((b.n_pages, Hk, 16, 2 * d), device="cuda", dtype=BF)
    x = torch.randn((b.N, Hq + 2 * Hk, d), device="cuda").to(BF)
    args = (x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], None, None, freqs(d), b.cu, b.kv_lens, b.table)
    kp, vp = torch.zeros_like(b.k_pool), torch.zeros_like(b.v_pool)
    jet.jet_attn_rope_append(*args, kp, vp)
    jet.jet_attn_rope_append(*args, kv[..., :d], kv[..., d:])
    assert torch.equal(kv[..., :d], kp) and torch.equal(kv[..., d:], vp)
    with pytest.raises(jet.JetError):
        jet.jet_attn_rope_append(*args, kv[..., :d], kv[..., d // 2:d + d // 2])
    torch.cuda.synchronize()
