"""jet_attn_rope_append: elements that are not rotated have no partner, so a
non-finite one stays where it is; in a rotated pair it reaches its partner
only."""
import pytest
import torch

from attn_testlib import BF, F32, HALF_STEP, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


def rotated(x, pos, f, interleaved):
    """The rotation in 64 bits; elements from 2 len(f) on as they are."""
    y = x.double().clone()
    if f is not None:
        h = f.numel()
        i = torch.arange(h, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        t = pos.double()[:, None, None] * f.double()
        c, s = torch.cos(t), torch.sin(t)
        ya, yb = x.double()[..., a], x.double()[..., b]
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y


def same(got, want, dtype, what):
    """Equal where not finite; elsewhere rounded once, with 16 float32 roundings of a pair's magnitude (values up to 16)."""
    want = want.to(got.device)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), what
    assert torch.equal(got[~fin].double().nan_to_num(nan=7.0, posinf=8.0, neginf=9.0),
                       want[~fin].nan_to_num(nan=7.0, posinf=8.0, neginf=9.0)), what
    err = (got[fin].double() - want[fin]).abs() - 1.01 * HALF_STEP[dtype] * want[fin].abs() - 16 * 2.0 ** -24 * 32
    assert err.amax().item() <= 0, what


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot", [(128, 64), (128, 0), (96, 40), (64, 0), (48, 8), (80, 64), (16, 8), (112, 0)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_non_finite_element_behind_the_rotated_part_stays_alone(jet, interleaved, value, d, rot, dtype):
    b = Batch([3, 30], [5, 40], 4, 2, d, 16, dtype, seed=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((b.N, 8, d), generator=g, device="cuda").clamp(-8, 8).to(dtype)
    for row in range(b.N):                     # one element of every head of every token, all columns in turn
        for h in range(8):
            x[row, h, rot + (row * 8 + h) % (d - rot)] = value
    f = None if rot == 0 else (0.3 ** torch.arange(rot // 2, dtype=torch.float64)).float().cuda()
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(b.new, b.kv)]).cuda()
    q = torch.empty((b.N, 4, d), device="cuda", dtype=dtype)
    jet.jet_attn_rope_append(x[:, :4], x[:, 4:6], x[:, 6:], None, None, f, b.cu, b.kv_lens, b.table, b.k_pool, b.v_pool, q,
                             interleaved=interleaved)
    same(q, rotated(x[:, :4], pos, f, interleaved), dtype, "q")
    want = rotated(x[:, 4:6], pos, f, interleaved)
    at = 0
    for s, (n, L) in enumerate(zip(b.new, b.kv)):
        for i in range(n):
            p = L - n + i
            pg = int(b.host_table[s, p // 16])
            same(b.k_pool[pg, :, p % 16], want[at + i], dtype, f"k of token {i} of sequence {s}")
        at += n
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rot", [0, 64, 128])
def test_an_infinite_element_under_the_norm(jet, rot, dtype):
    """The mean of squares is infinite: x / sqrt(inf) is zero everywhere but at the infinity itself."""
    d = 128
    b = Batch([6], [3], 2, 1, d, 16, dtype, seed=3)
    x = torch.ones((b.N, 4, d), device="cuda", dtype=dtype)
    x[:, :, d - 1] = float("inf")
    gamma = torch.full((d,), 2.0, device="cuda")
    f = None if rot == 0 else torch.full((rot // 2,), 0.01, device="cuda")
    q = torch.empty((b.N, 2, d), device="cuda", dtype=dtype)
    jet.jet_attn_rope_append(x[:, :2], x[:, 2:3], x[:, 3:], gamma, gamma, f, b.cu, b.kv_lens, b.table, b.k_pool, b.v_pool, q)
    odd = [d - 1] + ([d // 2 - 1] if rot == d else [])        # with the whole row rotated, its partner too
    keep = [i for i in range(d) if i not in odd]
    assert (q[:, :, keep] == 0).all()
    assert torch.isnan(q[:, :, odd]).all()
