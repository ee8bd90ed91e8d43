"""jet_attn_rope_append against the formula in 64 bits, and its part in a
prompt that is appended and attended to piece by piece."""
import pytest
import torch

from attn_testlib import BF, F32, HALF_STEP, Batch, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


def freqs(rot, base=1e6):
    return (base ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))).float().cuda()


def reference(x, gamma, eps, pos, inv_freq, interleaved):
    """(y, a): norm and rotation in 64 bits, and the sum of the magnitudes that each result is made of."""
    y = x.double()
    if gamma is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gamma.double()
    out, mag = y.clone(), y.abs().clone()
    if inv_freq is not None:
        h = inv_freq.numel()
        t = pos.double()[:, None] * inv_freq.double()[None]
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        i = torch.arange(h, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, mag


def close(got, want, mag, dtype):
    # rounded once (half a step of the value); float32 arithmetic: the norm's d products and a
    # rotation's few roundings, and sines of a reduced angle, within 16 roundings of each term
    bound = 1.01 * HALF_STEP[dtype] * want.abs() + 16 * 2.0 ** -24 * mag + 1e-30
    bad = ((got.double() - want).abs() - bound).amax().item()
    assert bad <= 0, f"above the bound by {bad:.3e}"


def run_case(jet, b, rot, norm=True, interleaved=False, fused=True, inplace=False, eps=1e-6, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(100 + seed)
    N, Hq, Hk, d = b.N, b.Hq, b.Hk, b.d
    if fused:
        x = (torch.randn((N, Hq + 2 * Hk, d), generator=g, device="cuda") * 3).to(b.dtype)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    else:
        q, k, v = ((torch.randn((N, h, d), generator=g, device="cuda") * 3).to(b.dtype) for h in (Hq, Hk, Hk))
    gq = torch.randn(d, generator=g, device="cuda") if norm else None
    gk = torch.randn(d, generator=g, device="cuda") if norm else None
    f = freqs(rot) if rot else None
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    before_k, before_v = b.k_pool.clone(), b.v_pool.clone()
    q_out = q if inplace else torch.full((N, Hq, d), 7.0, device="cuda", dtype=b.dtype)
    r = jet.jet_attn_rope_append(q, k, v, gq, gk, f, b.cu, b.kv_lens, b.table, b.k_pool, b.v_pool, q_out, eps=eps,
                                 interleaved=interleaved)
    assert r is q_out
    torch.cuda.synchronize()
    want_k, want_v = before_k, before_v
    seen = torch.zeros(N, dtype=torch.bool, device="cuda")
    for s, (n, L) in enumerate(zip(b.new, b.kv)):
        if n == 0:
            continue
        rows = slice(b.cu_host[s], b.cu_host[s] + n)
        pos = torch.arange(L - n, L, device="cuda")
        ok = pos >= 0
        seen[rows] = ok
        y, m = reference(q0[rows], gq, eps, pos, f, interleaved)
        close(q_out[rows][ok], y[ok], m[ok], b.dtype)
        y, m = reference(k0[rows], gk, eps, pos, f, interleaved)
        for i in range(n):
            p = L - n + i
            if p < 0:
                continue
            pg, row = int(b.host_table[s, p // b.page]), p % b.page
            close(b.k_pool[pg, :, row], y[i], m[i], b.dtype)
            assert torch.equal(b.v_pool[pg, :, row], v0[rows][i])
            want_k[pg, :, row], want_v[pg, :, row] = b.k_pool[pg, :, row], b.v_pool[pg, :, row]
    # nothing else was written
    same = lambda a, c: torch.equal(a.nan_to_num(12345.0), c.nan_to_num(12345.0))
    assert same(b.k_pool, want_k) and same(b.v_pool, want_v)
    assert torch.equal(q_out[~seen], q0[~seen] if inplace else torch.full_like(q_out[~seen], 7.0))
    if not inplace:
        assert torch.equal(q, q0)
    assert torch.equal(k, k0) and torch.equal(v, v0)


def batch(Hq, Hk, d, page=16, dtype=BF, seed=0, **kw):
    return Batch([1, 17, 0, 64, 3], [0, 30, 9, 1, 250], Hq, Hk, d, page, dtype, seed, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,d,rot", [(12, 2, 128, 128), (16, 2, 128, 64), (4, 2, 64, 64), (5, 5, 96, 96),
                                         (14, 2, 80, 40), (8, 1, 16, 16), (6, 3, 48, 8), (2, 1, 128, 0),
                                         (64, 1, 112, 112)])
def test_heads_and_rotated_parts(jet, Hq, Hk, d, rot, dtype):
    for interleaved in (False, True):
        run_case(jet, batch(Hq, Hk, d, dtype=dtype), rot, interleaved=interleaved)
    run_case(jet, batch(Hq, Hk, d, dtype=dtype), rot, norm=False)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["head", "token", "side", "wide"])
def test_layouts_and_in_place_queries(jet, layout, dtype):
    run_case(jet, batch(12, 2, 128, 32, dtype, layout=layout), 128, fused=False)
    run_case(jet, batch(12, 2, 128, 32, dtype, layout=layout), 128, inplace=True)
    run_case(jet, batch(4, 2, 64, 64, dtype, layout=layout, pad=5), 64, fused=False, inplace=True)


def test_many_tokens_and_far_positions(jet):
    b = Batch([2500, 1, 100], [0, 130000, 262000], 4, 1, 64, 64, seed=3)
    run_case(jet, b, 64)
    b = Batch([2500, 1, 100], [0, 30000, 62000], 3, 1, 128, 256, F32, seed=4)
    run_case(jet, b, 128, interleaved=True)


def test_tokens_without_a_position(jet):
    b = batch(4, 2, 64)
    b.kv[1] = 5
    b.kv_lens[1] = 5
    run_case(jet, b, 64)
    assert jet.jet_device_error() == 0


def test_zero_rows_and_small_values(jet):
    b = Batch([3], [4], 2, 1, 64, 16, F32)
    x = torch.zeros((3, 4, 64), device="cuda")
    x[1] = 1e-20
    x[2, :, 3] = 1e18
    g = torch.ones(64, device="cuda")
    o = jet.jet_attn_rope_append(x[:, :2], x[:, 2:3], x[:, 3:], g, g, None, b.cu, b.kv_lens, b.table, b.k_pool,
                                 b.v_pool)
    assert (o[0] == 0).all()
    assert torch.allclose(o[1], torch.full_like(o[1], 1e-17), rtol=1e-5)
    assert torch.allclose(o[2, :, 3], torch.full_like(o[2, :, 3], 8.0), rtol=1e-5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_pages_and_lengths_are_flagged_and_not_written(jet, dtype):
    assert jet.jet_device_error() == 0
    for what in ("page", "length", "offsets"):
        b = batch(4, 2, 64, dtype=dtype)
        if what == "page":
            b.table[4, 15] = b.n_pages           # position 250 on
        elif what == "length":
            b.kv_lens[4] = 16 * b.table.shape[1] + 1
        else:
            b.cu[5] = -3
        x = torch.randn((b.N, 8, 64), device="cuda").to(dtype)
        old_k = b.k_pool.clone()
        jet.jet_attn_rope_append(x[:, :4], x[:, 4:6], x[:, 6:], None, None, None, b.cu, b.kv_lens, b.table, b.k_pool,
                                 b.v_pool)
        if what != "offsets":
            assert jet.jet_device_error() == 6
            pages = b.host_table[4][b.host_table[4] >= 0].long()
            assert torch.equal(b.k_pool[pages].nan_to_num(9.0), old_k[pages].nan_to_num(9.0))
        else:
            jet.jet_device_error()
    assert jet.jet_device_error() == 0


def test_binding_refuses(jet):
    b = Batch([1, 2], [5, 6], 4, 2, 64, 16)
    x = torch.randn((3, 8, 64), device="cuda").to(BF)
    g = torch.ones(64, device="cuda")
    go = lambda **kw: jet.jet_attn_rope_append(**{**dict(
        q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], q_gamma=g, k_gamma=g, inv_freq=freqs(64), cu_q=b.cu, kv_lens=b.kv_lens,
        page_table=b.table, k_pool=b.k_pool, v_pool=b.v_pool), **kw})
    go()
    with pytest.raises(TypeError):
        go(q_gamma=g.to(BF))
    with pytest.raises(jet.JetError):
        go(k_gamma=None)
    with pytest.raises(jet.JetError):
        go(inv_freq=freqs(64)[:5])                 # rot 10
    with pytest.raises(jet.JetError):
        go(inv_freq=torch.ones(40, device="cuda"))     # rot 80 > d
    with pytest.raises(jet.JetError):
        go(q_out=x[:, 1:5])                        # overlaps its inputs
    with pytest.raises(jet.JetError):
        go(v_pool=b.k_pool)
    with pytest.raises(jet.JetError):
        go(eps=-1.0)
    with pytest.raises(ValueError):
        go(v=x[:, 5:])
    with pytest.raises(ValueError):
        go(k=x[:, 4:8:2])
    with pytest.raises(TypeError):
        go(k_pool=b.k_pool.float(), v_pool=b.v_pool.float())


@pytest.mark.parametrize("dtype,pieces", [(BF, [70, 1, 1, 129, 1]), (BF, [1] * 20), (F32, [33, 1, 50])])
@pytest.mark.parametrize("window", [0, 40])
def test_a_prompt_in_pieces_equals_the_prompt_at_once(jet, dtype, pieces, window):
    """Append and attend piece by piece, in place over the projection's
    output; every piece against the formula over all appended positions."""
    T, Hq, Hk, d, page = sum(pieces), 12, 2, 128, 16
    b = Batch([T], [0], Hq, Hk, d, page, dtype, seed=21)
    b.k_pool.fill_(float("nan"))
    b.v_pool.fill_(float("nan"))
    x = torch.randn((T, Hq + 2 * Hk, d), device="cuda").to(dtype)
    f, at, outs = freqs(d), 0, []
    for n in pieces:
        cu = torch.tensor([0, n], device="cuda", dtype=torch.int32)
        kv = torch.tensor([at + n], device="cuda", dtype=torch.int32)
        y = x[at:at + n].clone()
        q = jet.jet_attn_rope_append(y[:, :Hq], y[:, Hq:Hq + Hk], y[:, Hq + Hk:], None, None, f, cu, kv, b.table,
                                     b.k_pool, b.v_pool, y[:, :Hq])
        outs.append(jet.jet_attn_paged(q, b.k_pool, b.v_pool, cu, kv, b.table, n, window=window))
        b.q[at:at + n] = q
        at += n
    for p in range(T):
        pg, r = int(b.host_table[0, p // page]), p % page
        b.K[0][p], b.V[0][p] = b.k_pool[pg, :, r], b.v_pool[pg, :, r]
    check_attention(torch.cat(outs), b, window)
    assert jet.jet_device_error() == 0
