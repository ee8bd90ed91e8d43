"""jet_attn_paged against the formula in 64 bits: ragged batches, head
groups, head sizes, page sizes, windows, pool layouts, padding, empty
sequences, unused memory full of NaN, streams and captured graphs."""
import pytest
import torch

from attn_testlib import BF, F32, Batch, attention64, attention_bound, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


WIDE = False


@pytest.fixture(autouse=True, params=["narrow", "wide"])
def _tables(request):
    """Every test with the tables as narrow as they can be and with wide ones: the tables bound the lengths that the
    host knows of, and batches that can only be small take the decode kernel whatever their rows."""
    global WIDE
    WIDE = request.param == "wide"


def table_of(b):
    if not WIDE:
        return b.table
    cols = int(1.6e6 / (b.N * b.Hq)) // b.page + b.table.shape[1]
    t = torch.full((b.table.shape[0], cols), -1, dtype=torch.int32, device=b.device)
    t[:, :b.table.shape[1]] = b.table
    return t


def call(jet, b, max_new=None, **kw):
    o = torch.full((b.N, b.Hq, b.d), 7.0, device=b.device, dtype=b.dtype)
    jet.jet_attn_paged(b.q, b.k_pool, b.v_pool, b.cu, b.kv_lens, table_of(b), max(b.new) if max_new is None else max_new,
                       o, **kw)
    return o


DECODE = dict(new=[1, 1, 1, 1, 1], ctx=[0, 1, 62, 63, 700])
CHUNK = dict(new=[1, 37, 128, 300, 5], ctx=[0, 0, 64, 129, 1000])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,d", [(12, 2, 128), (16, 2, 128), (1, 1, 64), (6, 3, 64), (5, 5, 96), (14, 2, 80),
                                     (8, 1, 16), (40, 5, 48), (64, 1, 112), (34, 2, 128)])
def test_head_layouts(jet, Hq, Hk, d, dtype):
    for i, shape in enumerate((DECODE, CHUNK)):
        b = Batch(Hq=Hq, Hk=Hk, d=d, page=64, dtype=dtype, seed=i, **shape)
        check_attention(call(jet, b), b)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["head", "token", "side", "wide"])
def test_pages_and_pool_layouts(jet, page, layout, dtype):
    for i, shape in enumerate((DECODE, CHUNK)):
        b = Batch(Hq=4, Hk=2, d=64, page=page, dtype=dtype, seed=10 + i, layout=layout, **shape)
        check_attention(call(jet, b), b)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("window", [1, 2, 17, 64, 129, 500, 100000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_windows(jet, window, dtype):
    for i, shape in enumerate((DECODE, CHUNK)):
        b = Batch(Hq=12, Hk=2, d=128, page=32, dtype=dtype, seed=20 + i, **shape)
        check_attention(call(jet, b, window=window), b, window)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 3, 10, 11, 21, 22, 42, 43, 127, 128, 129, 255, 257])
def test_chunk_lengths_around_the_row_tiles(jet, n):
    for ctx in (0, 1, 127, 128, 500):
        b = Batch([n], [ctx], Hq=12, Hk=2, d=128, page=64, seed=n)
        check_attention(call(jet, b), b)
        check_attention(call(jet, b, window=100), b, 100)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("L", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023, 1025, 5000])
def test_decode_lengths(jet, L):
    b = Batch([1, 1], [L - 1, 3], Hq=16, Hk=2, d=128, page=16, seed=L)
    check_attention(call(jet, b), b)
    check_attention(call(jet, b, window=77), b, 77)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_new", [0, 1, 5000])
def test_max_new_only_chooses_the_kernel(jet, max_new, dtype):
    for i, shape in enumerate((DECODE, CHUNK)):
        b = Batch(Hq=6, Hk=2, d=128, page=64, dtype=dtype, seed=30 + i, **shape)
        check_attention(call(jet, b, max_new=max_new), b)


@pytest.mark.parametrize("max_new", [1, 0])
def test_a_long_cache_is_split_and_joined(jet, max_new):
    b = Batch([1, 3], [70001, 33], Hq=12, Hk=2, d=128, page=64, seed=5)
    check_attention(call(jet, b, max_new=max_new), b)
    b = Batch([2], [40000], Hq=2, Hk=1, d=64, page=32, seed=6)
    check_attention(call(jet, b, max_new=max_new), b)
    check_attention(call(jet, b, max_new=max_new, window=30000), b, 30000)


def test_long_chunk_over_a_long_cache(jet):
    b = Batch([700], [9000], Hq=12, Hk=2, d=128, page=64, seed=7)
    check_attention(call(jet, b), b)
    b = Batch([1500, 1, 1], [0, 3000, 10], Hq=8, Hk=2, d=96, page=128, seed=8)
    check_attention(call(jet, b), b)
    check_attention(call(jet, b, window=640), b, 640)


def test_many_sequences(jet):
    new = [1] * 300
    ctx = [(i * 37) % 500 for i in range(300)]
    b = Batch(new, ctx, Hq=4, Hk=2, d=64, page=16, seed=9)
    check_attention(call(jet, b), b)
    new = [(i * 7) % 5 for i in range(300)]
    b = Batch(new, ctx, Hq=4, Hk=2, d=64, page=16, seed=10)
    check_attention(call(jet, b), b)
    check_attention(call(jet, b, max_new=1), b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty_sequences_and_padding_rows(jet, dtype):
    b = Batch([0, 3, 0, 1, 0], [0, 5, 40, 0, 7], Hq=6, Hk=2, d=64, page=16, dtype=dtype, seed=11, pad=9)
    for max_new in (1, 3, 500):
        o = call(jet, b, max_new=max_new)
        check_attention(o, b)
        assert (o[b.cu_host[-1]:] == 7.0).all(), "rows behind the last sequence were written"
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_new", [1, 500])
def test_tokens_that_see_nothing_get_zeros(jet, dtype, max_new):
    b = Batch([4, 6], [30, 0], Hq=4, Hk=2, d=64, page=16, dtype=dtype, seed=12)
    # the second sequence holds two positions fewer than it has new tokens; the first holds none at all
    b.kv_lens[1] = 4
    b.kv[1] = 4
    b.K[1], b.V[1] = b.K[1][:4], b.V[1][:4]
    o = call(jet, b, max_new=max_new)
    assert (o[4:6] == 0).all()
    check_attention(o[:4], Batch_head(b, 4))
    want = attention64(tail(b))[0]
    assert torch.allclose(o[6:10].double(), want, atol=0.05)
    b.kv_lens[0] = 0
    o = call(jet, b, max_new=max_new)
    assert (o[:6] == 0).all()
    assert jet.jet_device_error() == 0


class _View:
    pass


def Batch_head(b, n):
    v = _View()
    v.__dict__.update(b.__dict__)
    v.new, v.kv, v.K, v.V, v.cu_host = [n], b.kv[:1], b.K[:1], b.V[:1], [0, n]
    return v


def tail(b):
    v = _View()
    v.__dict__.update(b.__dict__)
    v.new, v.kv, v.K, v.V, v.cu_host = [4], [4], b.K[1:], b.V[1:], [0, 4]
    v.q = b.q[6:10]
    return v


@pytest.mark.parametrize("max_new", [1, 500])
def test_pages_before_every_window_are_not_read(jet, max_new):
    b = Batch([3, 1], [400, 900], Hq=12, Hk=2, d=128, page=16, seed=13)
    W = 100
    for s, (n, L) in enumerate(zip(b.new, b.kv)):
        gone = (L - n - W + 1) // b.page
        for i in range(gone):
            pg = int(b.host_table[s, i])
            b.k_pool[pg], b.v_pool[pg] = float("nan"), float("nan")
            b.table[s, i] = -1
        # positions of the last page given up in part: outside every window, so they may hold anything
        for p in range(gone * b.page, L - n - W + 1):
            pg = int(b.host_table[s, p // b.page])
            b.k_pool[pg, :, p % b.page] = float("nan")
            b.v_pool[pg, :, p % b.page] = float("inf")
            b.K[s][p], b.V[s][p] = 0.0, 0.0
    check_attention(call(jet, b, max_new=max_new, window=W), b, W)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_new", [1, 500])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_a_token_masks_do_not_reach_it(jet, dtype, max_new, value):
    """A later token's value and an older one outside the window: they reach
    the tokens that see them and no other."""
    b = Batch([40, 3], [200, 20], Hq=4, Hk=2, d=64, page=16, dtype=dtype, seed=14)
    W = 64
    hot = [(0, 170), (0, 225), (1, 22)]           # (sequence, position)
    for s, p in hot:
        pg = int(b.host_table[s, p // b.page])
        b.v_pool[pg, 1, p % b.page, 5] = value
        b.V[s][p, 1, 5] = value
    o = call(jet, b, max_new=max_new, window=W).double()
    want, a = attention64(b, W)
    hit = torch.zeros_like(o, dtype=torch.bool)
    for s, p in hot:
        n, L, r = b.new[s], b.kv[s], b.cu_host[s]
        for i in range(n):
            at = L - n + i
            if p <= at and p > at - W:
                hit[r + i, 2:4, 5] = True
    assert not torch.isfinite(o[hit]).any(), "a value that is seen has to show"
    assert torch.isfinite(o[~hit]).all(), "a masked value reached a token"
    err = (o - want).abs() - attention_bound(want, a, dtype)
    assert err[~hit].amax().item() <= 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_new", [1, 500])
def test_large_logits_and_scales(jet, dtype, max_new):
    b = Batch([33, 1], [100, 300], Hq=4, Hk=2, d=64, page=32, dtype=dtype, seed=15)
    check_attention(call(jet, b, max_new=max_new, scale=1e-6), b, 0, 1e-6)
    # one key dominates by hundreds: the softmax is a selection
    for s in range(2):
        b.K[s].mul_(0)
        b.K[s][:, :, 0] = -40.0
        b.K[s][7, :, 0] = 40.0
        b.store(s, 0, b.K[s], b.V[s])
    b.q.zero_()
    b.q[:, :, 0] = 30.0
    o = call(jet, b, max_new=max_new)
    # scores of +150 and -150: the others' weights are exp(-300), zero in 32 bits
    for s in range(2):
        r = slice(b.cu_host[s], b.cu_host[s + 1])
        assert torch.equal(o[r], b.V[s][7].repeat_interleave(2, 0).expand(b.new[s], -1, -1))


def test_queries_with_a_token_stride_and_an_own_stream(jet):
    b = Batch(Hq=12, Hk=2, d=128, page=64, seed=16, **CHUNK)
    ref = call(jet, b)
    wide = torch.randn((b.N, 16, 128), device="cuda").to(BF)
    wide[:, :12] = b.q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t = table_of(b)
    side.wait_stream(torch.cuda.current_stream())
    o = jet.jet_attn_paged(wide[:, :12], b.k_pool, b.v_pool, b.cu, b.kv_lens, t, 300, stream=side)
    side.synchronize()
    assert torch.equal(o, ref)


@pytest.mark.parametrize("max_new", [1, 500])
def test_calls_repeat_bit_for_bit_and_with_a_dirty_workspace(jet, max_new):
    b = Batch([1, 2, 1], [9000, 40, 0], Hq=12, Hk=2, d=128, page=64, seed=17)
    n = jet.jet_attn_paged_workspace_size(3, b.N, 12, 2, 128)
    outs = []
    for fill in (0, 255, 77):
        ws = torch.full((max(n, 16),), fill, device="cuda", dtype=torch.uint8)
        outs.append(call(jet, b, max_new=max_new, workspace=ws))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("max_new,new", [(1, [1, 1, 1]), (200, [60, 1, 140])])
def test_a_captured_graph_follows_new_lengths(jet, max_new, new):
    b = Batch(new, [500, 300, 20], Hq=12, Hk=2, d=128, page=64, seed=18)
    ws = torch.empty(max(16, jet.jet_attn_paged_workspace_size(3, b.N, 12, 2, 128)), device="cuda", dtype=torch.uint8)
    o = torch.empty((b.N, 12, 128), device="cuda", dtype=BF)
    t = table_of(b)
    run = lambda: jet.jet_attn_paged(b.q, b.k_pool, b.v_pool, b.cu, b.kv_lens, t, max_new, o, ws)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    g.replay()
    check_attention(o, b)
    # fewer positions in the same tables
    for s, L in enumerate((b.kv[0] - 100, new[1], b.kv[2])):
        b.kv[s] = L
        b.K[s], b.V[s] = b.K[s][:L], b.V[s][:L]
    b.kv_lens.copy_(torch.tensor(b.kv, dtype=torch.int32))
    g.replay()
    check_attention(o, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("max_new", [1, 500])
def test_bad_device_data_is_flagged_and_reads_nothing(jet, dtype, max_new):
    assert jet.jet_device_error() == 0
    for what in ("page", "length", "offsets"):
        b = Batch([2, 3, 2], [50, 60, 70], Hq=4, Hk=2, d=64, page=16, dtype=dtype, seed=19)
        if what == "page":
            b.table[1, 1] = b.n_pages
            b.table[1, 2] = -5
        elif what == "length":
            b.kv_lens[1] = 2 ** 30 + 1              # no table holds that many
        else:
            b.cu[2] = b.N + 5
        o = call(jet, b, max_new=max_new)
        assert jet.jet_device_error() == 6
        want, a = attention64(b)
        good = slice(0, 2)
        assert ((o[good].double() - want[good]).abs() <= attention_bound(want, a, dtype)[good]).all()
        if what == "length":
            assert (o[2:5] == 7.0).all()
    assert jet.jet_device_error() == 0


def test_offsets_beyond_32_bits(jet):
    """A cache whose last pages lie behind 2^32 elements."""
    P, page, Hk, d = 2200000, 16, 1, 128
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    pool = torch.empty((P, 2, Hk, page, d), device="cuda", dtype=BF)
    assert pool.numel() > 2 ** 32
    b = Batch([2, 1], [100, 40], Hq=6, Hk=Hk, d=d, page=page, seed=20)
    shift = P - b.n_pages
    k, v = pool[:, 0], pool[:, 1]
    k[shift:], v[shift:] = b.k_pool, b.v_pool
    b.k_pool, b.v_pool = k, v
    b.table = torch.where(b.table >= 0, b.table + shift, b.table)
    for max_new in (1, 500):
        check_attention(call(jet, b, max_new=max_new), b)
    assert jet.jet_device_error() == 0


def test_binding_refuses(jet):
    b = Batch([1, 2], [5, 6], Hq=4, Hk=2, d=64, page=16)
    go = lambda **kw: jet.jet_attn_paged(**{**dict(q=b.q, k_pool=b.k_pool, v_pool=b.v_pool, cu_q=b.cu,
                                                   kv_lens=b.kv_lens, page_table=b.table), **kw})
    with pytest.raises(TypeError):
        go(q=b.q.half())
    with pytest.raises(TypeError):
        go(q=b.q.cpu())
    with pytest.raises(TypeError):
        go(k_pool=b.k_pool.float())
    with pytest.raises(TypeError):
        go(kv_lens=b.kv_lens.long())
    with pytest.raises(ValueError):
        go(kv_lens=b.kv_lens[:1])
    with pytest.raises(ValueError):
        go(q=b.q.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError):
        go(v_pool=b.v_pool.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        go(page_table=b.table.t())
    with pytest.raises(jet.JetError):
        go(o=b.q)
    with pytest.raises(jet.JetError):
        go(workspace=torch.empty(8, device="cuda", dtype=torch.uint8)[8:])
    with pytest.raises(jet.JetError):
        go(scale=0.0)
    with pytest.raises(jet.JetError):
        go(window=-1)
