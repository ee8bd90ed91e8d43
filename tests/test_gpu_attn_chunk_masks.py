"""Windows, given-up pages and non-finite values in the tcgen05 attention
kernel (csrc/k_attn_chunk.cuh). The host picks the kernel by a bound on rows
times positions, so small windowed batches would take the decode kernel: the
tables here are wide enough, and max_new large enough, that they do not, and
every test asserts which kernel was launched."""
import pytest
import torch

from attn_testlib import BF, Batch, attention64, attention_bound, check_attention, launched

pytestmark = pytest.mark.gpu

ANY = 1 << 20          # new tokens that the host may assume: the window bounds nothing then


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


def call(jet, b, window, kernel="attn_chunk_kernel"):
    """The attention with a table so wide that rows times positions pass 1.6 million, by the kernel of this name."""
    cols = int(1.6e6 / (b.N * b.Hq)) // b.page + b.table.shape[1]
    t = torch.full((b.table.shape[0], cols), -1, dtype=torch.int32, device=b.device)
    t[:, :b.table.shape[1]] = b.table
    o = torch.full((b.N, b.Hq, b.d), 7.0, device=b.device, dtype=b.dtype)
    ws = torch.empty(jet.jet_attn_paged_workspace_size(len(b.new), b.N, b.Hq, b.Hk, b.d, b.dtype), device=b.device,
                     dtype=torch.uint8)
    run = lambda: jet.jet_attn_paged(b.q, b.k_pool, b.v_pool, b.cu, b.kv_lens, t, ANY, o, ws, window=window)
    names = launched(run)
    assert any(kernel in n for n in names), names
    o.fill_(7.0)
    run()
    return o


def put(b, s, p, h, col, value, kv="v"):
    pg = int(b.host_table[s, p // b.page])
    (b.v_pool if kv == "v" else b.k_pool)[pg, h, p % b.page, col] = value
    (b.V if kv == "v" else b.K)[s][p, h, col] = value


def check_hits(b, o, hot, W):
    """Elements that see a non-finite value are not finite, all others are within the bound."""
    o = o[:b.cu_host[-1]].double()
    want, a = attention64(b, W)
    hit = torch.zeros_like(o, dtype=torch.bool)
    G = b.Hq // b.Hk
    for s, p, h, col in hot:
        n, L, r = b.new[s], b.kv[s], b.cu_host[s]
        for i in range(n):
            at = L - n + i
            if p <= at and (not W or p > at - W):
                hit[r + i, h * G:(h + 1) * G, col] = True
    assert hit.any() and not torch.isfinite(o[hit]).any(), "a value that is seen has to show"
    assert torch.isfinite(o[~hit]).all(), "a masked value reached a token"
    err = (o - want).abs() - attention_bound(want, a, b.dtype)
    assert err[~hit].amax().item() <= 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("Hq,Hk,d,page", [(4, 2, 64, 16), (12, 2, 128, 64), (5, 1, 96, 256), (64, 1, 16, 32)])
@pytest.mark.parametrize("W", [0, 1, 64, 200])
def test_values_that_a_token_masks_do_not_reach_it(jet, W, Hq, Hk, d, page, value):
    b = Batch([40, 3, 300], [200, 20, 150], Hq, Hk, d, page, seed=14)
    # new tokens' own values, older ones at both ends of windows, several in one row of pages and in one column
    hot = [(0, 170, Hk - 1, 5), (0, 225, Hk - 1, 5), (0, 239, 0, d - 1), (1, 22, 0, 0), (2, 149, 0, 3), (2, 150, 0, 3),
           (2, 300, Hk - 1, d // 2), (2, 449, 0, 1)]
    for s, p, h, col in hot:
        put(b, s, p, h, col, value)
    check_hits(b, call(jet, b, W), hot, W)
    assert jet.jet_device_error() == 0


def test_infinities_of_both_signs_and_a_value_among_many_steps(jet):
    b = Batch([257], [2000], 12, 2, 128, 64, seed=15)
    hot = [(0, 2100, 1, 7), (0, 2101, 1, 7), (0, 1900, 1, 9), (0, 30, 0, 2)]
    for (s, p, h, col), v in zip(hot, (float("inf"), float("-inf"), float("nan"), float("inf"))):
        put(b, s, p, h, col, v)
    for W in (0, 400):
        seen = [x for x in hot if not W or x[1] > 2000 - W]
        check_hits(b, call(jet, b, W), seen, W)


@pytest.mark.parametrize("W", [1, 50, 100, 500])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_pages_before_every_window_are_not_read(jet, page, W):
    b = Batch([3, 1, 200], [400, 900, 700], 12, 2, 128, page, seed=13)
    for s, (n, L) in enumerate(zip(b.new, b.kv)):
        first = max(0, L - n - W + 1)
        gone = first // page
        for i in range(gone):
            pg = int(b.host_table[s, i])
            b.k_pool[pg], b.v_pool[pg] = float("nan"), float("nan")
            b.table[s, i] = -1
        for p in range(gone * page, first):      # the page that is given up in part
            for kv, v in (("k", float("nan")), ("v", float("inf"))):
                for h in range(b.Hk):
                    put(b, s, p, h, slice(None), v, kv)
            b.K[s][p], b.V[s][p] = 0.0, 0.0
    check_attention(call(jet, b, W), b, W)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 10, 11, 21, 22, 42, 43, 127, 128, 129, 257])
@pytest.mark.parametrize("W", [1, 100, 129])
def test_chunk_lengths_around_the_row_tiles(jet, n, W):
    for ctx in (0, 1, 127, 128, 500):
        b = Batch([n], [ctx], Hq=12, Hk=2, d=128, page=64, seed=n)
        check_attention(call(jet, b, W), b, W)
    assert jet.jet_device_error() == 0


@pytest.mark.parametrize("W", [1, 17, 64, 129, 500, 100000])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_over_a_ragged_batch(jet, W, d):
    b = Batch([1, 37, 0, 128, 300, 5, 1], [0, 0, 9, 64, 129, 1000, 3000], Hq=12, Hk=2, d=d, page=32, seed=21, pad=5)
    o = call(jet, b, W)
    check_attention(o, b, W)
    assert (o[b.cu_host[-1]:] == 7.0).all(), "rows behind the last sequence were written"
    assert jet.jet_device_error() == 0


def test_bad_pages_read_as_zeros(jet):
    b = Batch([60, 300], [50, 200], Hq=12, Hk=2, d=128, page=64, seed=19)
    b.table[1, 2], b.table[0, 0] = b.n_pages, -5
    b.K[1][128:192], b.V[1][128:192] = 0.0, 0.0
    b.K[0][:64], b.V[0][:64] = 0.0, 0.0
    for W in (0, 300):
        check_attention(call(jet, b, W), b, W)
        assert jet.jet_device_error() == 6


def test_the_decode_kernel_is_seen_as_such(jet):
    """The check of the kernel's name tells the two apart."""
    b = Batch([1, 1], [30, 500], Hq=12, Hk=2, d=128, page=64, seed=22)
    run = lambda: jet.jet_attn_paged(b.q, b.k_pool, b.v_pool, b.cu, b.kv_lens, b.table, 1)
    run()
    names = launched(run)
    assert any("attn_decode_kernel" in n for n in names) and not any("attn_chunk_kernel" in n for n in names), names
