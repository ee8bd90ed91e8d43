"""Sizes at which the work of jet_attn_paged could pass 64 bits are refused.
Without a GPU: every call is rejected before any launch, the accepted sizes
for want of a workspace."""
import pytest

from test_abi_attn_cpu import A, STEP, UNSUPPORTED, WORKSPACE, lib, paged  # noqa: F401

FAR = 1 << 44          # outputs far behind the longest queries


def status(lib, **kw):  # noqa: F811
    kw = {**dict(Hq=16, Hk=16, d=16, qs=256, ps=16 * 256 * 16, hs=256 * 16, rs=16, page=256, q=A, kp=A + FAR,
                 vp=A + 2 * FAR, o=A + 3 * FAR, ws=None, wsb=0), **kw}
    return paged(lib, **kw)


@pytest.mark.parametrize("nseq,N,positions,expect", [
    (1, 1 << 24, 1 << 30, WORKSPACE),                 # 2^58: the longest call of one sequence
    (256, 1 << 17, 1 << 24, WORKSPACE), (65535, 65535, 1 << 25, WORKSPACE), (1024, 1 << 18, 1 << 28, WORKSPACE),
    (65535, 1 << 17, 1 << 20, WORKSPACE),
    (65535, 1 << 24, 1 << 19, UNSUPPORTED), (65535, 1 << 13, 1 << 30, UNSUPPORTED), (1024, 1 << 24, 1 << 30, UNSUPPORTED),
])
def test_work_is_counted_in_64_bits(lib, nseq, N, positions, expect):  # noqa: F811
    assert status(lib, nseq=nseq, N=N, mp=positions // 256) == expect


def cost(n, L, heads, window, rows_tokens, c0):
    """The work of one sequence on the axis, as csrc/k_attn_sched.cuh adds it up, in exact integers."""
    older, tiles = max(0, L - n), -(-n // rows_tokens)
    first = tiles
    if window:
        first = min(tiles, -(-max(0, window - 1 - older) // rows_tokens))
    return heads * (first * (c0 + older) + rows_tokens * (first * (first + 1) // 2)
                    + (tiles - first) * (c0 + rows_tokens + window - 1))


def test_the_limit_covers_the_cost_of_every_batch():
    for n in (1, 5, 1000, 1 << 20, 1 << 24):
        for L in (0, 1, 1000, 1 << 30):
            for window in (0, 1, 500, 1 << 30, (1 << 31) - 1):
                for tokens in (1, 2, 16, 42, 256):
                    assert cost(n, L, 16, window, tokens, 384) <= n * 16 * (max(L, n) + 1024)
    # the chunks of a grid of up to 592 reach the end, whatever the rounding in float64
    for total in [1, 100, 147, 148, 2 ** 40 + 1, 2 ** 50 - 1, 2 ** 50 + 77, 2 ** 53 + 1, 2 ** 57 - 1, 2 ** 61 + 12345, 2 ** 62]:
        for grid in (1, 132, 147, 148, 296, 444, 592):
            chunk = int(float(total) / grid * (1.0 + 2.0 ** -50)) + 1
            assert chunk * grid > total and chunk - 1 <= total / grid * (1 + 1e-15) + 1
            if total <= 2 ** 40:
                assert chunk == total // grid + 1
