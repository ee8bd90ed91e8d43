"""Overlaps that the append refuses: queries turned in place while keys or
values lie among them, and pools whose rows overlap. Without a GPU: every call
is rejected before any launch. The layouts that only look like overlaps are in
test_gpu_attn_append_layouts.py."""
import pytest

from test_abi_attn_cpu import A, INVALID, STEP, append, lib  # noqa: F401

BF = 2          # bytes of an element
# the call's rows: 5 tokens of 4 heads of 64 queries, 2 heads of keys and values; in place, so q_out is q
PLACE = dict(qo=A, qs=512, qos=512)
FUSED = dict(PLACE, k=A + 256 * BF, ks=512, v=A + 384 * BF, vs=512)


@pytest.mark.parametrize("kw", [
    dict(qo=A, qs=256, qos=256, k=A, ks=256),                     # the keys are among the queries
    dict(qo=A, qs=256, qos=256, v=A + 128, vs=256),
    dict(qo=A, qs=256, qos=256, v=A + 128, vs=512),               # with another stride, across them
    dict(PLACE, k=A + 192 * BF, ks=512),                          # the last head of a row
    dict(PLACE, k=A + 448 * BF, ks=512),                          # behind a row, into the next
    dict(PLACE, k=A - 64 * BF, ks=512),                           # before a row, into it
    dict(FUSED, v=A + 248 * BF), dict(FUSED, k=A + 248 * BF),     # slices that start too early
    dict(vp=A + 4 * STEP + 16), dict(vp=A + 4 * STEP - 64), dict(vp=A + 4 * STEP + 56 * BF),     # V within rows of K
])
def test_real_overlaps(lib, kw):  # noqa: F811
    assert append(lib, **kw) == INVALID
