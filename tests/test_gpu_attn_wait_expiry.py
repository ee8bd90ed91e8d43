"""A wait of the tensor-core attention kernel that runs out, on the GPU,
without faulting it: a test build with a 2 ms limit leaves the first scores of
a tile out, so that the threads that wait for them give up. The call returns,
the error word says so, every role winds down, and the next call is correct."""
import ctypes
import time

import pytest
import torch

from attn_testlib import Batch, check_attention

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 5


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    import linear_attention_lm_gen_b200 as jet
    build.build()
    jet.load_library()
    path = str(tmp_path_factory.mktemp("waittest") / "libjet_waittest.so")
    build.build(force=True, extra=["-DJET_TEST_WAIT_EXPIRY", "-DJET_WAIT_LIMIT_NS=2000000ull"], out=path)
    L = jet.declare(ctypes.CDLL(path))
    L.jet_test_skip_scores.argtypes = [ctypes.c_int]
    L.jet_test_skip_scores.restype = ctypes.c_int
    return jet, L


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_correct(libs, monkeypatch):
    jet, L = libs
    b = Batch([300, 1, 60], [200, 700, 0], Hq=12, Hk=2, d=128, page=64, seed=3)
    run = lambda: jet.jet_attn_paged(b.q, b.k_pool, b.v_pool, b.cu, b.kv_lens, b.table, 300)
    with monkeypatch.context() as m:
        m.setattr(jet, "_lib", L)
        check_attention(run(), b)
        assert jet.jet_device_error() == OK
        assert L.jet_test_skip_scores(1) == 0
        t = time.time()
        run()
        torch.cuda.synchronize()
        assert time.time() - t < 2.0
        assert jet.jet_device_error() == TIMEOUT
        assert L.jet_test_skip_scores(0) == 0
        check_attention(run(), b)
        assert jet.jet_device_error() == OK
    check_attention(run(), b)
    assert jet.jet_device_error() == OK
