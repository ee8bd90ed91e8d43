"""A launch that CUDA refuses is the error of that call alone: the next one
is judged by its own launches. The refusal here is a stream whose capture has
been invalidated (by a synchronisation inside it)."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


class Invalidated:
    """A stream in a capture that nothing can be added to."""

    def __enter__(self):
        self.cu, self.s = ctypes.CDLL("libcuda.so.1"), torch.cuda.Stream()
        self.raw = ctypes.c_void_p(self.s.cuda_stream)
        assert self.cu.cuStreamBeginCapture_v2(self.raw, 1) == 0       # checks of this thread only
        assert self.cu.cuStreamSynchronize(self.raw) != 0
        return self.s

    def __exit__(self, *exc):
        graph = ctypes.c_void_p()
        assert self.cu.cuStreamEndCapture(self.raw, ctypes.byref(graph)) != 0 and not graph.value
        return False


def test_the_next_call_succeeds(jet):
    pool = torch.arange(32, device="cuda", dtype=torch.float32).view(8, 4)
    x, w1, w2 = (torch.randn(s, device="cuda") for s in ((1, 8, 64), (64, 32), (32, 8)))
    table = torch.tensor([[6, 2]], device="cuda", dtype=torch.int32)
    lens = torch.tensor([20], device="cuda", dtype=torch.int32)
    calls = [lambda s: jet.jet_cache_copy([pool], [1], [5], stream=s),
             lambda s: jet.jet_kernel_gen(x, w1, w2, 2, stream=s),
             lambda s: jet.jet_cache_compact([pool], table, lens, 16, stream=s)]
    for call in calls:
        call(None)
    for after in calls:
        torch.cuda.synchronize()
        with Invalidated() as s:
            with pytest.raises(jet.JetError, match="CUDA"):
                calls[0](s)
        after(None)
    torch.cuda.synchronize()
    assert torch.equal(pool[5], pool[1]) and jet.jet_device_error() == 0
