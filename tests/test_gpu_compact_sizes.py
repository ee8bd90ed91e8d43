"""jet_cache_compact at the sizes where its plan's bitmap passes the shared
memory that a kernel has without asking, and at the largest cache."""
import numpy as np
import pytest
import torch

from test_gpu_cache_ops import expect_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


# in increasing order: a larger call before a smaller one would have asked for more
@pytest.mark.parametrize("P", [262144, 262145, 385024, 385056, 392192, 392800, 393216, 393217, 600001, 1 << 20])
def test_page_numbers_up_to_the_limit(jet, P):
    r = np.random.default_rng(P)
    page, seqs, width = 16, 40, 50
    kv = [int(x) for x in r.integers(1, width * page, size=seqs)]
    ids = r.choice(P, size=seqs * width, replace=False)
    ids[:3] = P - 1, P - 2, 0
    table = np.full((seqs, width), -1, dtype=np.int32)
    for s in range(seqs):
        n = -(-kv[s] // page)
        table[s, :n] = ids[s * width:s * width + n]
    table[7, 0] = table[0, 0]                  # a page that two sequences share
    want, n, to = expect_np(table, kv, page, P)
    pool = torch.arange(P, device="cuda", dtype=torch.int32).view(P, 1).expand(P, 4).contiguous()
    out, live = jet.jet_cache_compact([pool], torch.from_numpy(table).cuda(),
                                      torch.tensor(kv, dtype=torch.int32, device="cuda"), page)
    assert int(live) == n
    assert np.array_equal(out.cpu().numpy(), want)
    a, b = torch.tensor(list(to)), torch.tensor(list(to.values()))
    assert torch.equal(pool[b.cuda()].cpu(), a.int().view(-1, 1).expand(-1, 4))
    assert jet.jet_device_error() == 0
