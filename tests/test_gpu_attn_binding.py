"""The two ways through the Python binding of the attention and cache calls:
with outputs and workspace given (checked natively) and through the Python
checks; both make the same call and refuse the same arguments."""
import pytest
import torch

from attn_testlib import BF, F32, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_attention_lm_gen_b200 import build
    build.build()
    import linear_attention_lm_gen_b200 as m
    m.load_library()
    return m


class Case:
    def __init__(self, jet, dtype=BF, layout="head", new=(1, 5, 1), ctx=(30, 2, 100)):
        self.jet = jet
        self.b = b = Batch(list(new), list(ctx), 4, 2, 64, 16, dtype, seed=1, layout=layout)
        g = torch.Generator(device="cuda")
        g.manual_seed(2)
        self.x = torch.randn((b.N, 8, 64), generator=g, device="cuda").to(dtype)
        self.gamma = torch.ones(64, device="cuda")
        self.freq = torch.rand(32, generator=g, device="cuda")
        self.o = torch.empty((b.N, 4, 64), device="cuda", dtype=dtype)
        self.ws = torch.empty(jet.jet_attn_paged_workspace_size(len(new), b.N, 4, 2, 64, dtype), device="cuda",
                              dtype=torch.uint8)

    def append(self, **kw):
        x, b = self.x, self.b
        return self.jet.jet_attn_rope_append(**{**dict(
            q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], q_gamma=self.gamma, k_gamma=self.gamma, inv_freq=self.freq, cu_q=b.cu,
            kv_lens=b.kv_lens, page_table=b.table, k_pool=b.k_pool, v_pool=b.v_pool, q_out=self.o), **kw})

    def paged(self, **kw):
        b = self.b
        return self.jet.jet_attn_paged(**{**dict(q=b.q, k_pool=b.k_pool, v_pool=b.v_pool, cu_q=b.cu, kv_lens=b.kv_lens,
                                                 page_table=b.table, max_new=5, o=self.o, workspace=self.ws), **kw})


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["head", "token", "side", "wide"])
def test_both_ways_make_the_same_call(jet, dtype, layout):
    c = Case(jet, dtype, layout)
    here = torch.cuda.current_stream()
    first = c.paged(window=20, scale=0.2).clone()
    c.o.zero_()
    assert torch.equal(c.paged(window=20, scale=0.2, stream=here), first)
    assert torch.equal(c.paged(window=20, scale=0.2, o=None, workspace=None), first)
    assert torch.equal(c.paged(), c.paged(scale=64 ** -0.5))
    q1 = c.append(interleaved=True).clone()
    k1 = c.b.k_pool.clone()
    c.o.zero_()
    assert torch.equal(c.append(interleaved=True, stream=here), q1)
    assert torch.equal(c.append(interleaved=True, q_out=None), q1)
    assert torch.equal(c.b.k_pool.nan_to_num(9.0), k1.nan_to_num(9.0))
    assert torch.equal(c.append(inv_freq=None, q_gamma=None, k_gamma=None), c.x[:, :4])
    assert jet.jet_device_error() == 0


def test_one_token_and_one_head(jet):
    c = Case(jet, new=(1,), ctx=(40,))
    a = c.paged().clone()
    assert torch.equal(a, c.paged(workspace=None))
    q = torch.randn((1, 1, 64), device="cuda").to(BF)
    pool = c.b.k_pool[:, :1].contiguous()
    o = torch.empty_like(q)
    args = (q, pool, pool, c.b.cu, c.b.kv_lens, c.b.table, 1)
    jet.jet_attn_paged(*args, o, c.ws)
    assert torch.equal(o, jet.jet_attn_paged(*args))


def test_both_ways_refuse_the_same(jet):
    c = Case(jet)
    b = c.b
    for kw, err in [
            (dict(q=b.q.half()), TypeError), (dict(q=b.q.cpu()), TypeError), (dict(q=None), TypeError),
            (dict(k_pool=b.k_pool.float()), TypeError), (dict(kv_lens=b.kv_lens.long()), TypeError),
            (dict(kv_lens=b.kv_lens[:1]), ValueError), (dict(o=c.o[1:]), ValueError), (dict(o=c.o.float()), TypeError),
            (dict(page_table=b.table.t()), ValueError), (dict(page_table=b.table[0]), ValueError),
            (dict(v_pool=b.v_pool[1:]), ValueError), (dict(cu_q=b.cu.cpu()), TypeError),
            (dict(workspace=c.ws.cpu()), TypeError), (dict(workspace=c.ws[:100]), jet.JetError),
            (dict(o=b.q), jet.JetError), (dict(window=-1), jet.JetError), (dict(scale=-1.0), jet.JetError),
            (dict(max_new=-1), jet.JetError)]:
        for stream in (None, torch.cuda.current_stream()):
            with pytest.raises(err):
                c.paged(stream=stream, **kw)
    x = c.x
    for kw, err in [
            (dict(q=x[:, :4].cpu()), TypeError), (dict(v=x[:, 5:]), ValueError), (dict(k=x[:, 4:8:2]), ValueError),
            (dict(q_gamma=c.gamma.to(BF)), TypeError), (dict(q_gamma=c.gamma[:32]), ValueError),
            (dict(q_gamma=None), jet.JetError), (dict(inv_freq=c.freq[:3]), jet.JetError),
            (dict(inv_freq=c.freq.double()), TypeError), (dict(q_out=x[:, 1:5]), jet.JetError),
            (dict(q_out=c.o.float()), TypeError), (dict(eps=-1.0), jet.JetError), (dict(v_pool=b.k_pool), jet.JetError)]:
        for stream in (None, torch.cuda.current_stream()):
            with pytest.raises(err):
                c.append(stream=stream, **kw)
    table, lens = b.table, b.kv_lens
    ws = torch.empty(jet.jet_cache_compact_workspace_size(b.n_pages), device="cuda", dtype=torch.uint8)
    out, live = torch.empty_like(table), torch.empty(1, device="cuda", dtype=torch.int32)
    pools = [b.k_pool, b.v_pool]
    for stream in (None, torch.cuda.current_stream()):
        go = lambda *a: jet.jet_cache_compact(*a, stream=stream)
        with pytest.raises(jet.JetError):
            go(pools, table, lens, 17, out, live, ws)
        with pytest.raises(jet.JetError):
            go(pools, table, lens, 16, out, live, ws[:16])
        with pytest.raises(TypeError):
            go(pools, table, lens, 16, out.long(), live, ws)
        with pytest.raises(ValueError):
            go(pools, table, lens, 16, out[1:], live, ws)
        with pytest.raises(ValueError):
            go([b.k_pool, b.v_pool[1:]], table, lens, 16, out, live, ws)
        with pytest.raises(jet.JetError):
            jet.jet_cache_copy(pools, [0], [b.n_pages], stream=stream)
        with pytest.raises(ValueError):
            jet.jet_cache_copy(pools, [0, 1], [2], stream=stream)
        with pytest.raises((TypeError, OverflowError)):
            jet.jet_cache_copy(pools, [0], [1 << 40], stream=stream)
        with pytest.raises(TypeError):
            jet.jet_cache_copy(pools, [0.5], [1], stream=stream)
    torch.cuda.synchronize()
    assert jet.jet_device_error() == 0
