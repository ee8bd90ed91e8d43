"""Shared by the tests of the softmax-attention and cache operators: ragged
paged batches with poisoned unused memory, and the formulas in 64 bits."""
from __future__ import annotations

import ctypes
import random

import torch

BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}      # half a rounding step, relative to the value


class Batch:
    """New tokens and cached context of a ragged batch, with its page tables.
    Pool rows that belong to no position hold NaN; pages come in random order."""

    def __init__(self, new, ctx, Hq, Hk, d, page, dtype=BF, seed=0, layout="head", spare=3, pad=0, device="cuda",
                 width=None):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.g, self.device, self.dtype = g, device, dtype
        self.new, self.kv = list(new), [a + b for a, b in zip(new, ctx)]
        self.Hq, self.Hk, self.d, self.page = Hq, Hk, d, page
        need = [-(-x // page) for x in self.kv]
        self.n_pages = sum(need) + spare
        order = list(range(self.n_pages))
        random.Random(seed).shuffle(order)
        width = width or max(1, max(need))
        table = torch.full((len(new), width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            for i in range(n):
                table[s, i] = order.pop()
        self.host_table = table
        self.table = table.to(device)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu_host = cu
        self.N = cu[-1] + pad
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32, device=device)
        self.k_pool, self.v_pool = self.pools(layout)
        self.K = [self.randn((L, Hk, d)) for L in self.kv]
        self.V = [self.randn((L, Hk, d)) for L in self.kv]
        for s in range(len(new)):
            self.store(s, 0, self.K[s], self.V[s])
        self.q = self.randn((self.N, Hq, d)) if self.N else torch.empty((0, Hq, d), device=device, dtype=dtype)
        if pad:
            self.q[cu[-1]:] = float("nan")

    def randn(self, shape, std=1.0):
        return (torch.randn(shape, generator=self.g, device=self.device) * std).to(self.dtype)

    def pools(self, layout):
        P, H, p, d = self.n_pages, self.Hk, self.page, self.d
        nan = lambda *s: torch.full(s, float("nan"), device=self.device, dtype=self.dtype)
        if layout == "head":          # pages of head-major rows
            return nan(P, H, p, d), nan(P, H, p, d)
        if layout == "token":         # token-major pages
            return nan(P, p, H, d).transpose(1, 2), nan(P, p, H, d).transpose(1, 2)
        if layout == "side":          # K and V of a page side by side
            kv = nan(P, 2, H, p, d)
            return kv[:, 0], kv[:, 1]
        if layout == "wide":          # rows with a gap behind them
            return nan(P, H, p, d + 16)[..., :d], nan(P, H, p, d + 16)[..., :d]
        raise ValueError(layout)

    def store(self, s, p0, k, v):
        if k.shape[0]:
            p = torch.arange(p0, p0 + k.shape[0])
            pg, r = self.host_table[s, p // self.page].long().to(self.device), (p % self.page).to(self.device)
            self.k_pool[pg, :, r], self.v_pool[pg, :, r] = k, v


def attention64(b: Batch, window=0, scale=None):
    """(o, a): the attention of every new token in 64 bits, and the same with
    |v| in the place of v (what roundings of the weights scale with)."""
    scale = b.d ** -0.5 if scale is None else scale
    G = b.Hq // b.Hk
    o = torch.zeros((b.cu_host[-1], b.Hq, b.d), dtype=torch.float64, device=b.device)
    a = torch.zeros_like(o)
    for s, (n, L) in enumerate(zip(b.new, b.kv)):
        if n == 0 or L == 0:
            continue
        q = b.q[b.cu_host[s]:b.cu_host[s] + n].double()
        k, v = b.K[s].double(), b.V[s].double()
        p = torch.arange(L - n, L, device=b.device)[:, None]
        j = torch.arange(L, device=b.device)[None, :]
        seen = j <= p
        if window:
            seen &= j > p - window
        for h in range(b.Hq):
            x = (q[:, h] @ k[:, h // G].T) * scale
            w = torch.where(seen, torch.exp(x - torch.where(seen, x, -1e300).amax(1, keepdim=True).clamp(min=-1e200)),
                            torch.zeros_like(x))
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
            # a masked value has no part, whatever it holds
            clean = lambda t: t.nan_to_num(0.0, 0.0, 0.0)
            r = slice(b.cu_host[s], b.cu_host[s] + n)
            o[r, h] = w @ clean(v[:, h // G])
            a[r, h] = w @ clean(v[:, h // G]).abs()
    return o, a


def attention_bound(o, a, dtype):
    """What the kernels' roundings can add up to, per element: the weights
    rounded to the storage type (half a step of each: half a step of a), the
    result rounded once (half a step of |o|), and float32 arithmetic. The last
    moves a logit by at most d products' roundings, 128 * 2^-24 of
    sum |q k| scale, about 10 for unit-normal q and k: 8e-5, twice that in a
    weight; 2e-4 of a leaves room for the exponential's own error and the sums."""
    h = HALF_STEP[dtype]
    return 1.01 * h * (a + o.abs()) + 2e-4 * a + 1e-30


def check_attention(got, b, window=0, scale=None):
    o, a = attention64(b, window, scale)
    got = got[:b.cu_host[-1]].double()
    assert torch.isfinite(got).all(), "non-finite outputs"
    bad = ((got - o).abs() - attention_bound(o, a, b.dtype)).amax().item() if o.numel() else 0.0
    assert bad <= 0.0, f"error above its bound by {bad:.3e}; largest error {(got - o).abs().amax().item():.3e}"


class _KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 7), ("params", ctypes.c_void_p),
                ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launched(run):
    """Names (mangled) of the kernels that run() launches: captured into a graph, whose nodes are looked at; not replayed."""
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        run()
    cu = ctypes.CDLL("libcuda.so.1")
    P, graph = ctypes.c_void_p, ctypes.c_void_p(g.raw_cuda_graph())

    def ok(status):
        assert status == 0, f"driver call returned {status}"
    n = ctypes.c_size_t()
    ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
    nodes = (P * n.value)()
    ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
    names = []
    for node in nodes:
        kind = ctypes.c_int()
        ok(cu.cuGraphNodeGetType(P(node), ctypes.byref(kind)))
        if kind.value == 0:                    # a kernel
            p, name = _KernelNode(), ctypes.c_char_p()
            ok(cu.cuGraphKernelNodeGetParams_v2(P(node), ctypes.byref(p)))
            ok(cu.cuFuncGetName(ctypes.byref(name), P(p.func)) if p.func
               else cu.cuKernelGetName(ctypes.byref(name), P(p.kern)))
            names.append(name.value.decode())
    return names
