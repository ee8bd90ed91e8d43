"""The softmax-attention operators beside the JetBlock mixer, as a benchmark:
their cases, their inputs and their plain forms.

Operators (names of the calls in linear_attention_lm_gen_b200):
  attn     jet_attn_paged        attention of a chunk of new tokens per sequence (one token: decode)
                                 over a paged key/value cache, causal, optionally in a sliding window
  append   jet_attn_rope_append  RMSNorm of queries and keys per head, position rotation, and the
                                 append of keys and values to the paged cache, in one pass
  copy     jet_cache_copy        entries of cache pools copied onto others (forks of sequences: pages
                                 of a key/value cache, or the recurrent states of the mixer)
  compact  jet_cache_compact     live pages of a paged cache moved to its lowest entries

`own` chooses between the plain torch forms (float32 arithmetic, rounded once)
and the library's calls. A paged cache is a pair of pools [pages, Hk, page, d];
position p of sequence s is row p % page of page page_table[s][p // page], and
kv_lens[s] counts the positions of s with the new tokens included.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short conversation, one new token: latency alone (2B-shape attention heads: 12 over 2, d 128)
        dict(name="attn_decode_b1_517", op="attn", dtype="bf16", Hq=12, Hk=2, d=128, page=64, window=0,
             batch=1, new_lo=1, new_hi=1, ctx_lo=516, ctx_hi=516),
        # a serving batch in decode: 256 sequences of every age
        dict(name="attn_decode_b256_ragged", op="attn", dtype="bf16", Hq=12, Hk=2, d=128, page=64, window=0,
             batch=256, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=8191),
        # long-context decode, few sequences: the work has to be split along the cache
        # (4B-shape heads: 16 over 2; the 262144-token context of the long prefill workload)
        dict(name="attn_decode_b2_262144", op="attn", dtype="bf16", Hq=16, Hk=2, d=128, page=64, window=0,
             batch=2, new_lo=1, new_hi=1, ctx_lo=262143, ctx_hi=262143),
        # chunked prefill: a 4096-token piece of a long prompt over what is already cached
        dict(name="attn_chunk_4096_over_28672", op="attn", dtype="bf16", Hq=12, Hk=2, d=128, page=64, window=0,
             batch=1, new_lo=4096, new_hi=4096, ctx_lo=28672, ctx_hi=28672),
        # a sliding-window layer over a mixed batch: prompt pieces and single tokens together
        dict(name="attn_window_mixed_b24", op="attn", dtype="bf16", Hq=16, Hk=2, d=128, page=32, window=2048,
             batch=24, new_lo=1, new_hi=1500, ctx_lo=0, ctx_hi=9000),
        # float32 path, small heads, odd lengths
        dict(name="attn_f32_b3", op="attn", dtype="f32", Hq=6, Hk=3, d=64, page=16, window=0,
             batch=3, new_lo=100, new_hi=333, ctx_lo=0, ctx_hi=700),
        # the new tokens of a decode batch enter the cache
        dict(name="append_decode_b256", op="append", dtype="bf16", Hq=12, Hk=2, d=128, rot=128, page=64,
             norm=True, interleaved=False, batch=256, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=2047),
        # a round of chunked prefill enters the cache: ragged pieces, far positions
        dict(name="append_chunk_b5_ragged", op="append", dtype="bf16", Hq=16, Hk=2, d=128, rot=128, page=64,
             norm=True, interleaved=False, batch=5, new_lo=1000, new_hi=4096, ctx_lo=0, ctx_hi=200000),
        # parallel samples of a prompt: 8 sequences fork, their last pages are copied in 4 attention layers
        dict(name="copy_pages_8x8", op="copy", dtype="bf16", kind="pages", pools=8, entries=512, n=8, Hk=2, d=128,
             page=64, H=0, dk=0, dv=0),
        # beams over the recurrent states: 64 of 256 sequences fork (2B-shape states, 1.18 MB each)
        dict(name="copy_states_64", op="copy", dtype="bf16", kind="states", pools=2, entries=256, n=64, Hk=0, d=0,
             page=0, H=12, dk=96, dv=256),
        # a small cache after a few sequences ended
        dict(name="compact_300_pages", op="compact", dtype="bf16", pools=2, pages=300, Hk=2, d=128, page=16,
             batch=9, ctx_hi=250, shared=2),
        # a large cache at half load, 4 attention layers
        dict(name="compact_8192_pages", op="compact", dtype="bf16", pools=8, pages=8192, Hk=2, d=128, page=64,
             batch=120, ctx_hi=4000, shared=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "copy", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hk = rng.choice([1, 2, 2, 4, 5])
    Hq = Hk * rng.choice([1, 2, 3, 6, 7, 8])
    d = rng.choice([64, 80, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "attn":
        form = rng.choice(["decode", "chunk", "mixed"])
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        batch = _log(rng, 1, 200) if form == "decode" else _log(rng, 1, 12)
        new = 1 if form == "decode" else _log(rng, 2, 1500)
        ctx = _log(rng, 1, 100000 if batch * Hk < 8 and new <= 128 else 6000)
        if dtype == "f32":
            batch, new, ctx = min(batch, 16), min(new, 400), min(ctx, 3000)
        return dict(op=op, dtype=dtype, Hq=Hq, Hk=Hk, d=d, page=page, window=window, batch=batch,
                    new_lo=1 if form == "mixed" else (new + 1) // 2, new_hi=new, ctx_lo=0, ctx_hi=ctx)
    if op == "append":
        decode = rng.random() < 0.4
        batch = _log(rng, 1, 512) if decode else _log(rng, 1, 8)
        new = 1 if decode else _log(rng, 2, 2500)
        return dict(op=op, dtype=dtype, Hq=Hq, Hk=Hk, d=d, rot=rng.choice([d, d, d // 2]), page=page,
                    norm=rng.random() < 0.75, interleaved=rng.random() < 0.3, batch=batch, new_lo=(new + 1) // 2,
                    new_hi=new, ctx_lo=0, ctx_hi=_log(rng, 10, 4000 if batch > 16 else 100000))
    if op == "copy":
        if rng.random() < 0.5:
            return dict(op=op, dtype=dtype, kind="pages", pools=rng.choice([2, 4, 8]), entries=1000,
                        n=_log(rng, 1, 400), Hk=Hk, d=d, page=page, H=0, dk=0, dv=0)
        return dict(op=op, dtype=dtype, kind="states", pools=2, entries=128, n=_log(rng, 1, 60), Hk=0, d=0, page=0,
                    H=rng.choice([1, 2, 5, 12, 16]), dk=rng.choice([16, 64, 96, 128]), dv=rng.choice([32, 128, 256]))
    ctx = _log(rng, 20, 3000)
    batch = _log(rng, 1, 100)
    pages = int(batch * ctx / page * rng.uniform(1.1, 1.8)) + 2 * batch + 5
    return dict(op=op, dtype=dtype, pools=rng.choice([2, 4]), pages=pages, Hk=Hk, d=d, page=page, batch=batch,
                ctx_hi=ctx, shared=rng.randint(0, batch // 2))


# ------------------------------------------------------------------ inputs
def _lens(case):
    """New tokens and cached context of each sequence, fixed by the case. In a
    ragged case the first sequence takes both upper ends, the second both
    lower ones."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    if case["new_hi"] > 1 and case["new_lo"] == 1:      # a mixed batch: two of three sequences decode
        new = [n if i % 3 == 0 else 1 for i, n in enumerate(new)]
    new[0], ctx[0] = case["new_hi"], case["ctx_hi"]
    if case["batch"] > 1:
        new[1], ctx[1] = case["new_lo"], case["ctx_lo"]
    return new, ctx


def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed * 1000003 + 17)
    return g


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32).mul_(std).to(dtype)


def _pages(seed, kv, page):
    """A cache of a little more than the pages in use, handed out in random order."""
    need = [-(-n // page) for n in kv]
    total = sum(need) + 3 + sum(need) // 16
    order = list(range(total))
    random.Random(seed * 31 + 5).shuffle(order)
    table = np.full((len(kv), max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, total


def prepare(case, seed):
    op, dt = case["op"], DT[case["dtype"]]
    g = _gen(seed)
    st = dict(case=case)
    if own:
        import linear_attention_lm_gen_b200 as jet
        jet.load_library()
        st["jet"] = jet
    if op in ("attn", "append"):
        new, ctx = _lens(case)
        kv = [a + b for a, b in zip(new, ctx)]
        table, total = _pages(seed, kv, case["page"])
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        N, Hq, Hk, d, page = int(cu[-1]), case["Hq"], case["Hk"], case["d"], case["page"]
        st.update(new=new, kv=kv, N=N, cu=torch.from_numpy(cu).cuda(),
                  kv_lens=torch.tensor(kv, dtype=torch.int32).cuda(), table=torch.from_numpy(table).cuda(),
                  k_pool=_randn(g, (total, Hk, page, d), dt), v_pool=_randn(g, (total, Hk, page, d), dt),
                  q_out=torch.empty((N, Hq, d), device="cuda", dtype=dt))
        if op == "attn":
            # normalised queries times a learned gain: logits of standard deviation about 1.5
            st["q"] = _randn(g, (N, Hq, d), dt, 1.5)
            if own:
                n = st["jet"].jet_attn_paged_workspace_size(len(new), N, Hq, Hk, d, dt)
                st["ws"] = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
        else:
            # q, k and v as the one projection leaves them, [N, Hq + 2 Hk, d], unnormalised
            st["qkv"] = _randn(g, (N, Hq + 2 * Hk, d), dt, 2.0)
            st["gq"] = _randn(g, (d,), torch.float32, 0.2).add_(1.0) if case["norm"] else None
            st["gk"] = _randn(g, (d,), torch.float32, 0.2).add_(1.0) if case["norm"] else None
            half = case["rot"] // 2
            st["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
            st["seq_of"] = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
            st["pos"] = torch.cat([torch.arange(b, a + b) for a, b in zip(new, ctx)]).cuda()
        return st
    r = random.Random(seed * 101 + 3)
    if op == "copy":
        if case["kind"] == "pages":
            shapes = [((case["entries"], case["Hk"], case["page"], case["d"]), dt)] * case["pools"]
        else:
            shapes = [((case["entries"], case["H"], case["dv"], case["dk"]), torch.float32),
                      ((case["entries"], 3, case["H"], case["dv"]), dt)]
        st["pools"] = [_randn(g, s, t) for s, t in shapes]
        ids = list(range(case["entries"]))
        r.shuffle(ids)
        st["dst"] = ids[:case["n"]]
        live = ids[case["n"]:]
        st["src"] = [live[i // 2 % len(live)] for i in range(case["n"])]      # every source forks twice
        st["pairs"] = torch.tensor([st["src"], st["dst"]]).cuda()
        return st
    st["pools"] = [_randn(g, (case["pages"], case["Hk"], case["page"], case["d"]), dt) for _ in range(case["pools"])]
    table, kv = _compact_tables(case, seed)
    st["table"], st["kv_lens"] = torch.from_numpy(table).cuda(), torch.tensor(kv, dtype=torch.int32).cuda()
    if own:
        n = st["jet"].jet_cache_compact_workspace_size(case["pages"])
        st["ws"] = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
        st["table_out"] = torch.empty_like(st["table"])
        st["n_live"] = torch.empty(1, device="cuda", dtype=torch.int32)
    return st


def _compact_tables(case, seed):
    """Page tables of sequences that outlived others; the last `shared` ones
    are forks that hold the first half of an earlier sequence's pages."""
    r = random.Random(seed * 101 + 3)
    B, page = case["batch"], case["page"]
    kv = [r.randint(1, case["ctx_hi"]) for _ in range(B)]
    ids = list(range(case["pages"]))
    r.shuffle(ids)
    width = -(-case["ctx_hi"] // page)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for s in range(B):
        need = -(-kv[s] // page)
        first = 0
        if s >= B - case["shared"]:
            parent = s - (B - case["shared"])
            if parent < B - case["shared"]:
                first = min(need, -(-kv[parent] // page) // 2)
                table[s, :first] = table[parent, :first]
        take = min(need - first, len(ids) - at)
        table[s, first:first + take] = ids[at:at + take]
        at += take
        kv[s] = min(kv[s], (first + take) * page)
    return table, kv


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    return (_own if own else _plain)[op](st)


def _plain_attn(st):
    c = st["case"]
    Hq, Hk, d, page, W = c["Hq"], c["Hk"], c["d"], c["page"], c["window"]
    G, scale = Hq // Hk, 1.0 / math.sqrt(d)
    out, at = st["q_out"], 0
    for s, (n, L) in enumerate(zip(st["new"], st["kv"])):
        first = L - n
        step = max(1, (1 << 28) // (Hq * L))
        for a in range(0, n, step):
            b = min(n, a + step)
            lo = max(0, first + a - W + 1) if W else 0
            lo, hi = lo // page * page, first + b
            pages = st["table"][s, lo // page:-(-hi // page)].long()
            K = st["k_pool"][pages].float().transpose(0, 1).reshape(Hk, -1, d)[:, :hi - lo]
            V = st["v_pool"][pages].float().transpose(0, 1).reshape(Hk, -1, d)[:, :hi - lo]
            Q = st["q"][at + a:at + b].float().view(b - a, Hk, G, d).permute(1, 2, 0, 3).reshape(Hk, -1, d)
            S = (Q @ K.transpose(1, 2)).mul_(scale).view(Hk, G, b - a, hi - lo)
            p = torch.arange(first + a, first + b, device="cuda")[:, None]
            j = torch.arange(lo, hi, device="cuda")[None, :]
            hide = j > p
            if W:
                hide |= j <= p - W
            S.masked_fill_(hide, float("-inf"))
            S.sub_(S.amax(-1, keepdim=True)).exp_()
            O = (S.view(Hk, -1, hi - lo) @ V).view(Hk, G, b - a, d) / S.sum(-1, keepdim=True)
            out[at + a:at + b] = O.permute(2, 0, 1, 3).reshape(b - a, Hq, d)
        at += n
    return out


def _plain_append(st):
    c = st["case"]
    Hq, Hk, d, rot, page = c["Hq"], c["Hk"], c["d"], c["rot"], c["page"]
    half = rot // 2
    x = st["qkv"].float()
    qk, v = x[:, :Hq + Hk], st["qkv"][:, Hq + Hk:]
    if c["norm"]:
        w = torch.cat([st["gq"].expand(Hq, d), st["gk"].expand(Hk, d)])
        qk = qk * torch.rsqrt((qk * qk).mean(-1, keepdim=True) + 1e-6) * w
    ang = st["pos"].double()[:, None] * st["inv_freq"].double()[None, :]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    y = qk.clone()
    if c["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = qk[..., :half], qk[..., half:rot]
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    st["q_out"].copy_(y[:, :Hq])
    pid, row = st["table"][st["seq_of"], st["pos"] // page].long(), st["pos"] % page
    st["k_pool"][pid, :, row] = y[:, Hq:].to(st["k_pool"].dtype)
    st["v_pool"][pid, :, row] = v
    return [st["q_out"], st["k_pool"], st["v_pool"]]


def _plain_copy(st):
    for p in st["pools"]:
        p[st["pairs"][1]] = p[st["pairs"][0]]
    return st["pools"]


def _plain_compact(st):
    pages, page = st["case"]["pages"], st["case"]["page"]
    table, kv = st["table"], st["kv_lens"]
    need = (kv + page - 1) // page
    used = (torch.arange(table.shape[1], device="cuda")[None, :] < need[:, None]) & (table >= 0)
    live = torch.zeros(pages, dtype=torch.bool, device="cuda")
    live[table[used].long()] = True
    n = live.sum()
    ids = torch.arange(pages, device="cuda")
    src, dst = ids[live & (ids >= n)], ids[~live & (ids < n)]
    to = ids.clone()
    to[src] = dst
    for p in st["pools"]:
        p[dst] = p[src]
    out = torch.where(used, to[table.clamp(min=0).long()].int(), torch.full_like(table, -1))
    return [out, n.int().view(1)] + st["pools"]


def _own_attn(st):
    c = st["case"]
    return st["jet"].jet_attn_paged(st["q"], st["k_pool"], st["v_pool"], st["cu"], st["kv_lens"], st["table"],
                                    max(st["new"]), st["q_out"], st["ws"], window=c["window"])


def _own_append(st):
    c = st["case"]
    Hq, Hk, x = c["Hq"], c["Hk"], st["qkv"]
    st["jet"].jet_attn_rope_append(x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:], st["gq"], st["gk"], st["inv_freq"],
                                   st["cu"], st["kv_lens"], st["table"], st["k_pool"], st["v_pool"], st["q_out"],
                                   eps=1e-6, interleaved=c["interleaved"])
    return [st["q_out"], st["k_pool"], st["v_pool"]]


def _own_copy(st):
    st["jet"].jet_cache_copy(st["pools"], st["src"], st["dst"])
    return st["pools"]


def _own_compact(st):
    st["jet"].jet_cache_compact(st["pools"], st["table"], st["kv_lens"], st["case"]["page"], st["table_out"],
                                st["n_live"], st["ws"])
    return [st["table_out"], st["n_live"]] + st["pools"]


_plain = dict(attn=_plain_attn, append=_plain_append, copy=_plain_copy, compact=_plain_compact)
_own = dict(attn=_own_attn, append=_own_append, copy=_own_copy, compact=_own_compact)


# ------------------------------------------------------------------ work
def work(case):
    """Bytes and operations of one pass that no form can do without."""
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "attn":
        new, ctx = _lens(case)
        W = case["window"]
        nbytes, pairs = 0, 0
        for n, c in zip(new, ctx):
            L = c + n
            keys = min(L, n + W - 1) if W else L          # positions that some new token reads
            nbytes += 2 * keys * case["Hk"] * case["d"] * es + 2 * n * case["Hq"] * case["d"] * es
            if W:
                full = max(0, min(n, L - W + 1 if L >= W else 0))    # tokens that see a whole window
                m = n - full                                         # tokens whose window reaches position 0
                pairs += full * W + m * c + m * (m + 1) // 2
            else:
                pairs += n * c + n * (n + 1) // 2
        return dict(bytes=nbytes, flops=4 * case["d"] * case["Hq"] * pairs)
    if op == "append":
        new, _ = _lens(case)
        N = sum(new)
        el = N * (case["Hq"] + 2 * case["Hk"]) * case["d"]
        return dict(bytes=2 * el * es, flops=8 * el)
    if op == "copy":
        distinct = -(-case["n"] // 2)
        if case["kind"] == "pages":
            entry = case["pools"] * case["Hk"] * case["page"] * case["d"] * es
        else:
            entry = case["H"] * case["dv"] * (case["dk"] * 4 + 3 * es)
        return dict(bytes=(distinct + case["n"]) * entry, flops=0)
    table, kv = _compact_tables(case, 0)
    live = np.unique(table[table >= 0])
    moved = int((live >= len(live)).sum())
    entry = case["pools"] * case["Hk"] * case["page"] * case["d"] * es
    return dict(bytes=2 * moved * entry + 8 * table.size, flops=0)


# ------------------------------------------------------------------ exact values (64 bits)
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return dict(attn=_exact_attn, append=_exact_append, copy=_exact_copy, compact=_exact_compact)[case["op"]](st)


def _exact_attn(st):
    """Token by token and key by key: o = sum_j softmax_j(q k_j / sqrt(d)) v_j, a block of tokens at a time."""
    c = st["case"]
    Hq, Hk, d, page, W = c["Hq"], c["Hk"], c["d"], c["page"], c["window"]
    if work(c)["flops"] > 4e12:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    table = st["table"].cpu().numpy()
    at = 0
    for s, (n, L) in enumerate(zip(st["new"], st["kv"])):
        where = torch.tensor([int(table[s, p // page]) * page + p % page for p in range(L)], device="cuda")
        token = torch.arange(n, device="cuda") + (L - n)
        for h in range(Hk):
            k = st["k_pool"][:, h].reshape(-1, d)[where].double()
            v = st["v_pool"][:, h].reshape(-1, d)[where].double()
            rows = max(1, (1 << 26) // L)
            for head in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                for a in range(0, n, rows):
                    t = token[a:a + rows]
                    w = torch.einsum("nd,ld->nl", st["q"][at + a:at + a + len(t), head].double(), k) / d ** 0.5
                    key = torch.arange(L, device="cuda")
                    seen = key <= t[:, None]
                    if W:
                        seen = seen & (t[:, None] - key < W)
                    w = torch.softmax(torch.where(seen, w, torch.full_like(w, -math.inf)), dim=1)
                    out[at + a:at + a + len(t), head] = torch.einsum("nl,ld->nd", w, v)
        at += n
    return out


def _exact_append(st):
    c = st["case"]
    Hq, Hk, d, rot, page = c["Hq"], c["Hk"], c["d"], c["rot"], c["page"]
    x = st["qkv"].double()
    heads = []
    for h in range(Hq + Hk):
        y = x[:, h]
        if c["norm"]:
            y = y / torch.sqrt(y.pow(2).sum(1, keepdim=True) / d + 1e-6)
            y = y * (st["gq"] if h < Hq else st["gk"]).double()
        # a rotation is a product with e^(i angle) of the pairs taken as complex numbers
        first = [2 * i if c["interleaved"] else i for i in range(rot // 2)]
        second = [2 * i + 1 if c["interleaved"] else i + rot // 2 for i in range(rot // 2)]
        z = torch.complex(y[:, first], y[:, second])
        ang = torch.outer(st["pos"].double(), st["inv_freq"].double())
        z = z * torch.polar(torch.ones_like(ang), ang)
        y = y.clone()
        y[:, first], y[:, second] = z.real, z.imag
        heads.append(y)
    y = torch.stack(heads, 1)
    k, v = st["k_pool"].double(), st["v_pool"].double()
    flat = st["table"].long()[st["seq_of"], torch.div(st["pos"], page, rounding_mode="floor")] * page \
        + torch.remainder(st["pos"], page)
    for h in range(Hk):
        for pool, rows in ((k, y[:, Hq + h]), (v, x[:, Hq + Hk + h])):
            plane = pool[:, h].reshape(-1, d)
            plane[flat] = rows
            pool[:, h] = plane.view(-1, page, d)
    return [y[:, :Hq].contiguous(), k, v]


def _exact_copy(st):
    out = [p.clone() for p in st["pools"]]
    for a, b in zip(st["src"], st["dst"]):
        for new, old in zip(out, st["pools"]):
            new[b].copy_(old[a])
    return out


def _exact_compact(st):
    page = st["case"]["page"]
    table, kv = st["table"].cpu().numpy(), st["kv_lens"].cpu().numpy()
    held = set()
    for s in range(len(kv)):
        held.update(int(table[s, i]) for i in range(-(-int(kv[s]) // page)) if table[s, i] >= 0)
    holes = [i for i in range(len(held)) if i not in held]
    to = dict(zip(sorted(i for i in held if i >= len(held)), holes))
    out = np.full_like(table, -1)
    for s in range(len(kv)):
        for i in range(-(-int(kv[s]) // page)):
            if table[s, i] >= 0:
                out[s, i] = to.get(int(table[s, i]), int(table[s, i]))
    pools = [p.clone() for p in st["pools"]]
    for a, b in to.items():
        for new, old in zip(pools, st["pools"]):
            new[b].copy_(old[a])
    return [torch.from_numpy(out).cuda(), torch.tensor([len(held)], dtype=torch.int32).cuda()] + pools
