"""A serving cache for the softmax-attention layers of the hybrid model.

Between its JetBlock layers the model keeps a few softmax-attention layers,
some with a sliding window (Jet-Nemotron paper, section 3.1 and appendix A.1).
Where a JetBlock layer's state has a fixed size (engine.JetEngine), theirs
grows with the sequence; this module keeps it in pages:

  admit(seq)   an empty sequence
  begin({seq: n, ...})  make room for n new tokens of each of these sequences
               (a piece of a prompt, or one decode token, mixed freely) and
               return the step's batch
  attend(layer, batch, q, k, v)  one layer of the step: norm, rotation and
               append (jet_attn_rope_append), then attention over the cache
               (jet_attn_paged); q, k and v hold the sequences' new tokens one
               after another, in the batch's order
  fork(parent, children)  sequences that continue from the parent: whole pages
               are shared, the last one, which the next token writes to, is
               copied in every layer (jet_cache_copy, one launch)
  release(seq) give the pages up that no other sequence holds
  compact()    move the live pages to the lowest entries (jet_cache_compact),
               so that the tail of the pools is free

All layers share the page numbering: page i is entry i of every layer's pools.
If every layer has a window, pages that lie before all windows are given up as
the sequences advance. One layer that sees everything keeps every page, for
the windowed layers too: a model that mixes the two (as the 2B and 4B ones do)
saves their memory with two engines, one for the layers without a window and
one for those with, each with its own pages, whose begin, fork and release are
called alike. The host keeps the page tables and reference counts;
each step sends its tables to the GPU in one copy. Everything is issued on
torch's current stream. Steps on two streams share no scratch memory, but the
pages: a step that gives pages up or takes them has to be ordered with the
others, as with any tensor. Between a step's begin and its last attend, do not
fork or release its sequences, nor begin another step of them, not even one
that is refused for want of room; a batch from before a compact() is refused,
since its pages have moved.
"""
from __future__ import annotations

import heapq
from dataclasses import dataclass

import numpy as np
import torch

from . import (jet_attn_paged, jet_attn_paged_workspace_size, jet_attn_rope_append, jet_cache_compact, jet_cache_copy)


@dataclass
class AttnBatch:
    """One step's new tokens: the sequences in order and, on the GPU, what the library's calls take."""
    seqs: list
    new: list              # new tokens per sequence
    cu_q: torch.Tensor     # [n + 1] int32
    kv_lens: torch.Tensor  # [n] int32, the new tokens included
    page_table: torch.Tensor   # [n, width] int32
    epoch: int             # compactions before it

    @property
    def tokens(self) -> int:
        return sum(self.new)


class JetAttnEngine:
    def __init__(self, n_layers: int, Hq: int, Hk: int, d: int, n_pages: int, page_size: int = 64, max_seqs: int = 256,
                 max_len: int = 65536, *, windows=None, inv_freq=None, gammas=None, eps: float = 1e-6,
                 interleaved: bool = False, scale: float | None = None, dtype=torch.bfloat16, device="cuda"):
        """windows: per layer, the positions a token sees (0 or None: all).
        inv_freq [rot/2] float32 or None; gammas: per layer (q_gamma, k_gamma)
        [d] float32, or None."""
        if min(n_layers, Hq, Hk, d, n_pages, page_size, max_seqs, max_len) <= 0:
            raise ValueError("sizes must be positive")
        self.windows = [int(w or 0) for w in (windows or [0] * n_layers)]
        self.gammas = list(gammas) if gammas is not None else [(None, None)] * n_layers
        if len(self.windows) != n_layers or len(self.gammas) != n_layers:
            raise ValueError(f"windows and gammas need one entry for each of the {n_layers} layers")
        self.Hq, self.Hk, self.d, self.page, self.n_pages = Hq, Hk, d, page_size, n_pages
        self.inv_freq, self.eps, self.interleaved, self.scale = inv_freq, eps, interleaved, scale
        self.device, self.dtype = torch.device(device), dtype
        shape = (n_pages, Hk, page_size, d)
        self.k = [torch.zeros(shape, device=device, dtype=dtype) for _ in range(n_layers)]
        self.v = [torch.zeros(shape, device=device, dtype=dtype) for _ in range(n_layers)]
        self._table = np.full((max_seqs, -(-max_len // page_size)), -1, dtype=np.int32)
        self._rows = list(range(max_seqs - 1, -1, -1))      # pop() hands out the lowest row first
        self._free = list(range(n_pages))                   # a heap: the lowest page first
        self._ref = np.zeros(n_pages, dtype=np.int32)       # sequences that hold a page
        self.row: dict = {}                                 # sequence id -> row of the tables
        self.len: dict = {}                                 # sequence id -> positions in the cache
        self._first: dict = {}                              # sequence id -> first page still held
        self._epoch = 0                                     # compactions so far

    # ---------------------------------------------------------------- sequences and pages
    @property
    def free_pages(self) -> int:
        return len(self._free)

    @property
    def pools(self) -> list:
        return self.k + self.v

    def admit(self, seq) -> None:
        """An empty sequence."""
        if seq in self.row:
            raise KeyError(f"sequence {seq!r} is already admitted")
        if not self._rows:
            raise RuntimeError("no room for another sequence")
        self.row[seq] = self._rows.pop()
        self.len[seq] = self._first[seq] = 0

    def _drop(self, pages) -> None:
        for p in pages:
            self._ref[p] -= 1
            if self._ref[p] == 0:
                heapq.heappush(self._free, int(p))

    def release(self, seq) -> None:
        """Forget the sequence; its pages that no other sequence holds are free."""
        r = self.row.pop(seq)
        t = self._table[r]
        self._drop(t[t >= 0])
        t.fill(-1)
        self._rows.append(r)
        del self.len[seq], self._first[seq]

    def _known(self, seqs) -> None:
        unknown = [s for s in seqs if s not in self.row]
        if unknown:
            raise KeyError(f"sequences that are not admitted: {sorted(map(str, unknown))}")

    def fork(self, parent, children) -> None:
        """Admit `children` as continuations of `parent`: they share its whole
        pages and get a copy of the last one if it is not full."""
        children = list(children)
        self._known([parent])
        if len(set(children)) != len(children) or any(c in self.row for c in children):
            raise KeyError("a child is already admitted or appears twice")
        n, tail = divmod(self.len[parent], self.page)
        if len(children) > len(self._rows):
            raise RuntimeError("no room for another sequence")
        if tail and len(children) > len(self._free):
            raise RuntimeError("page cache is full")
        t = self._table[self.row[parent]]
        # the copies first: if one fails, nothing has changed but free pages
        dst = heapq.nsmallest(len(children), self._free) if tail else []
        if dst:
            pools = self.pools
            for i in range(0, len(pools), 64):              # pools per call
                jet_cache_copy(pools[i:i + 64], [int(t[n])] * len(dst), dst)
        shared = t[:n][t[:n] >= 0]
        for c in children:
            self.admit(c)
            tc = self._table[self.row[c]]
            tc[:n] = t[:n]
            self._ref[shared] += 1
            if tail:
                tc[n] = heapq.heappop(self._free)           # as in dst
                self._ref[tc[n]] = 1
            self.len[c], self._first[c] = self.len[parent], self._first[parent]

    def compact(self) -> int:
        """Move the live pages to the lowest entries of the pools; returns
        their number. Reads the new tables back (waits for the GPU)."""
        seqs = list(self.row)
        if not seqs:
            return 0
        rows = [self.row[s] for s in seqs]
        table = torch.from_numpy(self._table[rows]).to(self.device)
        lens = torch.tensor([self.len[s] for s in seqs], dtype=torch.int32).to(self.device)
        pools = self.pools
        out, live = None, None
        for i in range(0, len(pools), 64):                  # the plan depends on the tables alone
            out, live = jet_cache_compact(pools[i:i + 64], table, lens, self.page)
        self._epoch += 1
        self._table[rows] = out.cpu().numpy()
        n = int(live.item())
        self._ref[:] = 0
        held = self._table[rows]
        np.add.at(self._ref, held[held >= 0], 1)
        self._free = list(range(n, self.n_pages))           # ascending: a heap
        return n

    # ---------------------------------------------------------------- steps
    def begin(self, new: dict) -> AttnBatch:
        """Room for new[seq] >= 1 new tokens of each sequence, in the order of
        `new`. The checks come before any change. Pages that no window of
        these sequences will see again are then given up, which makes room;
        if there is still too little, no page is taken (RuntimeError)."""
        seqs = list(new)
        self._known(seqs)
        if not seqs or any(int(n) < 1 for n in new.values()):
            raise ValueError("a step needs at least one new token of each of its sequences")
        need = 0
        for s in seqs:
            total = self.len[s] + new[s]
            if -(-total // self.page) > self._table.shape[1]:
                raise ValueError(f"sequence {s!r} would outgrow the cache's longest sequence")
            need += -(-total // self.page) - -(-self.len[s] // self.page)
        keep = max(self.windows) if all(self.windows) else 0
        if keep:                                            # pages before every window of the step's tokens
            for s in seqs:
                f = max(0, self.len[s] - keep + 1) // self.page
                if f > self._first[s]:
                    t = self._table[self.row[s]][self._first[s]:f]
                    self._drop(t[t >= 0])
                    t.fill(-1)
                    self._first[s] = f
        if need > len(self._free):
            raise RuntimeError("page cache is full")
        for s in seqs:
            t = self._table[self.row[s]]
            for i in range(-(-self.len[s] // self.page), -(-(self.len[s] + new[s]) // self.page)):
                t[i] = heapq.heappop(self._free)
                self._ref[t[i]] = 1
            self.len[s] += new[s]
        n = len(seqs)
        lens = np.array([self.len[s] for s in seqs], dtype=np.int32)
        width = int(-(-lens.max() // self.page))
        host = np.empty(2 * n + 1 + n * width, dtype=np.int32)
        host[0] = 0
        host[1:n + 1] = np.cumsum([new[s] for s in seqs])
        host[n + 1:2 * n + 1] = lens
        host[2 * n + 1:] = self._table[[self.row[s] for s in seqs], :width].ravel()
        dev = torch.from_numpy(host).to(self.device, non_blocking=True)
        return AttnBatch(seqs, [int(new[s]) for s in seqs], dev[:n + 1], dev[n + 1:2 * n + 1],
                         dev[2 * n + 1:].view(n, width), self._epoch)

    def attend(self, layer: int, batch: AttnBatch, q, k, v) -> torch.Tensor:
        """One layer of a step: q [N,Hq,d], k, v [N,Hk,d] of the batch's new
        tokens (slices of one projection's output will do). Their keys and
        values enter the cache; returns o [N,Hq,d]."""
        if q.shape[0] != batch.tokens:
            raise ValueError(f"the batch has {batch.tokens} new tokens, q has {q.shape[0]}")
        if batch.epoch != self._epoch:
            raise ValueError("the batch is from before a compaction: its pages have moved")
        gq, gk = self.gammas[layer]
        kp, vp = self.k[layer], self.v[layer]
        y = torch.empty((batch.tokens, self.Hq, self.d), device=self.device, dtype=self.dtype)
        y = jet_attn_rope_append(q, k, v, gq, gk, self.inv_freq, batch.cu_q, batch.kv_lens, batch.page_table, kp, vp, y,
                                 eps=self.eps, interleaved=self.interleaved)
        need = jet_attn_paged_workspace_size(len(batch.seqs), batch.tokens, self.Hq, self.Hk, self.d, self.dtype)
        # of its own: a batch on another stream, or another captured graph, has another one
        ws = torch.empty(need, device=self.device, dtype=torch.uint8)
        return jet_attn_paged(y, kp, vp, batch.cu_q, batch.kv_lens, batch.page_table, max(batch.new),
                              torch.empty_like(y), ws, window=self.windows[layer], scale=self.scale)
