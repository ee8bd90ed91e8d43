// Copies of whole entries (pages of a key/value cache, or per-sequence
// states) inside cache pools, and the compaction of a paged cache.
//
// Both are bandwidth-bound: every moved byte is read once and written once.
// A block moves pieces of 16 KB, each thread four 16-byte loads in flight
// before the first store. 64 states of 1.2 MB (32 read, 64 written), other
// states every time: 20 us, 5.8 TB/s (the same ones again 17 us, part of them
// then in L2); a compaction that moves 0.54 GB of 8192 pages: 174 to 178 us,
// 6.1 to 6.2 TB/s, the plan of one block before it included. That plan is
// what a smaller one waits for: 4096 pages, half of them live, 28 us of 20.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace jet {
namespace cache {

constexpr int MAX_POOLS = 64;        // pools of one call
constexpr int THREADS = 256;
constexpr int PIECE = THREADS * 16 * 4;

struct Pools {
    unsigned char* base[MAX_POOLS];
    long long stride[MAX_POOLS];     // bytes between entries
    long long bytes[MAX_POOLS];      // bytes of an entry
    int n;
};

__device__ __forceinline__ void copy_piece(const unsigned char* src, unsigned char* dst, long long left) {
    uint4 r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const long long off = (long long)(u * THREADS + threadIdx.x) * 16;
        if (off < left) r[u] = __ldcs(reinterpret_cast<const uint4*>(src + off));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const long long off = (long long)(u * THREADS + threadIdx.x) * 16;
        if (off < left) __stcs(reinterpret_cast<uint4*>(dst + off), r[u]);
    }
}

// n pairs, the pair of index i given by pair(i); the pieces of all pools in
// one index space, pool by pool
template <typename PairFn>
__device__ __forceinline__ void copy_pairs(const Pools& p, int n, PairFn pair) {
    long long w = blockIdx.x;
    for (int k = 0; k < p.n; ++k) {
        const long long per = (p.bytes[k] + PIECE - 1) / PIECE, total = per * n;
        for (; w < total; w += gridDim.x) {
            const long long i = w / per, off = (w - i * per) * PIECE;
            const int2 e = pair((int)i);
            copy_piece(p.base[k] + e.x * p.stride[k] + off, p.base[k] + e.y * p.stride[k] + off, p.bytes[k] - off);
        }
        w -= total;
    }
}

template <int CAP> struct Pairs {
    int2 e[CAP];      // (source, destination)
};

// The pairs travel in the kernel's parameters: no host-to-device copy.
template <int CAP>
__global__ void __launch_bounds__(THREADS)
copy_kernel(const __grid_constant__ Pools p, const __grid_constant__ Pairs<CAP> pairs, int n) {
    pdl_wait();
    pdl_trigger();
    copy_pairs(p, n, [&](int i) { return pairs.e[i]; });
}

// ---------------------------------------------------------------- compaction
// With n live pages, the live pages at or above n move, in increasing order,
// to the free ones below n, in increasing order: the fewest moves, the same
// result every time, and no page is both a source and a destination.
//   plan: one block marks the live pages in a bitmap in shared memory and
//     writes the moves and each moved page's new index to the workspace;
//   move: all blocks copy the pages and rewrite the tables.
constexpr int PLAN_THREADS = 1024;

struct PlanOut {
    int* n_moves;      // [1]
    int2* moves;       // [n_pages / 2]
    int* to;           // [n_pages], written for moved pages only
};

__global__ void __launch_bounds__(PLAN_THREADS)
compact_plan_kernel(const int* __restrict__ table, const int* __restrict__ kv_lens, int nseq, int max_pages,
                    int page_shift, int n_pages, PlanOut out, int* __restrict__ n_live) {
    extern __shared__ uint32_t bits[];
    __shared__ int part[PLAN_THREADS / 32];
    __shared__ int total_s;
    const int words = (n_pages + 31) / 32;
    for (int i = threadIdx.x; i < words; i += PLAN_THREADS) bits[i] = 0u;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int s = warp; s < nseq; s += PLAN_THREADS / 32) {
        const int L = kv_lens[s];
        if (lane == 0 && (L < 0 || (long long)L > ((long long)max_pages << page_shift))) flag_error(DEVERR_DATA);
        const int need = min(max_pages, (int)(((long long)max(L, 0) + (1 << page_shift) - 1) >> page_shift));
        for (int i = lane; i < need; i += 32) {
            const int pg = table[(long long)s * max_pages + i];
            if ((unsigned)pg < (unsigned)n_pages) atomicOr(&bits[pg >> 5], 1u << (pg & 31));
            else if (pg != -1) flag_error(DEVERR_DATA);
        }
    }
    __syncthreads();
    // thread i takes a run of consecutive words; exclusive prefix of the live counts
    const int per = (words + PLAN_THREADS - 1) / PLAN_THREADS;
    const int w0 = min(words, (int)threadIdx.x * per), w1 = min(words, w0 + per);
    int cnt = 0;
    for (int i = w0; i < w1; ++i) cnt += __popc(bits[i]);
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int v = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        part[lane] = v;
        if (lane == 31) total_s = v;
    }
    __syncthreads();
    const int n = total_s;
    const int before = inc - cnt + (warp ? part[warp - 1] : 0);     // live pages before word w0
    // live pages below n; the first mover's rank is subtracted from the others'
    __shared__ int live_below;
    if (threadIdx.x == 0) live_below = 0;
    __syncthreads();
    if (n > 0 && n < n_pages) {
        const int wn = n >> 5;
        if (wn >= w0 && wn < w1) {
            int x = before;
            for (int i = w0; i < wn; ++i) x += __popc(bits[i]);
            live_below = x + __popc(bits[wn] & ((1u << (n & 31)) - 1u));
        }
    } else if (threadIdx.x == 0) {
        live_below = n;
    }
    __syncthreads();
    int rank = before;
    for (int i = w0; i < w1; ++i) {
        const uint32_t w = bits[i];
        for (int k = 0; k < 32; ++k) {
            const int pg = i * 32 + k;
            if (pg >= n_pages) break;
            const bool live = (w >> k) & 1u;
            if (live && pg >= n) out.moves[rank - live_below].x = pg;
            if (!live && pg < n) out.moves[pg - rank].y = pg;
            rank += live;
        }
    }
    __syncthreads();
    const int moves = n - live_below;
    __threadfence_block();
    for (int i = threadIdx.x; i < moves; i += PLAN_THREADS) {
        const int2 m = out.moves[i];
        out.to[m.x] = m.y;
    }
    if (threadIdx.x == 0) {
        *out.n_moves = moves;
        *n_live = n;
    }
}

// table and table_out may be the same array
__global__ void __launch_bounds__(THREADS)
compact_move_kernel(const __grid_constant__ Pools p, const int* table, int* table_out,
                    const int* __restrict__ kv_lens, int nseq, int max_pages, int page_shift, int n_pages,
                    const int* __restrict__ n_live, PlanOut plan) {
    pdl_wait();
    pdl_trigger();
    const int n = *n_live;
    const long long cells = (long long)nseq * max_pages;
    for (long long i = (long long)blockIdx.x * THREADS + threadIdx.x; i < cells; i += (long long)gridDim.x * THREADS) {
        const int s = (int)(i / max_pages), j = (int)(i - (long long)s * max_pages);
        const int pg = table[i];
        int to = -1;
        if ((unsigned)pg < (unsigned)n_pages && ((long long)j << page_shift) < kv_lens[s])
            to = pg < n ? pg : plan.to[pg];
        table_out[i] = to;
    }
    copy_pairs(p, *plan.n_moves, [&](int i) { return plan.moves[i]; });
}

}  // namespace cache
}  // namespace jet
