// How the attention kernels divide a ragged batch among a fixed grid.
//
// An item is a tile of query rows of one sequence and one cache head: `tpt`
// tokens times `gt` of the G query heads that share the head (`hs` such head
// parts, one unless G exceeds the tile's rows). Its cost is taken as the
// positions it reads plus a constant c0. The items lie one after another on
// an axis, sequence by sequence, head by head, tile by tile, and CTA c works
// on the interval [c * chunk, (c + 1) * chunk): every CTA gets the same cost
// whatever the lengths are, a long sequence is split along the cache as a
// matter of course, and the grid needs no length on the host. An item that
// lies in one interval is finished by its CTA; the parts of an item that is
// cut go to the workspace (each CTA has at most one part of an item that
// began before its interval, slot 0, and one of an item that goes on behind
// it, slot 1) and a second kernel joins them in order, so results do not
// depend on timing and the workspace not on the lengths.
//
// The cost of tile i of a sequence with A = max(0, L - n) older positions is
// c0 + A + (i + 1) tpt, or c0 + tpt + window - 1 once the window cuts the
// first positions off, so that sums over tiles have a closed form.
#pragma once
#include "k_attn_common.cuh"

namespace jet {
namespace attn {

struct Work {
    Batch b;
    Cache c;
    int Hk, G, window;
    int tpt, gt, hs;      // tokens and heads of a tile, head parts
    int kt;               // positions of a step along the cache (a power of two)
    int c0, min_chunk;
};

// one sequence on the axis
struct SeqAxis {
    Seq q;
    int A, tiles, first;       // older positions, tiles, first tile that the window cuts (tiles: none)

    __device__ __forceinline__ SeqAxis() {}
    __device__ __forceinline__ SeqAxis(const Work& w, const Seq& seq) : q(seq) {
        A = max(0, q.L - q.n);
        tiles = (int)((unsigned)(q.n + w.tpt - 1) / (unsigned)w.tpt);
        first = tiles;
        if (w.window > 0) {
            const unsigned ahead = A < w.window - 1 ? (unsigned)(w.window - 1 - A) : 0u;     // tokens it does not cut
            first = min(tiles, (int)((ahead + w.tpt - 1) / (unsigned)w.tpt));
        }
    }
    __device__ __forceinline__ long long upto(const Work& w, int i) const {       // cost of tiles 0 .. i-1
        const long long m = min(i, first);
        return m * (w.c0 + A) + w.tpt * (m * (m + 1) / 2) + (i - m) * ((long long)w.c0 + w.tpt + w.window - 1);
    }
    __device__ __forceinline__ long long tile(const Work& w, int i) const {       // cost of tile i
        return i < first ? (long long)w.c0 + A + (long long)(i + 1) * w.tpt : (long long)w.c0 + w.tpt + w.window - 1;
    }
};

// one item: its place on the axis and what it covers
struct Item {
    SeqAxis ax;
    int s, hh, i;              // sequence, head * hs + head part, tile
    long long a, cost;         // start and length on the axis
    int t0, nt;                // first token, tokens
    int p_first;               // position of the first token
    int lo, hi;                // positions read (lo a multiple of the step), empty if hi <= 0
    int steps;

    __device__ __forceinline__ void fill(const Work& w) {
        cost = ax.tile(w, i);
        t0 = i * w.tpt;
        nt = min(w.tpt, ax.q.n - t0);
        p_first = ax.q.L - ax.q.n + t0;
        lo = first_key(p_first, w.window) & ~(w.kt - 1);
        hi = p_first + nt;
        steps = hi > lo ? (int)((unsigned)(hi - lo + w.kt - 1) / (unsigned)w.kt) : 0;
    }
    // first step at or behind place x of the axis. In float64: any monotone
    // function of x serves, as long as every caller computes the same.
    __device__ __forceinline__ int step_at(long long x) const {
        if (x <= a) return 0;
        if (x >= a + cost) return steps;
        return min(steps, (int)((double)(x - a) * (double)steps / (double)cost));
    }
    __device__ __forceinline__ void next(const Work& w) {
        a += cost;
        if (++i >= ax.tiles) {
            i = 0;
            if (++hh >= w.Hk * w.hs) {
                hh = 0;
                Seq q;
                do {
                    if (++s >= w.b.nseq) return;
                    q = load_seq(w.b, w.c, s, false);
                } while (q.n == 0);
                ax = SeqAxis(w, q);
            }
        }
        fill(w);
    }
};

// The axis's length and step, and the item at place index * chunk of it.
// Every thread of the block (THREADS of them) calls it; `item` is the same in
// all of them. Returns false where the place lies behind the end.
template <int THREADS>
__device__ __forceinline__ bool block_locate(const Work& w, int n_cta, int index, long long& chunk, long long& total,
                                             Item& item) {
    __shared__ long long part[THREADS / 32];
    __shared__ long long found_a;
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (w.b.nseq + THREADS - 1) / THREADS;
    const int s0 = min(w.b.nseq, tid * per), s1 = min(w.b.nseq, s0 + per);
    long long sum = 0;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        const SeqAxis ax(w, load_seq(w.b, w.c, s, true));
        sum += ax.upto(w, ax.tiles) * (w.Hk * w.hs);
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    long long before = inc - sum;
    total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) before += part[i];
        total += part[i];
    }
    // n_cta chunks reach behind the end: the factor outweighs float64's roundings where the 1 no longer does
    chunk = (long long)((double)total / n_cta * (1.0 + 0x1p-50)) + 1;
    chunk = max((long long)w.min_chunk, chunk);
    const long long x = chunk * index;
    if (x >= total) return false;
    if (x >= before && x < before + sum) {
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
            const SeqAxis ax(w, load_seq(w.b, w.c, s, false));
            const long long per_head = ax.upto(w, ax.tiles), cost = per_head * (w.Hk * w.hs);
            if (x < before + cost) {
                int hh = 0;
                long long rem = x - before;
                for (; rem >= per_head; ++hh) rem -= per_head;
                int lo = 0, hi = ax.tiles - 1;                 // largest tile that starts at or before rem
#pragma unroll 1
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (ax.upto(w, mid) <= rem) lo = mid;
                    else hi = mid - 1;
                }
                found[0] = s;
                found[1] = hh;
                found[2] = lo;
                found_a = before + hh * per_head + ax.upto(w, lo);
                break;
            }
            before += cost;
        }
    }
    __syncthreads();
    item.s = found[0];
    item.hh = found[1];
    item.i = found[2];
    item.a = found_a;
    item.ax = SeqAxis(w, load_seq(w.b, w.c, item.s, false));
    item.fill(w);
    return true;
}

// What a CTA leaves for the join: the item that starts in its interval and is
// cut at its end, if there is one, and which of its slots it filled.
struct Cut {
    int row0, nt;              // first row of q and tokens of that item
    int head0, heads;          // first query head and heads
    int last;                  // the CTA with the item's end; -1: no such item
    int has0, has1;
    int pad;
};

// Workspace: per CTA two slots, each `rows` rows of d float32 sums and the
// rows' (maximum, sum) pairs, in units of base-2 logits, and a Cut.
struct Slots {
    float* o;          // [n_cta * 2][rows][d]
    float2* ml;        // [n_cta * 2][rows]
    Cut* cut;          // [n_cta]
    int rows;
};

// Enter an item of CTA `me` (interval x0 .. x1, its steps b0 .. b1) into the
// CTA's Cut; the slot its part goes to, or -1 if all steps are here.
__device__ __forceinline__ int note_item(const Work& w, const Item& it, int me, long long x0, long long x1, long long chunk,
                                         int b0, int b1, Cut& cut) {
    const bool part = b0 < b1 && !(b0 == 0 && b1 == it.steps);
    const bool older = it.a < x0;
    if (older && part) cut.has0 = 1;
    if (!older && it.a + it.cost > x1) {
        const long long end = it.a + it.cost - 1;
        int last = (int)((double)end / (double)chunk);          // to within one
        if (chunk * (last + 1) <= end) ++last;
        if (chunk * last > end) --last;
        cut.row0 = it.ax.q.r0 + it.t0;
        cut.nt = it.nt;
        cut.head0 = it.hh / w.hs * w.G + it.hh % w.hs * w.gt;
        cut.heads = min(w.gt, w.G - it.hh % w.hs * w.gt);
        cut.last = last;
        cut.has1 = part;
    }
    return part ? me * 2 + (older ? 0 : 1) : -1;
}

// element offset of row r of an item in the packed [N, Hq, d] outputs, or -1
__device__ __forceinline__ long long out_row(const Work& w, const Item& it, int r, int d) {
    const int tok = r / w.gt, g = r - tok * w.gt;
    const int part = it.hh % w.hs, h = it.hh / w.hs;
    const int head = part * w.gt + g;
    if (tok >= it.nt || head >= w.G) return -1;
    return ((long long)(it.ax.q.r0 + it.t0 + tok) * (w.Hk * w.G) + h * w.G + head) * d;
}

// Joins the parts of the items that were cut, in the order of the CTAs: block
// x of the grid takes the item that was cut at the end of CTA x's interval, if
// it started there. A warp takes RW rows at once, a lane four columns of each;
// the parts' weights are computed by lanes in parallel, 32 parts at a time,
// and their rows added PB parts at a time, all their loads in flight. Bound by
// latency, and by reading the parts once: a chunk's item has two or three
// parts of up to 256 rows (RW 4, PB 2, four blocks to an SM: 4096 new tokens
// 87 -> 81 us against PB 4 and two blocks), a decode's up to one part per CTA
// of few rows (RW 1, PB 16). Several warps to a row were measured: 2 x 262144
// positions gain 2 us, 64 x 1000 lose 1 to 4 us to the larger grid.
constexpr int JOIN_WARPS = 8;
constexpr int MAX_PARTS = 1024;

template <typename T, int RW, int PB, int BLOCKS>
__global__ void __launch_bounds__(JOIN_WARPS * 32, BLOCKS)
attn_join_kernel(Slots sl, T* __restrict__ o, int Hq, int d, int gt) {
    __shared__ int part_slot[MAX_PARTS + PB];
    __shared__ int n_parts;
    pdl_wait();
    pdl_trigger();
    const int first = blockIdx.x;
    const Cut me = sl.cut[first];
    if (me.last <= first) return;
    const int rows = me.nt * gt;
    if ((int)blockIdx.y * JOIN_WARPS * RW >= rows) return;
    if (threadIdx.x < 32) {
        int n = 0;
        for (int k0 = first; k0 <= me.last; k0 += 32) {
            const int k = k0 + threadIdx.x;
            const bool on = k <= me.last && (k == first ? me.has1 : sl.cut[min(k, me.last)].has0);
            const unsigned m = __ballot_sync(0xffffffffu, on);
            if (on) part_slot[n + __popc(m & ((1u << threadIdx.x) - 1u))] = k * 2 + (k == first ? 1 : 0);
            n += __popc(m);
        }
        if (threadIdx.x == 0) n_parts = n;
    }
    __syncthreads();
    const int n = n_parts;
    if (n == 0) return;                  // one CTA had all steps after all, and wrote the rows
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r0 = (blockIdx.y * JOIN_WARPS + warp) * RW;
    const bool col = lane * 4 < d;
    const int rmax = min(rows, sl.rows) - 1;
    float M[RW], l[RW], acc[RW][4];
#pragma unroll
    for (int u = 0; u < RW; ++u) {
        M[u] = -INFINITY;
        l[u] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][e] = 0.f;
    }
    for (int k = lane; k < n; k += 32) {
#pragma unroll
        for (int u = 0; u < RW; ++u) M[u] = fmaxf(M[u], sl.ml[(long long)part_slot[k] * sl.rows + min(r0 + u, rmax)].x);
    }
#pragma unroll
    for (int u = 0; u < RW; ++u) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) M[u] = fmaxf(M[u], __shfl_xor_sync(0xffffffffu, M[u], m));
        if (M[u] == -INFINITY) M[u] = 0.f;
    }
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += 32) {
        float wt[RW];
#pragma unroll
        for (int u = 0; u < RW; ++u) {
            wt[u] = 0.f;
            if (k0 + lane < n) {
                const float2 ml = sl.ml[(long long)part_slot[k0 + lane] * sl.rows + min(r0 + u, rmax)];
                wt[u] = exp2f(ml.x - M[u]);
                l[u] += wt[u] * ml.y;
            }
        }
#pragma unroll 1
        for (int j = 0; j < min(32, n - k0); j += PB) {
            float4 v[PB][RW];
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int u = 0; u < RW; ++u) {
                    v[p][u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (col && k0 + j + p < n)
                        v[p][u] = *reinterpret_cast<const float4*>(
                            sl.o + ((long long)part_slot[k0 + j + p] * sl.rows + min(r0 + u, rmax)) * d + lane * 4);
                }
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int u = 0; u < RW; ++u) {
                    const float x = __shfl_sync(0xffffffffu, wt[u], j + p);
                    acc[u][0] = fmaf(x, v[p][u].x, acc[u][0]);
                    acc[u][1] = fmaf(x, v[p][u].y, acc[u][1]);
                    acc[u][2] = fmaf(x, v[p][u].z, acc[u][2]);
                    acc[u][3] = fmaf(x, v[p][u].w, acc[u][3]);
                }
        }
    }
#pragma unroll
    for (int u = 0; u < RW; ++u) l[u] = warp_sum(l[u]);
#pragma unroll
    for (int u = 0; u < RW; ++u) {
        const float inv = l[u] == 0.f ? 0.f : 1.f / l[u];
        const int r = r0 + u, tok = r / gt, g = r - tok * gt;
        if (r >= rows || g >= me.heads || !col) continue;
        T* dst = o + ((long long)(me.row0 + tok) * Hq + me.head0 + g) * d + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) Elem<T>::st(dst + e, acc[u][e] * inv);
    }
}

}  // namespace attn
}  // namespace jet
