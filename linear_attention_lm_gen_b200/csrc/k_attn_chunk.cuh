// Attention of a chunk of new tokens per sequence over a paged cache (bf16),
// on tcgen05: prompt pieces, and batches that mix them with decode tokens.
//
// An item is two tiles of 128 query rows (A and B) of one cache head; a row
// is (token, query head of the group), so all heads that share the cache head
// are in the same tile and read it once. Per step of 128 positions and tile:
//   S = Q K^T (fp32, TMEM); P = exp2(scale2 (S - m)) (bf16, over S in TMEM);
//   O += P V (fp32, TMEM, P as the TMEM operand).
// The matrix products of a step and tile take about 1024 tensor cycles, its
// 128 x 128 exponentials 1024 cycles of the SM's special-function unit, so
// the two tiles alternate: while one is in its softmax the other's products
// run. Neither unit is full: a step takes 3650 cycles, 56 % of either, since a
// tile's softmax (1930 cycles) and products follow one another through two
// hand-overs.
//
//   warps 0-3, 4-7  softmax of tile A, B: one thread per row, the row's 128
//                   scores in registers, no exchange between threads. The
//                   maximum m is kept until a score exceeds it by 8 binades
//                   (weights up to 2^8 are harmless in bf16 and float32), so O
//                   is rescaled, by the same threads, only then. They also
//                   write the item's results.
//   warp 8          one lane issues all products
//   warp 9          the TMA loads: the item's queries; K and V, one box per
//                   page (up to 128 rows) and lane, page indices a step ahead,
//                   through a ring of stages that runs ahead into the next item
//   warp 10         cleans V at the ends of the range (below)
//   warp 11         one lane walks the axis of the work and hands the items to
//                   the other roles through a queue of four, so that the walk's
//                   64-bit arithmetic exists once (inlined into every role it made
//                   the kernel 190 KB long, and each switch of items waited for
//                   instructions)
//
// Order of the products: S_A(0) S_B(0) | PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) ...
// S(j+1) overwrites P(j) in TMEM; products of one thread execute in order.
//
// A masked weight is exactly zero, but zero times a non-finite value is not.
// In steps where not every row sees every position, warp 10 zeroes the rows
// of V outside the item's range (stale memory) and every non-finite value,
// before the product reads the stage. If it found one inside the range, the
// rows that do see that value get it added when the results are written.
//
// Work is divided as k_attn_sched.cuh says, one CTA to an SM. 4096 new tokens
// over 28672 (12 heads over 2, d 128): 618 us in bursts of about 20 calls (1.25
// PFLOP/s), 716 us in a long run of calls (1.08), where the power limit lowers
// the clock; the products alone take 2050 of a step's cycles. 4096 over nothing
// 77 us, 512 over 2048 33 us: there the ends of items and the join weigh most.
#pragma once
#include <cuda.h>

#include "k_attn_decode.cuh"
#include "sm100.cuh"

namespace jet {
namespace attn {

using namespace sm100;

constexpr int CH_THREADS = 384, CH_KT = 128;
constexpr int CH_MMA = 256, CH_LOAD = 288, CH_FIX = 320, CH_WALK = 352;       // first threads of warps 8 to 11

template <int NB> struct ChSmem {                              // NB: 64-column blocks of d
    static constexpr int STAGES = NB == 2 ? 4 : 8;
    static constexpr uint32_t TILE = NB * 16384;
    static constexpr uint32_t Q = 0;                           // [2] tiles
    static constexpr uint32_t KV = Q + 2 * TILE;               // [STAGES] of K or V
    static constexpr uint32_t OUT = KV + STAGES * TILE;        // [8 warps] of 4 KB, results on their way out
    static constexpr uint32_t BAR = OUT + 8 * 4096;
    static constexpr uint32_t MISC = BAR + 384;
    static constexpr uint32_t ITEMS = MISC + 64;               // [4] of the item queue
    static constexpr uint32_t BYTES = ITEMS + 4 * 48;
    static_assert(BYTES <= 232448 - 1024, "shared memory budget (with the static part of block_locate)");
};

template <int NB> struct ChBar {
    static constexpr int ST = ChSmem<NB>::STAGES;
    static constexpr int FULL = 0, EMPTY = ST, FIX = 2 * ST, S = 3 * ST, P = S + 2, Q = P + 2, O = Q + 1, QE = O + 2, END = QE + 1, IF = END + 1, IE = IF + 4, N = IE + 4;
};

// D[tmem] (+)= A * B[smem], A in shared memory or in TMEM, where `one` holds.
// The lane is chosen inside the instruction, so that the code around it stays
// uniform and its addresses in uniform registers.
__device__ __forceinline__ void mma_ss_if(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
        :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t one, uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n"
        :: "r"(smem_u32(bar)), "r"(one) : "memory");
}
// 32 lanes x 16 columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// the largest of three
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, uint64_t* bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;        // suspends the thread for a while by itself
        if ((i & 15u) == 0) {
            if (*abort_flag) return false;
            if (global_ns() - t0 > limit_ns) break;
        }
    }
    *abort_flag = 1;
    flag_error(DEVERR_TIMEOUT);
    return false;
}
// Wait for a phase, bounded in time; false once any role gave up.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort_flag, kWaitLimitNs);
}

// What the roles need of an item, as the queue holds it.
struct ChItem {
    int s, hk, row0, nt;            // sequence, cache head, first row of q, tokens (-1: no more items)
    int lo, hi, b0, b1;             // positions, and the steps of this CTA (b0 == b1: rows that see nothing)
    int p_first, lo_all, lo_last;   // position of the first token, first positions of the first and the last token
    int slot;                       // workspace slot of the part, -1: all steps are here
    __device__ __forceinline__ bool partial(int step) const {      // not every row sees every position of the step
        const int k0 = lo + step * CH_KT;
        return k0 < lo_last || k0 + CH_KT > p_first + 1;
    }
};
constexpr int CH_QUEUE = 4;
constexpr int CH_READERS = 11;      // warps that read the queue: softmax, products, loads, V
// Arrivals that free a stage of the ring: its products' completion, and warp
// 10's once it has seen the stage. Its waits tell phases apart by parity only,
// so the ring must not run two phases ahead of it.
constexpr int CH_RELEASES = 2;

#ifdef JET_TEST_WAIT_EXPIRY
// test builds only: leave out the first scores of tile A, so that the wait for them runs out
__device__ int g_test_skip_scores;
#endif

template <int NB>
__global__ void __launch_bounds__(CH_THREADS, 1)
attn_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_q, const Work w, const Slots sl,
                  __nv_bfloat16* __restrict__ o, int d, float scale2) {
    typedef ChSmem<NB> SM;
    typedef ChBar<NB> B;
    constexpr int ST = SM::STAGES;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::BAR);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + SM::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + SM::MISC + 16);
    volatile int* odd_flag = reinterpret_cast<volatile int*>(sm + SM::MISC + 32);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(sm) & 1023u) {                           // whole CTA, before any barrier
        if (tid == 0) flag_error(DEVERR_DATA);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < B::N; ++i)
            mbar_init(&bars[i], i >= B::EMPTY && i < B::EMPTY + ST ? CH_RELEASES
                                : i >= B::P && i < B::P + 2        ? 4
                                : i >= B::IE && i < B::IE + 4      ? CH_READERS
                                                                   : 1);
        *abort_flag = 0;
        *odd_flag = 0;
        fence_mbar_init();
    }
    if (tid == CH_LOAD) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_q);
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    {   // the rows of a query tile behind its last token's heads: never loaded, zero
        const int idle = 128 - w.tpt / 2 * w.gt;
        for (int e = tid; e < 2 * NB * idle * 8; e += CH_THREADS) {
            const int blk = e / (idle * 8), rest = e - blk * idle * 8;
            *reinterpret_cast<uint4*>(sm + SM::Q + blk * 16384 + (128 - idle + rest / 8) * 128 + (rest & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot;
    pdl_wait();
    pdl_trigger();
    long long chunk, total;
    Item it;
    const bool inside = block_locate<CH_THREADS>(w, gridDim.x, blockIdx.x, chunk, total, it);
    const long long x0 = chunk * blockIdx.x, x1 = min(total, x0 + chunk);
    const int rows = w.tpt / 2 * w.gt;                    // query rows of a tile
    const int page = 1 << w.c.page_shift;

    uint32_t n_it = 0;                                    // items this role has taken
    ChItem im;
    // the next item of the queue: false at the end, or if a role gave up
    auto next_item = [&]() -> bool {
        const uint32_t k = n_it % CH_QUEUE;
        if (!__all_sync(0xffffffffu, wait_for(&bars[B::IF + k], n_it / CH_QUEUE & 1, abort_flag))) return false;
        im = *reinterpret_cast<const ChItem*>(sm + SM::ITEMS + k * sizeof(ChItem));
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B::IE + k]);
        ++n_it;
        return im.nt >= 0;
    };
    const int half = w.tpt / 2;                           // tokens of a tile

    if (!inside) {
        if (tid == 0) sl.cut[blockIdx.x] = Cut{0, 0, 0, 0, -1, 0, 0, 0};
    } else if (warp < 8) {
        // 256 x 200 + 128 x 96 registers of the 384 x 168 that the block starts with
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ------------------------------------------------------------ softmax, queries, results
        const int tile = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32;
        const uint32_t tS = taddr_of(tb, lanes, tile * 128), tO = taddr_of(tb, lanes, 256 + tile * 128);
        uint32_t nS = 0, nO = 0;
        bool ok = true;
        while (ok && next_item()) {
            const bool two = im.nt > half;
            if (tile == 1 && !two) continue;
            // row r of the tile: its token, its offset in the outputs (-1: none)
            const int tok = tile * half + r / w.gt;
            const long long dst = r < rows && tok < im.nt
                                      ? ((long long)(im.row0 + tok) * (w.Hk * w.G) + im.hk * w.G + r % w.gt) * d : -1;
            if (im.b0 == im.b1) {                         // every row sees nothing
                if (dst >= 0)
                    for (int e = 0; e < d; e += 8) *reinterpret_cast<uint4*>(o + dst + e) = make_uint4(0, 0, 0, 0);
                continue;
            }
            const int pos = im.p_first + min(tok, im.nt - 1), lo = first_key(pos, w.window);
            float m = -INFINITY, l = 0.f;
            for (int step = im.b0; step < im.b1; ++step, ++nS) {
                ok = __all_sync(0xffffffffu, wait_for(&bars[B::S + tile], nS & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int u = 0; u < 4; ++u) tmem_ld32(tS + u * 32, s + u * 32);
                tmem_ld_wait();
                if (im.partial(step)) {                  // columns outside bot .. top to -inf, by a bit mask of each 32
                    const int k0 = im.lo + step * CH_KT, top = pos - k0, bot = lo - k0;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int a = min(32, max(0, bot - u * 32)), b = min(32, max(0, top + 1 - u * 32));
                        const uint32_t seen = (uint32_t)((1ull << b) - 1) & ~(uint32_t)((1ull << a) - 1);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(seen & (1u << c))) s[u * 32 + c] = 0xff800000u;
                    }
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(s[c]);
#pragma unroll
                for (int c = 4; c < 124; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = max3(mx[e], __uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e]));
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(s[124 + e]));
                const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                if (step == im.b0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, (top - m) * scale2 > 8.f)) {
                    // S(step) is complete, so PV(step - 1), issued before it, is too
                    const float mn = fmaxf(m, top);
                    const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * scale2);
                    m = mn;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < d; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(tO + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                        tmem_st16(tO + c, v);
                    }
                }
                const float base = m == -INFINITY ? 0.f : m * scale2;
                const uint64_t sc2 = pair(scale2, scale2), nb2 = pair(-base, -base);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint64_t x = fma2(pair(__uint_as_float(s[u * 32 + 2 * c]), __uint_as_float(s[u * 32 + 2 * c + 1])),
                                                sc2, nb2);
                        float a, b;
                        unpair(x, a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[c & 3] = add2(sum[c & 3], pair(a, b));
                        pk[c] = Vec16<__nv_bfloat16>::pack2(a, b);
                    }
                    tmem_st16(tS + u * 16, pk);
                }
                {
                    float a, b;
                    unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
                    l += a + b;
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B::P + tile]);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait_for(&bars[B::O + tile], nO & 1, abort_flag));
            if (!ok) break;
            ++nO;
            tc_fence_after();
            const bool whole = im.slot < 0;
            const long long srow = (long long)im.slot * sl.rows + tile * rows + r;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (*odd_flag) {
                // values that were cleaned out of V: a row gets the non-finite ones that it sees
#pragma unroll 1
                for (int c = 0; c < d; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tO + c, v);
                    tmem_ld_wait();
                    for (int step = im.b0; step < im.b1 && dst >= 0; ++step) {
                        if (!im.partial(step)) continue;
                        const int k0 = im.lo + step * CH_KT;
                        for (int j = max(k0, lo); j < min(k0 + CH_KT, pos + 1); ++j) {
                            const int pg = load_page(w.c, im.s, j);
                            if (pg < 0) continue;
                            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(w.c.v) + pg * w.c.page_stride +
                                                       im.hk * w.c.head_stride + (j & (page - 1)) * w.c.row_stride + c;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float x = __bfloat162float(src[e]);
                                if (!(fabsf(x) < INFINITY)) v[e] = __float_as_uint(__uint_as_float(v[e]) + x);
                            }
                        }
                    }
                    __syncwarp();
                    tmem_st16(tO + c, v);
                    tmem_st_wait();
                }
            }
            // 32 columns at a time: rows to shared memory, then out with consecutive lanes on a row
            uint8_t* stage = sm + SM::OUT + warp * 4096;
            const long long out = whole ? dst : dst < 0 ? -1 : srow * d;
#pragma unroll 1
            for (int c = 0; c < d; c += 32) {
                float v[32];
                tmem_ld32(tO + c, reinterpret_cast<uint32_t*>(v));
                tmem_ld_wait();
                const int nc = min(32, d - c);
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[e * 8 + k] *= inv;
                        *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ (lane >> 1 & 3)) << 4)) =
                            Vec16<__nv_bfloat16>::pack(v + e * 8);
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = k * 8 + (lane >> 2), ch = lane & 3;
                        const long long to = __shfl_sync(0xffffffffu, out, row);
                        const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 64 + ((ch ^ (row >> 1 & 3)) << 4));
                        if (to >= 0 && ch * 8 < nc) *reinterpret_cast<uint4*>(o + to + c + ch * 8) = x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                            make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = k * 4 + (lane >> 3), ch = lane & 7;
                        const long long to = __shfl_sync(0xffffffffu, out, row);
                        const float4 x = *reinterpret_cast<const float4*>(stage + row * 128 + ((ch ^ (row & 7)) << 4));
                        if (to >= 0 && ch * 4 < nc) *reinterpret_cast<float4*>(sl.o + to + c + ch * 4) = x;
                    }
                }
                __syncwarp();
            }
            if (!whole && dst >= 0) sl.ml[srow] = make_float2(m * scale2, l);
            // the loads of O above are complete (waited for); the next item's products may
            // overwrite it once this thread has let them
            tc_fence_before();
        }
        if (!ok) *abort_flag = 1;
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == CH_MMA / 32) {
        // ------------------------------------------------------------ products: the warp waits as one, one
        // elected lane issues
        const uint32_t id_s = idesc_bf16(128, 128, false, false), id_o = idesc_bf16(128, d, false, true);
        const uint64_t dQ = sw128_desc(smem_u32(sm + SM::Q), 16, 1024);
        const uint64_t dK = sw128_desc(smem_u32(sm + SM::KV), 16, 1024);
        const uint64_t dV = sw128_desc(smem_u32(sm + SM::KV), 16384, 1024);
        const int ks = d >> 4;
        const uint32_t one = elect_one();
        // ring position (stage, phase) of the next K or V, and the phases of the other barriers
        uint32_t slot = 0, ph = 0, fix = 0, phQ = 0, phP[2] = {0, 0};
        bool ok = true;
        auto wait = [&](int bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, wait_for(&bars[bar], parity, abort_flag));
            return ok;
        };
        auto advance = [&]() {
            if (++slot == ST) { slot = 0; ph ^= 1; }
        };
        auto issue_s = [&](int tile, uint32_t sl_) {
            const uint64_t a = dQ + (tile * SM::TILE >> 4), b = dK + (sl_ * SM::TILE >> 4);
#pragma unroll
            for (int k = 0; k < NB * 4; ++k)
                if (k < ks) {
                    const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                    mma_ss_if(one, tb + tile * 128, a + off, b + off, id_s, k > 0);
                }
            commit_if(one, &bars[B::S + tile]);
        };
        auto issue_o = [&](int tile, uint32_t sl_, bool fresh) {
            const uint64_t b = dV + (sl_ * SM::TILE >> 4);
#pragma unroll
            for (int k = 0; k < CH_KT / 16; ++k)
                mma_ts_if(one, tb + 256 + tile * 128, tb + tile * 128 + k * 8, b + (k * 2048 >> 4), id_o, !fresh || k > 0);
        };
        auto release = [&](uint32_t bar) { commit_if(one, &bars[bar]); };
        while (ok && next_item()) {
            if (im.b0 == im.b1) continue;
            const bool two = im.nt > half;
            if (!wait(B::FULL + slot, ph)) break;
            if (!wait(B::Q, phQ)) break;
            phQ ^= 1;
            tc_fence_after();
#ifdef JET_TEST_WAIT_EXPIRY
            if (!*reinterpret_cast<volatile int*>(&g_test_skip_scores))
#endif
            issue_s(0, slot);
            if (two) issue_s(1, slot);
            release(B::EMPTY + slot);
            if (im.b0 + 1 == im.b1) release(B::QE);
            advance();
            for (int step = im.b0; step < im.b1 && ok; ++step) {
                const bool more = step + 1 < im.b1, fresh = step == im.b0;
                const uint32_t vs = slot;
                wait(B::FULL + vs, ph);
                if (im.partial(step)) {
                    wait(B::FIX + vs, fix >> vs & 1);
                    fix ^= 1u << vs;
                }
                advance();
                if (more) wait(B::FULL + slot, ph);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if ((i == 1 && !two) || !wait(B::P + i, phP[i])) break;
                    phP[i] ^= 1;
                    tc_fence_after();
                    issue_o(i, vs, fresh);
                    if (more) issue_s(i, slot);
                    else release(B::O + i);
                    if (i == 1 || !two) {
                        release(B::EMPTY + vs);
                        if (more) release(B::EMPTY + slot);
                        if (step + 2 == im.b1) release(B::QE);      // the item's last scores: its queries are done
                    }
                }
                if (more) advance();
            }
        }
        if (!ok) *abort_flag = 1;
        // every product has completed before the CTA frees its memory
        if (one) {
            mma_commit(&bars[B::END]);
            mbar_wait(&bars[B::END], 0);
        }
    } else if (warp == CH_LOAD / 32) {
        // ------------------------------------------------------------ loads: lane e issues box e of a step
        uint32_t kv = 0, nQ = 0;
        bool ok = true;
        const int box = min(page, CH_KT);
        while (ok && next_item()) {
            if (im.b0 == im.b1) continue;
            // this lane's page of a step, or -1: no positions of the range in its box
            auto fetch = [&](int step) -> int {
                const int k0 = im.lo + step * CH_KT, p = k0 + lane * box;
                if (step >= im.b1 || lane * box >= CH_KT || p >= im.hi || p + box <= im.lo_all) return -1;
                const int pg = load_page(w.c, im.s, p);
                return pg < 0 ? w.c.n_pages : pg;                 // a bad index: behind the pool, reads zeros
            };
            int pg = fetch(im.b0);
            // the item's queries, once the last item's scores are complete
            if (lane == 0) {
                if (nQ > 0) ok = wait_for(&bars[B::QE], (nQ - 1) & 1, abort_flag);
                if (ok) {
                    const bool two = im.nt > half;
                    mbar_expect_tx(&bars[B::Q], (uint32_t)(two ? 2 : 1) * NB * rows * 128);
                    for (int e = 0; e < (two ? 2 : 1) * NB; ++e)
                        tma_load_3d(sm + SM::Q + e * 16384, &tm_q, &bars[B::Q], e % NB * 64, im.hk * w.G,
                                    im.row0 + e / NB * half);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++nQ;
            for (int step = im.b0; step < im.b1 && ok; ++step) {
                const int next = fetch(step + 1);
                const int p = im.lo + step * CH_KT + lane * box;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, pg >= 0)) * box * 128 * NB;
                for (int v = 0; v < 2; ++v, ++kv) {
                    const uint32_t slot = kv % ST;
                    uint64_t* bar = &bars[B::FULL + slot];
                    if (lane == 0) {
                        if (kv >= ST) ok = wait_for(&bars[B::EMPTY + slot], (kv / ST - 1) & 1, abort_flag);
                        if (ok) mbar_expect_tx(bar, bytes);
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* dst = sm + SM::KV + slot * SM::TILE + lane * box * 128;
                    if (pg >= 0)
#pragma unroll
                        for (int c = 0; c < NB; ++c)
                            tma_load_4d(dst + c * 16384, v ? &tm_v : &tm_k, bar, c * 64, p & (page - 1), im.hk, pg);
                }
                pg = next;
            }
        }
        if (!ok) *abort_flag = 1;
        // every issued load has landed before the CTA frees its memory
        if (lane == 0 && nQ > 0) mbar_wait(&bars[B::Q], (nQ - 1) & 1);
        if (lane == 0)
            for (uint32_t i = kv > ST ? kv - ST : 0; i < kv; ++i) mbar_wait(&bars[B::FULL + i % ST], (i / ST) & 1);
    } else if (tid >= CH_FIX && tid < CH_FIX + 32) {
        // ------------------------------------------------------------ V at the ends of the range
        uint32_t kv = 0;
        bool ok = true;
        while (ok && next_item()) {
            if (im.b0 == im.b1) continue;
            for (int step = im.b0; step < im.b1 && ok; ++step, kv += 2) {
                // every stage in its turn: a wait that skipped one could take an older phase for its own
                const uint32_t vi = kv + 1, slot = vi % ST;
                ok = wait_for(&bars[B::FULL + kv % ST], (kv / ST) & 1, abort_flag) &&
                     wait_for(&bars[B::FULL + slot], (vi / ST) & 1, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive(&bars[B::EMPTY + kv % ST]);
                if (!im.partial(step)) {
                    if (lane == 0) mbar_arrive(&bars[B::EMPTY + slot]);
                    continue;
                }
                const int k0 = im.lo + step * CH_KT;
                uint8_t* V = sm + SM::KV + slot * SM::TILE;
                // rows outside the range to zero
                const int ra = max(0, im.lo_all - k0), rb = min(CH_KT, im.hi - k0);
#pragma unroll 1
                for (int row = lane >> 3; row < CH_KT; row += 4)
                    if (row < ra || row >= rb)
#pragma unroll
                        for (int c = 0; c < NB; ++c)
                            *reinterpret_cast<uint4*>(V + c * 16384 + row * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                __syncwarp();
                // then all looked at: a magnitude of 0x7f80 and up is not finite
                uint32_t top = 0;
                if (im.nt > 1) {
#pragma unroll 8
                    for (int u = 0; u < NB * 32; ++u) {
                        const uint4 x = *reinterpret_cast<const uint4*>(V + u * 512 + lane * 16);
                        top = __vimax3_u16x2(top, x.x & 0x7fff7fffu, x.y & 0x7fff7fffu);
                        top = __vimax3_u16x2(top, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu);
                    }
                }
                const bool odd = (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u;
                if (odd) {
#pragma unroll 1
                    for (int u = 0; u < NB * 32 * 8; ++u) {
                        uint16_t* at = reinterpret_cast<uint16_t*>(V + (u >> 3) * 512 + lane * 16) + (u & 7);
                        if ((*at & 0x7fffu) >= 0x7f80u) *at = 0;
                    }
                }
                if (odd) *odd_flag = 1;
                __threadfence_block();
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[B::FIX + slot]);
                    mbar_arrive(&bars[B::EMPTY + slot]);
                }
            }
        }
        if (!ok) *abort_flag = 1;
    } else if (tid == CH_WALK) {
        // ------------------------------------------------------------ the walk along the axis
        Cut cut{0, 0, 0, 0, -1, 0, 0, 0};
        bool ok = true, more = true;
        while (more && ok) {
            const uint32_t k = n_it % CH_QUEUE;
            more = it.s < w.b.nseq && it.a < x1;
            bool mine = true;
            im.nt = -1;
            if (more) {
                const int b0 = it.step_at(x0), b1 = it.step_at(x1);
                mine = it.steps == 0 ? it.a >= x0 : b0 < b1;
                im = ChItem{it.s, it.hh, it.ax.q.r0 + it.t0, it.nt, it.lo, it.hi, b0, b1, it.p_first,
                            first_key(it.p_first, w.window), first_key(it.hi - 1, w.window),
                            note_item(w, it, blockIdx.x, x0, x1, chunk, b0, b1, cut)};
            }
            if (mine) {
                // the others may be at work on one long item all the while: a longer limit, and their own ends it too
                if (n_it >= CH_QUEUE)
                    ok = wait_on(&bars[B::IE + k], (n_it / CH_QUEUE - 1) & 1, abort_flag, 64 * kWaitLimitNs);
                if (!ok) break;
                *reinterpret_cast<ChItem*>(sm + SM::ITEMS + k * sizeof(ChItem)) = im;
                mbar_arrive(&bars[B::IF + k]);
                ++n_it;
            }
            if (more) it.next(w);
        }
        sl.cut[blockIdx.x] = cut;
    }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tb, 512);
}

}  // namespace attn
}  // namespace jet
