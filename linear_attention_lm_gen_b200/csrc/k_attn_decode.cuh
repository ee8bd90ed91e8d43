// Attention of few query rows per cache head over a paged cache (bf16): the
// decode step of a serving batch, one token or a few per sequence.
//
// Bound by reading the cache once (4 d Hk bytes per position and sequence,
// against 4 d Hq operations: 6 operations a byte at the 2B shape's 12 heads
// over 2), so the products need only keep up with HBM and the G heads that
// share a cache head form the rows of one 16-row tile, as m16n8k16 products
// take them. A CTA has four warps. Each warp takes 16 of every 64 positions
// on its own: a private ring of stages filled with 16-byte asynchronous
// copies, its own running maximum, sum and output tile, no block barrier
// until the item ends, when the four are joined through shared memory. A
// stage lies in one page, so each costs a warp one page-table entry, read a
// step ahead. Work is divided as k_attn_sched.cuh says: two CTAs to an SM.
// 256 sequences of up to 8192 positions (1.04 GB): 169 us, 6.2 TB/s, 94% of the
// copy rate; one CTA with six stages 225 us, three with two stages 168 us.
//
// Positions outside the item's range are filled with zeros, never read. The
// weights are rounded to bf16 for the second product (the type the tensor
// cores take): half a step of each weight, on the order of the rounding of
// the result itself; sums and maxima stay float32. A masked weight is zero,
// and zero times a non-finite value would reach the row all the same: where
// rows of a tile see different positions, the step's values are looked at and
// a non-finite one sends the step through scalar code that leaves masked
// values out.
#pragma once
#include "k_attn_sched.cuh"

namespace jet {
namespace attn {

constexpr int DEC_ROWS = 16, DEC_WARPS = 4, DEC_THREADS = DEC_WARPS * 32, DEC_KT = 64, DEC_KEYS = 16;

template <int DP> struct DecCfg {                       // DP: d rounded up to 64 or 128
    static constexpr int ROW = DP * 2;                  // bytes of a row in shared memory
    static constexpr int TILE = DEC_KEYS * ROW;         // K or V of one stage
    static constexpr int STAGES = DP == 64 ? 4 : 3;
    static constexpr int CTAS = DP == 64 ? 3 : 2;       // per SM
    static constexpr int SMEM = DEC_WARPS * STAGES * 2 * TILE;
};

__device__ __forceinline__ uint32_t dec_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// any non-finite bf16 among the two of w
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int DP>
__global__ void __launch_bounds__(DEC_THREADS, DecCfg<DP>::CTAS)
attn_decode_kernel(const __nv_bfloat16* __restrict__ q, long long q_stride, Work w, Slots sl,
                   __nv_bfloat16* __restrict__ o, int d, float scale2) {
    typedef DecCfg<DP> C;
    constexpr int KS = DP / 16, NT = DP / 8;            // k-steps of the first product, column tiles of the second
    constexpr int ST = C::STAGES;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    unsigned char* ring = smem + warp * (ST * 2 * C::TILE);
    const uint32_t ring_a = dec_smem(ring);
    pdl_wait();
    pdl_trigger();
    long long chunk, total;
    Item it;
    Cut cut{0, 0, 0, 0, -1, 0, 0, 0};
    if (!block_locate<DEC_THREADS>(w, gridDim.x, blockIdx.x, chunk, total, it)) {
        if (tid == 0) sl.cut[blockIdx.x] = cut;
        return;
    }
    const long long x0 = chunk * blockIdx.x, x1 = min(total, x0 + chunk);
    const unsigned char* kp = static_cast<const unsigned char*>(w.c.k);
    const unsigned char* vp = static_cast<const unsigned char*>(w.c.v);
    const int page_mask = (1 << w.c.page_shift) - 1;

    for (; it.s < w.b.nseq && it.a < x1; it.next(w)) {
        const int b0 = it.step_at(x0), b1 = it.step_at(x1);
        const int slot = note_item(w, it, blockIdx.x, x0, x1, chunk, b0, b1, cut);
        if (it.steps == 0) {                            // every row sees nothing: the CTA with the item's start
            if (it.a >= x0)
                for (int r = warp; r < DEC_ROWS; r += DEC_WARPS) {
                    const long long dst = out_row(w, it, r, d);
                    if (dst >= 0)
                        for (int e = lane; e < d; e += 32) o[dst + e] = __float2bfloat16_rn(0.f);
                }
            continue;
        }
        if (b0 >= b1) continue;
        const int hk = it.hh / w.hs;
        const long long head_off = hk * w.c.head_stride;
        const int p_first = it.p_first;
        const int lo_all = first_key(p_first, w.window);
        const int lo_last = first_key(it.hi - 1, w.window);       // the last token's first position
        auto page_of = [&](int step) -> int {           // -1 behind the part, or for a bad index
            const int p = it.lo + step * DEC_KT + warp * DEC_KEYS;
            if (step >= b1 || p >= it.hi || p + DEC_KEYS <= lo_all) return -1;
            return load_page(w.c, it.s, p);
        };
        auto issue = [&](int step, int pg) {            // fill the stage of `step`; always one copy group
            if (step < b1) {
                const int p = it.lo + step * DEC_KT + warp * DEC_KEYS;
                const uint32_t st = ring_a + (step % ST) * (2 * C::TILE);
                const long long base = pg < 0 ? 0 : pg * w.c.page_stride + head_off + (p & page_mask) * w.c.row_stride;
#pragma unroll
                for (int u = 0; u < DEC_KEYS * (C::ROW / 16) / 32; ++u) {
                    const int e = u * 32 + lane, row = e / (C::ROW / 16), ch = e % (C::ROW / 16);
                    const bool on = pg >= 0 && p + row < it.hi && p + row >= lo_all && ch * 8 < d;
                    const long long off = on ? (base + row * w.c.row_stride + ch * 8) * 2 : 0;
                    const uint32_t dst = st + row * C::ROW + ((ch ^ (row & 7)) << 4);
                    cp16(dst, kp + off, on);
                    cp16(dst + C::TILE, vp + off, on);
                }
            }
            cp_commit();
        };
        int pg = page_of(b0);
#pragma unroll
        for (int u = 0; u < ST - 1; ++u) {
            const int nx = page_of(b0 + u + 1);
            issue(b0 + u, pg);
            pg = nx;
        }
        // the tile's queries as product fragments: rows g and g + 8
        uint32_t qf[KS][4];
        int prow[2];                                    // the rows' positions
        {
            const int h = hk * w.G + (it.hh % w.hs) * w.gt;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = g + 8 * half, tok = r / w.gt, hd = r - tok * w.gt;
                const bool on = tok < it.nt && (it.hh % w.hs) * w.gt + hd < w.G;
                prow[half] = p_first + min(tok, it.nt - 1);
                const __nv_bfloat16* src = q + (it.ax.q.r0 + it.t0 + tok) * q_stride + (long long)(h + hd) * d;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int col = k * 16 + c * 8 + 2 * t;
                        qf[k][half + 2 * c] = on && col < d ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
                    }
            }
        }
        float acc[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;

        for (int step = b0; step < b1; ++step) {
            const int nx = page_of(step + ST);
            cp_wait<ST - 2>();
            __syncwarp();
            issue(step + ST - 1, pg);
            pg = nx;
            const int p = it.lo + step * DEC_KT + warp * DEC_KEYS;
            if (p >= it.hi || p + DEC_KEYS <= lo_all) continue;
            const uint32_t kt = ring_a + (step % ST) * (2 * C::TILE), vt = kt + C::TILE;
            // scores of 16 rows and 16 positions
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                // matrices: positions 0-7 / 8-15, columns 16k .. +7 / +8 .. +15
                const int row = (lane & 7) + ((lane >> 4) << 3), ch = 2 * k + ((lane >> 3) & 1);
                uint32_t b[4];
                ldsm4(b, kt + row * C::ROW + ((ch ^ (row & 7)) << 4));
                mma16816(s[0], qf[k], b[0], b[1]);
                mma16816(s[1], qf[k], b[2], b[3]);
            }
            const bool partial = p < lo_last || p + DEC_KEYS > p_first + 1;
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y = s[n][e] * scale2;
                    if (partial) {
                        const int j = p + n * 8 + 2 * t + (e & 1), pr = prow[e >> 1];
                        if (j > pr || j < first_key(pr, w.window)) y = -INFINITY;
                    }
                    s[n][e] = y;
                    mx[e >> 1] = fmaxf(mx[e >> 1], y);
                }
            bool moved = false;
            float base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                moved |= mx[h] > m[h];
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mn = fmaxf(m[h], mx[h]);
                    const float r = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
                    m[h] = mn;
                    l[h] *= r;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[n][2 * h] *= r;
                        acc[n][2 * h + 1] *= r;
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) base[h] = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = ex2(s[n][e] - base[e >> 1]);
                    l[e >> 1] += s[n][e];
                }
            bool odd = false;
            if (partial && it.nt > 1) {
#pragma unroll
                for (int u = 0; u < C::TILE / 512; ++u) {
                    const uint4 v = *reinterpret_cast<const uint4*>(ring + (vt - ring_a) + (u * 32 + lane) * 16);
                    odd |= nonfinite2(v.x) || nonfinite2(v.y) || nonfinite2(v.z) || nonfinite2(v.w);
                }
            }
            if (__any_sync(0xffffffffu, odd)) {
                for (int j = 0; j < DEC_KEYS; ++j) {
                    const int from = (lane & ~3) | ((j & 7) >> 1);
                    const float a0 = j < 8 ? s[0][0] : s[1][0], a1 = j < 8 ? s[0][1] : s[1][1];
                    const float c0 = j < 8 ? s[0][2] : s[1][2], c1 = j < 8 ? s[0][3] : s[1][3];
                    const float w0 = __shfl_sync(0xffffffffu, j & 1 ? a1 : a0, from);
                    const float w1 = __shfl_sync(0xffffffffu, j & 1 ? c1 : c0, from);
                    const int at = p + j;
                    const bool on0 = at <= prow[0] && at >= first_key(prow[0], w.window);
                    const bool on1 = at <= prow[1] && at >= first_key(prow[1], w.window);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t v = *reinterpret_cast<const uint32_t*>(
                            ring + (vt - ring_a) + j * C::ROW + ((n ^ (j & 7)) << 4) + t * 4);
                        const float v0 = __uint_as_float(v << 16), v1 = __uint_as_float(v & 0xffff0000u);
                        if (on0) { acc[n][0] = fmaf(w0, v0, acc[n][0]); acc[n][1] = fmaf(w0, v1, acc[n][1]); }
                        if (on1) { acc[n][2] = fmaf(w1, v0, acc[n][2]); acc[n][3] = fmaf(w1, v1, acc[n][3]); }
                    }
                }
                continue;
            }
            uint32_t pf[4];
            pf[0] = Vec16<__nv_bfloat16>::pack2(s[0][0], s[0][1]);
            pf[1] = Vec16<__nv_bfloat16>::pack2(s[0][2], s[0][3]);
            pf[2] = Vec16<__nv_bfloat16>::pack2(s[1][0], s[1][1]);
            pf[3] = Vec16<__nv_bfloat16>::pack2(s[1][2], s[1][3]);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                // transposed matrices: positions 0-7 / 8-15, columns 8n .. +7 / +8 .. +15
                const int row = (lane & 7) + (((lane >> 3) & 1) << 3), ch = n + (lane >> 4);
                uint32_t b[4];
                ldsm4t(b, vt + row * C::ROW + ((ch ^ (row & 7)) << 4));
                mma16816(acc[n], pf, b[0], b[1]);
                mma16816(acc[n + 1], pf, b[2], b[3]);
            }
        }
        cp_wait<0>();
        __syncwarp();
        // the four warps' parts: sums in the warp's own ring, [16][DP + 4] floats, then maximum and sum
        constexpr int LD = DP + 4;
        float* wo = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (t == 0) {
                wo[DEC_ROWS * LD + 2 * (g + 8 * h)] = m[h];
                wo[DEC_ROWS * LD + 2 * (g + 8 * h) + 1] = l[h];
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float2*>(wo + (g + 8 * h) * LD + n * 8 + 2 * t) =
                    make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
        }
        __syncthreads();
        {
            const bool whole = slot < 0;
            const int r = tid / 8, c8 = tid % 8;                    // 16 rows, 8 lanes each
            const long long dst = out_row(w, it, r, d);
            if (dst >= 0) {
                float M = -INFINITY, ww[DEC_WARPS], L = 0.f;
#pragma unroll
                for (int k = 0; k < DEC_WARPS; ++k)
                    M = fmaxf(M, reinterpret_cast<const float*>(smem + k * (ST * 2 * C::TILE))[DEC_ROWS * LD + 2 * r]);
                const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int k = 0; k < DEC_WARPS; ++k) {
                    const float* f = reinterpret_cast<const float*>(smem + k * (ST * 2 * C::TILE)) + DEC_ROWS * LD + 2 * r;
                    ww[k] = ex2(f[0] - base);
                    L += ww[k] * f[1];
                }
                const float inv = L == 0.f ? 0.f : 1.f / L;
                for (int c = c8 * 8; c < d; c += 64) {
                    float v[8] = {};
#pragma unroll
                    for (int k = 0; k < DEC_WARPS; ++k) {
                        const float* f = reinterpret_cast<const float*>(smem + k * (ST * 2 * C::TILE)) + r * LD + c;
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = fmaf(ww[k], f[e], v[e]);
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] *= inv;
                        *reinterpret_cast<uint4*>(o + dst + c) = Vec16<__nv_bfloat16>::pack(v);
                    } else {
                        float4* to = reinterpret_cast<float4*>(sl.o + ((long long)slot * sl.rows + r) * d + c);
                        to[0] = make_float4(v[0], v[1], v[2], v[3]);
                        to[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                }
                if (!whole && c8 == 0) sl.ml[(long long)slot * sl.rows + r] = make_float2(M, L);
            }
        }
        __syncthreads();
    }
    if (tid == 0) sl.cut[blockIdx.x] = cut;
}

}  // namespace attn
}  // namespace jet
