// Attention over a paged cache in float32, on the CUDA cores.
//
// An item is 32 query rows of one cache head (tokens times the heads that
// share it); a step is 64 positions, copied asynchronously into padded rows
// of shared memory: the next K while the values are summed, the next V while
// the next scores are computed. A thread computes 4 x 4 scores and holds 4
// rows x 4 or 8 columns of the result; a row's 16 threads are half a warp, so the
// running maximum and sum need four shuffles. A product is 64 fused
// multiply-adds for every 8 loads of 16 bytes, which broadcast within a warp:
// bound by the multiply-adds, those of masked positions and empty rows
// included. 3 sequences of 100 to 333 new tokens 40 us (as packed pairs 43 us)
// where the visible positions alone are 7.3 us of multiply-adds; 512 new tokens
// over 2048 (12 heads over 2, d 128) 279 us of 101. The tile is the same for a
// decode token, whose few rows leave most of it empty: 64 x 4000 positions 288
// us where the bytes are 80. Work is divided as k_attn_sched.cuh says, four
// CTAs to an SM for d <= 64 and two above.
//
// Positions outside the item's range are zero-filled, never read. A masked
// weight is stored as -1 and left out of the sum by a test (only in steps
// where rows see different positions), so a non-finite value reaches exactly
// the rows that see it.
#pragma once
#include "k_attn_decode.cuh"

namespace jet {
namespace attn {

constexpr int F32_ROWS = 32, F32_KT = 64, F32_THREADS = 128;

template <int DP> struct F32Cfg {                       // DP: d rounded up to 64 or 128
    static constexpr int CTAS = DP == 64 ? 4 : 2;       // per SM
    static constexpr int LD = DP + 4, PLD = F32_KT + 4;
    static constexpr int SMEM = 4 * (F32_ROWS * LD + 2 * F32_KT * LD + F32_ROWS * PLD) + 8 * 2 * F32_KT;
};

template <int DP>
__global__ void __launch_bounds__(F32_THREADS, F32Cfg<DP>::CTAS)
attn_f32_kernel(const float* __restrict__ q, long long q_stride, Work w, Slots sl, float* __restrict__ o, int d,
                float scale2) {
    constexpr int F32_LD = F32Cfg<DP>::LD, F32_PLD = F32Cfg<DP>::PLD, NC = DP / 64, CH = DP / 4;
    extern __shared__ __align__(128) float sf[];
    float* Q = sf;
    float* K = Q + F32_ROWS * F32_LD;
    float* V = K + F32_KT * F32_LD;
    float* P = V + F32_KT * F32_LD;
    long long* offs = reinterpret_cast<long long*>(P + F32_ROWS * F32_PLD);     // [2][64] offsets of the steps' rows
    const int tid = threadIdx.x, kt = tid & 15, rt = tid >> 4;          // keys kt + 16 i, rows 4 rt + i
    pdl_wait();
    pdl_trigger();
    long long chunk, total;
    Item it;
    Cut cut{0, 0, 0, 0, -1, 0, 0, 0};
    if (!block_locate<F32_THREADS>(w, gridDim.x, blockIdx.x, chunk, total, it)) {
        if (tid == 0) sl.cut[blockIdx.x] = cut;
        return;
    }
    const long long x0 = chunk * blockIdx.x, x1 = min(total, x0 + chunk);
    const float* kp = static_cast<const float*>(w.c.k);
    const float* vp = static_cast<const float*>(w.c.v);
    const int page_mask = (1 << w.c.page_shift) - 1, per = d >> 2;

    for (; it.s < w.b.nseq && it.a < x1; it.next(w)) {
        const int b0 = it.step_at(x0), b1 = it.step_at(x1);
        const int slot = note_item(w, it, blockIdx.x, x0, x1, chunk, b0, b1, cut);
        if (it.steps == 0) {                            // every row sees nothing
            if (it.a >= x0)
                for (int r = rt; r < F32_ROWS; r += F32_THREADS / 16) {
                    const long long dst = out_row(w, it, r, d);
                    if (dst >= 0)
                        for (int e = kt; e < d; e += 16) o[dst + e] = 0.f;
                }
            continue;
        }
        if (b0 >= b1) continue;
        const int hk = it.hh / w.hs;
        const int lo_all = first_key(it.p_first, w.window), lo_last = first_key(it.hi - 1, w.window);
        // offset of row `tid` of a step, -1 outside the range
        auto find = [&](int step) {
            if (tid < F32_KT) {
                const int p = it.lo + step * F32_KT + tid;
                long long off = -1;
                if (step < b1 && p >= lo_all && p < it.hi) {
                    const int pg = load_page(w.c, it.s, p);
                    if (pg >= 0) off = pg * w.c.page_stride + hk * w.c.head_stride + (p & page_mask) * w.c.row_stride;
                }
                offs[(step & 1) * F32_KT + tid] = off;
            }
        };
        auto fetch = [&](const float* src, float* to, int step) {      // one copy group, by all threads
            if (step < b1)
                for (int e = tid; e < F32_KT * CH; e += F32_THREADS) {
                    const int row = e / CH, ch = e % CH;
                    if (ch >= per) continue;
                    const long long off = offs[(step & 1) * F32_KT + row];
                    cp16(dec_smem(to + row * F32_LD + ch * 4), src + (off < 0 ? 0 : off + ch * 4), off >= 0);
                }
            cp_commit();
        };
        find(b0);
        for (int e = tid; e < F32_ROWS * CH; e += F32_THREADS) {
            const int row = e / CH, ch = e % CH, tok = row / w.gt, hd = row - tok * w.gt;
            if (ch >= per) continue;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (tok < it.nt && it.hh % w.hs * w.gt + hd < w.G)
                v = *reinterpret_cast<const float4*>(q + (it.ax.q.r0 + it.t0 + tok) * q_stride +
                                                     (long long)(hk * w.G + it.hh % w.hs * w.gt + hd) * d + ch * 4);
            *reinterpret_cast<float4*>(Q + row * F32_LD + ch * 4) = v;
        }
        int pos[4];
        float m[4], l[4], acc[4][4 * NC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pos[i] = it.p_first + min((rt * 4 + i) / w.gt, it.nt - 1);
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < 4 * NC; ++c) acc[i][c] = 0.f;
        }
        __syncthreads();
        fetch(kp, K, b0);
        fetch(vp, V, b0);
        for (int step = b0; step < b1; ++step) {
            const int k0 = it.lo + step * F32_KT;
            find(step + 1);
            cp_wait<1>();                               // K of this step
            __syncthreads();
            float s[4][4] = {};
#pragma unroll 4
            for (int c = 0; c < per; ++c) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = *reinterpret_cast<const float4*>(Q + (rt * 4 + i) * F32_LD + c * 4);
                    b[i] = *reinterpret_cast<const float4*>(K + (kt + 16 * i) * F32_LD + c * 4);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
            }
            const bool partial = k0 < lo_last || k0 + F32_KT > it.p_first + 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = k0 + kt + 16 * j;
                    s[i][j] *= scale2;
                    if (partial && (p > pos[i] || p < first_key(pos[i], w.window))) s[i][j] = -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[i] - base);
                m[i] = mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = k0 + kt + 16 * j;
                    float e = exp2f(s[i][j] - base);
                    sum += e;
                    if (partial && (p > pos[i] || p < first_key(pos[i], w.window))) e = -1.f;
                    P[(rt * 4 + i) * F32_PLD + kt + 16 * j] = e;
                }
                l[i] = l[i] * f + sum;
#pragma unroll
                for (int c = 0; c < 4 * NC; ++c) acc[i][c] *= f;
            }
            __syncthreads();                            // K is done, P is there
            fetch(kp, K, step + 1);
            cp_wait<1>();                               // V of this step
            __syncthreads();
#pragma unroll 2
            for (int j = 0; j < F32_KT; j += 4) {
                float4 p4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p4[i] = *reinterpret_cast<const float4*>(P + (rt * 4 + i) * F32_PLD + j);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    float v[4 * NC];
#pragma unroll
                    for (int h = 0; h < NC; ++h) {
                        const float4 x = *reinterpret_cast<const float4*>(V + (j + jj) * F32_LD + h * 64 + kt * 4);
                        v[4 * h] = x.x;
                        v[4 * h + 1] = x.y;
                        v[4 * h + 2] = x.z;
                        v[4 * h + 3] = x.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = jj == 0 ? p4[i].x : jj == 1 ? p4[i].y : jj == 2 ? p4[i].z : p4[i].w;
                        if (!partial || !(p < 0.f)) {
#pragma unroll
                            for (int c = 0; c < 4 * NC; ++c) acc[i][c] = fmaf(p, v[c], acc[i][c]);
                        }
                    }
                }
            }
            __syncthreads();                            // V and P are done
            fetch(vp, V, step + 1);
        }
        cp_wait<0>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            const int r = rt * 4 + i;
            const long long dst = out_row(w, it, r, d);
            if (dst < 0) continue;
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
            float* to = slot < 0 ? o + dst : sl.o + ((long long)slot * sl.rows + r) * d;
            const float f = slot < 0 ? inv : 1.f;
#pragma unroll
            for (int h = 0; h < NC; ++h)
                if (h * 64 + kt * 4 < d)
                    *reinterpret_cast<float4*>(to + h * 64 + kt * 4) =
                        make_float4(acc[i][h * 4] * f, acc[i][h * 4 + 1] * f, acc[i][h * 4 + 2] * f, acc[i][h * 4 + 3] * f);
            if (slot >= 0 && kt == 0) sl.ml[(long long)slot * sl.rows + r] = make_float2(m[i], l[i]);
        }
    }
    if (tid == 0) sl.cut[blockIdx.x] = cut;
}

}  // namespace attn
}  // namespace jet
