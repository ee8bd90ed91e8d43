// Attention over a paged cache on the CUDA cores, for float32 and for shapes
// off the tensor-core kernels. One warp per (token, query head): 32 keys at a
// time, each lane the product of one key with the query (kept in shared
// memory), a running maximum and sum in float32, then the 32 weighted value
// rows summed with each lane holding its columns. Keys outside the token's
// range are never read.
#pragma once
#include "k_attn_common.cuh"

namespace jet {
namespace attn {

constexpr int SIMT_WARPS = 4;

template <typename T>
__global__ void __launch_bounds__(SIMT_WARPS * 32)
attn_simt_kernel(const T* __restrict__ q, long long q_stride, Cache c, Batch b, T* __restrict__ o, int Hq, int Hk,
                 int d, int window, float scale) {
    __shared__ float qs[SIMT_WARPS][128];
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = block_find_seq(b, t);
    if (s >= b.nseq) return;
    const Seq sq = load_seq(b, c, s, threadIdx.x == 0);
    const int i = t - sq.r0;
    if (i < 0 || i >= sq.n) return;
    const int p = sq.L - sq.n + i;
    const int page = 1 << c.page_shift;
    const T* kp = static_cast<const T*>(c.k);
    const T* vp = static_cast<const T*>(c.v);
    for (int h = blockIdx.y * SIMT_WARPS + warp; h < Hq; h += gridDim.y * SIMT_WARPS) {
        const int hk = h / (Hq / Hk);
        __syncwarp();
        for (int e = lane; e < d; e += 32) qs[warp][e] = Elem<T>::ld(q + t * q_stride + (long long)h * d + e) * scale;
        __syncwarp();
        float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j0 = first_key(p, window); j0 <= p; j0 += 32) {
            const int j = j0 + lane;
            float x = -INFINITY;
            long long off = -1;
            if (j <= p) {
                const int pg = load_page(c, s, j);
                x = 0.f;
                if (pg >= 0) {
                    off = pg * c.page_stride + hk * c.head_stride + (j & (page - 1)) * c.row_stride;
                    for (int e = 0; e < d; e += Vec16<T>::N) {
                        float f[Vec16<T>::N];
                        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(kp + off + e), f);
#pragma unroll
                        for (int u = 0; u < Vec16<T>::N; ++u) x = fmaf(f[u], qs[warp][e + u], x);
                    }
                }
            }
            float mx = x;
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float m_new = fmaxf(m, mx);
            const float base = m_new == -INFINITY ? 0.f : m_new;     // every score so far is -inf
            const float r = expf(m - base), w = j <= p ? expf(x - base) : 0.f;
            l = l * r + warp_sum(w);
            m = m_new;
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[u] *= r;
            const int cnt = min(32, p - j0 + 1);
            for (int k = 0; k < cnt; ++k) {
                const float pk = __shfl_sync(0xffffffffu, w, k);
                const long long vo = __shfl_sync(0xffffffffu, off, k);
                if (vo < 0) continue;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (lane + 32 * u < d) acc[u] = fmaf(pk, Elem<T>::ld(vp + vo + lane + 32 * u), acc[u]);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;     // a row that sees nothing is zero
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (lane + 32 * u < d) Elem<T>::st(o + ((long long)t * Hq + h) * d + lane + 32 * u, acc[u] * inv);
    }
}

}  // namespace attn
}  // namespace jet
