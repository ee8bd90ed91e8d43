// RMSNorm of queries and keys per head, position rotation, and the append of
// keys and values to the paged cache, in one pass over the new tokens.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma            (per head; skipped without gammas)
//   the first `rot` elements of y are rotated in pairs by the angle p * inv_freq[i]:
//   pair i is (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) when interleaved
//
// Memory-bound: every element is read once and written once. A block takes TB
// tokens; a group of LPR lanes (16, or 8 for d <= 64) takes one row (token,
// head) at a time, each lane one unit of 8 elements: the 4 of the first and
// the 4 of the second half of 4 rotation pairs, so that a rotation needs no
// exchange between lanes and the norm LPR lanes' shuffles. The sines are
// computed once per token and shared through shared memory. The angle is
// formed and reduced to a fraction of a turn in float64: at position 200000
// a float32 product would be off by up to 0.008 rad, more than a bf16 step.
#pragma once
#include "k_attn_common.cuh"

namespace jet {
namespace attn {

constexpr int APPEND_THREADS = 256;

struct AppendArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride, qo_stride;     // elements between tokens
    const float *q_gamma, *k_gamma, *inv_freq;
    void* q_out;
    int Hq, Hk, d, rot, interleaved;
    float eps;
};

template <typename T> struct Vec4;      // 4 elements of a storage type
template <> struct Vec4<float> {
    typedef float4 raw;
    static __device__ __forceinline__ void unpack(const raw& r, float* f) {
        f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
    }
    static __device__ __forceinline__ raw pack(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <> struct Vec4<__nv_bfloat16> {
    typedef uint2 raw;
    static __device__ __forceinline__ void unpack(const raw& r, float* f) {
        f[0] = __uint_as_float(r.x << 16); f[1] = __uint_as_float(r.x & 0xffff0000u);
        f[2] = __uint_as_float(r.y << 16); f[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    static __device__ __forceinline__ raw pack(const float* f) {
        return make_uint2(Vec16<__nv_bfloat16>::pack2(f[0], f[1]), Vec16<__nv_bfloat16>::pack2(f[2], f[3]));
    }
};

template <typename T, int TB, int LPR>
__global__ void __launch_bounds__(APPEND_THREADS)
append_kernel(AppendArgs a, Cache c, Batch b) {
    typedef typename Vec4<T>::raw raw;
    constexpr int GROUPS = APPEND_THREADS / LPR;
    __shared__ float2 cs[TB][64];
    __shared__ long long page_off[TB];      // element offset of the token's cache row (head 0), -1: none
    __shared__ int live[TB];                // the token belongs to a sequence and has a position
    pdl_wait();
    pdl_trigger();
    const int t0 = blockIdx.x * TB;
    const int half = a.rot / 2;
    // the sequences of the block's tokens
    const int s0 = block_find_seq(b, t0);
    if (threadIdx.x < TB) {
        const int t = t0 + threadIdx.x;
        int s = s0;
        while (s < b.nseq && b.cu_q[s + 1] <= t) ++s;
        int ok = 0;
        long long off = -1;
        if (t < b.N && s < b.nseq) {
            const Seq sq = load_seq(b, c, s, true);
            const int i = t - sq.r0, p = sq.L - sq.n + i;
            if (i >= 0 && i < sq.n && p >= 0) {
                ok = 1;
                const int pg = load_page(c, s, p);
                if (pg >= 0) off = pg * c.page_stride + (p & ((1 << c.page_shift) - 1)) * c.row_stride;
                cs[threadIdx.x][0].x = __int_as_float(p);
            }
        }
        live[threadIdx.x] = ok;
        page_off[threadIdx.x] = off;
    }
    __syncthreads();
    int pos[TB];
#pragma unroll
    for (int u = 0; u < TB; ++u) pos[u] = __float_as_int(cs[u][0].x);
    __syncthreads();
    for (int e = threadIdx.x; e < TB * half; e += APPEND_THREADS) {
        const int u = e / half, i = e - u * half;
        int p = 0;
#pragma unroll
        for (int w = 0; w < TB; ++w)
            if (w == u) p = pos[w];
        if (live[u]) {
            // fraction of a turn in float64, its sine and cosine in float32
            double turn = (double)p * (double)a.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
            turn -= rint(turn);
            float sn, cn;
            sincospif((float)(2.0 * turn), &sn, &cn);
            cs[u][i] = make_float2(cn, sn);
        }
    }
    __syncthreads();
    const int group = threadIdx.x / LPR, unit = threadIdx.x % LPR;
    const int rows_per_token = a.Hq + 2 * a.Hk;
    const bool active = unit * 8 < a.d;
    // this lane's 8 elements: a pair unit of the rotated part, or 8 elements behind it
    const bool rotated = unit * 8 < a.rot;
    const int e0 = !rotated || a.interleaved ? unit * 8 : unit * 4;
    const int e1 = !rotated || a.interleaved ? unit * 8 + 4 : half + unit * 4;
    const int total = TB * rows_per_token;
    for (int r = group; r < (total + GROUPS - 1) / GROUPS * GROUPS; r += GROUPS) {
        const int u = r / rows_per_token, h = r - u * rows_per_token, t = t0 + u;
        const bool on = r < total && live[r < total ? u : 0];
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hk;
        raw x0{}, x1{};
        if (on && active) {
            const T* src = is_q ? static_cast<const T*>(a.q) + t * a.q_stride + (long long)h * a.d
                         : is_v ? static_cast<const T*>(a.v) + t * a.v_stride + (long long)(h - a.Hq - a.Hk) * a.d
                                : static_cast<const T*>(a.k) + t * a.k_stride + (long long)(h - a.Hq) * a.d;
            x0 = *reinterpret_cast<const raw*>(src + e0);
            x1 = *reinterpret_cast<const raw*>(src + e1);
        }
        if (!is_v) {
            float f0[4], f1[4];
            Vec4<T>::unpack(x0, f0);
            Vec4<T>::unpack(x1, f1);
            const float* gamma = is_q ? a.q_gamma : a.k_gamma;
            if (a.q_gamma) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) ss = fmaf(f0[e], f0[e], fmaf(f1[e], f1[e], ss));
#pragma unroll
                for (int w = LPR / 2; w > 0; w >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, w);
                const float inv = 1.f / sqrtf(ss / (float)a.d + a.eps);
                if (active) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f0[e] *= inv * gamma[e0 + e];
                        f1[e] *= inv * gamma[e1 + e];
                    }
                }
            }
            if (on && rotated) {
                const float2* tc = cs[u] + unit * 4;
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float2 ca = tc[e / 2], cb = tc[2 + e / 2];
                        const float a0 = f0[e], a1 = f0[e + 1], b0 = f1[e], b1 = f1[e + 1];
                        f0[e] = a0 * ca.x - a1 * ca.y;
                        f0[e + 1] = a1 * ca.x + a0 * ca.y;
                        f1[e] = b0 * cb.x - b1 * cb.y;
                        f1[e + 1] = b1 * cb.x + b0 * cb.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = f0[e], y = f1[e];
                        f0[e] = x * tc[e].x - y * tc[e].y;
                        f1[e] = y * tc[e].x + x * tc[e].y;
                    }
                }
            }
            x0 = Vec4<T>::pack(f0);
            x1 = Vec4<T>::pack(f1);
        }
        if (!on || !active) continue;
        T* dst;
        if (is_q) {
            dst = static_cast<T*>(a.q_out) + t * a.qo_stride + (long long)h * a.d;
        } else {
            if (page_off[u] < 0) continue;
            const int hk = is_v ? h - a.Hq - a.Hk : h - a.Hq;
            dst = static_cast<T*>(const_cast<void*>(is_v ? c.v : c.k)) + page_off[u] + hk * c.head_stride;
        }
        *reinterpret_cast<raw*>(dst + e0) = x0;
        *reinterpret_cast<raw*>(dst + e1) = x1;
    }
}

}  // namespace attn
}  // namespace jet
