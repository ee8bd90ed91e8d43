// RMSNorm of queries and keys per head, position rotation, and the append of
// keys and values to the paged cache, in one pass over the new tokens.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma            (per head; skipped without gammas)
//   the first `rot` elements of y are rotated in pairs by the angle p * inv_freq[i]:
//   pair i is (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) when interleaved
//
// Memory-bound: every element is read once and written once. A block takes TB
// tokens; a group of LPR lanes takes rows (token, head), three of them in
// flight and the first three on their way before the block looks its sequences
// up. Each lane has one unit of 2 E elements of a row: E of the first and E of
// the second half of E rotation pairs, so that a rotation needs no exchange
// between lanes and the norm LPR lanes' shuffles. E is 8 (16-byte accesses in
// bf16: half the instructions per element of E = 4, which were the limit there)
// where the rotated part is a multiple of 16, else 4. The sines are computed
// once per token and shared through shared memory. The angle is formed and
// reduced to a fraction of a turn in float64: at position 200000 a float32
// product would be off by up to 0.008 rad, more than a bf16 step.
#pragma once
#include "k_attn_common.cuh"

namespace jet {
namespace attn {

constexpr int APPEND_THREADS = 128;

struct AppendArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride, qo_stride;     // elements between tokens
    const float *q_gamma, *k_gamma, *inv_freq;
    void* q_out;
    int Hq, Hk, d, rot, interleaved;
    float eps;
};

// E elements of a storage type as they are moved
template <typename T, int E> struct Part {
    static constexpr int W = E * (int)sizeof(T) / 4;        // 2, 4 or 8 words
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
        if (W == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                w[(4 * i) % W] = v.x; w[(4 * i + 1) % W] = v.y; w[(4 * i + 2) % W] = v.z; w[(4 * i + 3) % W] = v.w;
            }
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if (W == 2) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i)
                reinterpret_cast<uint4*>(p)[i] =
                    make_uint4(w[(4 * i) % W], w[(4 * i + 1) % W], w[(4 * i + 2) % W], w[(4 * i + 3) % W]);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void get(float* f) const {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (sizeof(T) == 4) {
                f[i % E] = __uint_as_float(w[i]);
            } else {
                f[(2 * i) % E] = __uint_as_float(w[i] << 16);
                f[(2 * i + 1) % E] = __uint_as_float(w[i] & 0xffff0000u);
            }
    }
    __device__ __forceinline__ void put(const float* f) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = sizeof(T) == 4 ? __float_as_uint(f[i % E])
                                  : Vec16<__nv_bfloat16>::pack2(f[(2 * i) % E], f[(2 * i + 1) % E]);
    }
};

// the lanes of this lane's group (a power of two of one warp)
template <int LPR> __device__ __forceinline__ unsigned group_mask() {
    return ((1u << LPR) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
}

template <typename T, int TB, int LPR, int E>
__global__ void __launch_bounds__(APPEND_THREADS)
append_kernel(AppendArgs a, Cache c, Batch b) {
    constexpr int GROUPS = APPEND_THREADS / LPR;
    constexpr int U = 3;                    // rows in flight per group
    __shared__ __align__(16) float2 cs[TB][64];
    __shared__ long long page_off[TB];      // element offset of the token's cache row (head 0), -1: none
    __shared__ int pos[TB];                 // the token's position, -1: it has none
    const int t0 = blockIdx.x * TB;
    const int half = a.rot / 2;
    const int group = threadIdx.x / LPR, unit = threadIdx.x % LPR;
    const int rpt = a.Hq + 2 * a.Hk;        // rows per token
    const bool active = unit * 2 * E < a.d;
    // this lane's 2 E elements: a pair unit of the rotated part, or 2 E elements behind it
    const bool rotated = unit * 2 * E < a.rot;
    const int e0 = !rotated || a.interleaved ? unit * 2 * E : unit * E;
    const int e1 = !rotated || a.interleaved ? unit * 2 * E + E : half + unit * E;
    const int tokens = min(TB, b.N - t0);
    pdl_wait();
    pdl_trigger();
    Part<T, E> x[U][2];
    auto load = [&](int u, int h) {         // rows (u, h), (u, h + GROUPS) ...
#pragma unroll
        for (int k = 0; k < U; ++k) {
            x[k][0].zero();
            x[k][1].zero();
            if (u < tokens && active) {
                const int t = t0 + u;
                const T* src = h < a.Hq ? static_cast<const T*>(a.q) + t * a.q_stride + h * a.d
                             : h >= a.Hq + a.Hk ? static_cast<const T*>(a.v) + t * a.v_stride + (h - a.Hq - a.Hk) * a.d
                                                : static_cast<const T*>(a.k) + t * a.k_stride + (h - a.Hq) * a.d;
                x[k][0].load(src + e0);
                x[k][1].load(src + e1);
            }
            for (h += GROUPS; h >= rpt; h -= rpt) ++u;
        }
    };
    int u0 = group / rpt, h0 = group - u0 * rpt;
    load(u0, h0);                           // on their way while the positions are looked up
    // the sequences of the block's tokens
    const int s0 = block_find_seq(b, t0);
    if (threadIdx.x < TB) {
        const int t = t0 + threadIdx.x;
        int s = s0, p = -1;
        while (s < b.nseq && b.cu_q[s + 1] <= t) ++s;
        long long off = -1;
        if (t < b.N && s < b.nseq) {
            const Seq sq = load_seq(b, c, s, true);
            const int i = t - sq.r0;
            if (i >= 0 && i < sq.n) p = max(-1, sq.L - sq.n + i);
            if (p >= 0) {
                const int pg = load_page(c, s, p);
                if (pg >= 0) off = pg * c.page_stride + (p & ((1 << c.page_shift) - 1)) * c.row_stride;
            }
        }
        pos[threadIdx.x] = p;
        page_off[threadIdx.x] = off;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < TB * half; e += APPEND_THREADS) {
        const int u = e / half, i = e - u * half;
        if (pos[u] >= 0) {
            // fraction of a turn in float64, its sine and cosine in float32
            double turn = (double)pos[u] * (double)a.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
            turn -= rint(turn);
            float sn, cn;
            sincospif((float)(2.0 * turn), &sn, &cn);
            cs[u][i] = make_float2(cn, sn);
        }
    }
    __syncthreads();
    const int rounds = (tokens * rpt + U * GROUPS - 1) / (U * GROUPS);      // the same in every group
    for (int round = 0; round < rounds; ++round) {
        if (round > 0) load(u0, h0);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int u = min(u0, TB - 1), h = h0, t = t0 + u;
            const bool on = u0 < tokens && pos[u] >= 0;
            for (h0 += GROUPS; h0 >= rpt; h0 -= rpt) ++u0;
            const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hk;
            if (!on) continue;              // a whole group
            if (!is_v) {
                float f0[E], f1[E];
                x[k][0].get(f0);
                x[k][1].get(f1);
                if (a.q_gamma) {
                    const float* gamma = is_q ? a.q_gamma : a.k_gamma;
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) ss = fmaf(f0[e], f0[e], fmaf(f1[e], f1[e], ss));
#pragma unroll
                    for (int w = LPR / 2; w > 0; w >>= 1) ss += __shfl_xor_sync(group_mask<LPR>(), ss, w);
                    const float inv = 1.f / sqrtf(ss / (float)a.d + a.eps);
                    if (active) {
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            f0[e] *= inv * __ldg(gamma + e0 + e);
                            f1[e] *= inv * __ldg(gamma + e1 + e);
                        }
                    }
                }
                if (rotated) {
                    const float2* tc = cs[u] + unit * E;
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            const float2 ca = tc[e / 2], cb = tc[E / 2 + e / 2];
                            const float a0 = f0[e], a1 = f0[e + 1], b0 = f1[e], b1 = f1[e + 1];
                            f0[e] = a0 * ca.x - a1 * ca.y;
                            f0[e + 1] = a1 * ca.x + a0 * ca.y;
                            f1[e] = b0 * cb.x - b1 * cb.y;
                            f1[e + 1] = b1 * cb.x + b0 * cb.y;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            const float4 cc = *reinterpret_cast<const float4*>(tc + e);
                            const float y0 = f0[e], z0 = f1[e], y1 = f0[e + 1], z1 = f1[e + 1];
                            f0[e] = y0 * cc.x - z0 * cc.y;
                            f1[e] = z0 * cc.x + y0 * cc.y;
                            f0[e + 1] = y1 * cc.z - z1 * cc.w;
                            f1[e + 1] = z1 * cc.z + y1 * cc.w;
                        }
                    }
                }
                x[k][0].put(f0);
                x[k][1].put(f1);
            }
            if (!active || (!is_q && page_off[u] < 0)) continue;
            T* dst = is_q ? static_cast<T*>(a.q_out) + t * a.qo_stride + h * a.d
                          : static_cast<T*>(const_cast<void*>(is_v ? c.v : c.k)) + page_off[u] +
                                (h - a.Hq - (is_v ? a.Hk : 0)) * c.head_stride;
            x[k][0].store(dst + e0);
            x[k][1].store(dst + e1);
        }
    }
}

}  // namespace attn
}  // namespace jet
