// RMSNorm of queries and keys per head, position rotation, and the append of
// keys and values to the paged cache, in one pass over the new tokens.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma            (per head; skipped without gammas)
//   the first `rot` elements of y are rotated in pairs by the angle p * inv_freq[i]:
//   pair i is (y_i, y_{i + rot/2}), or (y_2i, y_2i+1) when interleaved
//
// Memory-bound: every element is read once and written once. A block takes TB
// tokens; a group of LPR lanes takes every S-th row (head) of one token, two
// of them in flight and the first two on their way before the block looks its
// sequences up. Each lane has one unit of 2 E elements of a row: E of the first
// and E of the second half of E rotation pairs, so that a rotation needs no
// exchange between lanes and the norm LPR lanes' shuffles. E is 8 (16-byte
// accesses in bf16) where the rotated part is a multiple of 16, else 4. Gammas,
// cosines and sines are multiplied once per token into two coefficients an
// element, kept in shared memory: applied row by row they made instructions the
// limit, and in registers the occupancy. 14463 tokens of 20 heads: 38 to 40
// us, 3.9 TB/s, of which the rows alone take 27; in float32 59 us, 5.0 TB/s;
// 256 tokens: 3.7 to 4.1 us.
// The angle is formed and reduced to a fraction of a turn in float64: at
// position 200000 a float32 product would be off by up to 0.008 rad, more than
// a bf16 step.
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
    int Hq, Hk, d, rot;
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
    // as pairs of consecutive elements
    __device__ __forceinline__ void get(uint64_t* f) const {
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            f[i] = sizeof(T) == 4 ? pair(__uint_as_float(w[(2 * i) % W]), __uint_as_float(w[(2 * i + 1) % W]))
                                  : pair(__uint_as_float(w[i % W] << 16), __uint_as_float(w[i % W] & 0xffff0000u));
    }
    __device__ __forceinline__ void put(const uint64_t* f) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            float a, b;
            unpair(f[i], a, b);
            if (sizeof(T) == 4) {
                w[(2 * i) % W] = __float_as_uint(a);
                w[(2 * i + 1) % W] = __float_as_uint(b);
            } else {
                w[i % W] = Vec16<__nv_bfloat16>::pack2(a, b);
            }
        }
    }
};

// the lanes of this lane's group (a power of two of one warp)
template <int LPR> __device__ __forceinline__ unsigned group_mask() {
    return ((1u << LPR) - 1u) << ((threadIdx.x & 31) / LPR * LPR);
}

template <typename T, int TB, int LPR, int E, bool INTER>
__global__ void __launch_bounds__(APPEND_THREADS, sizeof(T) == 2 ? 8 : 6)
append_kernel(AppendArgs a, Cache c, Batch b) {
    constexpr int S = APPEND_THREADS / LPR / TB;            // groups per token
    constexpr int U = 2;                                    // rows in flight per group
    // out = own * element + other * its partner in the rotation: the gammas times the
    // cosines and sines, for queries (0) and keys (1) of each token
    __shared__ __align__(16) float own[TB][2][128], other[TB][2][128];
    __shared__ float gs[2][128], fs[64];
    __shared__ long long page_off[TB];      // element offset of the token's cache row (head 0), -1: none
    __shared__ int pos[TB];                 // the token's position, -1: it has none
    const int t0 = blockIdx.x * TB;
    const int half = a.rot / 2;
    const int group = threadIdx.x / LPR, unit = threadIdx.x % LPR;
    const int u = group / S, first = group % S, t = t0 + u;             // this group's token and first row
    const int rows = a.Hq + 2 * a.Hk;
    const bool active = unit * 2 * E < a.d && t < b.N;
    // this lane's 2 E elements: a pair unit of the rotated part, or 2 E elements behind it
    const bool rotated = unit * 2 * E < a.rot;
    const int e0 = !rotated || INTER ? unit * 2 * E : unit * E;
    const int e1 = !rotated || INTER ? unit * 2 * E + E : half + unit * E;
    const T* qt = static_cast<const T*>(a.q) + t * a.q_stride;
    const T* kt = static_cast<const T*>(a.k) + t * a.k_stride;
    const T* vt = static_cast<const T*>(a.v) + t * a.v_stride;
    pdl_wait();
    pdl_trigger();
    Part<T, E> x[U][2];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < U; ++k, h += S) {
            x[k][0].zero();
            x[k][1].zero();
            if (active && h < rows) {
                const T* src = h < a.Hq ? qt + h * a.d : h < a.Hq + a.Hk ? kt + (h - a.Hq) * a.d
                                                                         : vt + (h - a.Hq - a.Hk) * a.d;
                x[k][0].load(src + e0);
                x[k][1].load(src + e1);
            }
        }
    };
    // on their way while the positions are looked up
    load(first);
    if ((int)threadIdx.x < a.d) {
        gs[0][threadIdx.x] = a.q_gamma ? a.q_gamma[threadIdx.x] : 1.f;
        gs[1][threadIdx.x] = a.q_gamma ? a.k_gamma[threadIdx.x] : 1.f;
    }
    if ((int)threadIdx.x < half) fs[threadIdx.x] = a.inv_freq[threadIdx.x];
    // the sequences of the block's tokens
    const int s0 = block_find_seq(b, t0);
    int s = s0, p = -1;
    if (threadIdx.x < TB) {
        const int tt = t0 + threadIdx.x;
        while (s < b.nseq && b.cu_q[s + 1] <= tt) ++s;
        if (tt < b.N && s < b.nseq) {
            const Seq sq = load_seq(b, c, s, true);
            const int i = tt - sq.r0;
            if (i >= 0 && i < sq.n) p = max(-1, sq.L - sq.n + i);
        }
        pos[threadIdx.x] = p;
    }
    __syncthreads();
    const int pg = p >= 0 ? load_page(c, s, p) : -1;        // needed only when the rows are stored
    for (int e = threadIdx.x; e < TB * half; e += APPEND_THREADS) {
        const int w = e / half, i = e - w * half;
        if (pos[w] >= 0) {
            // fraction of a turn in float64, its sine and cosine in float32
            double turn = (double)pos[w] * (double)fs[i] * 0.15915494309189533577;   // 1 / (2 pi)
            turn -= rint(turn);
            float sn, cn;
            sincospif((float)(2.0 * turn), &sn, &cn);
            const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + half;       // the pair
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const float ga = gs[z][ia], gb = gs[z][ib];
                own[w][z][ia] = ga * cn;
                own[w][z][ib] = gb * cn;
                other[w][z][ia] = -gb * sn;
                other[w][z][ib] = ga * sn;
            }
        }
    }
    for (int e = a.rot + threadIdx.x; e < a.d; e += APPEND_THREADS)
#pragma unroll
        for (int w = 0; w < TB; ++w)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                own[w][z][e] = gs[z][e];
                other[w][z][e] = 0.f;
            }
    if (threadIdx.x < TB)
        page_off[threadIdx.x] = pg >= 0 ? pg * c.page_stride + (p & ((1 << c.page_shift) - 1)) * c.row_stride : -1;
    __syncthreads();
    if (pos[u] < 0 || t >= b.N) return;     // a whole group
    T* const qo = static_cast<T*>(a.q_out) + t * a.qo_stride;
    const long long off = page_off[u];
    const float inv_d = 1.f / (float)a.d;
    for (int h0 = first; h0 < rows; h0 += U * S) {
        if (h0 > first) load(h0);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = h0 + k * S;
            if (h >= rows) break;
            T* dst = qo + h * a.d;
            if (h >= a.Hq) {
                const bool is_v = h >= a.Hq + a.Hk;
                dst = static_cast<T*>(const_cast<void*>(is_v ? c.v : c.k)) + off + (h - a.Hq - (is_v ? a.Hk : 0)) * c.head_stride;
            }
            if (h < a.Hq + a.Hk) {
                uint64_t f[2][E / 2];
                x[k][0].get(f[0]);
                x[k][1].get(f[1]);
                if (a.q_gamma) {
                    uint64_t sq[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        sq[0] = fma2(f[0][i], f[0][i], sq[0]);
                        sq[1] = fma2(f[1][i], f[1][i], sq[1]);
                    }
                    float sa, sb;
                    unpair(add2(sq[0], sq[1]), sa, sb);
                    float ss = sa + sb;
#pragma unroll
                    for (int w = LPR / 2; w > 0; w >>= 1) ss += __shfl_xor_sync(group_mask<LPR>(), ss, w);
                    const float inv = rsqrtf(fmaf(ss, inv_d, a.eps));
                    const uint64_t inv2 = pair(inv, inv);
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        f[0][i] = mul2(f[0][i], inv2);
                        f[1][i] = mul2(f[1][i], inv2);
                    }
                }
                const float* po = own[u][h < a.Hq ? 0 : 1];
                const float* pt = other[u][h < a.Hq ? 0 : 1];
                uint64_t y[2][E / 2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < E / 2; i += 2) {
                        const int e = (j ? e1 : e0) + 2 * i;
                        const ulonglong2 co = *reinterpret_cast<const ulonglong2*>(po + e);
                        const ulonglong2 cp = *reinterpret_cast<const ulonglong2*>(pt + e);
                        uint64_t pa = f[j ^ 1][i], pb = f[j ^ 1][i + 1];
                        if (INTER) {
                            float lo, hi;
                            unpair(f[j][i], lo, hi);
                            pa = pair(hi, lo);
                            unpair(f[j][i + 1], lo, hi);
                            pb = pair(hi, lo);
                        }
                        if (!rotated) pa = pb = 0;          // no partner: zero times a non-finite one would not be zero
                        y[j][i] = fma2(f[j][i], co.x, mul2(pa, cp.x));
                        y[j][i + 1] = fma2(f[j][i + 1], co.y, mul2(pb, cp.y));
                    }
                x[k][0].put(y[0]);
                x[k][1].put(y[1]);
            }
            if (!active || (h >= a.Hq && off < 0)) continue;
            x[k][0].store(dst + e0);
            x[k][1].store(dst + e1);
        }
    }
}

}  // namespace attn
}  // namespace jet
