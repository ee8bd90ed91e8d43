// Softmax attention over a paged key/value cache: what its kernels share.
//
// A cache is two pools of pages, [n_pages][Hk][page][d] with arbitrary page,
// head and row strides (elements). Position p of sequence s is row p % page
// of pool page page_table[s][p / page]. A call brings the new tokens of every
// sequence packed along the token axis (sequence s: rows cu_q[s] ..
// cu_q[s+1]-1) and kv_lens[s], the positions of s with the new ones included;
// token i of the n new ones of s is at position kv_lens[s] - n + i and sees
// positions max(0, p - window + 1) .. p (window 0: all up to p).
//
// cu_q, kv_lens and page_table live on the device (a captured graph can be
// replayed with new lengths), so they are checked there: a sequence whose
// offsets or length are out of range is skipped and a page index out of range
// reads as zeros; both set the device error word.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace jet {
namespace attn {

// packed float32 arithmetic on pairs
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

struct Cache {
    const void* k;
    const void* v;
    long long page_stride, head_stride, row_stride;   // elements, the same for both pools
    const int* page_table;                            // [nseq][max_pages]
    int max_pages, n_pages, page_shift;               // page size = 1 << page_shift
};

struct Batch {
    const int* cu_q;      // [nseq + 1]
    const int* kv_lens;   // [nseq]
    int nseq, N;          // sequences, rows of q
};

// New tokens and positions of one sequence (n = 0: nothing to do or bad data).
struct Seq {
    int r0, n, L;
};

__device__ __forceinline__ Seq load_seq(const Batch& b, const Cache& c, int s, bool flag) {
    const int r0 = b.cu_q[s], r1 = b.cu_q[s + 1], L = b.kv_lens[s];
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= b.N && L >= 0 &&
                    (long long)L <= ((long long)c.max_pages << c.page_shift);
    if (!ok) {
        if (flag) flag_error(DEVERR_DATA);
        return Seq{0, 0, 0};
    }
    return Seq{r0, r1 - r0, L};
}

// page of position p of sequence s, or -1 (bad index: sets the error word)
__device__ __forceinline__ int load_page(const Cache& c, int s, int p) {
    const int pg = c.page_table[(long long)s * c.max_pages + (p >> c.page_shift)];
    if ((unsigned)pg < (unsigned)c.n_pages) return pg;
    flag_error(DEVERR_DATA);
    return -1;
}

// first visible position of a token at position p
__device__ __forceinline__ int first_key(int p, int window) {
    return window > 0 && p >= window ? p - window + 1 : 0;
}

// Sequence of row t of the packed tokens: the number of sequences that end at
// or before t. Every thread of the block calls it; nseq if t is behind the
// last sequence.
__device__ __forceinline__ int block_find_seq(const Batch& b, int t) {
    int s = 0;
    for (int base = 0; base < b.nseq; base += blockDim.x) {
        const int i = base + threadIdx.x;
        s += __syncthreads_count(i < b.nseq && b.cu_q[i + 1] <= t);
    }
    return s;
}

}  // namespace attn
}  // namespace jet
