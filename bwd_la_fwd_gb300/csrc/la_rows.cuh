// la_rows.cuh -- what the operators over rows of channels (norm, short convolution, selective scan) share: 16-byte
// vectors of a row, sequences that lie end to end, the logistic function, sums over a call's blocks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "la_internal.h"
#include "la_tc_common.cuh"
#include "la_views.h"

namespace la {
namespace rows {

constexpr int kMaxRows = 0x7fffffff - 1024;  // the end of a block of rows is an int

struct Op {
    const void *p;
    long long sb, sn;  // batch, row stride in elements
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// V neighbouring elements of a row, as the row holds them (rows begin at 16 bytes, no more).
template <typename T, int V> struct __align__(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Vec {
    T e[V];
};

// Elements [0, n) of a vector (the others zero): one access where all V are there, and at a vector's place.
template <typename T, int V> __device__ __forceinline__ Vec<T, V> load_vec(const T *p, int n, bool aligned = true) {
    if (n >= V && aligned) return *(const Vec<T, V> *)p;
    Vec<T, V> r;
#pragma unroll
    for (int k = 0; k < V; ++k) r.e[k] = k < n ? p[k] : T(0.f);
    return r;
}
// A whole vector loaded into `r` where `on` holds, for use after other work: the load stays where it is written (a plain one
// may be moved down to its first use) and has no branch, whose end would wait for it.
template <typename T, int V> __device__ __forceinline__ void load_ahead(Vec<T, V> &r, const T *p, bool on) {
    constexpr int WORDS = (int)sizeof(T) * V / 4;
    uint32_t *w = (uint32_t *)&r;
    if constexpr (WORDS == 1) {
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\n@p ld.global.b32 %0, [%1];\n}" : "+r"(w[0]) : "l"(p), "r"((int)on));
    } else if constexpr (WORDS == 2) {
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %3, 0;\n@p ld.global.v2.b32 {%0, %1}, [%2];\n}"
                     : "+r"(w[0]), "+r"(w[1])
                     : "l"(p), "r"((int)on));
    } else {
#pragma unroll
        for (int k = 0; k < WORDS; k += 4)
            asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %5, 0;\n@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n}"
                         : "+r"(w[k]), "+r"(w[k + 1]), "+r"(w[k + 2]), "+r"(w[k + 3])
                         : "l"((const char *)p + 4 * k), "r"((int)on));
    }
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &x, int n, bool aligned = true) {
    if (n >= V && aligned) {
        *(Vec<T, V> *)p = x;
        return;
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
        if (k < n) p[k] = x.e[k];
}

// Two values rounded together, four to a vector.
__device__ __forceinline__ void put2(float *p, float x, float y) { p[0] = x, p[1] = y; }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float x, float y) { *(__nv_bfloat162 *)p = __floats2bfloat162_rn(x, y); }
template <typename T> __device__ __forceinline__ Vec<T, 4> rounded4(const float (&x)[4]) {
    Vec<T, 4> r;
    put2(r.e, x[0], x[1]);
    put2(r.e + 2, x[2], x[3]);
    return r;
}

// e^x by the hardware's 2^x: within 2 ulp, and half a step of the product x log2 e, which is |x| half steps of the result.
__device__ __forceinline__ float exp_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269502f));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {  // within 1 ulp; 0 from 2^126 on
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-x): (|x| + 8) half steps, as e^-x is; 0 below -87, where it is under 2^-125.
__device__ __forceinline__ float sigmoid(float x) { return rcp_fast(1.f + exp_fast(-x)); }
// The derivative of x sigmoid(x), from s = sigmoid(x).
__device__ __forceinline__ float silu_grad(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// Sequences one behind another: nseq of N rows each, a batch (off null), or packed into T rows with sequence i at
// off[i] ... off[i + 1] - 1.
struct Seqs {
    const int *off;    // device, [nseq + 1]
    int nseq, N, T;    // T: all rows
    uint32_t *status;  // workspace status word (packed)
};

// Whether the offsets run in order within [0, T], and for how many sequences f(i, first row) holds; the same answers for
// every thread of a block, which all call it.  (Sequences out of order would read and write rows that others have.)
template <typename F> __device__ __forceinline__ bool offsets_in_order(const Seqs &Q, int &count, F f) {
    int bad = 0, n = 0;
    for (int i0 = 0; i0 < Q.nseq; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        bool here = false;
        if (i < Q.nseq) {
            const int lo = Q.off[i], hi = Q.off[i + 1];
            bad |= lo < 0 || hi < lo || hi > Q.T;
            here = f(i, lo);
        }
        n += __syncthreads_count(here);
    }
    bad = __syncthreads_or(bad);
    count = n;
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0)
        tc::report(Q.status, kDevBounds, 0x0FF6u);
    return !bad;
}

// f(sequence, the first and last row of the stretch within it, its length, whether it begins there) for each stretch of
// the block's rows r0 ... r1 - 1, for sequences without rows too (those behind the last row belong to the block that ends
// there); false where the offsets are out of order.  All threads of the block call it.
template <typename F> __device__ __forceinline__ bool for_stretches(const Seqs &Q, int r0, int r1, F f) {
    int k;  // sequences that begin before the block
    if (!Q.off) k = Q.N > 0 ? (int)(((long long)r0 + Q.N - 1) / Q.N) : 0;
    else if (!offsets_in_order(Q, k, [&](int, int lo) { return lo < r0; })) return false;
    auto begin = [&](int i) { return Q.off ? Q.off[i] : i * Q.N; };
    if (k > 0) {  // the sequence that began before
        const int lo = begin(k - 1), hi = begin(k);
        if (hi > r0) f(k - 1, r0 - lo, min(r1, hi) - lo, hi - lo, false);
    }
    for (; k < Q.nseq; ++k) {
        const int lo = begin(k);
        if (lo >= r1 && r1 < Q.T) break;
        const int hi = begin(k + 1);
        f(k, 0, min(r1, hi) - lo, hi - lo, true);
    }
    return true;
}
// A sequence's first row in an operand.
template <typename T> __device__ __forceinline__ T *rows_of(const Seqs &Q, const Op &o, int seq) {
    return (T *)o.p + (Q.off ? Q.off[seq] * o.sn : seq * o.sb);
}

// out[m] = sum over p of part[p M + m], p in a fixed order: the first n0 sums go to out0, the next n1 to out1, the others to
// out2 (any of which may be null).
cudaError_t sum_parts(const float *part, int parts, long long M, float *out0, long long n0, float *out1, long long n1,
                      float *out2, cudaStream_t s);

// A [B,N,C] operand's view; strides: its (batch, row), or null for contiguous rows.
inline int rows_view(View &v, const void *p, long long B, long long N, long long C, int elem, const long long *strides) {
    if (!p || ((uintptr_t)p & 15)) return LA_ERR_INVALID_ARG;
    v = View{p, {B, N, 1}, {}, C, elem};
    const long long dense[3] = {N * C, C, C}, given[3] = {strides ? strides[0] : 0, strides ? strides[1] : 0, C};
    return set_view(v, strides ? given : dense, dense);
}

// A contiguous array among a call's operands.
struct Range {
    const void *p;
    size_t bytes;
};
inline bool meets(const View &v, const Range &r) { return r.p && ranges_meet(v.p, view_bytes(v), r.p, r.bytes); }
inline bool meets(const Range &a, const Range &b) { return a.p && b.p && ranges_meet(a.p, a.bytes, b.p, b.bytes); }
// Whether one of the outputs meets an input or another output (views and arrays; those without a pointer count for nothing).
__attribute__((noinline)) static bool outputs_meet(const View *in, int n_in, const View *out, int n_out, const Range *rin, int n_rin,
                         const Range *rout, int n_rout) {
    for (int o = 0; o < n_out; ++o) {
        if (!out[o].p) continue;
        for (int k = 0; k < n_in; ++k)
            if (in[k].p && views_meet(out[o], in[k])) return true;
        for (int k = o + 1; k < n_out; ++k)
            if (out[k].p && views_meet(out[o], out[k])) return true;
        for (int k = 0; k < n_rin; ++k)
            if (meets(out[o], rin[k])) return true;
    }
    for (int o = 0; o < n_rout; ++o) {
        for (int k = 0; k < n_in; ++k)
            if (in[k].p && meets(in[k], rout[o])) return true;
        for (int k = 0; k < n_out; ++k)
            if (out[k].p && meets(out[k], rout[o])) return true;
        for (int k = 0; k < n_rin; ++k)
            if (meets(rin[k], rout[o])) return true;
        for (int k = o + 1; k < n_rout; ++k)
            if (meets(rout[k], rout[o])) return true;
    }
    return false;
}

}  // namespace rows
}  // namespace la
