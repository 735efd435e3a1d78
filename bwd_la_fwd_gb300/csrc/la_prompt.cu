// la_prompt.cu -- the causal head over packed prompts with grouped heads (la_prompt): argument checks, and the
// CUDA-core form, which serves fp32 and the bf16 head sizes without a tensor-core form.
//
// Sequences of different lengths lie end to end in T rows; query head h reads key/value head h / r.  Per sequence:
//   O_i = (a + S^T q_i + sum_{j<=i} W_ij v_j) / (n + q_i . z + sum_{j<=i} W_ij),   W_ij = 1 + q_i . k_j
// with (S, z, a, n) the state of all rows before the block of rows that i and j lie in; the state at the end is what
// la_decode_step_grouped continues from.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "la_f32x2.cuh"
#include "la_prompt.h"
#include "la_views.h"

namespace cg = cooperative_groups;

namespace la {
namespace prompt {

// ----------------------------------------------------------------------------------------------------------------
// CUDA-core form.  grid = (sequences x key/value heads, column blocks, parts): a cluster has one head of one sequence,
// its CTAs E columns of S each and a part of the rows each, which they walk 32 rows at a time.  First every CTA sums its
// part; the parts' sums are added up through distributed shared memory, each CTA a share of the elements over all parts;
// and every CTA then walks its rows again, for O, from the state before them.  In a block of rows warp w has rows w,
// w + 8, ..., one lane per column (and per row j of W), so a query head's rows stay within a warp.
//
// fp32 tokens keep an fp64 state, as la_decode_step does, but this GPU has two fp64 multiply-adds per SM and clock;
// a sum of rows is therefore two floats here (the product's and the sum's rounding errors, exact in fp32 by Dekker's and
// Knuth's steps, are gathered in the low one), good to 2^-46, and becomes a double once, when it is added to the state that
// the sequence started from.  O is formed in fp32 from the high floats, so the second walk sums in plain fp32.  1,500 tokens
// in 7 sequences, 8 query and 4 key/value heads of 64, fp32: 66 us (one walk for both, one CTA to a sequence: 405 us; the
// whole exchange in every CTA and scalar multiply-adds: 92 us).
// Bound by fp32 arithmetic, ten operations for a product of the sums, in the SMs that have the longest sequence's
// cluster: a block of 32 rows takes a CTA 4 us for the sums and 5 us for O, and up to three share an SM.
// ----------------------------------------------------------------------------------------------------------------
constexpr int kMaxRows = 0x7fffffff - 256;  // a chunk that begins at a row ends at an int
constexpr int kThreads = 256, kWarps = 8, kRows = 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// A running sum: a float (bf16 tokens), or a float and the sum of its rounding errors (fp32 tokens).
template <typename T> struct Sum;
template <> struct Sum<__nv_bfloat16> {  // (one float)
    using Acc = float;
    float hi;
    __device__ void set(float x) { hi = x; }
    __device__ void add(float x) { hi += x; }
    __device__ void fma(float x, float y) { hi = fmaf(x, y, hi); }
    __device__ void join(const Sum &s) { hi += s.hi; }
    __device__ float get() const { return hi; }
};
template <> struct Sum<float> {
    using Acc = double;
    float hi, lo;
    __device__ void set(double x) {
        hi = (float)x;
        lo = (float)(x - (double)hi);
    }
    __device__ void add(float x) {
        const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
        hi = t;
    }
    __device__ void fma(float x, float y) {
        const float p = __fmul_rn(x, y), e = __fmaf_rn(x, y, -p);
        add(p);
        lo = __fadd_rn(lo, e);
    }
    __device__ void join(const Sum &s) {
        add(s.hi);
        lo = __fadd_rn(lo, s.lo);
    }
    // (an infinite sum's error is no number)
    __device__ double get() const { return fabsf(hi) < INFINITY ? (double)hi + (double)lo : (double)hi; }
};

// a += x.x y, b += x.y y; the two floats of each in ten packed operations.  -p is formed as x (-y), and differences as
// multiply-adds with -1, which are exact products.
__device__ __forceinline__ void fma_pair(Sum<__nv_bfloat16> &a, Sum<__nv_bfloat16> &b, float2 x, float y) {
    const float2 r = fma2(x, both(y), make_float2(a.hi, b.hi));
    a.hi = r.x, b.hi = r.y;
}
__device__ __forceinline__ void fma_pair(Sum<float> &a, Sum<float> &b, float2 x, float y) {
    const float2 hi = make_float2(a.hi, b.hi), minus = both(-1.f);
    const float2 np = mul2(x, both(-y)), e = fma2(x, both(y), np);
    const float2 s = fma2(np, minus, hi), d = fma2(hi, minus, s);  // hi + p, and what of it p brought
    const float2 lost = fma2(add2(np, d), minus, fma2(fma2(d, minus, s), minus, hi));
    const float2 lo = add2(add2(make_float2(a.lo, b.lo), lost), e);
    a.hi = s.x, b.hi = s.y, a.lo = lo.x, b.lo = lo.y;
}

template <typename T, int D> struct Tile {
    static constexpr int E = D < 32 ? D : 32;       // columns of S in a CTA
    static constexpr int LD = D + 4;                // row pitch of Q and K: 16-byte loads of 8 rows meet all banks
    static constexpr int RE = 32 / E;               // halves of a warp that share the sums of O (2 where E = 16)
    static constexpr int NS = D * E / kThreads;     // elements of S of a thread: column t % E, rows from t / E * NS
    static constexpr int PER = kRows / kWarps;      // rows of a block of a warp
    static constexpr int PER_SM = D <= 64 ? 3 : D == 128 ? 2 : 1;  // CTAs that registers leave room for (of the case above: two 70 us)
    static constexpr size_t FLOATS = 2 * kRows * LD + kRows * E + kRows * kRows + D * E + D + E;
    static constexpr int SUMS = D * E + D + E;      // S, z and a of a CTA
    static constexpr size_t SMEM = sizeof(float) * FLOATS + sizeof(Sum<T>) * SUMS + sizeof(typename Sum<T>::Acc) * D;
    static_assert(FLOATS % 4 == 0 && SUMS % 2 == 0, "alignment of the sums and of z");
};

// `rows` rows of 32 (the others zero) of W elements each, global -> shared floats, 16 bytes at a time.
template <typename T, int W>
__device__ __forceinline__ void load_rows(float *dst, int pitch, const T *src, long long stride, int rows, int first, int step) {
    constexpr int V = 16 / (int)sizeof(T);
    for (int x = first; x < kRows * W / V; x += step) {
        const int j = x / (W / V), c = x % (W / V) * V;
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (j < rows) raw = *(const uint4 *)(src + j * stride + c);
        const T *e = (const T *)&raw;
#pragma unroll
        for (int k = 0; k < V; ++k) dst[j * pitch + c + k] = to_f(e[k]);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, Tile<T, D>::PER_SM) prompt_simt_kernel(const __grid_constant__ Args A) {
    using C = Tile<T, D>;
    using Acc = typename Sum<T>::Acc;
    constexpr int E = C::E, LD = C::LD, NS = C::NS, PER = C::PER;
    extern __shared__ __align__(16) float sm[];
    float *Ks = sm, *Qs = Ks + kRows * LD, *Vs = Qs + kRows * LD, *Ws = Vs + kRows * E, *Sf = Ws + kRows * kRows;
    float *zs = Sf + D * E, *as = zs + D;
    Sum<T> *of_part = (Sum<T> *)(sm + C::FLOATS);  // the part's sums: S, z, a
    Acc *z0 = (Acc *)(of_part + C::SUMS);          // z before the first row of this call
    if (!offsets_in_order(A)) return;               // the same for the whole grid
    cg::cluster_group cluster = cg::this_cluster();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int seq = blockIdx.x / A.Hkv, h = blockIdx.x % A.Hkv, e0 = blockIdx.y * E;
    const int parts = gridDim.z, part = blockIdx.z;
    const long long at = (long long)seq * A.Hkv + h;
    const int first = A.off[seq], len = A.off[seq + 1] - first;
    const int share = ((len + kRows - 1) / kRows + parts - 1) / parts * kRows;  // rows of a part
    const int lo = min(part * share, len), hi = min(lo + share, len);
    const T *K = (const T *)A.k + h * A.kh + first * A.kn, *V = (const T *)A.v + h * A.vh + first * A.vn + e0;
    Acc *S = A.S ? (Acc *)A.S + at * D * D : nullptr, *z = (Acc *)A.z + at * D, *a = (Acc *)A.a + at * D;
    const bool resume = A.resume && S;
    // this thread's elements of S: column t % E, rows d0 ...; thread t < D has z[t], t < E has a[e0 + t]
    const int e = t % E, d0 = t / E * NS;
    // ---- the part's sums
    {
        Sum<T> s[NS], zt, at_;
#pragma unroll
        for (int m = 0; m < NS; ++m) s[m].set(0);
        zt.set(0);
        at_.set(0);
        for (int row0 = lo; row0 < hi; row0 += kRows) {
            const int live = min(kRows, hi - row0);
            __syncthreads();
            load_rows<T, D>(Ks, LD, K + (long long)row0 * A.kn, A.kn, live, t, kThreads);
            load_rows<T, E>(Vs, E, V + (long long)row0 * A.vn, A.vn, live, t, kThreads);
            __syncthreads();
            // the block's own sums first: over a long sequence a sum then passes a rounding for every 32 rows
            Sum<T> bs[NS], bz, ba;
#pragma unroll
            for (int m = 0; m < NS; ++m) bs[m].set(0);
            bz.set(0);
            ba.set(0);
            for (int j = 0; j < live; ++j) {
                const float v = Vs[j * E + e];
                if constexpr (NS % 4 == 0) {
#pragma unroll
                    for (int m = 0; m < NS; m += 4) {
                        const float4 k4 = *(const float4 *)(Ks + j * LD + d0 + m);
                        fma_pair(bs[m], bs[m + 1], make_float2(k4.x, k4.y), v);
                        fma_pair(bs[m + 2], bs[m + 3], make_float2(k4.z, k4.w), v);
                    }
                } else {
#pragma unroll
                    for (int m = 0; m < NS; ++m) bs[m].fma(Ks[j * LD + d0 + m], v);
                }
                if (t < D) bz.add(Ks[j * LD + t]);
                if (t < E) ba.add(Vs[j * E + t]);
            }
#pragma unroll
            for (int m = 0; m < NS; ++m) s[m].join(bs[m]);
            zt.join(bz);
            at_.join(ba);
        }
#pragma unroll
        for (int m = 0; m < NS; ++m) of_part[(d0 + m) * E + e] = s[m];
        if (t < D) of_part[D * E + t] = zt;
        if (t < E) of_part[D * E + D + t] = at_;
    }
    // ---- the state before each part, and behind the last one.  Each CTA adds up its share of the elements over all parts
    // and leaves them in the parts' shared memory.
    const int n0 = resume ? A.n[at] : 0;
    if (resume && t < D) z0[t] = z[t];
    cluster.sync();  // every part's sums are there, and all have read z and n
    {
        const int per = (C::SUMS + parts - 1) / parts;
        for (int x = part * per + t; x < min((part + 1) * per, C::SUMS); x += kThreads) {
            const bool of_z = x >= D * E && x < D * E + D;
            Acc *state = x < D * E ? S + (long long)(x / E) * D + e0 + x % E : of_z ? z + (x - D * E) : a + e0 + (x - D * E - D);
            auto start = [&] { return resume ? of_z ? z0[x - D * E] : *state : (Acc)0; };
            float run = (float)start();  // the state before each part, as O takes it
            Sum<T> rows;              // the sum of all parts: added to the whole of an fp64 state, once
            rows.set(0);
            constexpr int kAhead = 8;
            for (int p0 = 0; p0 < parts; p0 += kAhead) {
                Sum<T> v[kAhead];
#pragma unroll
                for (int p = 0; p < kAhead; ++p)
                    if (p0 + p < parts) v[p] = *cluster.map_shared_rank(of_part + x, (p0 + p) * gridDim.y + blockIdx.y);
#pragma unroll
                for (int p = 0; p < kAhead; ++p)
                    if (p0 + p < parts) {
                        *cluster.map_shared_rank(Sf + x, (p0 + p) * gridDim.y + blockIdx.y) = run;  // Sf, zs, as in a row
                        run += v[p].hi;
                        rows.join(v[p]);
                    }
            }
            if (S && (!of_z || blockIdx.y == 0) && !(resume && len == 0))
                *state = sizeof(Acc) == 8 ? (Acc)(start() + rows.get()) : (Acc)run;
        }
        if (S && part == 0 && blockIdx.y == 0 && t == 0) A.n[at] = n0 + len;
    }
    cluster.sync();  // the parts have their states, and none is read any more
    // ---- O
    for (int row0 = lo; row0 < hi; row0 += kRows) {
        const int live = min(kRows, hi - row0);
        __syncthreads();  // the block before is done with K and V, and S, z, a are those after it
        load_rows<T, D>(Ks, LD, K + (long long)row0 * A.kn, A.kn, live, t, kThreads);
        load_rows<T, E>(Vs, E, V + (long long)row0 * A.vn, A.vn, live, t, kThreads);
        __syncthreads();
        const float nb = (float)(n0 + row0);
        for (int g = 0; g < A.r; ++g) {
            const int hq = h * A.r + g;
            const T *Q = (const T *)A.q + hq * A.qh + (first + (long long)row0) * A.qn;
            T *O = (T *)A.o + hq * A.oh + (first + (long long)row0) * A.on + e0;
            __syncwarp();
            // the warp's rows warp, warp + 8, ... stand one behind another in Qs
            float *Qw = Qs + warp * PER * LD;
            {
                constexpr int VW = 16 / (int)sizeof(T);
                for (int x = lane; x < PER * D / VW; x += 32) {
                    const int m = x / (D / VW), c = x % (D / VW) * VW, i = warp + kWarps * m;
                    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
                    if (i < live) raw = *(const uint4 *)(Q + i * A.qn + c);
                    const T *el = (const T *)&raw;
#pragma unroll
                    for (int k = 0; k < VW; ++k) Qw[m * LD + c + k] = to_f(el[k]);
                }
            }
            __syncwarp();
            // W and g: lane j of row i
            float2 w2[PER];
            float w[PER], gi[PER];
#pragma unroll
            for (int m = 0; m < PER; ++m) w2[m] = make_float2(1.f, 0.f), gi[m] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                const float4 k4 = *(const float4 *)(Ks + lane * LD + d);
#pragma unroll
                for (int m = 0; m < PER; ++m) {
                    const float4 q4 = *(const float4 *)(Qw + m * LD + d);
                    w2[m] = fma2(make_float2(q4.x, q4.y), make_float2(k4.x, k4.y), w2[m]);
                    w2[m] = fma2(make_float2(q4.z, q4.w), make_float2(k4.z, k4.w), w2[m]);
                }
            }
            for (int d = lane; d < D; d += 32) {
                const float zd = zs[d];
#pragma unroll
                for (int m = 0; m < PER; ++m) gi[m] = fmaf(Qw[m * LD + d], zd, gi[m]);
            }
#pragma unroll
            for (int m = 0; m < PER; ++m) {
                w[m] = lane <= warp + kWarps * m ? w2[m].x + w2[m].y : 0.f;
                Ws[(warp * PER + m) * kRows + lane] = w[m];
                gi[m] += w[m];
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) gi[m] += __shfl_xor_sync(0xffffffffu, gi[m], x);
            }
            __syncwarp();
            const int c = lane % E, half = lane / E;  // E = 16: the two half warps take half of the sums each
            float2 o2[PER];
#pragma unroll
            for (int m = 0; m < PER; ++m) o2[m] = make_float2(half ? 0.f : as[c], 0.f);
#pragma unroll 4
            for (int d = half * (D / C::RE); d < (half + 1) * (D / C::RE); d += 4) {
                const float s0 = Sf[d * E + c], s1 = Sf[(d + 1) * E + c], s2 = Sf[(d + 2) * E + c], s3 = Sf[(d + 3) * E + c];
#pragma unroll
                for (int m = 0; m < PER; ++m) {
                    const float4 q4 = *(const float4 *)(Qw + m * LD + d);
                    o2[m] = fma2(make_float2(q4.x, q4.y), make_float2(s0, s1), o2[m]);
                    o2[m] = fma2(make_float2(q4.z, q4.w), make_float2(s2, s3), o2[m]);
                }
            }
#pragma unroll 4
            for (int j = half * 4; j < kRows; j += 4 * C::RE) {
                const float v0 = Vs[j * E + c], v1 = Vs[(j + 1) * E + c], v2 = Vs[(j + 2) * E + c], v3 = Vs[(j + 3) * E + c];
#pragma unroll
                for (int m = 0; m < PER; ++m) {
                    const float4 w4 = *(const float4 *)(Ws + (warp * PER + m) * kRows + j);
                    o2[m] = fma2(make_float2(w4.x, w4.y), make_float2(v0, v1), o2[m]);
                    o2[m] = fma2(make_float2(w4.z, w4.w), make_float2(v2, v3), o2[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < PER; ++m) {
                const int i = warp + kWarps * m;
                float o = o2[m].x + o2[m].y;
                if (C::RE == 2) o += __shfl_xor_sync(0xffffffffu, o, 16);
                if (i < live && half == 0) put(O + (long long)i * A.on + c, o / (nb + gi[m]));
            }
        }
        if (row0 + kRows >= hi) break;
        __syncthreads();  // every warp has read S, z and a of before
        Sum<__nv_bfloat16> bs[NS];
        float bz = 0.f, ba = 0.f;
#pragma unroll
        for (int m = 0; m < NS; ++m) bs[m].set(0);
        for (int j = 0; j < live; ++j) {
            const float v = Vs[j * E + e];
            if constexpr (NS % 4 == 0) {
#pragma unroll
                for (int m = 0; m < NS; m += 4) {
                    const float4 k4 = *(const float4 *)(Ks + j * LD + d0 + m);
                    fma_pair(bs[m], bs[m + 1], make_float2(k4.x, k4.y), v);
                    fma_pair(bs[m + 2], bs[m + 3], make_float2(k4.z, k4.w), v);
                }
            } else {
#pragma unroll
                for (int m = 0; m < NS; ++m) bs[m].fma(Ks[j * LD + d0 + m], v);
            }
            if (t < D) bz += Ks[j * LD + t];
            if (t < E) ba += Vs[j * E + t];
        }
#pragma unroll
        for (int m = 0; m < NS; ++m) Sf[(d0 + m) * E + e] += bs[m].hi;
        if (t < D) zs[t] += bz;
        if (t < E) as[t] += ba;
    }
}

template <typename T, int D> cudaError_t launch_simt(const Args &A, cudaStream_t s) {
    using C = Tile<T, D>;
    static std::atomic<int> attr_state[kMaxDevices];
    if (!once_per_device(attr_state, [] {
            return cudaFuncSetAttribute(prompt_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)C::SMEM) == cudaSuccess &&
                   cudaFuncSetAttribute(prompt_simt_kernel<T, D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                       cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    // Parts: up to what a cluster holds, while that does not make more than three CTAs for each SM and leaves sequences
    // of the mean length a block of rows in a part.  (The case above: eight parts 106 us, four 116, two 179, before the
    // exchange was shared out; no more than two CTAs for each SM: 112 where three take 82.)
    constexpr int cols = D / C::E;
    const long long heads = (long long)A.nseq * A.Hkv;
    int parts = 1;
    while (2 * parts * cols <= 16 && 2 * parts * cols * heads <= 456 && (long long)A.T >= (long long)parts * kRows * A.nseq) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)heads, cols, parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = cols;
    attr[0].val.clusterDim.z = parts;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prompt_simt_kernel<T, D>, A);
}

cudaError_t simt(const Args &A, int dtype, cudaStream_t s) {
    cudaError_t e;
    if (dtype == LA_BF16) {
        e = A.D == 16 ? launch_simt<__nv_bfloat16, 16>(A, s) : launch_simt<__nv_bfloat16, 256>(A, s);
    } else {
        switch (A.D) {
            case 16: e = launch_simt<float, 16>(A, s); break;
            case 32: e = launch_simt<float, 32>(A, s); break;
            case 64: e = launch_simt<float, 64>(A, s); break;
            case 128: e = launch_simt<float, 128>(A, s); break;
            default: e = launch_simt<float, 256>(A, s);
        }
    }
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// T = 0: a sequence that starts empty leaves an empty state, one that is continued its own.
template <typename Acc> __global__ void __launch_bounds__(kThreads) no_rows_kernel(const __grid_constant__ Args A) {
    if (!offsets_in_order(A) || !A.S || A.resume) return;
    const long long at = blockIdx.x;
    for (int x = threadIdx.x; x < A.D * A.D; x += kThreads) ((Acc *)A.S)[at * A.D * A.D + x] = 0;
    for (int x = threadIdx.x; x < A.D; x += kThreads) ((Acc *)A.z)[at * A.D + x] = ((Acc *)A.a)[at * A.D + x] = 0;
    if (threadIdx.x == 0) A.n[at] = 0;
}

cudaError_t no_rows(const Args &A, int dtype, cudaStream_t s) {
    auto *k = dtype == LA_BF16 ? no_rows_kernel<float> : no_rows_kernel<double>;
    k<<<(unsigned)(A.nseq * A.Hkv), kThreads, 0, s>>>(A);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

bool supported_d(int D) { return D == 16 || D == 32 || D == 64 || D == 128 || D == 256; }

}  // namespace prompt
}  // namespace la

extern "C" {

size_t la_prompt_workspace_bytes(int T, int nseq, int Hq, int Hkv, int D, int dtype) {
    if (T < 0 || T > la::prompt::kMaxRows || nseq < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || !la::prompt::supported_d(D) ||
        (dtype != LA_F32 && dtype != LA_BF16))
        return 0;
    return la::prompt::tc_supported(D, dtype) ? la::prompt::tc_workspace_bytes(T, nseq, Hkv, Hq / Hkv, D) : 256;
}

int la_prompt(const void *Q, const void *K, const void *V, const int *seq_offsets, void *O, void *S, void *z, void *a,
              int *n, int resume, int T, int nseq, int Hq, int Hkv, int D, int dtype, const long long *strides,
              void *workspace, size_t workspace_bytes, void *stream) {
    using namespace la;
    using namespace la::prompt;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (T < 0 || T > kMaxRows || nseq < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || D < 1) return LA_ERR_INVALID_ARG;
    if (!supported_d(D)) return LA_ERR_UNSUPPORTED;
    if ((long long)T * Hq >= (1LL << 40) / D || (long long)nseq * Hkv >= (1LL << 31) / 16) return LA_ERR_INVALID_ARG;
    const int elem = dtype == LA_BF16 ? 2 : 4, acc = dtype == LA_BF16 ? 4 : 8;
    const bool any = S || z || a || n, all = S && z && a && n;
    if (any != all || (resume && !all)) return LA_ERR_INVALID_ARG;
    if (nseq == 0) return LA_OK;
    const size_t ws_need = la_prompt_workspace_bytes(T, nseq, Hq, Hkv, D, dtype);
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < ws_need) return LA_ERR_WORKSPACE;
    if (!seq_offsets || ((uintptr_t)seq_offsets & 3)) return LA_ERR_INVALID_ARG;
    const void *ptr[4] = {Q, K, V, O};
    View v[4];
    int rc;
    for (int k = 0; k < 4; ++k) {  // (Q, K, V, O) x (head, row)
        const int H = k == 0 || k == 3 ? Hq : Hkv;
        if (T > 0 && (!ptr[k] || ((uintptr_t)ptr[k] & 15))) return LA_ERR_INVALID_ARG;
        v[k] = View{ptr[k], {1, H, T}, {}, D, elem};
        const long long dense[3] = {D, D, (long long)H * D};
        const long long given[3] = {D, strides ? strides[2 * k] : 0, strides ? strides[2 * k + 1] : 0};
        if (T > 0 && (rc = set_view(v[k], strides ? given : dense, dense))) return rc;
    }
    const long long SH = (long long)nseq * Hkv;
    const void *st[4] = {S, z, a, n};
    const size_t sb[4] = {(size_t)SH * D * D * acc, (size_t)SH * D * acc, (size_t)SH * D * acc, (size_t)SH * 4};
    const size_t ob = (size_t)(nseq + 1) * 4;
    for (int k = 0; k < 3 && T > 0; ++k)
        if (views_meet(v[3], v[k])) return LA_ERR_INVALID_ARG;
    if (ranges_meet(workspace, ws_need, seq_offsets, ob)) return LA_ERR_INVALID_ARG;
    if (T > 0) {
        if (ranges_meet(O, view_bytes(v[3]), seq_offsets, ob)) return LA_ERR_INVALID_ARG;
        for (int k = 0; k < 4; ++k)
            if (ranges_meet(workspace, ws_need, ptr[k], view_bytes(v[k]))) return LA_ERR_INVALID_ARG;
    }
    for (int x = 0; x < 4 && all; ++x) {
        if ((uintptr_t)st[x] & 15) return LA_ERR_INVALID_ARG;
        for (int y = x + 1; y < 4; ++y)
            if (ranges_meet(st[x], sb[x], st[y], sb[y])) return LA_ERR_INVALID_ARG;
        for (int k = 0; k < 4 && T > 0; ++k)
            if (ranges_meet(st[x], sb[x], ptr[k], view_bytes(v[k]))) return LA_ERR_INVALID_ARG;
        if (ranges_meet(st[x], sb[x], seq_offsets, ob) || ranges_meet(st[x], sb[x], workspace, ws_need))
            return LA_ERR_INVALID_ARG;
    }
    Args A = {};
    A.q = Q;
    A.k = K;
    A.v = V;
    A.o = O;
    A.off = seq_offsets;
    A.S = S;
    A.z = z;
    A.a = a;
    A.n = n;
    A.resume = resume ? 1 : 0;
    A.T = T;
    A.nseq = nseq;
    A.Hq = Hq;
    A.Hkv = Hkv;
    A.r = Hq / Hkv;
    A.D = D;
    A.qh = v[0].st[1], A.qn = v[0].st[2], A.kh = v[1].st[1], A.kn = v[1].st[2];
    A.vh = v[2].st[1], A.vn = v[2].st[2], A.oh = v[3].st[1], A.on = v[3].st[2];
    A.status = (uint32_t *)workspace;
    cudaStream_t cs = (cudaStream_t)stream;
    const cudaError_t e = T == 0 ? no_rows(A, dtype, cs)
                          : tc_supported(D, dtype) ? tensor_cores(A, (unsigned char *)workspace, cs)
                                                   : simt(A, dtype, cs);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
