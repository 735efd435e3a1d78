// la_rotary.cu -- rotary positions on Q and K (la_rotary) and the gradient through them (la_rotary_backward).
//
// Pair i of a row at position p turns by theta = p f_i:  y1 = m (x1 cos - x2 sin),  y2 = m (x1 sin + x2 cos);
// the transposed map, which the gradient takes, turns by -theta.  A pair is channels (i, i + R / 2) of the R
// rotated ones, or (2 i, 2 i + 1) interleaved; channels past R are copied.
//
// The phase.  p f_i radians in fp32 is off by 0.06 at p = 10^6, and fp64 is slow on this GPU.  f_i / 2 pi is held
// instead as a 64-bit fixed-point fraction F of a turn: p F mod 2^64 is the phase, exact in its 64 bits for every
// p (negative ones too) but for F's own rounding (p 2^-54 turns), in two integer multiplies.
//
// Bound by HBM: every element is read and written once.  A block takes a few rows of one batch entry in all heads of Q and
// K, or in some: its threads form each sine and cosine once, into shared memory, and then turn one vector of pairs each in
// every kth head.  Thread and block indices are the coordinates themselves: with rows counted through and divided out
// again (64-bit divisions), a block's beginning took longer than its copying.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "la_f32x2.cuh"
#include "la_internal.h"
#include "la_views.h"

namespace la {
namespace rot {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // D <= 256
constexpr int kTable = 1024;    // sines of a block
constexpr int kAhead = 4;       // heads of a thread on their way
// A block's last row and a thread's last head on its way are ints.
constexpr int kMaxRows = 0x7fffffff - 1024, kMaxHeads = (1 << 30) - 1;

struct Side {  // Q or K: from, to, their (batch, head, row) strides in elements
    const void *x;
    void *y;
    long long xs[3], ys[3];
    int H;     // heads (K: possibly none)
    int copy;  // the channels past R are copied (not in place)
};

struct Params {
    Side side[2];
    const int *positions;  // nullptr: first + row
    long long pos_stride;  // between batch entries
    long long first;
    int B, N, R, D;
    int heads;             // heads of a block
    float magnitude;
    int inverse;
    unsigned long long freq[kMaxPairs];
};

template <typename T, int V> struct alignas(V * sizeof(T)) VecN { T e[V]; };

__device__ __forceinline__ float load_f(float x) { return x; }
__device__ __forceinline__ float load_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T round_to(float x);
template <> __device__ __forceinline__ float round_to<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// cos and sin of pair i at position p, times the magnitude.
__device__ __forceinline__ void turn(const Params &P, long long p, int i, float &c, float &s) {
    const long long phase = (long long)((unsigned long long)p * P.freq[i]);  // in 2^-64 turns, signed
    sincospif((float)phase * 0x1p-63f, &s, &c);
    c *= P.magnitude;
    s *= P.inverse ? -P.magnitude : P.magnitude;
}

// A vector of 4, 8 or 16 bytes, global -> shared.
template <typename T, int V> __device__ __forceinline__ void copy_async(VecN<T, V> *dst, const T *src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (sizeof(VecN<T, V>) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"((int)sizeof(VecN<T, V>)) : "memory");
}

// (y1, y2) of two pairs side by side: x1 c - x2 s and x1 s + x2 c.
__device__ __forceinline__ void turn2(float2 &x1, float2 &x2, float2 c, float2 s) {
    const float2 m = mul2(x2, s), y1 = fma2(x1, c, make_float2(-m.x, -m.y));
    x2 = fma2(x1, s, mul2(x2, c));
    x1 = y1;
}

// Block (units, rows, heads side by side), grid (row tiles, head groups, batch).
// INTER: unit u is the 16-byte vector u of the row, V / 2 pairs, the last ones copied.  Otherwise unit u < R / 2 / V
// holds pairs u V ... as a vector of the first and one of the second half, and the units after those are the copied
// vectors.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ Params P) {
    constexpr int NP = INTER ? V / 2 : V;  // pairs per unit
    constexpr bool ASYNC = V * sizeof(T) >= 4;  // vectors that cp.async can copy
    __shared__ float2 turns[kTable];            // [row of the block][pair]: cos, sin
    // each thread's own ring of vectors on their way: only so do enough bytes fly (with the next head's vectors in
    // registers 4.0 TB/s, so 5.8)
    __shared__ VecN<T, V> ring[ASYNC ? kAhead : 1][INTER ? 1 : 2][kThreads];
    const int me = threadIdx.x + blockDim.x * (threadIdx.y + blockDim.y * threadIdx.z);
    const int u = threadIdx.x, r = threadIdx.y, n = blockIdx.x * blockDim.y + r;
    const int Hq = P.side[0].H, H = Hq + P.side[1].H;
    const int head0 = blockIdx.y * P.heads + threadIdx.z, head1 = min((int)(blockIdx.y + 1) * P.heads, H);
    const int step = blockDim.z, pairs = P.R / 2, half_units = pairs / V;
    const bool live = n < P.N, turned = INTER ? u * V < P.R : u < half_units;
    const int at1 = INTER || turned ? u * V : P.R + (u - half_units) * V, at2 = pairs + u * V;
    for (int b = blockIdx.z; b < P.B; b += gridDim.z) {
        // the row's vector in head h of Q and K together
        const T *xq = (const T *)P.side[0].x + b * P.side[0].xs[0] + n * P.side[0].xs[2] + at1;
        const T *xk = (const T *)P.side[1].x + b * P.side[1].xs[0] + n * P.side[1].xs[2] + at1 - Hq * P.side[1].xs[1];
        T *yq = (T *)P.side[0].y + b * P.side[0].ys[0] + n * P.side[0].ys[2] + at1;
        T *yk = (T *)P.side[1].y + b * P.side[1].ys[0] + n * P.side[1].ys[2] + at1 - Hq * P.side[1].ys[1];
        VecN<T, V> va, vb;
        auto fetch = [&](int h, int slot) {
            if (live && h < head1) {
                const T *x = h < Hq ? xq + h * P.side[0].xs[1] : xk + h * P.side[1].xs[1];
                if constexpr (ASYNC) {
                    copy_async(&ring[slot][0][me], x);
                    if (!INTER && turned) copy_async(&ring[slot][INTER ? 0 : 1][me], x + at2 - at1);
                } else {
                    va = *(const VecN<T, V> *)x;
                    if (!INTER && turned) vb = *(const VecN<T, V> *)(x + at2 - at1);
                }
            }
            if constexpr (ASYNC) asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if constexpr (ASYNC) {  // on their way while the sines are formed
#pragma unroll
            for (int k = 0; k < kAhead; ++k) fetch(head0 + k * step, k);
        }
        if (live) {
            const long long pos = P.positions ? (long long)P.positions[b * P.pos_stride + n] : P.first + n;
            for (int i = u + blockDim.x * threadIdx.z; i < pairs; i += blockDim.x * blockDim.z) {
                float2 cs;
                turn(P, pos, i, cs.x, cs.y);
                turns[r * pairs + i] = cs;
            }
        }
        __syncthreads();
        float c[NP], s[NP];
        if (live && turned) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const float2 cs = turns[r * pairs + (INTER ? min(u * NP + j, pairs - 1) : u * NP + j)];
                c[j] = cs.x, s[j] = cs.y;
            }
        }
        int slot = 0;
        for (int h = head0; h < head1; h += step) {
            if constexpr (ASYNC) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
                va = ring[slot][0][me];
                if (!INTER) vb = ring[slot][INTER ? 0 : 1][me];
            } else {
                fetch(h, 0);
            }
            if (!live) continue;
            T *y = h < Hq ? yq + h * P.side[0].ys[1] : yk + h * P.side[1].ys[1];
            if (!turned) {  // copied, unless in place
                if (P.side[h >= Hq].copy) *(VecN<T, V> *)y = va;
            } else {
                if constexpr (INTER) {
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        if (2 * (u * NP + j) >= P.R) continue;  // copied as it is (no product with 1: NaN payloads, -0)
                        const float x1 = load_f(va.e[2 * j]), x2 = load_f(va.e[2 * j + 1]);
                        const float2 z = fma2(make_float2(x1, x2), both(c[j]), mul2(make_float2(x2, x1), make_float2(-s[j], s[j])));
                        va.e[2 * j] = round_to<T>(z.x);
                        va.e[2 * j + 1] = round_to<T>(z.y);
                    }
                } else if constexpr (V == 1) {
                    const float x1 = load_f(va.e[0]), x2 = load_f(vb.e[0]);
                    va.e[0] = round_to<T>(x1 * c[0] - x2 * s[0]);
                    vb.e[0] = round_to<T>(x1 * s[0] + x2 * c[0]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        float2 x1 = make_float2(load_f(va.e[j]), load_f(va.e[j + 1]));
                        float2 x2 = make_float2(load_f(vb.e[j]), load_f(vb.e[j + 1]));
                        turn2(x1, x2, make_float2(c[j], c[j + 1]), make_float2(s[j], s[j + 1]));
                        va.e[j] = round_to<T>(x1.x), va.e[j + 1] = round_to<T>(x1.y);
                        vb.e[j] = round_to<T>(x2.x), vb.e[j + 1] = round_to<T>(x2.y);
                    }
                }
                *(VecN<T, V> *)y = va;
                if (!INTER) *(VecN<T, V> *)(y + at2 - at1) = vb;
            }
            if constexpr (ASYNC) {
                fetch(h + kAhead * step, slot);
                slot = (slot + 1) % kAhead;
            }
        }
        __syncthreads();  // the sines have been read
    }
}

template <typename T, int V, bool INTER> cudaError_t launch(Params &P, cudaStream_t s) {
    // Units fit into a block: V = 1 only where R / 2 is odd, and then there are at most D - R / 2 < 256 of them.
    const int units = INTER ? P.D / V : P.R / 2 / V + (P.D - P.R) / V, H = P.side[0].H + P.side[1].H;
    auto ceil = [](long long a, long long b) { return (a + b - 1) / b; };
    // Rows of a block: two warps' worth of vectors of one head (8 rows of 8: 47 us at 4 x 4096 x 32 heads of 128 in bf16, 4
    // rows 48, one row 74), and what the table holds; the rest of its threads take heads.
    int tile = units < 64 ? 64 / units : 1;
    if (tile > P.N) tile = P.N;
    while (tile > 1 && tile * (P.R / 2) > kTable) --tile;
    int par = kThreads / (units * tile);
    if (par > H) par = H;
    if (par > 64) par = 64;
    // Heads of a block: all of them, or fewer while that leaves the GPU without four blocks on each SM.
    P.heads = H;
    while (P.heads > par && ceil(P.N, tile) * P.B * ceil(H, P.heads) < 608) P.heads = (P.heads + 1) / 2;
    const long long gx = ceil(P.N, tile), gy = ceil(H, P.heads);
    if (gy > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)gx, (unsigned)gy, P.B < 65535 ? P.B : 65535);
    rotary_kernel<T, V, INTER><<<grid, dim3(units, tile, par), 0, s>>>(P);
    return cudaGetLastError();
}

// The widest vectors that halves of R / 2 channels are made of; interleaved pairs lie in 16-byte vectors.
template <typename T> cudaError_t by_layout(Params &P, int interleaved, cudaStream_t s) {
    constexpr int W = 16 / (int)sizeof(T);
    if (interleaved) return launch<T, W, true>(P, s);
    const int half = P.R / 2;
    if (half % W == 0) return launch<T, W, false>(P, s);
    if (W > 4 && half % 4 == 0) return launch<T, 4, false>(P, s);
    if (half % 2 == 0) return launch<T, 2, false>(P, s);
    return launch<T, 1, false>(P, s);
}

int rotary(const void *Q, const void *K, void *Qr, void *Kr, const unsigned long long *freq, const int *positions,
           long long position_stride, long long first, int interleaved, float magnitude, int inverse, int B, int Hq,
           int Hk, int N, int D, int R, int dtype, const long long *strides, void *stream) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (B < 0 || N < 0 || N > kMaxRows || Hq < 1 || Hk < 0 || D < 1) return LA_ERR_INVALID_ARG;
    if ((long long)Hq + Hk > kMaxHeads) return LA_ERR_INVALID_ARG;
    const int elem = dtype == LA_BF16 ? 2 : 4;
    if (D > 2 * kMaxPairs || (D * elem) % 16 != 0) return LA_ERR_UNSUPPORTED;
    if (R < 2 || R > D || R % 2 != 0 || !freq) return LA_ERR_INVALID_ARG;
    if (!(magnitude == magnitude) || position_stride < 0) return LA_ERR_INVALID_ARG;
    const long long rows = (long long)B * N;
    if (rows * (Hq > Hk ? Hq : Hk) >= (1LL << 40) / D) return LA_ERR_INVALID_ARG;
    if (rows == 0) return LA_OK;
    if (positions && position_stride != 0 && position_stride < N) return LA_ERR_INVALID_ARG;
    if (positions && ((uintptr_t)positions & 3)) return LA_ERR_INVALID_ARG;
    const int ns = Hk > 0 ? 2 : 1;
    const void *xs[2] = {Q, K};
    void *ys[2] = {Qr, Kr};
    const int H[2] = {Hq, Hk};
    View vx[2], vy[2];
    int rc;
    for (int k = 0; k < ns; ++k) {
        if (!xs[k] || !ys[k] || ((uintptr_t)xs[k] & 15) || ((uintptr_t)ys[k] & 15)) return LA_ERR_INVALID_ARG;
        const long long dense[3] = {(long long)H[k] * N * D, (long long)N * D, D};
        vx[k] = View{xs[k], {B, H[k], N}, {}, D, elem};
        vy[k] = View{ys[k], {B, H[k], N}, {}, D, elem};
        // (Q, K, Qr, Kr) x (batch, head, row)
        if ((rc = set_view(vx[k], strides ? strides + 3 * k : nullptr, dense))) return rc;
        if ((rc = set_view(vy[k], strides ? strides + 6 + 3 * k : nullptr, dense))) return rc;
    }
    // an output is its own input (in place), or meets no input; outputs do not meet; positions are apart from both
    const size_t pos_bytes = positions ? ((size_t)(B - 1) * position_stride + N) * sizeof(int) : 0;
    for (int k = 0; k < ns; ++k) {
        for (int j = 0; j < ns; ++j)
            if (!(j == k && same_view(vx[j], vy[k])) && views_meet(vy[k], vx[j])) return LA_ERR_INVALID_ARG;
        if (ranges_meet(ys[k], view_bytes(vy[k]), positions, pos_bytes)) return LA_ERR_INVALID_ARG;
    }
    if (ns == 2 && views_meet(vy[0], vy[1])) return LA_ERR_INVALID_ARG;
    Params P;
    memset(&P, 0, sizeof(P));
    for (int k = 0; k < ns; ++k) {
        Side &S = P.side[k];
        S.x = xs[k];
        S.y = ys[k];
        for (int d = 0; d < 3; ++d) {
            S.xs[d] = vx[k].st[d];
            S.ys[d] = vy[k].st[d];
        }
        S.H = H[k];
        S.copy = !same_view(vx[k], vy[k]);
    }
    P.positions = positions;
    P.pos_stride = position_stride;
    P.first = first;
    P.B = B;
    P.N = N;
    P.R = R;
    P.D = D;
    P.magnitude = magnitude;
    P.inverse = inverse;
    memcpy(P.freq, freq, (size_t)(R / 2) * sizeof(*freq));
    const cudaError_t e = dtype == LA_BF16 ? by_layout<__nv_bfloat16>(P, interleaved, (cudaStream_t)stream)
                                           : by_layout<float>(P, interleaved, (cudaStream_t)stream);
    if (e == cudaErrorInvalidConfiguration) return LA_ERR_INVALID_ARG;
    if (e != cudaSuccess) return LA_ERR_CUDA;
    count_launches(1);
    return LA_OK;
}

}  // namespace rot
}  // namespace la

extern "C" {

int la_rotary_frequencies(int rotary_dim, double base, int scaling, double factor, double original_length,
                          double low_turns, double high_turns, unsigned long long *frequencies) {
    const double two_pi = 6.283185307179586476925;
    if (!frequencies || rotary_dim < 2 || rotary_dim % 2 != 0) return LA_ERR_INVALID_ARG;
    if (rotary_dim > 2 * la::rot::kMaxPairs) return LA_ERR_UNSUPPORTED;
    if (!(base >= 1.0) || !isfinite(base)) return LA_ERR_INVALID_ARG;
    if (scaling != LA_ROTARY_NONE && scaling != LA_ROTARY_LINEAR && scaling != LA_ROTARY_BY_TURNS)
        return LA_ERR_INVALID_ARG;
    if (scaling != LA_ROTARY_NONE && (!(factor >= 1.0) || !isfinite(factor))) return LA_ERR_INVALID_ARG;
    if (scaling == LA_ROTARY_BY_TURNS &&
        (!(original_length > 0.0) || !isfinite(original_length) || !(low_turns >= 0.0) || !(high_turns > low_turns) ||
         !isfinite(high_turns)))
        return LA_ERR_INVALID_ARG;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rotary_dim);
        if (scaling == LA_ROTARY_LINEAR) f /= factor;
        if (scaling == LA_ROTARY_BY_TURNS) {
            double t = (original_length * f / two_pi - low_turns) / (high_turns - low_turns);
            t = t < 0.0 ? 0.0 : t > 1.0 ? 1.0 : t;
            f = (1.0 - t) * f / factor + t * f;
        }
        frequencies[i] = (unsigned long long)llrint(ldexp(f / two_pi, 64));  // f <= 1: below 2^62
    }
    return LA_OK;
}

int la_rotary(const void *Q, const void *K, void *Qr, void *Kr, const unsigned long long *frequencies,
              const int *positions, long long position_stride, long long first_position, int interleaved,
              float magnitude, int B, int Hq, int Hk, int N, int D, int rotary_dim, int dtype,
              const long long *strides, void *stream) {
    return la::rot::rotary(Q, K, Qr, Kr, frequencies, positions, position_stride, first_position, interleaved,
                           magnitude, 0, B, Hq, Hk, N, D, rotary_dim, dtype, strides, stream);
}

int la_rotary_backward(const void *dQr, const void *dKr, void *dQ, void *dK, const unsigned long long *frequencies,
                       const int *positions, long long position_stride, long long first_position, int interleaved,
                       float magnitude, int B, int Hq, int Hk, int N, int D, int rotary_dim, int dtype,
                       const long long *strides, void *stream) {
    return la::rot::rotary(dQr, dKr, dQ, dK, frequencies, positions, position_stride, first_position, interleaved,
                           magnitude, 1, B, Hq, Hk, N, D, rotary_dim, dtype, strides, stream);
}

}  // extern "C"
