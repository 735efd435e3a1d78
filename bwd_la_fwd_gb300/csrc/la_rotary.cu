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
// Bound by HBM: every element is read and written once.  A block takes a few rows (tokens) in all heads of Q and K, or in
// some: its threads form each sine and cosine once, into shared memory, and then turn one vector of pairs each in every
// kth head.  (With the sines formed by each thread for the 8 heads it turned, they took as long as the copying.)
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "la_internal.h"
#include "la_views.h"

namespace la {
namespace rot {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // D <= 256
constexpr int kTable = 2048;    // sines of a block

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
    long long rows;        // B N
    int N, R, D;
    int units;             // vectors a row is cut into
    int tile;              // rows of a block
    int par;               // heads turned side by side
    int heads, groups;     // heads of a block, blocks that a row's heads are spread over
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

// INTER: unit u is the 16-byte vector u of the row, V / 2 pairs, the last ones copied.  Otherwise unit u < R / 2 / V
// holds pairs u V ... as a vector of the first and one of the second half, and the units after those are the copied
// vectors.  Threads run over units, then rows, then heads, so that a warp's accesses are whole row pieces.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const __grid_constant__ Params P) {
    constexpr int NP = INTER ? V / 2 : V;  // pairs per unit
    constexpr int BATCH = 4;               // heads in flight
    __shared__ float2 turns[kTable];       // [row of the block][pair]: cos, sin
    const long long row0 = (long long)(blockIdx.x / (unsigned)P.groups) * P.tile;
    const int head0 = (int)(blockIdx.x % (unsigned)P.groups) * P.heads, H = P.side[0].H + P.side[1].H;
    const int head1 = min(head0 + P.heads, H);
    const int t = threadIdx.x, u = t % P.units, r = t / P.units % P.tile, lane = t / (P.units * P.tile);
    const long long row = row0 + r;
    const bool live = lane < P.par && row < P.rows;
    const long long b = row / P.N, n = row - b * P.N;
    const int half_units = P.R / 2 / V;
    const bool turned = INTER ? u * V < P.R : u < half_units;
    const int at1 = INTER || turned ? u * V : P.R + (u - half_units) * V, at2 = INTER ? 0 : P.R / 2 + u * V;
    // this thread's vectors in head h of Q and K together
    auto from = [&](int h) {
        const bool k = h >= P.side[0].H;
        const Side &S = P.side[k];
        return (const T *)S.x + b * S.xs[0] + n * S.xs[2] + (k ? h - P.side[0].H : h) * S.xs[1];
    };
    VecN<T, V> v1[BATCH], v2[BATCH];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (live && h + k * P.par < head1) {
                const T *x = from(h + k * P.par);
                v1[k] = *(const VecN<T, V> *)(x + at1);
                if (!INTER && turned) v2[k] = *(const VecN<T, V> *)(x + at2);
            }
    };
    load(head0 + lane);  // on their way while the sines are formed
    const int pairs = P.R / 2;
    for (int i = t; i < P.tile * pairs; i += kThreads) {
        const long long at = row0 + i / pairs;
        if (at >= P.rows) break;
        const long long ab = at / P.N, an = at - ab * P.N;
        const long long pos = P.positions ? (long long)P.positions[ab * P.pos_stride + an] : P.first + an;
        float2 cs;
        turn(P, pos, i % pairs, cs.x, cs.y);
        turns[i] = cs;
    }
    __syncthreads();
    float c[NP], s[NP];
    if (turned && live) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            const int i = u * NP + j;
            const float2 cs = turns[r * pairs + (INTER ? min(i, pairs - 1) : i)];
            c[j] = cs.x, s[j] = cs.y;
        }
    }
    for (int h = head0 + lane; h < head1; h += BATCH * P.par) {
        if (h != head0 + lane) load(h);
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (h + k * P.par < head1) {
                const int hh = h + k * P.par;
                const bool is_k = hh >= P.side[0].H;
                const Side &S = P.side[is_k];
                T *y = (T *)S.y + b * S.ys[0] + n * S.ys[2] + (is_k ? hh - P.side[0].H : hh) * S.ys[1];
                if (!turned) {
                    if (S.copy) *(VecN<T, V> *)(y + at1) = v1[k];
                    continue;
                }
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    T &e1 = INTER ? v1[k].e[2 * j] : v1[k].e[j];
                    T &e2 = INTER ? v1[k].e[2 * j + 1] : v2[k].e[j];
                    if (INTER && 2 * (u * NP + j) >= P.R) continue;  // copied as it is (no product with 1: NaN payloads, -0)
                    const float x1 = load_f(e1), x2 = load_f(e2);
                    e1 = round_to<T>(x1 * c[j] - x2 * s[j]);
                    e2 = round_to<T>(x1 * s[j] + x2 * c[j]);
                }
                *(VecN<T, V> *)(y + at1) = v1[k];
                if (!INTER) *(VecN<T, V> *)(y + at2) = v2[k];
            }
    }
}

template <typename T, int V, bool INTER> cudaError_t launch(Params &P, cudaStream_t s) {
    P.units = INTER ? P.D / V : P.R / 2 / V + (P.D - P.R) / V;
    // Rows of a block: as many as its threads take of one head (contiguous pieces of 8 KB and more: with 1 KB, 4 rows of 8
    // heads at a time, DRAM gave 2.9 instead of 3.6 TB/s), as the table holds, and so that every SM has two blocks.
    // Units fit into a block: V = 1 only where R / 2 is odd, and then there are at most D - R / 2 < 256 of them.
    P.tile = kThreads / P.units;
    while (P.tile > 1 && (P.tile * (P.R / 2) > kTable || (P.rows + P.tile - 1) / P.tile < 304)) P.tile = (P.tile + 1) / 2;
    P.par = kThreads / (P.units * P.tile);
    // Heads of a block: all of them, or fewer while that leaves the GPU without two blocks on each SM.
    const int H = P.side[0].H + P.side[1].H;
    const long long blocks = (P.rows + P.tile - 1) / P.tile;
    P.heads = H;
    while (P.heads > P.par && blocks * ((H + P.heads - 1) / P.heads) < 304) P.heads = (P.heads + 1) / 2;
    P.groups = (H + P.heads - 1) / P.heads;
    if (blocks * P.groups >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    rotary_kernel<T, V, INTER><<<(unsigned)(blocks * P.groups), kThreads, 0, s>>>(P);
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
    if (B < 0 || N < 0 || Hq < 1 || Hk < 0 || D < 1) return LA_ERR_INVALID_ARG;
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
    P.rows = rows;
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
