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
// Bound by HBM: every element is read and written once.  One thread turns the same V pairs of one token in several
// heads of Q and K, so that a sine and a cosine serve up to kHeads rows.
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

struct Side {  // Q or K: from, to, their (batch, head, row) strides in elements
    const void *x;
    void *y;
    long long xs[3], ys[3];
    int H;     // heads
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
    int heads;             // heads of each thread
    int groups_q, groups;  // head groups of Q; of Q and K together
    float magnitude;
    int inverse;
    unsigned long long freq[kMaxPairs];
};

template <typename T> struct alignas(16) Vec16 { T e[16 / sizeof(T)]; };
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
// vectors.  Threads run over units, then rows, so that a warp's accesses are whole row pieces.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params P) {
    constexpr int NP = INTER ? V / 2 : V;  // pairs per unit
    constexpr int BATCH = 4;               // heads in flight
    const unsigned group = blockIdx.x % (unsigned)P.groups;
    const long long f = (long long)(blockIdx.x / (unsigned)P.groups) * kThreads + threadIdx.x;
    const long long row = f / P.units;
    const int u = (int)(f - row * P.units);
    if (row >= P.rows) return;
    const bool is_k = (int)group >= P.groups_q;
    const Side &S = P.side[is_k ? 1 : 0];
    const int h0 = ((int)group - (is_k ? P.groups_q : 0)) * P.heads;
    const int h1 = min(h0 + P.heads, S.H);
    const long long b = row / P.N, n = row - b * P.N;
    const T *x = (const T *)S.x + b * S.xs[0] + n * S.xs[2];
    T *y = (T *)S.y + b * S.ys[0] + n * S.ys[2];
    const int half_units = P.R / 2 / V;
    if (INTER ? u * V >= P.R : u >= half_units) {  // nothing but copied channels
        if (!S.copy) return;
        const int at = INTER ? u * V : P.R + (u - half_units) * V;
        for (int h = h0; h < h1; ++h)
            *(VecN<T, V> *)(y + h * S.ys[1] + at) = *(const VecN<T, V> *)(x + h * S.xs[1] + at);
        return;
    }
    const long long pos = P.positions ? (long long)P.positions[b * P.pos_stride + n] : P.first + n;
    float c[NP], s[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int i = u * NP + j;
        if (!INTER || 2 * i < P.R) turn(P, pos, i, c[j], s[j]);
        else c[j] = 1.f, s[j] = 0.f;
    }
    const int at1 = u * V, at2 = INTER ? u * V : P.R / 2 + u * V;
    for (int h = h0; h < h1; h += BATCH) {
        VecN<T, V> v1[BATCH], v2[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (h + k < h1) {
                v1[k] = *(const VecN<T, V> *)(x + (h + k) * S.xs[1] + at1);
                if (!INTER) v2[k] = *(const VecN<T, V> *)(x + (h + k) * S.xs[1] + at2);
            }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (h + k < h1) {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    T &e1 = INTER ? v1[k].e[2 * j] : v1[k].e[j];
                    T &e2 = INTER ? v1[k].e[2 * j + 1] : v2[k].e[j];
                    if (INTER && 2 * (u * NP + j) >= P.R) continue;  // copied as it is (no product with 1: NaN payloads, -0)
                    const float a = load_f(e1), d = load_f(e2);
                    e1 = round_to<T>(a * c[j] - d * s[j]);
                    e2 = round_to<T>(a * s[j] + d * c[j]);
                }
                *(VecN<T, V> *)(y + (h + k) * S.ys[1] + at1) = v1[k];
                if (!INTER) *(VecN<T, V> *)(y + (h + k) * S.ys[1] + at2) = v2[k];
            }
    }
}

template <typename T, int V, bool INTER> cudaError_t launch(Params &P, cudaStream_t s) {
    P.units = INTER ? P.D / V : P.R / 2 / V + (P.D - P.R) / V;
    const long long threads = P.rows * P.units;
    const long long blocks = (threads + kThreads - 1) / kThreads;
    // Heads per thread: up to 8, so that a sine serves 8 rows, fewer while that leaves the GPU without some 1024
    // threads on each SM: a token of a small batch is then one load, one turn and one store deep.
    const int sms = 152;
    P.heads = 8;
    auto groups = [&](int H) { return (H + P.heads - 1) / P.heads; };
    while (P.heads > 1 && threads * (groups(P.side[0].H) + groups(P.side[1].H)) < (long long)sms * 1024) P.heads /= 2;
    P.groups_q = groups(P.side[0].H);
    P.groups = P.groups_q + groups(P.side[1].H);
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
