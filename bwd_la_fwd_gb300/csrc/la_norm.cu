// la_norm.cu -- root-mean-square norm of rows with the residual's addition (la_rms_norm), with an output in 8 bits and
// scales (la_rms_norm_8bit), and its gradients (la_rms_norm_backward).
//
//   r = x + residual,  y = w r rstd,  rstd = (mean r^2 + eps)^-1/2
//   backward, at r as stored: g = w dy,  dx = dr + rstd (g - r rstd^2 mean(g r)),  dw = sum over rows of dy r rstd
//
// A row is read once into registers: TPR threads with NV 16-byte vectors each.  What bounds it is HBM (forward x, residual,
// r, y; backward r, dy, dr, dx).  The blocks stand on all SMs at once and walk the rows, one or two at a time for each group of
// TPR threads, the next ones' loads on their way meanwhile and the weights in registers (4 x 4096 x 2048 with a residual, bf16:
// 45.1 us, 5.9 TB/s; without loads ahead and with eight blocks to an SM 94; four blocks for three change nothing).  The
// gradient of 8 x 2048 x 2048 takes 60 us (4.5 TB/s): two sums a row and the parts of dw, 304 rows of them, added by a second
// launch.  r is normed as the fp32 sum, not as rounded to the tokens' type: y then passes one rounding.
#include <math.h>

#include <type_traits>

#include "la_rows.cuh"

namespace la {
namespace norm {

using namespace rows;

constexpr int kMaxC = 16384;
constexpr int kBlock = 128;        // channels of an 8-bit scale (else the whole row)
constexpr float kTop = 448.f;      // the largest e4m3 value
constexpr float kLeast = 7.888609e-31f;  // 2^-100: a scale stands for at least so much, so that 448 / it is a number
constexpr int kSMs = 152;

struct Params {
    Op x, res, r, y, dr;       // forward: r the sum's output; backward: x = r as stored, y = dy, r = dx
    const float *w;
    unsigned char *y8;         // 8-bit output, contiguous
    float *scales;             // contiguous [rows][groups]
    float *part;               // backward: partial sums of dw
    long long rows;
    int N, C, groups;
    float eps;
};

enum : int { kPlain = 0, kRow8, kBlock8 };  // kinds of output

template <typename T, int TPR_, int NV_> struct Shape {
    static constexpr int V = 16 / (int)sizeof(T), TPR = TPR_, NV = NV_;
    static constexpr int THREADS = TPR > 256 ? TPR : 256;
    static constexpr int GROUPS = THREADS / TPR;  // rows at a time of a block
    static constexpr int RPI = NV == 1 ? 2 : 1;  // rows at a time of a group
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// K values for each of the TPR threads of a group, combined over them; all threads of the block call it.
template <int TPR, int THREADS, int K, bool MAX> __device__ __forceinline__ void combine(float (&x)[K], float *sm) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float o = __shfl_xor_sync(0xffffffffu, x[k], d);
            x[k] = MAX ? max_nan(x[k], o) : x[k] + o;
        }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5, group = warp / W;
        __syncthreads();  // the last values have been read
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) sm[k * (THREADS / 32) + warp] = x[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float a = sm[k * (THREADS / 32) + group * W];
#pragma unroll
            for (int j = 1; j < W; ++j) {
                const float o = sm[k * (THREADS / 32) + group * W + j];
                a = MAX ? max_nan(a, o) : a + o;
            }
            x[k] = a;
        }
    }
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// N = 0: the batch entries' rows lie evenly spaced, one entry behind another.
template <typename T> __device__ __forceinline__ T *row_of(const Op &o, long long row, int N) {
    if (N == 0) return (T *)o.p + row * o.sn;
    const long long b = row / N;
    return (T *)o.p + b * o.sb + (row - b * N) * o.sn;
}

// Blocks on an SM, which walk all rows.
template <int TPR> constexpr int back_per_sm() { return TPR > 256 ? 1 : 2; }  // each leaves sums of dw
template <int TPR> constexpr int per_sm() { return TPR > 256 ? 1 : 3; }

template <typename T, int TPR, int NV, int KIND>
__global__ void __launch_bounds__(Shape<T, TPR, NV>::THREADS, per_sm<TPR>()) forward_kernel(const __grid_constant__ Params P) {
    using S = Shape<T, TPR, NV>;
    constexpr int V = S::V, R = S::RPI;
    __shared__ float sm[R * S::THREADS / 32];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const float per = 1.f / (float)P.C;
    float w[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (i * TPR + t) * V + k;
            w[i][k] = c < P.C ? P.w[c] : 0.f;
        }
    const long long step = (long long)gridDim.x * S::GROUPS * R;
    Vec<T, V> x[R][NV], a[R][NV];  // the next rows, on their way while the last are normed
    auto fetch = [&](long long first) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * V;
                const bool on = first + j < P.rows && P.C - c >= V;
                load_ahead(x[j][i], row_of<T>(P.x, first + j, P.N) + c, on);
                if (P.res.p) load_ahead(a[j][i], row_of<T>(P.res, first + j, P.N) + c, on);
            }
    };
    fetch((long long)blockIdx.x * S::GROUPS * R + group * R);
    for (long long base = (long long)blockIdx.x * S::GROUPS * R; base < P.rows; base += step) {
        const long long first = base + group * R;
        float r[R][NV][V], ss[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            ss[j] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * V, n = P.C - c;
                const bool in = first + j < P.rows && n > 0;
                if (in && n < V) {  // the last channels, where they are no whole vector
                    x[j][i] = load_vec<T, V>(row_of<T>(P.x, first + j, P.N) + c, n);
                    if (P.res.p) a[j][i] = load_vec<T, V>(row_of<T>(P.res, first + j, P.N) + c, n);
                }
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float v = to_f(x[j][i].e[k]);
                    if (P.res.p) v += to_f(a[j][i].e[k]);
                    r[j][i][k] = in ? v : 0.f;
                    ss[j] = fmaf(r[j][i][k], r[j][i][k], ss[j]);
                }
            }
        }
        fetch(first + step);
        if (P.r.p)
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (i * TPR + t) * V, n = first + j < P.rows ? P.C - c : 0;
                    if (n <= 0) continue;
                    Vec<T, V> o;
#pragma unroll
                    for (int k = 0; k < V; k += 2) put2(o.e + k, r[j][i][k], r[j][i][k + 1]);
                    store_vec<T, V>(row_of<T>(P.r, first + j, P.N) + c, o, n);
                }
        combine<TPR, S::THREADS, R, false>(ss, sm);
        float top[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float rstd = rsqrtf(fmaf(ss[j], per, P.eps));
            top[j] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    r[j][i][k] *= rstd * w[i][k];
                    if (KIND == kRow8) top[j] = max_nan(top[j], fabsf(r[j][i][k]));
                }
        }
        if (KIND == kRow8) combine<TPR, S::THREADS, R, true>(top, sm);
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * V, n = first + j < P.rows ? P.C - c : 0;
                if (KIND == kPlain) {
                    if (n <= 0) continue;
                    Vec<T, V> o;
#pragma unroll
                    for (int k = 0; k < V; k += 2) put2(o.e + k, r[j][i][k], r[j][i][k + 1]);
                    store_vec<T, V>(row_of<T>(P.y, first + j, P.N) + c, o, n);
                } else {
                    float a = top[j];
                    if (KIND == kBlock8) {  // kBlock channels are neighbouring lanes
                        a = 0.f;
#pragma unroll
                        for (int k = 0; k < V; ++k) a = max_nan(a, fabsf(r[j][i][k]));
#pragma unroll
                        for (int d = kBlock / V / 2; d > 0; d >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, d));
                    }
                    a = max_nan(a, kLeast);
                    if (n <= 0) continue;
                    const int at = KIND == kRow8 ? 0 : c / kBlock;
                    if (c % (KIND == kRow8 ? kMaxC : kBlock) == 0) P.scales[(first + j) * P.groups + at] = __fdividef(a, kTop);
                    const float s = kTop / a;  // (an infinite a: 0, and its own value NaN)
                    unsigned char *out = P.y8 + (first + j) * P.C + c;
                    uint32_t q[V / 4];
#pragma unroll
                    for (int k = 0; k < V; k += 4)
                        q[k / 4] = e4m3x4(r[j][i][k] * s, r[j][i][k + 1] * s, r[j][i][k + 2] * s, r[j][i][k + 3] * s);
                    if (n >= V && ((uintptr_t)out % V) == 0) {
                        if constexpr (V == 8) *(uint2 *)out = make_uint2(q[0], q[1]);
                        else *(uint32_t *)out = q[0];
                    } else {
#pragma unroll
                        for (int k = 0; k < V; ++k)
                            if (k < n) out[k] = (unsigned char)(q[k / 4] >> (8 * (k % 4)));
                    }
                }
            }
    }
}

template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(Shape<T, TPR, NV>::THREADS, back_per_sm<TPR>()) backward_kernel(const __grid_constant__ Params P) {
    using S = Shape<T, TPR, NV>;
    constexpr int V = S::V, R = S::RPI;
    __shared__ float sm[2 * R * S::THREADS / 32];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const float per = 1.f / (float)P.C;
    float w[NV][V], dw[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (i * TPR + t) * V + k;
            w[i][k] = c < P.C ? P.w[c] : 0.f;
            dw[i][k] = 0.f;
        }
    const long long step = (long long)gridDim.x * S::GROUPS * R;
    Vec<T, V> nr[R][NV], ny[R][NV], nd[R][NV];  // the next rows, on their way meanwhile
    auto fetch = [&](long long first) {
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * V;
                const bool on = first + j < P.rows && P.C - c >= V;
                load_ahead(nr[j][i], row_of<T>(P.x, first + j, P.N) + c, on);
                load_ahead(ny[j][i], row_of<T>(P.y, first + j, P.N) + c, on);
                if (P.dr.p) load_ahead(nd[j][i], row_of<T>(P.dr, first + j, P.N) + c, on);
            }
    };
    fetch((long long)blockIdx.x * S::GROUPS * R + group * R);
    for (long long base = (long long)blockIdx.x * S::GROUPS * R; base < P.rows; base += step) {
        const long long first = base + group * R;
        Vec<T, V> r[R][NV], dy[R][NV], dr[R][NV];
        float sums[2 * R];  // of r^2, of g r
#pragma unroll
        for (int j = 0; j < R; ++j) {
            sums[j] = sums[R + j] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * V, n = first + j < P.rows ? P.C - c : 0;
                r[j][i] = nr[j][i], dy[j][i] = ny[j][i], dr[j][i] = nd[j][i];
                if (n > 0 && n < V) {  // the last channels, where they are no whole vector
                    r[j][i] = load_vec<T, V>(row_of<T>(P.x, first + j, P.N) + c, n);
                    dy[j][i] = load_vec<T, V>(row_of<T>(P.y, first + j, P.N) + c, n);
                    if (P.dr.p) dr[j][i] = load_vec<T, V>(row_of<T>(P.dr, first + j, P.N) + c, n);
                }
                if (n <= 0)
#pragma unroll
                    for (int k = 0; k < V; ++k) r[j][i].e[k] = dy[j][i].e[k] = T(0.f);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float x = to_f(r[j][i].e[k]);
                    sums[j] = fmaf(x, x, sums[j]);
                    sums[R + j] = fmaf(w[i][k] * to_f(dy[j][i].e[k]), x, sums[R + j]);
                }
            }
        }
        fetch(first + step);
        combine<TPR, S::THREADS, 2 * R, false>(sums, sm);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float rstd = rsqrtf(fmaf(sums[j], per, P.eps)), m = sums[R + j] * per * rstd * rstd;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * V, n = first + j < P.rows ? P.C - c : 0;
                if (n <= 0) continue;
                Vec<T, V> o;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float x = to_f(r[j][i].e[k]), d = to_f(dy[j][i].e[k]);
                    dw[i][k] = fmaf(d, x * rstd, dw[i][k]);
                    const float dx = rstd * fmaf(-x, m, w[i][k] * d);
                    put(&o.e[k], P.dr.p ? dx + to_f(dr[j][i].e[k]) : dx);
                }
                store_vec<T, V>(row_of<T>(P.r, first + j, P.N) + c, o, n);
            }
        }
    }
    float *part = P.part + ((long long)blockIdx.x * S::GROUPS + group) * P.C;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = (i * TPR + t) * V + k;
            if (c < P.C) part[c] = dw[i][k];
        }
}

template <typename T, int TPR, int NV> cudaError_t launch_forward(const Params &P, int kind, cudaStream_t s) {
    using S = Shape<T, TPR, NV>;
    const long long need = (P.rows + S::GROUPS * S::RPI - 1) / (S::GROUPS * S::RPI);
    const int most = per_sm<TPR>() * kSMs;
    const unsigned grid = (unsigned)(need < most ? need : most);
    auto *k = kind == kPlain ? forward_kernel<T, TPR, NV, kPlain>
              : kind == kRow8 ? forward_kernel<T, TPR, NV, kRow8>
                              : forward_kernel<T, TPR, NV, kBlock8>;
    k<<<grid, S::THREADS, 0, s>>>(P);
    return cudaGetLastError();
}

template <typename T, int TPR, int NV> int parts_of(long long rows) {
    using S = Shape<T, TPR, NV>;
    const long long need = (rows + S::GROUPS * S::RPI - 1) / (S::GROUPS * S::RPI);
    constexpr int most = back_per_sm<TPR>() * kSMs;
    return (int)(need < most ? need : most) * S::GROUPS;
}

template <typename T, int TPR, int NV> cudaError_t launch_backward(const Params &P, float *dw, cudaStream_t s) {
    using S = Shape<T, TPR, NV>;
    const int parts = parts_of<T, TPR, NV>(P.rows);
    backward_kernel<T, TPR, NV><<<(unsigned)(parts / S::GROUPS), S::THREADS, 0, s>>>(P);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : sum_parts(P.part, parts, P.C, dw, P.C, nullptr, 0, nullptr, s);
}

// f(TPR, NV) for rows of n vectors of V elements: as few threads as hold a row in one to four vectors each (in eight, the
// widest fp32 rows).
template <int V, typename F> auto by_shape(int n, F f) {
    using std::integral_constant;
    if (n <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (n <= 64) return f(integral_constant<int, 32>(), integral_constant<int, 2>());
    if (n <= 128) return f(integral_constant<int, 128>(), integral_constant<int, 1>());
    if (n <= 256) return f(integral_constant<int, 256>(), integral_constant<int, 1>());
    if (n <= 512) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (n <= 1024) return f(integral_constant<int, 512>(), integral_constant<int, 2>());
    if (V == 8 || n <= 2048) return f(integral_constant<int, 512>(), integral_constant<int, 4>());
    return f(integral_constant<int, 512>(), integral_constant<int, V == 8 ? 4 : 8>());
}

template <typename T> cudaError_t forward(const Params &P, int kind, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    return by_shape<V>((P.C + V - 1) / V, [&](auto tpr, auto nv) { return launch_forward<T, tpr.value, nv.value>(P, kind, s); });
}
template <typename T> cudaError_t backward(const Params &P, float *dw, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    return by_shape<V>((P.C + V - 1) / V, [&](auto tpr, auto nv) { return launch_backward<T, tpr.value, nv.value>(P, dw, s); });
}

// Sums of dw that a call may leave, whatever its type and rows.
int most_parts(int C) {
    auto parts = [](auto tpr, auto) { return back_per_sm<tpr.value>() * kSMs * (tpr.value >= 256 ? 1 : 256 / tpr.value); };
    const int a = by_shape<8>((C + 7) / 8, parts), b = by_shape<4>((C + 3) / 4, parts);
    return a > b ? a : b;
}

int check_sizes(int B, int N, int C, float eps, int dtype, bool *empty) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (B < 0 || N < 0 || N > kMaxRows || C < 1 || !(eps >= 0.f) || !(eps < INFINITY)) return LA_ERR_INVALID_ARG;
    if ((long long)B * N >= (1LL << 40) / C) return LA_ERR_INVALID_ARG;
    if (C > kMaxC) return LA_ERR_UNSUPPORTED;
    *empty = B == 0 || N == 0;
    return LA_OK;
}

// Whether the batch entries' rows follow one another evenly in all operands.
bool flat(const View *const *v, int n, int B, int N) {
    for (int k = 0; k < n; ++k)
        if (v[k]->p && B > 1 && (N == 1 ? false : v[k]->st[0] != N * v[k]->st[1])) return false;
    return B == 1 || N > 1;
}

// The forward calls: y is a view of the tokens' type, or y8 and its scales.
int forward_call(const void *X, const void *residual, const float *weight, void *sum, void *Y, unsigned char *y8,
                 float *scales, int group, int B, int N, int C, float eps, int dtype, const long long *strides,
                 cudaStream_t s) {
    bool empty;
    int rc = check_sizes(B, N, C, eps, dtype, &empty);
    if (rc) return rc;
    if (y8 && group != 0 && group != kBlock) return LA_ERR_INVALID_ARG;
    if ((residual != nullptr) != (sum != nullptr)) return LA_ERR_INVALID_ARG;
    if (empty) return LA_OK;
    const int elem = dtype == LA_BF16 ? 2 : 4;
    View x = {}, res = {}, r = {}, y = {};
    auto st = [&](int k) { return strides ? strides + 2 * k : nullptr; };
    if ((rc = rows_view(x, X, B, N, C, elem, st(0)))) return rc;
    if (residual && (rc = rows_view(res, residual, B, N, C, elem, st(1)))) return rc;
    if (sum && (rc = rows_view(r, sum, B, N, C, elem, st(2)))) return rc;
    if (!y8 && (rc = rows_view(y, Y, B, N, C, elem, st(3)))) return rc;
    if (!weight || ((uintptr_t)weight & 15)) return LA_ERR_INVALID_ARG;
    const long long n = (long long)B * N;
    const int groups = y8 && group ? (C + kBlock - 1) / kBlock : 1;
    const Range rin[1] = {{weight, (size_t)C * 4}};
    const Range rout[2] = {{y8, (size_t)n * C}, {scales, (size_t)n * groups * 4}};
    if (y8 && (((uintptr_t)y8 & 15) || !scales || ((uintptr_t)scales & 3))) return LA_ERR_INVALID_ARG;
    // A row is read before any of it is written, so an output may be an input itself; else they are apart.
    const View in[2] = {x, res}, out[2] = {r, y};
    for (int o = 0; o < 2; ++o)
        for (int k = 0; k < 2; ++k)
            if (out[o].p && in[k].p && !same_view(out[o], in[k]) && views_meet(out[o], in[k])) return LA_ERR_INVALID_ARG;
    if (outputs_meet(nullptr, 0, out, 2, rin, 1, rout, 2)) return LA_ERR_INVALID_ARG;
    if (outputs_meet(in, 2, nullptr, 0, nullptr, 0, rout, 2)) return LA_ERR_INVALID_ARG;
    Params P = {};
    P.x = Op{X, x.st[0], x.st[1]};
    P.res = Op{residual, res.st[0], res.st[1]};
    P.r = Op{sum, r.st[0], r.st[1]};
    P.y = Op{Y, y.st[0], y.st[1]};
    P.w = weight;
    P.y8 = y8;
    P.scales = scales;
    P.rows = n;
    const View *const ops[4] = {&x, &res, &r, &y};
    P.N = flat(ops, 4, B, N) ? 0 : N, P.C = C, P.groups = groups, P.eps = eps;
    const int kind = !y8 ? kPlain : group ? kBlock8 : kRow8;
    const cudaError_t e = dtype == LA_BF16 ? forward<__nv_bfloat16>(P, kind, s) : forward<float>(P, kind, s);
    if (e != cudaSuccess) return LA_ERR_CUDA;
    count_launches(1);
    return LA_OK;
}

}  // namespace norm

namespace rows {

constexpr int kSumCols = 32, kSumRows = 16;

__global__ void __launch_bounds__(kSumCols *kSumRows) sum_parts_kernel(const float *part, int parts, long long M, float *out0,
                                                                       long long n0, float *out1, long long n1, float *out2) {
    __shared__ float sm[kSumRows][kSumCols + 1];
    const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;
    const long long m = (long long)blockIdx.x * kSumCols + col;
    float a = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the launch before, which left the parts, is done
    if (m < M) {
#pragma unroll 8
        for (int p = row; p < parts; p += kSumRows) a += part[p * M + m];
    }
    sm[row][col] = a;
    __syncthreads();
    if (row == 0 && m < M) {
#pragma unroll
        for (int k = 1; k < kSumRows; ++k) a += sm[k][col];
        float *o = m < n0 ? out0 : m < n0 + n1 ? out1 : out2;
        if (o) o[m < n0 ? m : m < n0 + n1 ? m - n0 : m - n0 - n1] = a;
    }
}

cudaError_t sum_parts(const float *part, int parts, long long M, float *out0, long long n0, float *out1, long long n1,
                      float *out2, cudaStream_t s) {
    const long long blocks = (M + kSumCols - 1) / kSumCols;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    // Begun while the launch before it ends (8 x 2048 x 2048 gradient of the norm: 63.5 us without this).
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kSumCols * kSumRows);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, sum_parts_kernel, part, parts, M, out0, n0, out1, n1, out2);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace rows
}  // namespace la

extern "C" {

int la_rms_norm(const void *X, const void *residual, const float *weight, void *sum, void *Y, int B, int N, int C,
                float eps, int dtype, const long long *strides, void *stream) {
    return la::norm::forward_call(X, residual, weight, sum, Y, nullptr, nullptr, 0, B, N, C, eps, dtype, strides,
                                  (cudaStream_t)stream);
}

int la_rms_norm_8bit(const void *X, const void *residual, const float *weight, void *sum, unsigned char *Y8,
                     float *scales, int group, int B, int N, int C, float eps, int dtype, const long long *strides,
                     void *stream) {
    if (!Y8 && B > 0 && N > 0) return LA_ERR_INVALID_ARG;
    static unsigned char none;  // an empty call's place: checks only
    return la::norm::forward_call(X, residual, weight, sum, nullptr, Y8 ? Y8 : &none, scales, group, B, N, C, eps, dtype,
                                  strides, (cudaStream_t)stream);
}

size_t la_rms_norm_workspace_bytes(int C) {
    if (C < 1 || C > la::norm::kMaxC) return 0;
    return 256 + (size_t)la::norm::most_parts(C) * C * sizeof(float);
}

int la_rms_norm_backward(const void *R, const float *weight, const void *dY, const void *dR, void *dX, float *dweight,
                         int B, int N, int C, float eps, int dtype, const long long *strides, void *workspace,
                         size_t workspace_bytes, void *stream) {
    using namespace la;
    using namespace la::norm;
    bool empty;
    int rc = check_sizes(B, N, C, eps, dtype, &empty);
    if (rc) return rc;
    const int elem = dtype == LA_BF16 ? 2 : 4;
    if (!weight || ((uintptr_t)weight & 15) || !dweight || ((uintptr_t)dweight & 15)) return LA_ERR_INVALID_ARG;
    const size_t need = la_rms_norm_workspace_bytes(C);
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need) return LA_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    const Range rin[1] = {{weight, (size_t)C * 4}}, rout[2] = {{dweight, (size_t)C * 4}, {workspace, need}};
    if (outputs_meet(nullptr, 0, nullptr, 0, rin, 1, rout, 2)) return LA_ERR_INVALID_ARG;
    if (empty) {  // no rows: their sum is zero
        return sum_parts(nullptr, 0, C, dweight, C, nullptr, 0, nullptr, s) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    View r = {}, dy = {}, dr = {}, dx = {};
    auto st = [&](int k) { return strides ? strides + 2 * k : nullptr; };
    if ((rc = rows_view(r, R, B, N, C, elem, st(0)))) return rc;
    if ((rc = rows_view(dy, dY, B, N, C, elem, st(1)))) return rc;
    if (dR && (rc = rows_view(dr, dR, B, N, C, elem, st(2)))) return rc;
    if ((rc = rows_view(dx, dX, B, N, C, elem, st(3)))) return rc;
    const View in[3] = {r, dy, dr};
    for (const View &v : in)
        if (v.p && !same_view(dx, v) && views_meet(dx, v)) return LA_ERR_INVALID_ARG;
    if (outputs_meet(in, 3, nullptr, 0, nullptr, 0, rout, 2)) return LA_ERR_INVALID_ARG;
    if (outputs_meet(nullptr, 0, &dx, 1, rin, 1, rout, 2)) return LA_ERR_INVALID_ARG;
    Params P = {};
    P.x = Op{R, r.st[0], r.st[1]};
    P.y = Op{dY, dy.st[0], dy.st[1]};
    P.dr = Op{dR, dr.st[0], dr.st[1]};
    P.r = Op{dX, dx.st[0], dx.st[1]};
    P.w = weight;
    P.part = (float *)((char *)workspace + 256);
    P.rows = (long long)B * N;
    const View *const ops[4] = {&r, &dy, &dr, &dx};
    P.N = flat(ops, 4, B, N) ? 0 : N, P.C = C, P.eps = eps;
    const cudaError_t e = dtype == LA_BF16 ? backward<__nv_bfloat16>(P, dweight, s) : backward<float>(P, dweight, s);
    if (e != cudaSuccess) return LA_ERR_CUDA;
    count_launches(1);
    return LA_OK;
}

}  // extern "C"
