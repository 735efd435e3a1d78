// la_conv.cu -- short causal convolution over time, each channel by itself (la_short_conv), its gradients
// (la_short_conv_backward) and one token of it (la_short_conv_step).
//
//   p_t = bias + sum_j w_j x_{t-K+1+j},  o = p or p sigmoid(p);  K taps; before a sequence's first row stand the K - 1
//   rows of its state, or zeros; its last K - 1 inputs are the state that it leaves
//   backward: dp = do (o's derivative at p),  dx_t = sum_j w_j dp_{t+K-1-j},  dw_j = sum_t dp_t x_{t-K+1+j}
//
// A thread has four channels and walks a run of rows, the last K - 1 of them in registers as fp32 pairs and the next ones on
// their way, so each row is read once (and K - 1 rows again at a run's start).  Runs are as long as lets all blocks stand on the
// SMs at once.  HBM and issue slots (56 %) bound it alike: 12,000 x 4096, bf16, four taps: 45 us, 4.4 TB/s (runs of 32 rows 53 us, each
// tap's conversion by itself 47).  The backward walk is the same with a second window, of dp: dx of a row is complete K - 1
// rows later, so a run computes dp of the K - 1 rows behind it again (2 x 2047 x 2048, fp32: 32 us, of which the sums of the runs'
// dw are a second launch).  Sums are fp32.
#include "la_f32x2.cuh"
#include "la_rows.cuh"

namespace la {
namespace conv {

using namespace rows;

constexpr int kThreads = 128;
constexpr int kRun = 8;           // rows of a run at least
constexpr int kMaxParts = 256;    // runs of the backward walk
constexpr int kMaxK = 4;
constexpr int kAhead = 4, kFwdAhead = 8;  // rows loaded together
constexpr int kV = 4;            // channels of a thread
constexpr int kSMs = 152, kPerSM = 4, kBackPerSM = 3;  // blocks on an SM, all at once

struct Params {
    Op x, o, dO;                  // forward: x, o; backward: x, do, and o is dx
    const float *w, *bias;        // [C][K], [C] or null
    const void *first;            // [nseq][K - 1][C], or null: zeros
    void *last;                   // [nseq][K - 1][C], or null: not written
    Seqs seq;
    int C, run;                   // rows of a run
    float *part;                  // backward: [parts][C][K], then [C], of each part
};

// Taps and bias of a thread's channels, in pairs.
template <int K> struct Taps {
    float2 w[K][kV / 2], bias[kV / 2];
    __device__ __forceinline__ Taps(const Params &P, int c) {
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const bool in = c + k < P.C;
            float t[K];
            if constexpr (K == 4) {
                const float4 f = in ? *(const float4 *)(P.w + (long long)(c + k) * K) : make_float4(0.f, 0.f, 0.f, 0.f);
                t[0] = f.x, t[1] = f.y, t[2] = f.z, t[3] = f.w;
            } else {
#pragma unroll
                for (int j = 0; j < K; ++j) t[j] = in ? P.w[(long long)(c + k) * K + j] : 0.f;
            }
            const float b = in && P.bias ? P.bias[c + k] : 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j) (k & 1 ? w[j][k / 2].y : w[j][k / 2].x) = t[j];
            (k & 1 ? bias[k / 2].y : bias[k / 2].x) = b;
        }
    }
    // p of a row whose taps are rows x[0] ... x[K - 1]
    __device__ __forceinline__ float2 sum(const float2 (*x)[kV / 2], int k) const {
        float2 p = bias[k];
#pragma unroll
        for (int j = 0; j < K; ++j) p = fma2(w[j][k], x[j][k], p);
        return p;
    }
};
template <typename T> __device__ __forceinline__ void widen(float2 (&to)[kV / 2], const Vec<T, kV> &x) {
#pragma unroll
    for (int k = 0; k < kV / 2; ++k) to[k] = make_float2(to_f(x.e[2 * k]), to_f(x.e[2 * k + 1]));
}
template <typename T> __device__ __forceinline__ Vec<T, kV> narrow(const float2 (&x)[kV / 2]) {
    Vec<T, kV> r;
#pragma unroll
    for (int k = 0; k < kV / 2; ++k) put2(r.e + 2 * k, x[k].x, x[k].y);
    return r;
}
__device__ __forceinline__ float2 sigmoid2(float2 p) { return make_float2(sigmoid(p.x), sigmoid(p.y)); }

// The row `place` of a sequence; negative: of the state before it.
template <typename T, int K, int V>
__device__ __forceinline__ Vec<T, V> row_at(const Params &P, const T *x, int seq, int place, int c) {
    const int n = P.C - c;
    if (place >= 0) return load_vec<T, V>(x + place * P.x.sn + c, n);
    if (P.first) return load_vec<T, V>((const T *)P.first + ((long long)seq * (K - 1) + (K - 1 + place)) * P.C + c, n, P.C % V == 0);
    Vec<T, V> z;
#pragma unroll
    for (int k = 0; k < V; ++k) z.e[k] = T(0.f);
    return z;
}

template <typename T, int K, bool SILU> __global__ void __launch_bounds__(kThreads, kPerSM) forward_kernel(const __grid_constant__ Params P) {
    constexpr int V = kV, A = kFwdAhead;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V, n = P.C - c;
    const int r0 = blockIdx.y * P.run, r1 = r0 + min(P.run, P.seq.T - r0);
    const Taps<K> taps(P, c);
    for_stretches(P.seq, r0, r1, [&](int seq, int t0, int t1, int len, bool begins) {
        if (n <= 0) return;
        const T *x = rows_of<const T>(P.seq, P.x, seq);
        T *o = rows_of<T>(P.seq, P.o, seq) + c;
        float2 win[K - 1 + A][V / 2];  // rows t - K + 1 ... t + A - 1
        Vec<T, V> next[A];             // those behind, on their way
        auto fetch = [&](int t) {
#pragma unroll
            for (int a = 0; a < A; ++a) load_ahead(next[a], x + (t + a) * P.x.sn + c, t + a < t1 && n >= V);
        };
        fetch(t0);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) widen(win[j], row_at<T, K, V>(P, x, seq, t0 - (K - 1) + j, c));
        for (int t = t0; t < t1; t += A) {
#pragma unroll
            for (int a = 0; a < A; ++a) {
                if (n < V && t + a < t1) next[a] = load_vec<T, V>(x + (t + a) * P.x.sn + c, n);  // no whole vector
                widen(win[K - 1 + a], next[a]);
            }
            fetch(t + A);
#pragma unroll
            for (int a = 0; a < A; ++a) {
                float2 p[V / 2];
#pragma unroll
                for (int k = 0; k < V / 2; ++k) {
                    p[k] = taps.sum(win + a, k);
                    if (SILU) p[k] = mul2(p[k], sigmoid2(p[k]));
                }
                if (t + a < t1) store_vec<T, V>(o + (t + a) * P.o.sn, narrow<T>(p), n);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int k = 0; k < V / 2; ++k) win[j][k] = win[j + A][k];
        }
        if (begins && P.last)  // (the state before is another array)
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                store_vec<T, V>((T *)P.last + ((long long)seq * (K - 1) + j) * P.C + c,
                                row_at<T, K, V>(P, x, seq, len - (K - 1) + j, c), n, P.C % V == 0);
    });
}

template <typename T, int K, bool SILU> __global__ void __launch_bounds__(kThreads, kBackPerSM) backward_kernel(const __grid_constant__ Params P) {
    constexpr int V = kV, A = kAhead;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V, n = P.C - c;
    const int r0 = blockIdx.y * P.run, r1 = r0 + min(P.run, P.seq.T - r0);
    const Taps<K> taps(P, c);
    float2 dw[K][V / 2] = {}, db[V / 2] = {};
    for_stretches(P.seq, r0, r1, [&](int seq, int t0, int t1, int len, bool) {
        if (n <= 0) return;
        const T *x = rows_of<const T>(P.seq, P.x, seq), *d = rows_of<const T>(P.seq, P.dO, seq) + c;
        T *dx = rows_of<T>(P.seq, P.o, seq) + c;
        const int end = min(t1 + K - 1, len);  // rows whose dp reaches the run's
        float2 win[K - 1 + A][V / 2], dp[K - 1 + A][V / 2];  // of rows t - K + 1 ... t + A - 1
        Vec<T, V> nx[A], nd[A];
        auto fetch = [&](int t) {
#pragma unroll
            for (int a = 0; a < A; ++a) {
                load_ahead(nx[a], x + (t + a) * P.x.sn + c, t + a < end && n >= V);
                load_ahead(nd[a], d + (t + a) * P.dO.sn, t + a < end && n >= V);
            }
        };
        fetch(t0);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            widen(win[j], row_at<T, K, V>(P, x, seq, t0 - (K - 1) + j, c));
#pragma unroll
            for (int k = 0; k < V / 2; ++k) dp[j][k] = both(0.f);
        }
        for (int t = t0; t < t1 + K - 1; t += A) {
#pragma unroll
            for (int a = 0; a < A; ++a) {
                if (n < V && t + a < end) {  // no whole vector
                    nx[a] = load_vec<T, V>(x + (t + a) * P.x.sn + c, n);
                    nd[a] = load_vec<T, V>(d + (t + a) * P.dO.sn, n);
                }
                widen(win[K - 1 + a], nx[a]);
                widen(dp[K - 1 + a], nd[a]);
            }
            fetch(t + A);
#pragma unroll
            for (int a = 0; a < A; ++a) {
                float2 e[V / 2];
#pragma unroll
                for (int k = 0; k < V / 2; ++k) {
                    float2 g = dp[K - 1 + a][k];
                    if (SILU) {
                        const float2 p = taps.sum(win + a, k), s = sigmoid2(p);
                        g = mul2(g, make_float2(silu_grad(p.x, s.x), silu_grad(p.y, s.y)));
                    }
                    if (t + a >= end) g = both(0.f);
                    if (t + a < t1) {
                        db[k] = add2(db[k], g);
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][k] = fma2(g, win[a + j][k], dw[j][k]);
                    }
                    dp[K - 1 + a][k] = g;
                    e[k] = mul2(taps.w[0][k], g);
#pragma unroll
                    for (int j = 1; j < K; ++j) e[k] = fma2(taps.w[j][k], dp[K - 1 + a - j][k], e[k]);
                }
                // the row whose last dp this was
                if (t + a - (K - 1) >= t0 && t + a < t1 + K - 1) store_vec<T, V>(dx + (t + a - (K - 1)) * P.o.sn, narrow<T>(e), n);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int k = 0; k < V / 2; ++k) win[j][k] = win[j + A][k], dp[j][k] = dp[j + A][k];
        }
    });
    float *part = P.part + (long long)blockIdx.y * P.C * (K + 1);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int j = 0; j < K; ++j) part[(long long)(c + k) * K + j] = k & 1 ? dw[j][k / 2].y : dw[j][k / 2].x;
        part[(long long)P.C * K + c + k] = k & 1 ? db[k / 2].y : db[k / 2].x;
    }
}

template <typename T, int K, bool SILU> __global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Params P) {
    constexpr int V = kV;
    const int per = (P.C + V - 1) / V;  // vectors of a row
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)P.seq.nseq * per) return;
    const int b = (int)(i / per), c = (int)(i - (long long)b * per) * V, n = P.C - c;
    T *st = (T *)P.last + (long long)b * (K - 1) * P.C + c;
    Vec<T, V> row[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row[j] = load_vec<T, V>(st + (long long)j * P.C, n, P.C % V == 0);
    row[K - 1] = load_vec<T, V>((const T *)P.x.p + b * P.x.sb + c, n);
    const Taps<K> taps(P, c);
    float2 win[K][V / 2], p[V / 2];
#pragma unroll
    for (int j = 0; j < K; ++j) widen(win[j], row[j]);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
        p[k] = taps.sum(win, k);
        if (SILU) p[k] = mul2(p[k], sigmoid2(p[k]));
    }
    store_vec<T, V>((T *)P.o.p + b * P.o.sb + c, narrow<T>(p), n);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_vec<T, V>(st + (long long)j * P.C, row[j + 1], n, P.C % V == 0);
}

enum : int { kForward = 0, kBackward, kStep };

template <int WHAT, typename T, int K, bool SILU> cudaError_t launch(const Params &P, dim3 grid, cudaStream_t s) {
    if constexpr (WHAT == kForward) forward_kernel<T, K, SILU><<<grid, kThreads, 0, s>>>(P);
    else if constexpr (WHAT == kBackward) backward_kernel<T, K, SILU><<<grid, kThreads, 0, s>>>(P);
    else step_kernel<T, K, SILU><<<grid, kThreads, 0, s>>>(P);
    return cudaGetLastError();
}
template <int WHAT, typename T> cudaError_t by_taps(const Params &P, int K, int act, dim3 grid, cudaStream_t s) {
    if (K == 2) return act ? launch<WHAT, T, 2, true>(P, grid, s) : launch<WHAT, T, 2, false>(P, grid, s);
    if (K == 3) return act ? launch<WHAT, T, 3, true>(P, grid, s) : launch<WHAT, T, 3, false>(P, grid, s);
    return act ? launch<WHAT, T, 4, true>(P, grid, s) : launch<WHAT, T, 4, false>(P, grid, s);
}
template <int WHAT> int run(const Params &P, int K, int act, int dtype, dim3 grid, void *stream) {
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == LA_BF16 ? by_taps<WHAT, __nv_bfloat16>(P, K, act, grid, s) : by_taps<WHAT, float>(P, K, act, grid, s);
    if (e != cudaSuccess) return LA_ERR_CUDA;
    count_launches(1);
    return LA_OK;
}

int runs_of(int T, int rows) { return (int)(((long long)T + rows - 1) / rows); }

// Rows of a run: as many as let all blocks stand on the SMs at once, and kRun at least.
int run_rows(int T, int across, int per_sm) {
    const int runs = across < per_sm * kSMs ? per_sm * kSMs / across : 1;
    int rows = (int)(((long long)T + runs - 1) / runs);
    if (rows < kRun) rows = kRun;
    while (runs_of(T, rows) > 65535) rows *= 2;
    return rows;
}

// Kinds and sizes; N rows each, or (packed) N rows in all.
int check_sizes(int nseq, int N, int C, int K, int act, int dtype, bool packed) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (act != LA_CONV_NONE && act != LA_CONV_SILU) return LA_ERR_INVALID_ARG;
    if (nseq < 0 || N < 0 || C < 1 || C >= 1 << 24 || K < 1) return LA_ERR_INVALID_ARG;
    const long long T = packed ? N : (long long)nseq * N;
    if (T > kMaxRows || T >= (1LL << 40) / C || (long long)nseq * kMaxK >= (1LL << 40) / C || nseq > kMaxRows) return LA_ERR_INVALID_ARG;
    if (K < 2 || K > kMaxK) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

int check_params(const float *W, const float *bias) {
    return !W || ((uintptr_t)W & 15) || ((uintptr_t)bias & 15) ? LA_ERR_INVALID_ARG : LA_OK;
}

// The offsets and the workspace of a packed call; both may be missing otherwise.
int check_packed(const int *off, void *workspace, size_t bytes) {
    if (!off) return LA_OK;
    if (!workspace || ((uintptr_t)workspace & 255) || bytes < 256) return LA_ERR_WORKSPACE;
    return ((uintptr_t)off & 3) ? LA_ERR_INVALID_ARG : LA_OK;
}

}  // namespace conv
}  // namespace la

extern "C" {

int la_short_conv(const void *X, const float *W, const float *bias, const void *state_in, void *O, void *state_out,
                  const int *seq_offsets, int nseq, int N, int C, int K, int activation, int dtype,
                  const long long *strides, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace la;
    using namespace la::conv;
    const bool packed = seq_offsets != nullptr;
    int rc = check_sizes(nseq, N, C, K, activation, dtype, packed);
    if (rc) return rc;
    if ((rc = check_params(W, bias)) || (rc = check_packed(seq_offsets, workspace, workspace_bytes))) return rc;
    if (((uintptr_t)state_in & 15) || ((uintptr_t)state_out & 15)) return LA_ERR_INVALID_ARG;
    const int elem = dtype == LA_BF16 ? 2 : 4, T = packed ? N : nseq * N;
    View x = {}, o = {};
    if (T > 0) {
        if ((rc = rows_view(x, X, packed ? 1 : nseq, N, C, elem, strides))) return rc;
        if ((rc = rows_view(o, O, packed ? 1 : nseq, N, C, elem, strides ? strides + 2 : nullptr))) return rc;
    }
    const size_t state = (size_t)nseq * (K - 1) * C * elem;
    const Range rin[4] = {{W, (size_t)C * K * 4}, {bias, (size_t)C * 4}, {state_in, state}, {seq_offsets, ((size_t)nseq + 1) * 4}};
    const Range rout[2] = {{state_out, state}, {packed ? workspace : nullptr, 256}};
    if (outputs_meet(&x, 1, &o, 1, rin, 4, rout, 2)) return LA_ERR_INVALID_ARG;
    if (nseq == 0 || (T == 0 && !state_out)) return LA_OK;
    Params P = {};
    P.x = Op{X, x.st[0], x.st[1]};
    P.o = Op{O, o.st[0], o.st[1]};
    P.w = W, P.bias = bias, P.first = state_in, P.last = state_out;
    P.seq = Seqs{seq_offsets, nseq, N, T, (uint32_t *)workspace};
    P.C = C;
    const unsigned across = (unsigned)((C + kThreads * kV - 1) / (kThreads * kV));
    P.run = run_rows(T, (int)across, kPerSM);
    const int runs = T > 0 ? runs_of(T, P.run) : 1;
    return run<kForward>(P, K, activation, dtype, dim3(across, (unsigned)runs), stream);
}

size_t la_short_conv_workspace_bytes(int C, int K) {
    if (C < 1 || C >= 1 << 24 || K < 2 || K > la::conv::kMaxK) return 0;
    return 256 + (size_t)la::conv::kMaxParts * C * (K + 1) * sizeof(float);
}

int la_short_conv_backward(const void *X, const float *W, const float *bias, const void *state_in, const void *dO,
                           void *dX, float *dW, float *dbias, const int *seq_offsets, int nseq, int N, int C, int K,
                           int activation, int dtype, const long long *strides, void *workspace, size_t workspace_bytes,
                           void *stream) {
    using namespace la;
    using namespace la::conv;
    const bool packed = seq_offsets != nullptr;
    int rc = check_sizes(nseq, N, C, K, activation, dtype, packed);
    if (rc) return rc;
    if ((rc = check_params(W, bias))) return rc;
    const size_t need = la_short_conv_workspace_bytes(C, K);
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need) return LA_ERR_WORKSPACE;
    if ((rc = check_packed(seq_offsets, workspace, workspace_bytes))) return rc;
    if (((uintptr_t)state_in & 15) || !dW || ((uintptr_t)dW & 15) || ((uintptr_t)dbias & 15)) return LA_ERR_INVALID_ARG;
    const int elem = dtype == LA_BF16 ? 2 : 4, T = packed ? N : nseq * N;
    View in[2] = {}, dx = {};
    const void *const ptr[2] = {X, dO};
    if (T > 0) {
        for (int k = 0; k < 2; ++k)
            if ((rc = rows_view(in[k], ptr[k], packed ? 1 : nseq, N, C, elem, strides ? strides + 2 * k : nullptr))) return rc;
        if ((rc = rows_view(dx, dX, packed ? 1 : nseq, N, C, elem, strides ? strides + 4 : nullptr))) return rc;
    }
    const Range rin[4] = {{W, (size_t)C * K * 4}, {bias, (size_t)C * 4}, {state_in, (size_t)nseq * (K - 1) * C * elem}, {seq_offsets, ((size_t)nseq + 1) * 4}};
    const Range rout[3] = {{dW, (size_t)C * K * 4}, {dbias, (size_t)C * 4}, {workspace, need}};
    if (outputs_meet(in, 2, &dx, 1, rin, 4, rout, 3)) return LA_ERR_INVALID_ARG;
    Params P = {};
    P.x = Op{X, in[0].st[0], in[0].st[1]};
    P.dO = Op{dO, in[1].st[0], in[1].st[1]};
    P.o = Op{dX, dx.st[0], dx.st[1]};
    P.w = W, P.bias = bias, P.first = state_in;
    P.seq = Seqs{seq_offsets, nseq, N, T, (uint32_t *)workspace};
    P.C = C;
    P.part = (float *)((char *)workspace + 256);
    const unsigned across = (unsigned)((C + kThreads * kV - 1) / (kThreads * kV));
    int parts = 0;
    if (nseq > 0 && T > 0) {
        P.run = run_rows(T, (int)across, kBackPerSM);
        if (runs_of(T, P.run) > kMaxParts) P.run = runs_of(T, kMaxParts);
        parts = runs_of(T, P.run);
        if ((rc = run<kBackward>(P, K, activation, dtype, dim3(across, (unsigned)parts), stream))) return rc;
    }
    const long long M = (long long)C * (K + 1);
    return sum_parts(P.part, parts, M, dW, (long long)C * K, dbias, C, nullptr, (cudaStream_t)stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

int la_short_conv_step(const void *x, const float *W, const float *bias, void *state, void *o, int nseq, int C, int K,
                       int activation, int dtype, const long long *strides, void *stream) {
    using namespace la;
    using namespace la::conv;
    int rc = check_sizes(nseq, 1, C, K, activation, dtype, false);
    if (rc) return rc;
    if ((rc = check_params(W, bias))) return rc;
    if (nseq == 0) return LA_OK;
    if (!state || ((uintptr_t)state & 15)) return LA_ERR_INVALID_ARG;
    const int elem = dtype == LA_BF16 ? 2 : 4;
    View vx = {}, vo = {};
    const long long sx[2] = {strides ? strides[0] : C, C}, so[2] = {strides ? strides[1] : C, C};
    if ((rc = rows_view(vx, x, nseq, 1, C, elem, sx)) || (rc = rows_view(vo, o, nseq, 1, C, elem, so))) return rc;
    const Range rin[2] = {{W, (size_t)C * K * 4}, {bias, (size_t)C * 4}}, rout[1] = {{state, (size_t)nseq * (K - 1) * C * elem}};
    if (outputs_meet(&vx, 1, &vo, 1, rin, 2, rout, 1)) return LA_ERR_INVALID_ARG;
    Params P = {};
    P.x = Op{x, vx.st[0], vx.st[1]};
    P.o = Op{o, vo.st[0], vo.st[1]};
    P.w = W, P.bias = bias, P.last = state;
    P.seq = Seqs{nullptr, nseq, 1, nseq, nullptr};
    P.C = C;
    const long long blocks = ((long long)nseq * ((C + kV - 1) / kV) + kThreads - 1) / kThreads;
    if (blocks >= (1LL << 31)) return LA_ERR_INVALID_ARG;
    return run<kStep>(P, K, activation, dtype, dim3((unsigned)blocks), stream);
}

}  // extern "C"
