// la_conv.cu -- short causal convolution over time, each channel by itself (la_short_conv), its gradients
// (la_short_conv_backward) and one token of it (la_short_conv_step).
//
//   p_t = bias + sum_j w_j x_{t-K+1+j},  o = p or p sigmoid(p);  K taps; before a sequence's first row stand the K - 1
//   rows of its state, or zeros; its last K - 1 inputs are the state that it leaves
//   backward: dp = do (o's derivative at p),  dx_t = sum_j w_j dp_{t+K-1-j},  dw_j = sum_t dp_t x_{t-K+1+j}
//
// A thread has one vector of channels and walks a run of rows, the last K - 1 of them in registers, so each row is read
// once (and K - 1 rows again at a run's start), which bounds it (HBM).  The backward walk is the same with a second window,
// of dp: dx of a row is complete K - 1 rows later, so a run computes dp of the K - 1 rows behind it again.  Sums are fp32.
#include "la_rows.cuh"

namespace la {
namespace conv {

using namespace rows;

constexpr int kThreads = 128;
constexpr int kRun = 32;          // rows of a forward run
constexpr int kMaxParts = 256;    // runs of the backward walk
constexpr int kMaxK = 4;
constexpr int kAhead = 4;         // rows loaded together
constexpr int kBackV = 4;         // channels of a thread in the backward walk, whose windows and sums take the registers
constexpr int kEnough = 608;      // blocks: four to an SM

struct Params {
    Op x, o, dO;                  // forward: x, o; backward: x, do, and o is dx
    const float *w, *bias;        // [C][K], [C] or null
    const void *first;            // [nseq][K - 1][C], or null: zeros
    void *last;                   // [nseq][K - 1][C], or null: not written
    Seqs seq;
    int C, run;                   // rows of a run
    float *part;                  // backward: [parts][C][K], then [C], of each part
};

// Taps and bias of a thread's channels.
template <int K, int V> __device__ __forceinline__ void load_taps(const Params &P, int c, float (&w)[K][V], float (&bias)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const bool in = c + k < P.C;
        if (K == 4) {
            const float4 f = in ? *(const float4 *)(P.w + (long long)(c + k) * K) : make_float4(0.f, 0.f, 0.f, 0.f);
            w[0][k] = f.x, w[1][k] = f.y, w[K - 2][k] = f.z, w[K - 1][k] = f.w;
        } else {
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][k] = in ? P.w[(long long)(c + k) * K + j] : 0.f;
        }
        bias[k] = in && P.bias ? P.bias[c + k] : 0.f;
    }
}

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

template <typename T, int K, bool SILU> __global__ void __launch_bounds__(kThreads) forward_kernel(const __grid_constant__ Params P) {
    constexpr int V = 16 / (int)sizeof(T);
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V, n = P.C - c;
    const int r0 = blockIdx.y * P.run, r1 = min(r0 + P.run, P.seq.T);
    float w[K][V], bias[V];
    load_taps<K, V>(P, c, w, bias);
    for_stretches(P.seq, r0, r1, [&](int seq, int t0, int t1, int len, bool begins) {
        if (n <= 0) return;
        const T *x = rows_of<const T>(P.seq, P.x, seq);
        T *o = rows_of<T>(P.seq, P.o, seq) + c;
        Vec<T, V> win[K - 1 + kAhead];  // rows t - K + 1 ... t + kAhead - 1
        Vec<T, V> next[kAhead];         // those behind, on their way
        auto fetch = [&](int t) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) load_ahead(next[a], x + (t + a) * P.x.sn + c, t + a < t1 && n >= V);
        };
        fetch(t0);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) win[j] = row_at<T, K, V>(P, x, seq, t0 - (K - 1) + j, c);
        for (int t = t0; t < t1; t += kAhead) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (n < V && t + a < t1) next[a] = load_vec<T, V>(x + (t + a) * P.x.sn + c, n);  // no whole vector
                win[K - 1 + a] = next[a];
            }
            fetch(t + kAhead);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (t + a >= t1) break;
                Vec<T, V> out;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float p = bias[k];
#pragma unroll
                    for (int j = 0; j < K; ++j) p = fmaf(w[j][k], to_f(win[a + j].e[k]), p);
                    put(&out.e[k], SILU ? p * sigmoid(p) : p);
                }
                store_vec<T, V>(o + (t + a) * P.o.sn, out, n);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) win[j] = win[j + kAhead];
        }
        if (begins && P.last)  // (the state before is another array)
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                store_vec<T, V>((T *)P.last + ((long long)seq * (K - 1) + j) * P.C + c,
                                row_at<T, K, V>(P, x, seq, len - (K - 1) + j, c), n, P.C % V == 0);
    });
}

template <typename T, int K, bool SILU> __global__ void __launch_bounds__(kThreads) backward_kernel(const __grid_constant__ Params P) {
    constexpr int V = kBackV;
    const int c = (blockIdx.x * kThreads + threadIdx.x) * V, n = P.C - c;
    const int r0 = blockIdx.y * P.run, r1 = min(r0 + P.run, P.seq.T);
    float w[K][V], bias[V], dw[K][V], db[V];
    load_taps<K, V>(P, c, w, bias);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        db[k] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][k] = 0.f;
    }
    for_stretches(P.seq, r0, r1, [&](int seq, int t0, int t1, int len, bool) {
        if (n <= 0) return;
        const T *x = rows_of<const T>(P.seq, P.x, seq), *d = rows_of<const T>(P.seq, P.dO, seq) + c;
        T *dx = rows_of<T>(P.seq, P.o, seq) + c;
        const int end = min(t1 + K - 1, len);  // rows whose dp reaches the run's
        Vec<T, V> win[K - 1 + kAhead], dO[kAhead], nx[kAhead], nd[kAhead];
        float dp[K - 1 + kAhead][V];  // of rows t - K + 1 ... t + kAhead - 1
        auto fetch = [&](int t) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                load_ahead(nx[a], x + (t + a) * P.x.sn + c, t + a < end && n >= V);
                load_ahead(nd[a], d + (t + a) * P.dO.sn, t + a < end && n >= V);
            }
        };
        fetch(t0);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            win[j] = row_at<T, K, V>(P, x, seq, t0 - (K - 1) + j, c);
#pragma unroll
            for (int k = 0; k < V; ++k) dp[j][k] = 0.f;
        }
        for (int t = t0; t < t1 + K - 1; t += kAhead) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (n < V && t + a < end) {  // no whole vector
                    nx[a] = load_vec<T, V>(x + (t + a) * P.x.sn + c, n);
                    nd[a] = load_vec<T, V>(d + (t + a) * P.dO.sn, n);
                }
                win[K - 1 + a] = nx[a];
                dO[a] = nd[a];
            }
            fetch(t + kAhead);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const bool in = t + a < end, mine = t + a < t1;
                Vec<T, V> out;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float g = 0.f;
                    if (in) {
                        g = to_f(dO[a].e[k]);
                        if (SILU) {
                            float p = bias[k];
#pragma unroll
                            for (int j = 0; j < K; ++j) p = fmaf(w[j][k], to_f(win[a + j].e[k]), p);
                            g *= silu_grad(p, sigmoid(p));
                        }
                        if (mine) {
                            db[k] += g;
#pragma unroll
                            for (int j = 0; j < K; ++j) dw[j][k] = fmaf(g, to_f(win[a + j].e[k]), dw[j][k]);
                        }
                    }
                    dp[K - 1 + a][k] = g;
                    float e = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) e = fmaf(w[j][k], dp[K - 1 + a - j][k], e);
                    put(&out.e[k], e);
                }
                // the row whose last dp this was
                if (t + a - (K - 1) >= t0 && t + a < t1 + K - 1) store_vec<T, V>(dx + (t + a - (K - 1)) * P.o.sn, out, n);
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                win[j] = win[j + kAhead];
#pragma unroll
                for (int k = 0; k < V; ++k) dp[j][k] = dp[j + kAhead][k];
            }
        }
    });
    float *part = P.part + (long long)blockIdx.y * P.C * (K + 1);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int j = 0; j < K; ++j) part[(long long)(c + k) * K + j] = dw[j][k];
        part[(long long)P.C * K + c + k] = db[k];
    }
}

template <typename T, int K, bool SILU> __global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Params P) {
    constexpr int V = 16 / (int)sizeof(T);
    const int per = (P.C + V - 1) / V;  // vectors of a row
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (long long)P.seq.nseq * per) return;
    const int b = (int)(i / per), c = (int)(i - (long long)b * per) * V, n = P.C - c;
    T *st = (T *)P.last + (long long)b * (K - 1) * P.C + c;
    Vec<T, V> win[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) win[j] = load_vec<T, V>(st + (long long)j * P.C, n, P.C % V == 0);
    win[K - 1] = load_vec<T, V>((const T *)P.x.p + b * P.x.sb + c, n);
    float w[K][V], bias[V];
    load_taps<K, V>(P, c, w, bias);
    Vec<T, V> out;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        float p = bias[k];
#pragma unroll
        for (int j = 0; j < K; ++j) p = fmaf(w[j][k], to_f(win[j].e[k]), p);
        put(&out.e[k], SILU ? p * sigmoid(p) : p);
    }
    store_vec<T, V>((T *)P.o.p + b * P.o.sb + c, out, n);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_vec<T, V>(st + (long long)j * P.C, win[j + 1], n, P.C % V == 0);
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

// Kinds and sizes; N rows each, or (packed) N rows in all.
int check_sizes(int nseq, int N, int C, int K, int act, int dtype, bool packed) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (act != LA_CONV_NONE && act != LA_CONV_SILU) return LA_ERR_INVALID_ARG;
    if (nseq < 0 || N < 0 || C < 1 || K < 1) return LA_ERR_INVALID_ARG;
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
    // Shorter runs where long ones would leave SMs without a block.
    const unsigned across = (unsigned)((C + kThreads * (16 / elem) - 1) / (kThreads * (16 / elem)));
    P.run = kRun;
    while (P.run > 8 && (long long)across * ((T + P.run - 1) / P.run) < kEnough) P.run /= 2;
    while ((T + P.run - 1) / P.run > 65535) P.run *= 2;
    const int runs = T > 0 ? (T + P.run - 1) / P.run : 1;
    return run<kForward>(P, K, activation, dtype, dim3(across, (unsigned)runs), stream);
}

size_t la_short_conv_workspace_bytes(int C, int K) {
    if (C < 1 || K < 2 || K > la::conv::kMaxK) return 0;
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
    // Runs of at least 16 rows, as few as fill the SMs, and no more than the workspace has places for.
    const unsigned across = (unsigned)((C + kThreads * kBackV - 1) / (kThreads * kBackV));
    int parts = (T + 15) / 16;
    if (parts > (kEnough + (int)across - 1) / (int)across) parts = (kEnough + (int)across - 1) / (int)across;
    if (parts > kMaxParts) parts = kMaxParts;
    if (nseq == 0 || T == 0) parts = 0;
    if (parts > 0) {
        P.run = (T + parts - 1) / parts;
        parts = (T + P.run - 1) / P.run;
        if ((rc = run<kBackward>(P, K, activation, dtype, dim3(across, (unsigned)parts), stream))) return rc;
    }
    const long long M = (long long)C * (K + 1);
    return sum_parts(P.part, parts, M, (long long)C * K, dW, dbias, (cudaStream_t)stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
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
    const int V = 16 / elem;
    const long long blocks = ((long long)nseq * ((C + V - 1) / V) + kThreads - 1) / kThreads;
    if (blocks >= (1LL << 31)) return LA_ERR_INVALID_ARG;
    return run<kStep>(P, K, activation, dtype, dim3((unsigned)blocks), stream);
}

}  // extern "C"
