// la_selective.cu -- selective state space scan (la_selective_scan), its gradients (la_selective_scan_backward) and one
// token of it (la_selective_scan_step).
//
//   d = softplus(dt + dt_bias) or dt + dt_bias,   h_t[c,n] = e^(d A[c,n]) h_{t-1}[c,n] + d x B_t[n]
//   y = sum_n C_t[n] h_t[c,n] + D x,   out = y z sigmoid(z)   (or y)
//   backward, with g = dout z sigmoid(z) and G_t = g C_t + a_{t+1} G_{t+1} (a = e^(d A)):
//   dx = d sum_n G B + D g,  dd = sum_n a h_{t-1} G A + x sum_n G B,  dA = sum_t d a h_{t-1} G,  dB = sum_c G d x,
//   dC = sum_c g h,  dD = sum_t g x,  dz = dout y (z sigmoid(z))'
//
// A scanning thread holds four states of two channels in registers, a warp four states of 64 channels, and the warps of the
// other states stand beside it.  They walk rows in tiles of 16, reading d, d x, B and C from shared memory and leaving each
// row's part of y there, while helping warps form d and d x of the next tile and write the outputs of the tile before; one
// barrier a tile.  x, dt, z, B and C come by asynchronous copies into a ring of tiles: loaded ahead into registers, behind
// branches, each waited for its own arrival (4 x 4096 x 2048, bf16: 1209 us; predicated 332; copies 287).  All is held in fp32.
// T C S exponentials (32 an SM and clock) and 4 T C S multiply-adds are 60 us there; what binds it are issue slots (some 270
// instructions for a row of 64 channels) and shared memory, whose 16-byte loads of B and C take two clocks of the SM each
// though all lanes ask for the same.  Two channels to a thread share them (1 x 65536 x 2048: 1.13 ms, one channel 1.33); one
// channel to a thread gives twice the warps where an SM has one CTA, and registers for operands three rows ahead (4 x 4096 x
// 2048: 240 us, one row ahead 250, two channels 287).
// Where there are few channels time is cut into parts: a first launch forms each part's last state, started from zero (the
// first part of a sequence: from its state), and the sum of its d, whose e^(A sum) is the part's decay; the second launch
// folds them into the state that each part starts from.
#include <math.h>

#include <type_traits>

#include "la_f32x2.cuh"
#include "la_rows.cuh"

namespace la {
namespace sel {

using namespace rows;

constexpr int kThreads = 256;  // of a step's block
constexpr int kMark = 8;       // rows between the states that a forward keeps for its backward, and of its tile
constexpr int kTile = 16;      // rows of a forward tile
constexpr int kGroup = 16;     // tiles whose sums of dA are added up by themselves
constexpr int kSMs = 152;
constexpr int kMaxParts = 64;  // of a sequence of the mean length (each folds in all before it, one by one)

struct GOp {                   // B, C: [.., G, S]
    const void *p;
    long long sb, sn, sg;
};

struct Params {
    Op x, dt, z, y;            // z.p null: no gate
    GOp B, C;
    const float *A, *D, *bias;
    const float *first;        // [nseq, C, S] or null
    float *last, *marks;       // [nseq, C, S], [slots, C, S], or null
    Seqs seq;
    int C_, G, cpg, bpg;       // channels, groups, channels and blocks of a group
    int part, parts;           // rows of a part (a multiple of the tile's); units in all
    int softplus;
    float *ends, *sums;        // [units, C, S], [units, C]: parts' last states and sums of d
    // backward
    Op dO, dx, ddt, dz;
    const float *dlast;        // [nseq, C, S] or null
    float *dfirst;
    float *pbc;                // [groups of 64 channels, T, G, 2 S]
    float *pa;                 // [walkers][C S of dA, C of dD, C of d(dt_bias)]
    int walkers, units;        // CTAs of a channel block, which walk all units
    uint32_t *valid;           // whether the offsets were in order, for the sums behind
};

constexpr float kLn2 = 0.693147181f, kLargest = 3.40282347e38f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v|; log(1 + e) = 2 artanh(s), s = e / (2 + e) <= 1/3, by its series to
// s^13 (the next term is 2^-26 of the sum): as exact for small e as for large.  NaN stays NaN.
__device__ __forceinline__ float2 softplus2(float2 v) {
    const float2 e = make_float2(exp_fast(-fabsf(v.x)), exp_fast(-fabsf(v.y)));
    const float2 s = mul2(e, make_float2(rcp_fast(2.f + e.x), rcp_fast(2.f + e.y))), q = mul2(s, s);
    float2 p = fma2(q, both(2.f / 13.f), both(2.f / 11.f));
    p = fma2(q, p, both(2.f / 9.f));
    p = fma2(q, p, both(2.f / 7.f));
    p = fma2(q, p, both(2.f / 5.f));
    p = fma2(q, p, both(2.f / 3.f));
    p = fma2(q, p, both(2.f));
    return fma2(s, p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float2 step_of(const Params &P, float2 v) { return P.softplus ? softplus2(v) : v; }

// Four states.
struct F4 {
    float2 a, b;
};
__device__ __forceinline__ F4 load4(const float *p) {
    const float4 v = *(const float4 *)p;
    return F4{make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ void store4(float *p, const F4 &v) { *(float4 *)p = make_float4(v.a.x, v.a.y, v.b.x, v.b.y); }
__device__ __forceinline__ F4 zero4() { return F4{both(0.f), both(0.f)}; }
__device__ __forceinline__ F4 mul4(const F4 &x, const F4 &y) { return F4{mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ F4 mul4(const F4 &x, float y) { return F4{mul2(x.a, both(y)), mul2(x.b, both(y))}; }
__device__ __forceinline__ F4 fma4(const F4 &x, const F4 &y, const F4 &z) { return F4{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)}; }
__device__ __forceinline__ F4 fma4(const F4 &x, float y, const F4 &z) { return F4{fma2(x.a, both(y), z.a), fma2(x.b, both(y), z.b)}; }
__device__ __forceinline__ float dot4(const F4 &x, const F4 &y) {
    const float2 s = fma2(x.b, y.b, mul2(x.a, y.a));
    return s.x + s.y;
}
// A log2 e, rounded towards zero: never infinite, so that a row with d = 0, or one that is not there, changes no state.  The
// constant is the float above log2 e, 1.2 half steps too large, so that the product is off by as much at most either way.
__device__ __forceinline__ float log2_rate(float a) { return __fmul_rz(a, 1.44269514f); }
__device__ __forceinline__ F4 rates4(const float *A) {
    const F4 a = load4(A);
    return F4{make_float2(log2_rate(a.a.x), log2_rate(a.a.y)), make_float2(log2_rate(a.b.x), log2_rate(a.b.y))};
}
// 2^(a2 d).  The hardware's 2^x is on the average too small, by 0.6 to 2.6e-8 for exponents between -2^-17 and -1/2, and a state
// that fades slowly gathers that of all rows it remembers.  So exponents are made kLift larger, within the one multiply-add that
// forms them: means between -1.1 and 1.0e-8, the same rms; 2^kLift is 1, so rows that are not there still leave a state as it
// is.  8 x 2048 x 2048: dA off by 0.92e-6 of its norm, 2.0e-6 without.
constexpr float kLift = 2.2351742e-8f;  // 3 2^-27
__device__ __forceinline__ F4 decay4(const F4 &a2, float d) {
    const F4 e = fma4(a2, d, F4{both(kLift), both(kLift)});
    return F4{make_float2(ex2(e.a.x), ex2(e.a.y)), make_float2(ex2(e.b.x), ex2(e.b.y))};
}

// 2^(a2 d) h + x, d a part's sum, by four factors: a part's growth, or its fading, may be beyond fp32's range where the state that
// it reaches is not.  A factor counts as the largest number at most, so what is 0 stays 0, as it does row by row.
__device__ __forceinline__ float finite(float f) { return fminf(f, kLargest); }
__device__ __forceinline__ F4 over_part(const F4 &a2, float d, const F4 &h, const F4 &x) {
    const F4 e = decay4(a2, 0.25f * d), f{make_float2(finite(e.a.x), finite(e.a.y)), make_float2(finite(e.b.x), finite(e.b.y))};
    return fma4(f, mul4(f, mul4(f, mul4(f, h))), x);
}

// Sums over L lanes (q of them this one's number, lanes STEP apart) of L values each; lane q gets value q's.
template <int L, int STEP> __device__ __forceinline__ float lanes_sum(float (&v)[L], int q) {
#pragma unroll
    for (int d = L / 2; d > 0; d /= 2) {
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const bool up = q & d;
            const float keep = up ? v[i + d] : v[i], send = up ? v[i] : v[i + d];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, d * STEP);
        }
    }
    return v[0];
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// A thread's share of a tile's copies: 16 bytes of a row, `bytes` of them there (the others zero), or none (-1).  The source has
// to lie at a multiple of 16 bytes even where nothing is read of it.
template <typename T> struct Copy {
    const T *src;         // of tile 0
    long long step;       // elements to the next tile
    uint32_t dst;         // of stage 0
    int stage, row, bytes;
    // `live`: the tile has the row; else zeros, and nothing is read
    __device__ __forceinline__ void issue(int tile, int st, bool live) const {
        if (bytes < 0) return;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + st * stage), "l"(src + (live ? tile * step : 0)),
                     "r"(live ? bytes : 0)
                     : "memory");
    }
};
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A forward CTA has 64 channels, CT of them to a scanning thread.
template <typename T, int S, int CT> struct Tile {
    static constexpr int R = kTile, CH = 64;
    static constexpr int QW = S / 4, CW = 32 * CT;                       // warps of a channel group, channels of a warp
    static constexpr int SCAN = 32 * QW * (CH / CW), HELP = R * CH / 4;  // threads; a vector of four channels to a helper
    static constexpr int THREADS = SCAN + HELP;
    static constexpr int PER_SM = THREADS <= 384 ? 2 : 1;
    static constexpr int STAGES = 5;                                     // tiles on their way, or read for d, y or the outputs
    struct Smem {
        T in[STAGES][3][R][CH];            // x, dt, z
        T bc_in[STAGES][2][R][S];
        float ds[2][R][CH], us[2][R][CH];  // d and d x
        float bc[2][2][R][S];
        float ys[2][QW][R][CH];            // parts of y (the last member: a launch for ends has none)
    };
};

// Parts of `part` that N rows (or sequences) have: one at least.
__host__ __device__ __forceinline__ int parts_of(int N, int part) { return (N - 1) / part + 1; }
// The unit's sequence and part.  A sequence's parts are units i + off[i] / part onwards: there are as many as it needs.
__device__ __forceinline__ bool unit_of(const Params &P, int unit, int &seq, int &j, int &len) {
    if (!P.seq.off) {
        const int per = parts_of(P.seq.N, P.part);
        seq = unit / per, j = unit - seq * per, len = P.seq.N;
        return true;
    }
    int n;
    if (!offsets_in_order(P.seq, n, [&](int i, int lo) { return i + lo / P.part <= unit; })) return false;
    seq = n - 1;
    if (seq < 0) {  // (the first sequence begins behind the first part)
        j = len = 0;
        seq = P.seq.nseq;
        return true;
    }
    const int lo = P.seq.off[seq];
    j = unit - (seq + lo / P.part), len = P.seq.off[seq + 1] - lo;
    return true;
}
// The same where the offsets are known to be in order; by each thread itself.
__device__ __forceinline__ void unit_at(const Params &P, int unit, int &seq, int &j, int &first, int &len) {
    if (!P.seq.off) {
        const int per = parts_of(P.seq.N, P.part);
        seq = unit / per, j = unit - seq * per, first = seq * P.seq.N, len = P.seq.N;
        return;
    }
    int lo = 0, hi = P.seq.nseq;  // units of sequences before lo begin at or before this one, those from hi on behind it
    while (lo < hi) {
        const int m = (lo + hi) / 2;
        if (m + P.seq.off[m] / P.part <= unit) lo = m + 1;
        else hi = m;
    }
    seq = lo - 1, j = first = len = 0;
    if (seq < 0) return;
    first = P.seq.off[seq], len = P.seq.off[seq + 1] - first;
    j = unit - (seq + first / P.part);
}
__device__ __forceinline__ long long mark_slot(const Params &P, int seq, int row) {
    const long long lo = P.seq.off ? P.seq.off[seq] : (long long)seq * P.seq.N;
    return seq + lo / kMark + row / kMark;
}

// ENDS: the first launch, which forms the parts' last states only.
template <typename T, int S, int CT, bool ENDS>
__global__ void __launch_bounds__(Tile<T, S, CT>::THREADS, Tile<T, S, CT>::PER_SM) forward_kernel(const __grid_constant__ Params P) {
    using K = Tile<T, S, CT>;
    constexpr int CH = K::CH, R = K::R, QW = K::QW, HELP = K::HELP, ST = K::STAGES;
    extern __shared__ __align__(16) unsigned char raw[];
    typename K::Smem &M = *(typename K::Smem *)raw;
    const int cblocks = P.G * P.bpg, unit = blockIdx.x / cblocks, cb = blockIdx.x - unit * cblocks;
    int seq, j, len;
    if (!unit_of(P, unit, seq, j, len)) return;
    if (seq >= P.seq.nseq) return;
    const long long t0 = (long long)j * P.part;
    if (j > 0 && t0 >= len) return;
    const int lo = (int)t0, hi = (int)min(t0 + P.part, (long long)len);
    if (ENDS && hi == len) return;  // nothing follows
    const int g = cb / P.bpg, c0 = g * P.cpg + (cb - g * P.bpg) * CH, nc = min(CH, (g + 1) * P.cpg - c0);
    const int tiles = (hi - lo + R - 1) / R, helper = (int)threadIdx.x - K::SCAN;
    if (helper >= 0) {
        const T *x = rows_of<const T>(P.seq, P.x, seq) + c0, *dt = rows_of<const T>(P.seq, P.dt, seq) + c0;
        const T *z = P.z.p ? rows_of<const T>(P.seq, P.z, seq) + c0 : nullptr;
        T *y = ENDS ? nullptr : rows_of<T>(P.seq, P.y, seq) + c0;
        const T *Bp = (const T *)P.B.p + (P.seq.off ? P.seq.off[seq] * P.B.sn : seq * P.B.sb) + g * P.B.sg;
        const T *Cp = (const T *)P.C.p + (P.seq.off ? P.seq.off[seq] * P.C.sn : seq * P.C.sb) + g * P.C.sg;
        const int row = helper / (CH / 4), col = helper % (CH / 4) * 4, n = nc - col;
        float bias[4], D[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bias[k] = P.bias && k < n ? P.bias[c0 + col + k] : 0.f;
            D[k] = P.D && k < n ? P.D[c0 + col + k] : 0.f;
        }
        // x, dt, z, B and C of a tile, 16 bytes a copy, zeros where there is no row or channel
        constexpr int E = 16 / (int)sizeof(T), VR = CH / E, VS = S / E, ROWS = R * VR, ALL = 3 * ROWS + 2 * R * VS;
        Copy<T> mine[(ALL + HELP - 1) / HELP];
#pragma unroll
        for (int i = 0; i < (ALL + HELP - 1) / HELP; ++i) {
            const int v = i * HELP + helper;
            if (v < 3 * ROWS) {
                const int op = v / ROWS, r = v % ROWS / VR, e = v % VR * E;
                const T *p = op == 0 ? x : op == 1 ? dt : z;
                const long long sn = op == 0 ? P.x.sn : op == 1 ? P.dt.sn : P.z.sn;
                mine[i] = Copy<T>{p + (lo + r) * sn + e, R * sn, smem_addr(&M.in[0][op][r][e]), (int)sizeof(M.in[0]), r,
                                  op == 2 && (ENDS || !z) ? -1 : max(0, min(16, (nc - e) * (int)sizeof(T)))};
            } else {
                const int w = v - 3 * ROWS, op = w / (R * VS) & 1, r = w % (R * VS) / VS, e = w % VS * E;
                const long long sn = op ? P.C.sn : P.B.sn;
                mine[i] = Copy<T>{(op ? Cp : Bp) + (lo + r) * sn + e, R * sn, smem_addr(&M.bc_in[0][op][r][e]), (int)sizeof(M.bc_in[0]), r,
                                  v < ALL && !(op && ENDS) ? 16 : -1};
            }
        }
        auto copy = [&](int k) {
#pragma unroll
            for (int i = 0; i < (ALL + HELP - 1) / HELP; ++i) mine[i].issue(k, k % ST, lo + k * R < hi - mine[i].row);
            copy_commit();
        };
        const bool whole = nc == CH;
        auto produce = [&](int k) {
            const int t = lo + k * R, buf = k & 1, st = k % ST;
            const Vec<T, 4> vx = *(const Vec<T, 4> *)&M.in[st][0][row][col], vd = *(const Vec<T, 4> *)&M.in[st][1][row][col];
            const float2 a = step_of(P, make_float2(to_f(vd.e[0]) + bias[0], to_f(vd.e[1]) + bias[1]));
            const float2 b = step_of(P, make_float2(to_f(vd.e[2]) + bias[2], to_f(vd.e[3]) + bias[3]));
            float4 d = make_float4(a.x, a.y, b.x, b.y);
            if (!(whole && t + R <= hi)) {  // no row or channel: nothing happens
                if (t + row >= hi || n < 1) d.x = 0.f;
                if (t + row >= hi || n < 2) d.y = 0.f;
                if (t + row >= hi || n < 3) d.z = 0.f;
                if (t + row >= hi || n < 4) d.w = 0.f;
            }
            *(float4 *)&M.ds[buf][row][col] = d;
            *(float4 *)&M.us[buf][row][col] = make_float4(d.x * to_f(vx.e[0]), d.y * to_f(vx.e[1]), d.z * to_f(vx.e[2]), d.w * to_f(vx.e[3]));
            constexpr int NB = (ENDS ? 1 : 2) * R * S / 4;
#pragma unroll
            for (int i = 0; i < (NB + HELP - 1) / HELP; ++i) {
                const int v = i * HELP + helper;
                if (NB % HELP != 0 && v >= NB) break;
                const Vec<T, 4> f = ((const Vec<T, 4> *)M.bc_in[st])[v];
                ((float4 *)M.bc[buf])[v] = make_float4(to_f(f.e[0]), to_f(f.e[1]), to_f(f.e[2]), to_f(f.e[3]));
            }
        };
        auto finish = [&](int k) {
            const int t = lo + k * R, buf = k & 1, st = k % ST;
            const Vec<T, 4> vx = *(const Vec<T, 4> *)&M.in[st][0][row][col], vz = *(const Vec<T, 4> *)&M.in[st][2][row][col];
            float4 s = *(const float4 *)&M.ys[buf][0][row][col];
#pragma unroll
            for (int w = 1; w < QW; ++w) {
                const float4 o = *(const float4 *)&M.ys[buf][w][row][col];
                s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
            }
            float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = fmaf(D[e], to_f(vx.e[e]), v[e]);
                if (z) {
                    const float ze = to_f(vz.e[e]);
                    v[e] *= ze * sigmoid(ze);
                }
            }
            if (t + row < hi && n > 0) store_vec<T, 4>(y + (t + row) * P.y.sn + col, rounded4<T>(v), n);
        };
        copy(0), copy(1), copy(2);
        copy_wait<2>();
        __syncthreads();
        if (tiles > 0) produce(0);
        copy_wait<1>();
        // Step k, while tile k is scanned: d of tile k + 1, the outputs of tile k - 1, and tile k + 3 on its way into the
        // place of tile k - 2.  Tile k + 2 is there when the next step begins.
        for (int k = 0; k <= tiles; ++k) {
            __syncthreads();
            if (k + 1 < tiles) produce(k + 1);
            copy(k + 3);
            if (!ENDS && k > 0) finish(k - 1);
            copy_wait<1>();
        }
        copy_wait<0>();
        return;
    }
    // four states of CT neighbouring channels
    const int warp = threadIdx.x >> 5, q = warp % QW, ch = warp / QW * K::CW + (threadIdx.x & 31) * CT, c = c0 + ch;
    F4 a2[CT], h[CT];
    float sum[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        a2[i] = h[i] = zero4();
        sum[i] = 0.f;
        if (ch + i >= nc) continue;
        const long long at = (long long)(c + i) * S + 4 * q;
        a2[i] = rates4(P.A + at);
        if (j == 0) {
            if (P.first) h[i] = load4(P.first + (long long)seq * P.C_ * S + at);
        } else if (!ENDS) {
            h[i] = load4(P.ends + (long long)(unit - j) * P.C_ * S + at);
#pragma unroll 4
            for (int p = unit - j + 1; p < unit; ++p)
                h[i] = over_part(a2[i], P.sums[(long long)p * P.C_ + c + i], h[i], load4(P.ends + (long long)p * P.C_ * S + at));
        }
    }
    __syncthreads();
    for (int k = 0; k <= tiles; ++k) {
        __syncthreads();
        if (k == tiles) break;
        const int buf = k & 1;
        float *mark = !ENDS && P.marks ? P.marks + (mark_slot(P, seq, lo + k * R) * P.C_ + c) * S + 4 * q : nullptr;
        // A row's operands are loaded ahead of it, before the parts of y of the rows between are stored (which the compiler has
        // to take for stores to them); as many rows as registers allow.
        constexpr int DEPTH = CT == 1 ? 4 : 2;
        struct Row {
            float d[CT], u[CT];
            F4 B, C;
        } ahead[DEPTH];
        auto load = [&](int r, Row &o) {
            if constexpr (CT == 2) {
                const float2 d = *(const float2 *)&M.ds[buf][r][ch], u = *(const float2 *)&M.us[buf][r][ch];
                o.d[0] = d.x, o.d[1] = d.y, o.u[0] = u.x, o.u[1] = u.y;
            } else {
                o.d[0] = M.ds[buf][r][ch], o.u[0] = M.us[buf][r][ch];
            }
            o.B = load4(&M.bc[buf][0][r][4 * q]);
            if (!ENDS) o.C = load4(&M.bc[buf][1][r][4 * q]);
        };
#pragma unroll
        for (int r = 0; r < DEPTH - 1; ++r) load(r, ahead[r]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r + DEPTH - 1 < R) load(r + DEPTH - 1, ahead[(r + DEPTH - 1) % DEPTH]);
            const Row &o = ahead[r % DEPTH];
            if (r % kMark == 0 && mark && lo + k * R + r < hi) {
                float *m = mark + (long long)(r / kMark) * P.C_ * S;
#pragma unroll
                for (int i = 0; i < CT; ++i)
                    if (ch + i < nc) store4(m + i * S, h[i]);
            }
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                h[i] = fma4(decay4(a2[i], o.d[i]), h[i], mul4(o.B, o.u[i]));
                if (ENDS) sum[i] += o.d[i];
            }
            if constexpr (!ENDS) {
                if constexpr (CT == 2) *(float2 *)&M.ys[buf][q][r][ch] = make_float2(dot4(o.C, h[0]), dot4(o.C, h[CT - 1]));
                else M.ys[buf][q][r][ch] = dot4(o.C, h[0]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        if (ch + i >= nc) continue;
        const long long at = (long long)(c + i) * S + 4 * q;
        if (ENDS) {
            store4(P.ends + (long long)unit * P.C_ * S + at, h[i]);
            if (q == 0) P.sums[(long long)unit * P.C_ + c + i] = sum[i];
        } else if (P.last && hi == len) {
            store4(P.last + (long long)seq * P.C_ * S + at, h[i]);
        }
    }
}

// ------------------------------------------------------------------------------------------------------- backward
// The same roles.  A tile is kMark rows, entered with the state that the forward kept: its states are formed again, in
// registers, and its rows walked from the last to the first with G.  Four states of two channels leave a row's parts of y,
// sum G B and sum a h G A in shared memory, where the helping warps add them up and form the gradients of rows; dB and dC are
// summed over the warp's 64 channels, in the thread and then by butterflies of shuffles that hand each lane a value of its
// own (8 values over 8 lanes, then four rows of them over the four groups of lanes), and over the channel blocks by a launch
// of its own.  Bound by issue slots (834 instructions for a row of 64 channels, 65 % of the slots of the SMs that have two
// CTAs) and by the scanning warps' latencies; shared memory takes 190 clocks for such a row.  8 x 2048 x 2048, bf16: 743 us.
// Values kept from the way forth to the way back (decays, d, B) spill: 1713 us where forming them again takes 778.  Components
// turned so that lanes need not choose what they exchange save 6 % of the instructions and cost as much in shared memory.
template <typename T, int S> struct Back {
    static constexpr int R = kMark, QW = S / 4, GW = QW > 4 ? 1 : 4 / QW, CH = 64 * GW;
    static constexpr int HELP = R * CH / 4, SCAN = 32 * QW * GW, THREADS = HELP + SCAN;  // a vector of four channels to a helper
    static constexpr int STAGES = 4;  // tiles on their way, or read for d and g, or for the gradients of rows
    struct Smem {
        T in[STAGES][4][R][CH];                          // x, dt, dO, z
        T bc_in[STAGES][2][R][S];
        float ds[3][R][CH], us[2][R][CH], gs[2][R][CH];  // d, d x, g
        float bc[2][2][R][S];
        float ys[2][QW][R][CH], ws[2][QW][R][CH], es[2][QW][R][CH];
        float4 dA[2][2][SCAN];                           // each scanning thread's sums: of a group of tiles, of all groups
    };
};

// ENDS: where time is cut into parts, a first launch, which forms what leaves each part's first row (from zero behind its
// last, the last part from dstate_out) and the sum of its d.
template <typename T, int S, bool ENDS>
__global__ void __launch_bounds__(Back<T, S>::THREADS, S == 16 ? 2 : 1) backward_kernel(const __grid_constant__ Params P) {
    using K = Back<T, S>;
    constexpr int CH = K::CH, R = K::R, QW = K::QW, HELP = K::HELP, ST = K::STAGES;
    extern __shared__ __align__(16) unsigned char raw[];
    typename K::Smem &M = *(typename K::Smem *)raw;
    const int cblocks = P.G * P.bpg, walker = blockIdx.x / cblocks, cb = blockIdx.x - walker * cblocks;
    const int g = cb / P.bpg, c0 = g * P.cpg + (cb - g * P.bpg) * CH, nc = min(CH, (g + 1) * P.cpg - c0);
    bool fine = true;
    if (P.seq.off) {
        int n;
        fine = offsets_in_order(P.seq, n, [](int, int) { return false; });
    }
    if (!ENDS && blockIdx.x == 0 && threadIdx.x == 0) *P.valid = fine;
    const int helper = (int)threadIdx.x - K::SCAN;
    if (helper >= 0) {
        const int row = helper / (CH / 4), col = helper % (CH / 4) * 4, n = nc - col;
        float bias[4], D[4], dD[4], dbias[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bias[e] = P.bias && e < n ? P.bias[c0 + col + e] : 0.f;
            D[e] = P.D && e < n ? P.D[c0 + col + e] : 0.f;
            dD[e] = dbias[e] = 0.f;
        }
        for (int unit = walker; unit < P.units && fine; unit += P.walkers) {
            int seq, j, first, all;
            unit_at(P, unit, seq, j, first, all);
            const long long t0 = (long long)j * P.part;
            if (seq < 0 || (j > 0 && t0 >= all) || (ENDS && j == 0)) continue;
            const int lo = (int)t0, len = (int)min(t0 + P.part, (long long)all);  // rows lo ... len - 1
            const T *x = rows_of<const T>(P.seq, P.x, seq) + c0, *dt = rows_of<const T>(P.seq, P.dt, seq) + c0;
            const T *z = P.z.p ? rows_of<const T>(P.seq, P.z, seq) + c0 : nullptr, *dO = rows_of<const T>(P.seq, P.dO, seq) + c0;
            T *dx = rows_of<T>(P.seq, P.dx, seq) + c0 + col, *ddt = rows_of<T>(P.seq, P.ddt, seq) + c0 + col;
            T *dz = z ? rows_of<T>(P.seq, P.dz, seq) + c0 + col : nullptr;
            const T *Bp = (const T *)P.B.p + (P.seq.off ? first * P.B.sn : seq * P.B.sb) + g * P.B.sg;
            const T *Cp = (const T *)P.C.p + (P.seq.off ? first * P.C.sn : seq * P.C.sb) + g * P.C.sg;
            const int tiles = (len - lo + R - 1) / R;
            // x, dt, dO, z, B and C of a tile, 16 bytes a copy, zeros where there is no row or channel
            constexpr int E = 16 / (int)sizeof(T), VR = CH / E, VS = S / E, ROWS = R * VR, ALL = 4 * ROWS + 2 * R * VS;
            Copy<T> mine[(ALL + HELP - 1) / HELP];
#pragma unroll
            for (int i = 0; i < (ALL + HELP - 1) / HELP; ++i) {
                const int v = i * HELP + helper;
                if (v < 4 * ROWS) {
                    const int op = v / ROWS, r = v % ROWS / VR, e = v % VR * E;
                    const T *p = op == 0 ? x : op == 1 ? dt : op == 2 ? dO : z;
                    const long long sn = op == 0 ? P.x.sn : op == 1 ? P.dt.sn : op == 2 ? P.dO.sn : P.z.sn;
                    const bool on = !((op == 3 && !z) || (op == 0 && ENDS));
                    mine[i] = Copy<T>{p + (lo + r) * sn + e, R * sn, smem_addr(&M.in[0][op][r][e]), (int)sizeof(M.in[0]), r,
                                      on ? max(0, min(16, (nc - e) * (int)sizeof(T))) : -1};
                } else {
                    const int w = v - 4 * ROWS, op = w / (R * VS) & 1, r = w % (R * VS) / VS, e = w % VS * E;
                    const long long sn = op ? P.C.sn : P.B.sn;
                    mine[i] = Copy<T>{(op ? Cp : Bp) + (lo + r) * sn + e, R * sn, smem_addr(&M.bc_in[0][op][r][e]), (int)sizeof(M.bc_in[0]), r,
                                      v < ALL && (op || !ENDS) ? 16 : -1};
                }
            }
            auto copy = [&](int k) {
                if (k >= 0)
#pragma unroll
                    for (int i = 0; i < (ALL + HELP - 1) / HELP; ++i) mine[i].issue(k, k % ST, lo + k * R < len - mine[i].row);
                copy_commit();
            };
            auto produce = [&](int k) {
                const int t = lo + k * R, st = k % ST;
                auto at = [&](int op) { return *(const Vec<T, 4> *)&M.in[st][op][row][col]; };
                const Vec<T, 4> vx = at(0), vd = at(1), vo = at(2), vz = at(3);
                const float2 a = step_of(P, make_float2(to_f(vd.e[0]) + bias[0], to_f(vd.e[1]) + bias[1]));
                const float2 b = step_of(P, make_float2(to_f(vd.e[2]) + bias[2], to_f(vd.e[3]) + bias[3]));
                float d[4] = {a.x, a.y, b.x, b.y}, gr[4];
                if (!(nc == CH && t + R <= len))  // no row or channel: nothing happens (what was copied there is zero)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (t + row >= len || e >= n) d[e] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    gr[e] = to_f(vo.e[e]);
                    if (z) {
                        const float ze = to_f(vz.e[e]);
                        gr[e] *= ze * sigmoid(ze);
                    }
                }
                *(float4 *)&M.ds[k % 3][row][col] = make_float4(d[0], d[1], d[2], d[3]);
                *(float4 *)&M.gs[k & 1][row][col] = make_float4(gr[0], gr[1], gr[2], gr[3]);
                if (!ENDS) *(float4 *)&M.us[k & 1][row][col] = make_float4(d[0] * to_f(vx.e[0]), d[1] * to_f(vx.e[1]), d[2] * to_f(vx.e[2]), d[3] * to_f(vx.e[3]));
                constexpr int NB = 2 * R * S / 4;
#pragma unroll
                for (int i = 0; i < (NB + HELP - 1) / HELP; ++i) {
                    const int v = i * HELP + helper;
                    if (NB % HELP != 0 && v >= NB) break;
                    const Vec<T, 4> f = ((const Vec<T, 4> *)M.bc_in[st])[v];
                    ((float4 *)M.bc[k & 1])[v] = make_float4(to_f(f.e[0]), to_f(f.e[1]), to_f(f.e[2]), to_f(f.e[3]));
                }
            };
            auto total = [&](const float (&parts)[QW][R][CH], float (&s)[4]) {
                float4 a = *(const float4 *)&parts[0][row][col];
#pragma unroll
                for (int w = 1; w < QW; ++w) {
                    const float4 o = *(const float4 *)&parts[w][row][col];
                    a.x += o.x, a.y += o.y, a.z += o.z, a.w += o.w;
                }
                s[0] = a.x, s[1] = a.y, s[2] = a.z, s[3] = a.w;
            };
            auto finish = [&](int k) {
                const int r = lo + k * R + row, st = k % ST;
                if (r >= len || n <= 0) return;
                auto in = [&](int op) { return *(const Vec<T, 4> *)&M.in[st][op][row][col]; };
                const Vec<T, 4> vx = in(0), vd = in(1), vo = in(2), vz = in(3);
                float w[4], es[4], ys[4];
                total(M.ws[k & 1], w), total(M.es[k & 1], es);
                if (z) total(M.ys[k & 1], ys);
                const float4 d4 = *(const float4 *)&M.ds[k % 3][row][col];
                const float d[4] = {d4.x, d4.y, d4.z, d4.w};
                float fx[4], fd[4], fz[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float xe = to_f(vx.e[e]), oe = to_f(vo.e[e]);
                    float gr = oe;
                    if (z) {
                        const float ze = to_f(vz.e[e]), sg = sigmoid(ze);
                        gr *= ze * sg;
                        fz[e] = oe * fmaf(D[e], xe, ys[e]) * silu_grad(ze, sg);
                    }
                    fx[e] = fmaf(d[e], w[e], D[e] * gr);
                    float s = fmaf(es[e], kLn2, xe * w[e]);
                    if (P.softplus) s *= sigmoid(to_f(vd.e[e]) + bias[e]);
                    fd[e] = s;
                    dbias[e] += s;
                    dD[e] = fmaf(gr, xe, dD[e]);
                }
                store_vec<T, 4>(dx + r * P.dx.sn, rounded4<T>(fx), n);
                store_vec<T, 4>(ddt + r * P.ddt.sn, rounded4<T>(fd), n);
                if (z) store_vec<T, 4>(dz + r * P.dz.sn, rounded4<T>(fz), n);
            };
            copy(tiles - 1), copy(tiles - 2);
            copy_wait<1>();
            __syncthreads();
            if (tiles > 0) produce(tiles - 1);
            copy_wait<0>();
            // while tile k is walked: d and g of tile k - 1, the gradients of tile k + 1, and tile k - 2 on its way into the place
            // of tile k + 2
            for (int k = tiles - 1; k >= -1; --k) {
                __syncthreads();
                if (k > 0) produce(k - 1);
                copy(k - 2);
                if (!ENDS && k + 1 < tiles) finish(k + 1);
                copy_wait<0>();
            }
            __syncthreads();  // the last tile's shared memory has been read
        }
        if constexpr (!ENDS) {
            // dD and the bias: over the tile's rows
#pragma unroll
            for (int e = 0; e < 4; ++e) M.us[0][row][col + e] = dD[e], M.gs[0][row][col + e] = dbias[e];
            __syncthreads();
            float *pd = P.pa + (long long)walker * P.C_ * (S + 2) + (long long)P.C_ * S;
            for (int v = helper; v < nc; v += HELP) {
                float s = 0.f, b = 0.f;
                for (int r = 0; r < R; ++r) s += M.us[0][r][v], b += M.gs[0][r][v];
                pd[c0 + v] = s;
                pd[P.C_ + c0 + v] = b;
            }
        }
        return;
    }
    // four states of two neighbouring channels
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp % QW, group = warp / QW, ch = group * 64 + lane * 2, c = c0 + ch;
    F4 a2[2] = {zero4(), zero4()}, dA[2] = {zero4(), zero4()};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (ch + i < nc) a2[i] = rates4(P.A + (long long)(c + i) * S + 4 * q);
        M.dA[0][i][threadIdx.x] = M.dA[1][i][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto flush = [&](bool group_ends) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float4 &s = M.dA[0][i][threadIdx.x], &all = M.dA[1][i][threadIdx.x];
            s = make_float4(s.x + dA[i].a.x, s.y + dA[i].a.y, s.z + dA[i].b.x, s.w + dA[i].b.y);
            dA[i] = zero4();
            if (!group_ends) continue;
            all = make_float4(all.x + s.x, all.y + s.y, all.z + s.z, all.w + s.w);
            s = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    for (int unit = walker; unit < P.units && fine; unit += P.walkers) {
        int seq, j, first, all;
        unit_at(P, unit, seq, j, first, all);
        const long long t0 = (long long)j * P.part;
        if (seq < 0 || (j > 0 && t0 >= all) || (ENDS && j == 0)) continue;
        const int lo = (int)t0, len = (int)min(t0 + P.part, (long long)all);
        const int tiles = (len - lo + R - 1) / R;
        F4 carry[2] = {zero4(), zero4()};  // a_{t+1} G_{t+1}
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (ch + i >= nc) continue;
            const long long at = (long long)(c + i) * S + 4 * q;
            if (P.dlast && len == all) carry[i] = load4(P.dlast + (long long)seq * P.C_ * S + at);
            if (ENDS || len == all) continue;
            const int last = unit + (all - lo - 1) / P.part;  // the sequence's last part, whose end has dstate_out in it
            carry[i] = load4(P.ends + (long long)last * P.C_ * S + at);
#pragma unroll 4
            for (int p = last - 1; p > unit; --p)
                carry[i] = over_part(a2[i], P.sums[(long long)p * P.C_ + c + i], carry[i], load4(P.ends + (long long)p * P.C_ * S + at));
        }
        float sum[2] = {0.f, 0.f};
        Vec<float, 4> mark[2] = {};
        auto fetch = [&](int k) {
            if (ENDS) return;
            const float *m = P.marks + (mark_slot(P, seq, lo + k * R) * P.C_ + c) * S + 4 * q;
            load_ahead(mark[0], m, k >= 0 && ch < nc);
            load_ahead(mark[1], m + S, k >= 0 && ch + 1 < nc);
        };
        fetch(tiles - 1);
        __syncthreads();
        // sums of dB (values 0 ... 3) and dC (4 ... 7) of the warp's states: a lane's value of a row of four
        float *pbc = P.pbc + ((long long)((cb - g * P.bpg) * K::GW + group) * P.seq.T + first) * P.G * 2 * S + g * 2 * S +
                     (lane & 4 ? S : 0) + 4 * q + (lane & 3);
        for (int k = tiles - 1; k >= -1; --k) {
            __syncthreads();
            if (k < 0) break;
            const int buf = k & 1;
            const auto &ds = M.ds[k % 3];
            if constexpr (ENDS) {
#pragma unroll
                for (int r = R - 1; r >= 0; --r) {
                    const float2 d = *(const float2 *)&ds[r][ch], gr = *(const float2 *)&M.gs[buf][r][ch];
                    const F4 C = load4(&M.bc[buf][1][r][4 * q]);
                    carry[0] = mul4(decay4(a2[0], d.x), fma4(C, gr.x, carry[0]));
                    carry[1] = mul4(decay4(a2[1], d.y), fma4(C, gr.y, carry[1]));
                    sum[0] += d.x, sum[1] += d.y;
                }
            } else {
                F4 h0[2];  // the tile's first state
#pragma unroll
                for (int i = 0; i < 2; ++i) h0[i] = F4{make_float2(mark[i].e[0], mark[i].e[1]), make_float2(mark[i].e[2], mark[i].e[3])};
                fetch(k - 1);
                auto advance = [&](int r, const F4(&h)[2], F4(&to)[2]) {
                    const float2 d = *(const float2 *)&ds[r][ch], u = *(const float2 *)&M.us[buf][r][ch];
                    const F4 B = load4(&M.bc[buf][0][r][4 * q]);
                    to[0] = fma4(decay4(a2[0], d.x), h[0], mul4(B, u.x));
                    to[1] = fma4(decay4(a2[1], d.y), h[1], mul4(B, u.y));
                };
#pragma unroll
                for (int half = R - 4; half >= 0; half -= 4) {
                    F4 hs[5][2];  // the states before each of four rows, and behind the last
                    hs[0][0] = h0[0], hs[0][1] = h0[1];
#pragma unroll
                    for (int r = 0; r < half; ++r) advance(r, hs[0], hs[0]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) advance(half + r, hs[r], hs[r + 1]);
                    asm volatile("" ::: "memory");  // d, d x, B and the decays are not kept for the way back: registers are short
                    // Four rows' results are stored together: a store ends what may be loaded early.
                    float four[4];
                    float2 w[4], e[4], y[4];
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        const int r = half + i;
                        const float2 d = *(const float2 *)&ds[r][ch], u = *(const float2 *)&M.us[buf][r][ch], gr = *(const float2 *)&M.gs[buf][r][ch];
                        const F4 B = load4(&M.bc[buf][0][r][4 * q]), C = load4(&M.bc[buf][1][r][4 * q]);
                        if (P.z.p) y[i] = make_float2(dot4(C, hs[i + 1][0]), dot4(C, hs[i + 1][1]));
                        const F4 G0 = fma4(C, gr.x, carry[0]), G1 = fma4(C, gr.y, carry[1]);
                        const F4 dB = fma4(G1, u.y, mul4(G0, u.x)), dC = fma4(hs[i + 1][1], gr.y, mul4(hs[i + 1][0], gr.x));
                        w[i] = make_float2(dot4(G0, B), dot4(G1, B));
                        carry[0] = mul4(decay4(a2[0], d.x), G0);
                        carry[1] = mul4(decay4(a2[1], d.y), G1);
                        const F4 e0 = mul4(carry[0], hs[i][0]), e1 = mul4(carry[1], hs[i][1]);
                        dA[0] = fma4(e0, d.x, dA[0]);
                        dA[1] = fma4(e1, d.y, dA[1]);
                        e[i] = make_float2(dot4(e0, a2[0]), dot4(e1, a2[1]));
                        float v[8] = {dB.a.x, dB.a.y, dB.b.x, dB.b.y, dC.a.x, dC.a.y, dC.b.x, dC.b.y};
                        four[i] = lanes_sum<8, 1>(v, lane & 7);
                    }
                    const float s = lanes_sum<4, 8>(four, lane >> 3);
                    const int at = lo + k * R + half + (lane >> 3);
                    if (at < len) pbc[(long long)at * P.G * 2 * S] = s;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        *(float2 *)&M.ws[buf][q][half + i][ch] = w[i];
                        *(float2 *)&M.es[buf][q][half + i][ch] = e[i];
                        if (P.z.p) *(float2 *)&M.ys[buf][q][half + i][ch] = y[i];
                    }
                }
                flush(k % kGroup == 0);  // (registers added to shared memory once in eight tiles: 752 us)
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (ch + i >= nc) continue;
            const long long at = (long long)(c + i) * S + 4 * q;
            if (ENDS) {
                store4(P.ends + (long long)unit * P.C_ * S + at, carry[i]);
                if (q == 0) P.sums[(long long)unit * P.C_ + c + i] = sum[i];
            } else if (P.dfirst && j == 0) {
                store4(P.dfirst + (long long)seq * P.C_ * S + at, carry[i]);
            }
        }
        __syncthreads();
    }
    if (ENDS) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (ch + i < nc) {  // (a walker's sums begin at 16 bytes where the channels are even)
            const float4 f = M.dA[1][i][threadIdx.x];
            store_vec(P.pa + (long long)walker * P.C_ * (S + 2) + (long long)(c + i) * S + 4 * q, Vec<float, 4>{{f.x, f.y, f.z, f.w}}, 4,
                      P.C_ % 2 == 0);
        }
    __syncthreads();
}

// dB and dC: the channel blocks' sums, rounded once.
template <typename T, int S> __global__ void __launch_bounds__(256) sum_bc_kernel(const __grid_constant__ Params P, T *dB, T *dC) {
    if (P.seq.off && *P.valid == 0) return;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, row_w = (long long)P.G * 2 * S, row = i / row_w;
    const int at = (int)(i - row * row_w);
    if (row >= P.seq.T) return;
    if (P.seq.off && (row < P.seq.off[0] || row >= P.seq.off[P.seq.nseq])) return;
    float s = 0.f;
#pragma unroll 4
    for (int b = 0; b < P.bpg * Back<T, S>::GW; ++b) s += P.pbc[(long long)b * P.seq.T * row_w + i];
    const int g = at / (2 * S), n = at % (2 * S);
    put((n < S ? dB : dC) + (row * P.G + g) * S + n % S, s);
}

// ----------------------------------------------------------------------------------------------------------- step
// S / 4 lanes to a channel; a block keeps its channels' A and walks `per` sequences, two states to a lane on their way.  Bound by
// the state's bytes: 256 x 4096 x 16, bf16: 31.5 us, 4.5 TB/s (one state on its way 37, four 37 with fewer blocks).
template <typename T, int S> __global__ void __launch_bounds__(kThreads, 4) step_kernel(const __grid_constant__ Params P, int per) {
    constexpr int L = S / 4;
    const int q = threadIdx.x % L, c = (int)((blockIdx.x * (long long)kThreads + threadIdx.x) / L);
    const bool mine = c < P.C_;
    const int cc = mine ? c : 0, g = cc / P.cpg;
    const F4 a2 = rates4(P.A + (long long)cc * S + 4 * q);
    const float bias = P.bias ? P.bias[cc] : 0.f, D = P.D ? P.D[cc] : 0.f;
    const int b1 = (int)min((blockIdx.y + 1) * (unsigned)per, (unsigned)P.seq.nseq);
    constexpr int U = 2;  // sequences whose states are on their way together
    for (int b0 = blockIdx.y * per; b0 < b1; b0 += U) {
        Vec<float, 4> h0[U];
        Vec<T, 4> vb[U], vc[U];
        T x[U], dt[U], z[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const long long b = min(b0 + i, b1 - 1);
            h0[i] = *(const Vec<float, 4> *)(P.last + (b * P.C_ + cc) * S + 4 * q);
            vb[i] = *(const Vec<T, 4> *)((const T *)P.B.p + b * P.B.sb + g * P.B.sg + 4 * q);
            vc[i] = *(const Vec<T, 4> *)((const T *)P.C.p + b * P.C.sb + g * P.C.sg + 4 * q);
            x[i] = ((const T *)P.x.p)[b * P.x.sb + cc];
            dt[i] = ((const T *)P.dt.p)[b * P.dt.sb + cc];
            if (P.z.p) z[i] = ((const T *)P.z.p)[b * P.z.sb + cc];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (b0 + i >= b1) break;  // the same for the block
            const long long b = b0 + i;
            const float xv = to_f(x[i]), d = step_of(P, both(to_f(dt[i]) + bias)).x;
            const F4 B{make_float2(to_f(vb[i].e[0]), to_f(vb[i].e[1])), make_float2(to_f(vb[i].e[2]), to_f(vb[i].e[3]))};
            const F4 C{make_float2(to_f(vc[i].e[0]), to_f(vc[i].e[1])), make_float2(to_f(vc[i].e[2]), to_f(vc[i].e[3]))};
            const F4 h = fma4(decay4(a2, d), F4{make_float2(h0[i].e[0], h0[i].e[1]), make_float2(h0[i].e[2], h0[i].e[3])}, mul4(B, d * xv));
            if (mine) store4(P.last + (b * P.C_ + cc) * S + 4 * q, h);
            float y = dot4(C, h);
#pragma unroll
            for (int k = L / 2; k > 0; k /= 2) y += __shfl_xor_sync(0xffffffffu, y, k);
            if (q == 0 && mine) {
                y = fmaf(D, xv, y);
                if (P.z.p) {
                    const float zv = to_f(z[i]);
                    y *= zv * sigmoid(zv);
                }
                put((T *)P.y.p + b * P.y.sb + cc, y);
            }
        }
    }
}

// ----------------------------------------------------------------------------------------------------------- host
constexpr int kForwardChannels = 64;
int back_channels(int S) { return S == 8 ? Back<float, 8>::CH : S == 16 ? Back<float, 16>::CH : Back<float, 32>::CH; }
int blocks_per_group(int C, int G, int channels) { return (C / G + channels - 1) / channels; }

// Rows of a part.  Where the sequences' channel blocks make fewer CTAs than one for two SMs, as many parts of a sequence of the
// mean length as stand on the SMs at once, two CTAs on each, of kLeastPart rows at least (1 x 65536 x 2048, bf16: 9 parts 1.13 ms,
// one 3.51 ms).  That is what fits with 8 states and with 16 in bf16; with 16 in fp32 (124,928 bytes of shared memory) and with 32
// (131,072 and 172,032) one CTA fits, and such parts stand in two rounds; these were not measured.  Else eight mean lengths: only
// packed sequences that are far longer than the others are cut, but a packed call of more than that in all makes the launch for
// the parts' last states in any case, as the host does not know the lengths.
constexpr int kLeastPart = 128;
int part_rows(int T, int nseq, int C, int G) {
    const long long n = nseq > 0 ? nseq : 1, ctas = n * G * blocks_per_group(C, G, kForwardChannels);
    const long long whole = ((long long)T + kTile) / kTile * kTile;
    long long part = 8 * ((T + n - 1) / n);
    if (ctas < kSMs / 2 && T / n >= 2 * kLeastPart) {
        long long want = 2 * kSMs / ctas;
        if (want > kMaxParts) want = kMaxParts;
        part = (T + n * want - 1) / (n * want);
    }
    if (part < kLeastPart) part = kLeastPart;
    part = (part + kTile - 1) / kTile * kTile;
    return (int)(part < whole ? part : whole);
}
long long units_of(int T, int nseq, int N, int part, bool packed) {
    if (packed) return (long long)nseq + T / part;
    return (long long)nseq * parts_of(N, part);
}
// CTAs of a channel block in the backward walk: four CTAs to an SM in all, or the units that there are at most (a batch has no
// more than the same sequences packed).
int walkers_of(int T, int nseq, int C, int G, int S) {
    const long long cblocks = (long long)G * blocks_per_group(C, G, back_channels(S)), want = (4 * kSMs + cblocks - 1) / cblocks;
    const long long units = units_of(T, nseq, 0, part_rows(T, nseq, C, G), true);
    return (int)(units < want ? units : want);
}
struct Space {  // byte offsets of the workspace's arrays
    size_t ends, sums, pbc, pa, bytes;
};
Space space_of(int T, int nseq, int C, int G, int S, bool back) {
    Space w = {};
    size_t at = 256;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) & ~(size_t)255;
        return here;
    };
    const int part = part_rows(T, nseq, C, G);
    if (part < T) {
        const size_t units = (size_t)units_of(T, nseq, 0, part, true) + 1;  // a batch has no more
        w.ends = take(units * C * S * 4);
        w.sums = take(units * C * 4);
    }
    if (back) {
        const size_t walkers = walkers_of(T, nseq, C, G, S);
        w.pbc = take((size_t)blocks_per_group(C, G, back_channels(S)) * (back_channels(S) / 64) * T * G * 2 * S * 4);
        w.pa = take(walkers * C * (S + 2) * 4);
    }
    w.bytes = at;
    return w;
}

int check_sizes(int nseq, int N, int C, int G, int S, int dtype, bool packed) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (nseq < 0 || N < 0 || C < 1 || C >= 1 << 24 || G < 1 || S < 1 || C % G != 0) return LA_ERR_INVALID_ARG;
    const long long T = packed ? N : (long long)nseq * N;
    if (T > kMaxRows || nseq > kMaxRows || T >= (1LL << 40) / C || (long long)nseq * S >= (1LL << 40) / C ||
        (long long)G * S >= (1LL << 31) / 2 || T >= (1LL << 40) / ((long long)G * S))
        return LA_ERR_INVALID_ARG;
    if ((S != 8 && S != 16 && S != 32) || (G > 1 && (C / G) % 8 != 0)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// A [B, N, G, S] operand.
int group_view(View &v, const void *p, int B, int N, int G, int S, int elem, const long long *strides) {
    if (!p || ((uintptr_t)p & 15)) return LA_ERR_INVALID_ARG;
    v = View{p, {B, N, G}, {}, S, elem};
    const long long dense[3] = {(long long)N * G * S, (long long)G * S, S};
    return set_view(v, strides ? strides : dense, dense);
}

// What the three calls share: parameters and views of (X, dt, z, Y or dO) x (batch, row), and B, C x (batch, row, group).
struct Call {
    Params P = {};
    View v[6] = {};
    Range rin[8] = {};
};
int take_inputs(Call &K, const void *X, const void *dt, const float *A, const void *B, const void *C, const float *D,
                const void *z, const float *bias, const void *other, const float *state, const int *off, int nseq, int N,
                int Cn, int G, int S, int softplus, int dtype, const long long *strides) {
    const bool packed = off != nullptr;
    const int elem = dtype == LA_BF16 ? 2 : 4, batch = packed ? 1 : nseq, T = packed ? N : nseq * N;
    if (!A || ((uintptr_t)A & 15) || ((uintptr_t)D & 15) || ((uintptr_t)bias & 15) || ((uintptr_t)state & 15) || ((uintptr_t)off & 3))
        return LA_ERR_INVALID_ARG;
    // Operands that have one row at most are never stepped, and the rows of a tile behind the last one are addressed, though not
    // read: their row stride is 0, as the width of one row need not be whole vectors.  Without rows A stands for them.
    const void *ptr[4] = {X, dt, z, other};
    if (T == 0) ptr[0] = ptr[1] = ptr[3] = B = C = A, ptr[2] = z ? A : nullptr;
    int rc;
    for (int k = 0; k < 4 && T > 0; ++k) {
        if (k == 2 && !z) continue;
        if ((rc = rows_view(K.v[k], ptr[k], batch, N, Cn, elem, strides ? strides + 2 * k : nullptr))) return rc;
    }
    if (T > 0) {
        if ((rc = group_view(K.v[4], B, batch, N, G, S, elem, strides ? strides + 8 : nullptr))) return rc;
        if ((rc = group_view(K.v[5], C, batch, N, G, S, elem, strides ? strides + 11 : nullptr))) return rc;
    }
    Params &P = K.P;
    const bool stepped = (packed ? T : N) > 1;
    auto op = [&](int k) { return Op{ptr[k], K.v[k].st[0], stepped ? K.v[k].st[1] : 0}; };
    P.x = op(0), P.dt = op(1), P.z = op(2), P.y = P.dO = op(3);
    P.y.p = other;
    auto group_op = [&](int k, const void *p) { return GOp{p, K.v[k].st[0], stepped ? K.v[k].st[1] : 0, K.v[k].st[2]}; };
    P.B = group_op(4, B), P.C = group_op(5, C);
    P.A = A, P.D = D, P.bias = bias, P.first = state;
    P.seq = Seqs{off, nseq, N, T, nullptr};
    P.C_ = Cn, P.G = G, P.cpg = Cn / G;
    P.softplus = softplus ? 1 : 0;
    K.rin[0] = {A, (size_t)Cn * S * 4};
    K.rin[1] = {D, (size_t)Cn * 4};
    K.rin[2] = {bias, (size_t)Cn * 4};
    K.rin[3] = {state, (size_t)nseq * Cn * S * 4};
    K.rin[4] = {off, ((size_t)nseq + 1) * 4};
    return LA_OK;
}

template <typename T, int S, int CT> cudaError_t launch_forward(const Params &P, long long blocks, bool split, cudaStream_t s) {
    using K = Tile<T, S, CT>;
    constexpr int all = (int)sizeof(typename K::Smem), some = (int)offsetof(typename K::Smem, ys);
    static std::atomic<int> attr_state[kMaxDevices];
    if (!once_per_device(attr_state, [] {
            return cudaFuncSetAttribute(forward_kernel<T, S, CT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, some) == cudaSuccess &&
                   cudaFuncSetAttribute(forward_kernel<T, S, CT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, all) == cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    if (split) {
        forward_kernel<T, S, CT, true><<<(unsigned)blocks, K::THREADS, some, s>>>(P);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    forward_kernel<T, S, CT, false><<<(unsigned)blocks, K::THREADS, all, s>>>(P);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}
// One channel to a scanning thread where each SM has one CTA at most, whose warps then are too few; else two.
template <typename T, int S> cudaError_t forward(const Params &P, long long units, bool split, cudaStream_t s) {
    const long long blocks = units * P.G * P.bpg;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    if (S <= 16 && blocks <= kSMs) return launch_forward<T, S, S <= 16 ? 1 : 2>(P, blocks, split, s);
    return launch_forward<T, S, 2>(P, blocks, split, s);
}
template <typename T> cudaError_t forward(const Params &P, int S, long long units, bool split, cudaStream_t s) {
    return S == 8 ? forward<T, 8>(P, units, split, s) : S == 16 ? forward<T, 16>(P, units, split, s) : forward<T, 32>(P, units, split, s);
}

template <typename T, int S> cudaError_t backward(const Params &P, bool split, void *dB, void *dC, float *dA, float *dD, float *dbias, cudaStream_t s) {
    using M = typename Back<T, S>::Smem;
    static std::atomic<int> attr_state[kMaxDevices];
    if (!once_per_device(attr_state, [] {
            return cudaFuncSetAttribute(backward_kernel<T, S, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(M)) == cudaSuccess &&
                   cudaFuncSetAttribute(backward_kernel<T, S, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(M)) == cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    const long long blocks = (long long)P.walkers * P.G * P.bpg;
    if (blocks > 0) {
        cudaError_t e;
        if (split) {
            backward_kernel<T, S, true><<<(unsigned)blocks, Back<T, S>::THREADS, sizeof(M), s>>>(P);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            count_launches(1);
        }
        backward_kernel<T, S, false><<<(unsigned)blocks, Back<T, S>::THREADS, sizeof(M), s>>>(P);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        count_launches(1);
        const long long sums = ((long long)P.seq.T * P.G * 2 * S + 255) / 256;
        if (sums >= (1LL << 31)) return cudaErrorInvalidConfiguration;
        if (sums > 0) {
            sum_bc_kernel<T, S><<<(unsigned)sums, 256, 0, s>>>(P, (T *)dB, (T *)dC);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            count_launches(1);
        }
    }
    const long long n = (long long)P.C_ * S;
    return sum_parts(P.pa, P.walkers, n + 2LL * P.C_, dA, n, dD, P.C_, dbias, s);
}
template <typename T> cudaError_t backward(const Params &P, int S, bool split, void *dB, void *dC, float *dA, float *dD, float *dbias, cudaStream_t s) {
    return S == 8 ? backward<T, 8>(P, split, dB, dC, dA, dD, dbias, s) : S == 16 ? backward<T, 16>(P, split, dB, dC, dA, dD, dbias, s)
                                                                       : backward<T, 32>(P, split, dB, dC, dA, dD, dbias, s);
}

template <typename T, int S> cudaError_t step(const Params &P, cudaStream_t s) {
    const long long across = ((long long)P.C_ * (S / 4) + kThreads - 1) / kThreads;
    // Sequences to a block, which read A once: as many as leave 16 blocks to an SM.
    int per = 1;
    while (per < 16 && across * parts_of(P.seq.nseq, 2 * per) >= 16 * kSMs) per *= 2;
    while (parts_of(P.seq.nseq, per) > 65535) per *= 2;
    step_kernel<T, S><<<dim3((unsigned)across, (unsigned)parts_of(P.seq.nseq, per)), kThreads, 0, s>>>(P, per);
    return cudaGetLastError();
}
template <typename T> cudaError_t step(const Params &P, int S, cudaStream_t s) {
    return S == 8 ? step<T, 8>(P, s) : S == 16 ? step<T, 16>(P, s) : step<T, 32>(P, s);
}

int status_of(cudaError_t e) { return e == cudaSuccess ? LA_OK : e == cudaErrorInvalidConfiguration ? LA_ERR_INVALID_ARG : LA_ERR_CUDA; }

}  // namespace sel
}  // namespace la

extern "C" {

size_t la_selective_scan_marks_bytes(int T, int nseq, int C, int S) {
    if (T < 0 || T > la::rows::kMaxRows || nseq < 0 || C < 1 || (S != 8 && S != 16 && S != 32)) return 0;
    return ((size_t)nseq + T / la::sel::kMark) * C * S * 4;
}

size_t la_selective_scan_workspace_bytes(int T, int nseq, int C, int G, int S, int dtype, int backward) {
    if (la::sel::check_sizes(nseq, T, C, G, S, dtype, true)) return 0;
    return la::sel::space_of(T, nseq, C, G, S, backward != 0).bytes;
}

int la_selective_scan(const void *X, const void *dt, const float *A, const void *B, const void *C, const float *D,
                      const void *z, const float *dt_bias, int softplus, const float *state_in, void *Y,
                      float *state_out, float *marks, const int *seq_offsets, int nseq, int N, int channels, int G,
                      int S, int dtype, const long long *strides, void *workspace, size_t workspace_bytes,
                      void *stream) {
    using namespace la;
    using namespace la::sel;
    const bool packed = seq_offsets != nullptr;
    int rc = check_sizes(nseq, N, channels, G, S, dtype, packed);
    if (rc) return rc;
    const int T = packed ? N : nseq * N;
    const Space w = space_of(T, nseq, channels, G, S, false);
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < w.bytes) return LA_ERR_WORKSPACE;
    Call K;
    if ((rc = take_inputs(K, X, dt, A, B, C, D, z, dt_bias, Y, state_in, seq_offsets, nseq, N, channels, G, S, softplus, dtype, strides)))
        return rc;
    if (((uintptr_t)state_out & 15) || ((uintptr_t)marks & 15)) return LA_ERR_INVALID_ARG;
    const View in[5] = {K.v[0], K.v[1], K.v[2], K.v[4], K.v[5]};
    const Range rout[3] = {{state_out, (size_t)nseq * channels * S * 4},
                           {marks, la_selective_scan_marks_bytes(T, nseq, channels, S)},
                           {workspace, w.bytes}};
    if (outputs_meet(in, 5, &K.v[3], 1, K.rin, 5, rout, 3)) return LA_ERR_INVALID_ARG;
    if (nseq == 0) return LA_OK;
    Params &P = K.P;
    P.last = state_out, P.marks = marks;
    P.bpg = blocks_per_group(channels, G, kForwardChannels);
    P.seq.status = (uint32_t *)workspace;
    P.part = part_rows(T, nseq, channels, G);
    const long long units = units_of(T, nseq, N, P.part, packed);
    const bool split = P.part < T && (packed || N > P.part);
    P.ends = (float *)((char *)workspace + w.ends), P.sums = (float *)((char *)workspace + w.sums);
    cudaStream_t s = (cudaStream_t)stream;
    return status_of(dtype == LA_BF16 ? forward<__nv_bfloat16>(P, S, units, split, s) : forward<float>(P, S, units, split, s));
}

int la_selective_scan_backward(const void *X, const void *dt, const float *A, const void *B, const void *C,
                               const float *D, const void *z, const float *dt_bias, int softplus, const void *dY,
                               const float *marks, const float *dstate_out, void *dX, void *ddt, float *dA, void *dB,
                               void *dC, float *dD, void *dz, float *ddt_bias, float *dstate_in,
                               const int *seq_offsets, int nseq, int N, int channels, int G, int S, int dtype,
                               const long long *strides, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace la;
    using namespace la::sel;
    const bool packed = seq_offsets != nullptr;
    int rc = check_sizes(nseq, N, channels, G, S, dtype, packed);
    if (rc) return rc;
    const int T = packed ? N : nseq * N, elem = dtype == LA_BF16 ? 2 : 4;
    const Space w = space_of(T, nseq, channels, G, S, true);
    if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < w.bytes) return LA_ERR_WORKSPACE;
    Call K;
    if ((rc = take_inputs(K, X, dt, A, B, C, D, z, dt_bias, dY, dstate_out, seq_offsets, nseq, N, channels, G, S, softplus, dtype, strides)))
        return rc;
    if (((uintptr_t)marks & 15) || (T > 0 && !marks) || !dA || ((uintptr_t)dA & 15) || ((uintptr_t)dD & 15) ||
        ((uintptr_t)ddt_bias & 15) || ((uintptr_t)dstate_in & 15) || ((z != nullptr) != (dz != nullptr) && T > 0))
        return LA_ERR_INVALID_ARG;
    View out[3] = {};
    void *const po[3] = {dX, ddt, dz};
    const long long dense[2] = {(long long)N * channels, channels};
    if (T > 0) {
        if (!dB || !dC || ((uintptr_t)dB & 15) || ((uintptr_t)dC & 15)) return LA_ERR_INVALID_ARG;
        for (int k = 0; k < 3; ++k)
            if (po[k] && (rc = rows_view(out[k], po[k], packed ? 1 : nseq, N, channels, elem, dense))) return rc;
        if (!dX || !ddt) return LA_ERR_INVALID_ARG;
    }
    const size_t bc = (size_t)T * G * S * elem;
    K.rin[5] = {marks, la_selective_scan_marks_bytes(T, nseq, channels, S)};
    const Range rout[7] = {{dA, (size_t)channels * S * 4}, {dB, bc}, {dC, bc}, {dD, (size_t)channels * 4},
                           {ddt_bias, (size_t)channels * 4}, {dstate_in, (size_t)nseq * channels * S * 4}, {workspace, w.bytes}};
    if (outputs_meet(K.v, 6, out, 3, K.rin, 6, rout, 7)) return LA_ERR_INVALID_ARG;
    Params &P = K.P;
    P.first = nullptr;
    P.bpg = blocks_per_group(channels, G, back_channels(S));
    P.dlast = dstate_out, P.dfirst = dstate_in, P.marks = (float *)marks;
    P.seq.status = (uint32_t *)workspace;
    P.valid = (uint32_t *)workspace + offsetof(WsHeader, reserved) / 4;
    P.dx = Op{dX, out[0].st[0], out[0].st[1]};
    P.ddt = Op{ddt, out[1].st[0], out[1].st[1]};
    P.dz = Op{dz, out[2].st[0], out[2].st[1]};
    P.part = part_rows(T, nseq, channels, G);
    const bool split = P.part < T && (packed || N > P.part);
    const long long units = units_of(T, nseq, N, P.part, packed);
    if (units >= (1LL << 31)) return LA_ERR_INVALID_ARG;
    P.units = (int)units;
    P.walkers = walkers_of(T, nseq, channels, G, S);
    P.ends = (float *)((char *)workspace + w.ends), P.sums = (float *)((char *)workspace + w.sums);
    P.pbc = (float *)((char *)workspace + w.pbc), P.pa = (float *)((char *)workspace + w.pa);
    cudaStream_t s = (cudaStream_t)stream;
    return status_of(dtype == LA_BF16 ? backward<__nv_bfloat16>(P, S, split, dB, dC, dA, dD, ddt_bias, s)
                                      : backward<float>(P, S, split, dB, dC, dA, dD, ddt_bias, s));
}

int la_selective_scan_step(const void *x, const void *dt, const float *A, const void *B, const void *C, const float *D,
                           const void *z, const float *dt_bias, int softplus, float *state, void *y, int nseq,
                           int channels, int G, int S, int dtype, const long long *strides, void *stream) {
    using namespace la;
    using namespace la::sel;
    int rc = check_sizes(nseq, 1, channels, G, S, dtype, false);
    if (rc) return rc;
    if (nseq == 0) return LA_OK;
    if (!state) return LA_ERR_INVALID_ARG;
    long long st[14];  // as take_inputs reads them: a row's strides are those of the sequence
    if (strides) {
        for (int k = 0; k < 4; ++k) st[2 * k] = strides[k], st[2 * k + 1] = channels;
        for (int k = 0; k < 2; ++k) st[8 + 3 * k] = strides[4 + 2 * k], st[9 + 3 * k] = G * S, st[10 + 3 * k] = strides[5 + 2 * k];
    }
    Call K;
    if ((rc = take_inputs(K, x, dt, A, B, C, D, z, dt_bias, y, nullptr, nullptr, nseq, 1, channels, G, S, softplus, dtype, strides ? st : nullptr)))
        return rc;
    if ((uintptr_t)state & 15) return LA_ERR_INVALID_ARG;
    const View in[5] = {K.v[0], K.v[1], K.v[2], K.v[4], K.v[5]};
    const Range rout[1] = {{state, (size_t)nseq * channels * S * 4}};
    if (outputs_meet(in, 5, &K.v[3], 1, K.rin, 5, rout, 1)) return LA_ERR_INVALID_ARG;
    K.P.last = state;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == LA_BF16 ? step<__nv_bfloat16>(K.P, S, s) : step<float>(K.P, S, s);
    if (e == cudaSuccess) count_launches(1);
    return status_of(e);
}

}  // extern "C"
