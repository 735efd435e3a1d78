// la_scan.cu -- the gated linear recurrence over time, per channel (la_gated_scan), its gradient
// (la_gated_scan_backward) and one step of it (la_gated_scan_step).
//
//   h_t = a_t h_{t-1} + b_t x_t      log gate: a = e^w, b = 1;  sigmoid gate: a = 1 / (1 + e^-w), b = 1 - a
//   G_t = dh_t + a_{t+1} G_{t+1},    dx = b G,  dw = a h_{t-1} G  or  a b (h_{t-1} - x) G,  dh0 = a_0 G_0
//
// A run of steps is an affine map h -> A h + V with A the product of its gates, and maps of neighbouring runs compose.
// A CTA walks a block of 64, 32 or 16 channels (two to a lane) through time in rounds.  In a round each warp has 1, 2 or 4
// runs, one behind another, and forms their maps with a and b x in registers; the warps' maps are applied one after another
// to the value that every lane keeps, and each warp then walks its rows again from the value it enters with.  Every input
// is read once and every output written once, which bounds it (HBM); the next round's rows are on their way (cp.async,
// each warp its own) meanwhile.  Two CTAs of 8 warps on an SM, because a round's phases wait for one another: one CTA of
// 16 warps gave 4.0 TB/s where these give 5.4 (64 x 1024 x 2048, bf16).
// Where batch and channels give too few CTAs even in blocks of 16 channels, time is cut into up to 16 parts, the CTAs of a
// cluster: each first forms its part's map (its warps side by side, without rounds), they exchange these once through
// distributed shared memory, and each walks its part as above, reading it again.  (Exchanging in every round instead, so
// that nothing is read twice, took three times as long: a cluster's barrier costs microseconds.)
//
// Everything is held in fp32.  A gate is within 5 (log) or 9 (sigmoid) half steps of 2^-24: the same gate at every step
// leaves an error of up to that many 2^-24 / (1 - a) of the value.  A gate of exactly 0 cuts: what came before, infinities
// and NaN included, has no part in what follows.  A product of nonzero gates that underflows is held at the smallest
// denormal for that.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "la_f32x2.cuh"
#include "la_internal.h"
#include "la_views.h"

namespace cg = cooperative_groups;

namespace la {
namespace scan {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxRows = 0x7fffffff - 1024;  // the end of a round, of at most 512 rows, is an int
constexpr int kMaxCluster = 16;  // parts that time is cut into
constexpr int kEnough = 228, kFew = 76;  // CTAs: three for two SMs, one for two SMs

struct Op {
    const void *p;
    long long sb, sn;  // batch, row stride in elements
};

enum : int { kX = 0, kW, kH, kdH, kdX, kdW, kOps };

struct Params {
    Op op[kOps];
    const float *first;  // [B, C], the value before the first row (forward h0, backward dh_last); null: 0
    float *last;         // [B, C], the value after the last one (forward h_last, backward dh0); null: not written
    const float *h0;     // backward: what stands before row 0 of H; null: 0
    int N, C, cblocks;   // channel blocks
    int rounds;          // of a part
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes global -> shared; bytes past `n` are zero.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two neighbouring channels of a row.
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p) { return __bfloat1622float2(*(const __nv_bfloat162 *)p); }
__device__ __forceinline__ float2 load2(const float *p) { return *(const float2 *)p; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y) { *(__nv_bfloat162 *)p = __floats2bfloat162_rn(x, y); }
__device__ __forceinline__ void store2(float *p, float x, float y) { *(float2 *)p = make_float2(x, y); }

// The larger of the two; NaN stays NaN.
__device__ __forceinline__ float at_least(float x, float least) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(least));
    return y;
}
// e^w: 2^(w log2 e) by the hardware's 2^x, within 2 ulp, and the product's rounding error put back: 5 half steps in all.
// Below 2^-126: 0; w is held where that error is a number (near the type's lowest value the product is infinite).  Where the
// power is infinite, infinite or NaN: grown() tells.
__device__ __forceinline__ float2 exp_of(float2 w) {
    w = make_float2(at_least(w.x, -200.f), at_least(w.y, -200.f));
    const float2 y = mul2(w, both(1.44269502f));
    float2 t = fma2(w, both(1.92596299e-8f), fma2(w, both(1.44269502f), make_float2(-y.x, -y.y)));
    t = mul2(t, both(0.693147182f));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
    return fma2(e, t, e);
}
// e^w where it may be infinite: at 88.7228394, whose product with log2 e rounds to 128, and above.
__device__ __forceinline__ float2 grown(float2 a, float2 w) {
    return make_float2(w.x >= 88.7228394f ? INFINITY : a.x, w.y >= 88.7228394f ? INFINITY : a.y);
}

// a and b of two gates.  The sigmoid's smaller half comes from e^-|w|, so that neither loses its leading digits.
template <int GATE> __device__ __forceinline__ void gate(float2 w, float2 &a, float2 &b) {
    if (GATE == LA_GATE_LOG) {
        a = exp_of(w);
        b = both(1.f);
    } else {
        const float2 e = exp_of(make_float2(-fabsf(w.x), -fabsf(w.y))), d = add2(e, both(1.f));
        float2 r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));  // of 1 ... 2, within 1 ulp
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
        const float2 s = mul2(e, r);
        a = make_float2(w.x >= 0.f ? r.x : s.x, w.y >= 0.f ? r.y : s.y);
        b = make_float2(w.x >= 0.f ? s.x : r.x, w.y >= 0.f ? s.y : r.y);
    }
}
// b x; an input that the gate shuts out (b = 0) has no part, whatever it is.
template <int GATE> __device__ __forceinline__ float gated(float b, float x) {
    return GATE == LA_GATE_LOG ? x : (b == 0.f ? 0.f : b * x);
}

// h -> a h + v, with a = 0 a cut.
__device__ __forceinline__ float apply(float a, float v, float h) { return a == 0.f ? v : fmaf(a, h, v); }
__device__ __forceinline__ float cut(float a, float h) { return a == 0.f ? 0.f : __fmul_rn(a, h); }
// The same with a product of gates, which may be beyond fp32: 0 stays 0.
__device__ __forceinline__ float enter(float a, float v, float h) { return a == 0.f || (h == 0.f && a > 0.f) ? v : fmaf(a, h, v); }
// A cut among the gates makes the product one, whatever the others are.
__device__ __forceinline__ float product(float a, float b) {
    const float p = a * b;
    return a == 0.f || b == 0.f ? 0.f : p == 0.f ? 1.4e-45f : p;
}

// The map of a run of steps on a lane's two channels.
struct Map2 {
    float a0, v0, a1, v1;
};
// Whether a map formed by plain products and sums is right as it is: nothing was cut, nothing overflowed or vanished.
__device__ __forceinline__ bool plain(const Map2 &m) {
    return m.a0 > 0.f && m.a0 < INFINITY && m.a1 > 0.f && m.a1 < INFINITY && fabsf(m.v0) < INFINITY && fabsf(m.v1) < INFINITY;
}
__device__ __forceinline__ Map2 then(const Map2 &f, const Map2 &g) {  // first f, then g
    return Map2{product(f.a0, g.a0), enter(g.a0, g.v0, f.v0), product(f.a1, g.a1), enter(g.a1, g.v1, f.v1)};
}

// CH: channels of a CTA.
template <typename T, int GATE, bool BACK, int CH> struct Shape {
    static constexpr bool PARTS = CH == 16;                             // time may be cut into parts
    static constexpr int NT = !BACK ? 2 : GATE == LA_GATE_LOG ? 3 : 4;  // operands read
    static constexpr int LANES = CH / 2, RUNS = 32 / LANES;             // lanes of a run, runs of a warp
    static constexpr int SEG = (NT == 4 ? 16 : 32) / (int)sizeof(T);    // rows of a run: 16 or 8 (bf16), 8 or 4 (fp32)
    // A run's rows in shared memory; with several runs to a warp a row between them keeps them on banks of their own.
    static constexpr int PITCH = (SEG + (RUNS > 1)) * CH;               // elements
    static constexpr int TILE = RUNS * PITCH * (int)sizeof(T);
    static constexpr int STAGES = 2;
    static constexpr int SMEM = STAGES * kWarps * NT * TILE;
};

template <typename T, int GATE, bool BACK, int CH>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(const __grid_constant__ Params P) {
    using S = Shape<T, GATE, BACK, CH>;
    constexpr int SEG = S::SEG, LANES = S::LANES, RUNS = S::RUNS;
    constexpr int VPR = CH * (int)sizeof(T) / 16;  // 16-byte vectors of a row
    constexpr int E = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ __align__(16) Map2 of_warp[2][kWarps][LANES];
    __shared__ __align__(16) Map2 of_cta[S::PARTS ? kMaxCluster : 1][LANES];
    int ncta = 1, rank = 0;
    if constexpr (S::PARTS) {
        ncta = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
        // A CTA's shared memory may be written by others once it has begun: said here, waited for before the first such write.
        if (ncta > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    }
    // Forward, rank is not to be known to be 0: row addresses are then formed where they are used (8 x 2048 x 2048, sigmoid,
    // bf16: 47.6 us where 49.5; the gradient is slower so, 79.5 where 77).
    if (!BACK) asm volatile("" : "+r"(rank));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int block = (int)(blockIdx.x / (unsigned)ncta);
    const long long b = block / P.cblocks;
    const int run = lane / LANES, pair = lane % LANES;  // of the warp's runs, of the block's channel pairs
    const int c0 = (block - (int)b * P.cblocks) * CH, c = c0 + 2 * pair;
    const bool in0 = c < P.C, in1 = c + 1 < P.C;
    // Ranks, rounds, warps and runs count in the direction of the walk: from the last row in the backward pass.  A warp's
    // runs are one block of rows; `place` is this lane's run's in it.
    const int R = P.rounds, place = BACK ? RUNS - 1 - run : run;
    const long long part = (long long)(BACK ? ncta - 1 - rank : rank) * R * kWarps;  // first block of the part
    auto row_of = [&](int k) { return (part + (BACK ? R * kWarps - 1 - k : k)) * (RUNS * SEG); };
    // operand of each slot of a stage; the rows of H are those before the gates'
    constexpr int op_of[4] = {kW, BACK ? kdH : kX, kH, kX};
    auto tile = [&](int at, int k) {
        return (T *)(stages + (((at % S::STAGES) * kWarps + warp) * S::NT + k) * S::TILE);
    };
    // the rows from t0 on, into stage `at`: the first nt operands
    auto fetch = [&](int at, long long t0, int nt) {
#pragma unroll
        for (int k = 0; k < S::NT; ++k) {
            if (k >= nt) break;
            const Op &o = P.op[op_of[k]];
            const T *base = (const T *)o.p + b * o.sb + c0;
            const long long shift = op_of[k] == kH ? -1 : 0;
            const uint32_t dst = smem_addr(tile(at, k));
#pragma unroll
            for (int v = 0; v < RUNS * SEG * VPR / 32; ++v) {
                const int x = v * 32 + lane, row = x / VPR, col = (x % VPR) * E;
                const long long t = t0 + row + shift;
                int n = (P.C - c0 - col) * (int)sizeof(T);
                n = n < 0 || t < 0 || t >= P.N ? 0 : n > 16 ? 16 : n;
                copy16(dst + (row / SEG * S::PITCH + row % SEG * CH + col) * (int)sizeof(T), n ? base + t * o.sn + col : base, n);
            }
        }
        copy_commit();
    };
    // gates, and b x (forward) or dh, of the rows in stage `at`; their map
    auto map_of = [&](int at, int live, float2 (&a)[SEG], float2 (&u)[SEG]) {
        const int mine = place * S::PITCH + 2 * pair;
        const T *wt = tile(at, 0) + mine, *ut = tile(at, 1) + mine;
#pragma unroll
        for (int j = 0; j < SEG; ++j) {
            const float2 w = load2(wt + j * CH);
            u[j] = load2(ut + j * CH);
            float2 g;
            gate<GATE>(w, a[j], g);
            if (!BACK && GATE == LA_GATE_SIGMOID) u[j] = mul2(u[j], g);
        }
        if (live < SEG) {
#pragma unroll
            for (int j = 0; j < SEG; ++j)
                if (j >= live) {  // no row: nothing happens
                    a[j] = make_float2(1.f, 1.f);
                    u[j] = make_float2(0.f, 0.f);
                }
        }
        // By plain products and sums.  Where these come to something finite and a product that is not 0 no gate has cut
        // anything off that matters; else (the warp together) once more, with cuts.
        float2 A = both(1.f), V = both(0.f);
#pragma unroll
        for (int i = 0; i < SEG; ++i) {
            const int j = BACK ? SEG - 1 - i : i;
            A = mul2(A, a[j]);
            V = BACK ? mul2(a[j], add2(u[j], V)) : fma2(a[j], V, u[j]);  // backwards a_j G_j leaves row j
        }
        Map2 m{A.x, V.x, A.y, V.y};
        if (__any_sync(0xffffffffu, !plain(m))) {
            if (GATE == LA_GATE_LOG) {
#pragma unroll
                for (int j = 0; j < SEG; ++j) a[j] = grown(a[j], load2(wt + j * CH));
            } else if (!BACK) {  // an input that the gate shuts out has no part
#pragma unroll
                for (int j = 0; j < SEG; ++j) {
                    float2 t, g;
                    gate<GATE>(load2(wt + j * CH), t, g);
                    if (g.x == 0.f) u[j].x = 0.f;
                    if (g.y == 0.f) u[j].y = 0.f;
                }
            }
            m = Map2{1.f, 0.f, 1.f, 0.f};
#pragma unroll
            for (int i = 0; i < SEG; ++i) {
                const int j = BACK ? SEG - 1 - i : i;
                m.a0 = product(m.a0, a[j].x);
                m.a1 = product(m.a1, a[j].y);
                m.v0 = BACK ? cut(a[j].x, u[j].x + m.v0) : apply(a[j].x, u[j].x, m.v0);
                m.v1 = BACK ? cut(a[j].y, u[j].y + m.v1) : apply(a[j].y, u[j].y, m.v1);
            }
        }
        return m;
    };
    // rows there are of this lane's run in the block from t0 on
    auto live_of = [&](long long t0) {
        const long long n = P.N - t0 - place * SEG;
        return n < 0 ? 0 : n < SEG ? (int)n : SEG;
    };
    auto shuffled = [&](const Map2 &m, int from) {
        return Map2{__shfl_sync(0xffffffffu, m.a0, from), __shfl_sync(0xffffffffu, m.v0, from),
                    __shfl_sync(0xffffffffu, m.a1, from), __shfl_sync(0xffffffffu, m.v1, from)};
    };
    // the maps of the warp's runs up to and with this lane's
    auto upto = [&](const Map2 &mine) {
        Map2 m = mine;
#pragma unroll
        for (int d = 1; d < RUNS; d *= 2) {
            const Map2 before = shuffled(m, (run - d) * LANES + pair);
            if (run >= d) m = then(before, m);
        }
        return m;
    };
    const int last_lane = (RUNS - 1) * LANES + pair;

    float2 carry = make_float2(0.f, 0.f);  // the value that the part starts with
    if (P.first) {
        if (in0) carry.x = P.first[b * P.C + c];
        if (in1) carry.y = P.first[b * P.C + c + 1];
    }
    if (S::PARTS && ncta > 1) {
        const cg::cluster_group cluster = cg::this_cluster();
        // the part's map: each warp R runs, one behind another, then the warps' in order
        Map2 m{1.f, 0.f, 1.f, 0.f};
#pragma unroll
        for (int r = 0; r < S::STAGES - 1; ++r)
            if (r < R) fetch(r, row_of(warp * R + r), 2);
            else copy_commit();
        for (int r = 0; r < R; ++r) {
            const int ahead = r + S::STAGES - 1;
            __syncwarp();  // every lane is done with the stage that is refilled now
            if (ahead < R) fetch(ahead, row_of(warp * R + ahead), 2);
            else copy_commit();
            copy_wait<S::STAGES - 1>();
            __syncwarp();
            float2 a[SEG], u[SEG];
            m = then(m, shuffled(upto(map_of(r, live_of(row_of(warp * R + r)), a, u)), last_lane));
        }
        copy_wait<0>();
        if (run == 0) of_warp[0][warp][pair] = m;
        __syncthreads();
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // every CTA of the cluster has begun
        if (warp == 0 && run == 0) {
            Map2 all{1.f, 0.f, 1.f, 0.f};
            for (int k = 0; k < kWarps; ++k) all = then(all, of_warp[0][k][pair]);
            for (int k = 0; k < ncta; ++k) *cluster.map_shared_rank(&of_cta[rank][pair], k) = all;
        }
        cluster.sync();  // the maps are there, and no CTA writes to another from here on
        for (int k = 0; k < rank; ++k) {
            const Map2 g = of_cta[k][pair];
            carry.x = enter(g.a0, g.v0, carry.x);
            carry.y = enter(g.a1, g.v1, carry.y);
        }
    }
#pragma unroll
    for (int r = 0; r < S::STAGES - 1; ++r)
        if (r < R) fetch(r, row_of(r * kWarps + warp), S::NT);
        else copy_commit();
    for (int r = 0; r < R; ++r) {
        const int ahead = r + S::STAGES - 1;
        __syncwarp();
        if (ahead < R) fetch(ahead, row_of(ahead * kWarps + warp), S::NT);
        else copy_commit();
        copy_wait<S::STAGES - 1>();
        __syncwarp();
        const long long b0 = row_of(r * kWarps + warp), t0 = b0 + place * SEG;
        const int live = live_of(b0);
        float2 a[SEG], u[SEG];
        const Map2 sofar = upto(map_of(r, live, a, u));
        if (run == RUNS - 1) of_warp[r & 1][warp][pair] = sofar;
        __syncthreads();  // (the maps of two rounds before have been read: all have passed the last round's)
        float2 h = carry, end = carry;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (k == warp) h = end;
            const Map2 g = of_warp[r & 1][k][pair];
            end = fma2(make_float2(g.a0, g.a1), end, make_float2(g.v0, g.v1));
        }
        if (__any_sync(0xffffffffu, !(fabsf(end.x) < INFINITY && fabsf(end.y) < INFINITY))) {  // once more, with cuts
            end = carry;
            for (int k = 0; k < kWarps; ++k) {
                if (k == warp) h = end;
                const Map2 g = of_warp[r & 1][k][pair];
                end = make_float2(enter(g.a0, g.v0, end.x), enter(g.a1, g.v1, end.y));
            }
        }
        carry = end;
        if (RUNS > 1) {  // through the warp's runs before this lane's
            const Map2 before = shuffled(sofar, (run - 1) * LANES + pair);
            if (run > 0) h = make_float2(enter(before.a0, before.v0, h.x), enter(before.a1, before.v1, h.y));
        }
        const bool whole = b0 + RUNS * SEG <= P.N && c0 + CH <= P.C;  // the same for the warp: no row or channel is missing
        // The rows from the value that they are entered with: plainly, and again with cuts where that ends in something
        // that is not finite (which no plain step leaves again).
        if (!BACK) {
            const Op &o = P.op[kH];
            T *out = (T *)o.p + b * o.sb + t0 * o.sn + c;
            auto row = [&](int j, float2 h) {
                if (in1) store2(out + j * o.sn, h.x, h.y);
                else if (in0) store1(out + j * o.sn, h.x);
            };
            float2 v = h;
            if (whole) {
#pragma unroll
                for (int j = 0; j < SEG; ++j) {
                    v = fma2(a[j], v, u[j]);
                    store2(out + j * o.sn, v.x, v.y);
                }
            } else {
#pragma unroll
                for (int j = 0; j < SEG; ++j) {
                    v = fma2(a[j], v, u[j]);
                    if (j < live) row(j, v);
                }
            }
            if (__any_sync(0xffffffffu, !(fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY))) {
#pragma unroll
                for (int j = 0; j < SEG; ++j) {
                    h = make_float2(apply(a[j].x, u[j].x, h.x), apply(a[j].y, u[j].y, h.y));
                    if (j < live) row(j, h);
                }
            }
        } else {
            const Op &ox = P.op[kdX], &ow = P.op[kdW];
            T *dx = (T *)ox.p + b * ox.sb + t0 * ox.sn + c, *dw = (T *)ow.p + b * ow.sb + t0 * ow.sn + c;
            const int mine = place * S::PITCH + 2 * pair;
            const T *wt = tile(r, 0) + mine, *ht = tile(r, 2) + mine, *xt = tile(r, S::NT - 1) + mine;
            auto walk = [&](float2 h, auto with_cuts) {
                constexpr bool CUTS = decltype(with_cuts)::value;
                float2 seen = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < SEG; ++i) {
                    const int j = SEG - 1 - i;
                    float2 hp = load2(ht + j * CH);
                    if (j == 0 && t0 == 0) {
                        hp = make_float2(0.f, 0.f);
                        if (P.h0 && in0) hp.x = P.h0[b * P.C + c];
                        if (P.h0 && in1) hp.y = P.h0[b * P.C + c + 1];
                    }
                    const float2 G = add2(u[j], h);
                    h = CUTS ? make_float2(cut(a[j].x, G.x), cut(a[j].y, G.y)) : mul2(a[j], G);
                    float2 ex = G, ew;  // gradients of x and w
                    if (GATE == LA_GATE_LOG) {
                        ew = mul2(hp, h);
                        if (CUTS && a[j].x == 0.f) ew.x = 0.f;
                        if (CUTS && a[j].y == 0.f) ew.y = 0.f;
                    } else {
                        float2 t, g;
                        gate<GATE>(load2(wt + j * CH), t, g);
                        ex = CUTS ? make_float2(gated<GATE>(g.x, G.x), gated<GATE>(g.y, G.y)) : mul2(g, G);
                        const float2 x = load2(xt + j * CH);
                        ew = mul2(add2(hp, make_float2(-x.x, -x.y)), mul2(a[j], ex));
                        if (CUTS && (t.x == 0.f || g.x == 0.f)) ew.x = 0.f;
                        if (CUTS && (t.y == 0.f || g.y == 0.f)) ew.y = 0.f;
                    }
                    seen = fma2(ew, both(0.f), seen);  // no number once something was not finite
                    if (whole) {
                        store2(dx + j * ox.sn, ex.x, ex.y);
                        store2(dw + j * ow.sn, ew.x, ew.y);
                        continue;
                    }
                    if (j < live) {
                        if (in1) {
                            store2(dx + j * ox.sn, ex.x, ex.y);
                            store2(dw + j * ow.sn, ew.x, ew.y);
                        } else if (in0) {
                            store1(dx + j * ox.sn, ex.x);
                            store1(dw + j * ow.sn, ew.x);
                        }
                    }
                }
                return seen.x == 0.f && seen.y == 0.f && fabsf(h.x) < INFINITY && fabsf(h.y) < INFINITY;
            };
            if (__any_sync(0xffffffffu, !walk(h, std::false_type{}))) walk(h, std::true_type{});
        }
    }
    if (P.last && rank == ncta - 1 && warp == 0 && run == 0) {
        if (in0) P.last[b * P.C + c] = carry.x;
        if (in1) P.last[b * P.C + c + 1] = carry.y;
    }
}

template <typename T, int GATE, bool BACK, int CH> cudaError_t launch(Params P, int B, cudaStream_t s) {
    using Sh = Shape<T, GATE, BACK, CH>;
    static std::atomic<int> attr_state[kMaxDevices];
    if (!once_per_device(attr_state, [] {
            return cudaFuncSetAttribute(scan_kernel<T, GATE, BACK, CH>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        Sh::SMEM) == cudaSuccess &&
                   cudaFuncSetAttribute(scan_kernel<T, GATE, BACK, CH>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                        1) == cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    // Parts of time, which are read twice: none where the channel blocks make a CTA for every other SM, else doubled until
    // there are three for two SMs, as long as each has two rounds.  (For 1, 2, 4, 8, 16 parts: 1 x 65536 x 512, fp32, 32
    // blocks: 339, 270, 151, 129, 157 us; 1 x 8192 x 1024, bf16, backward, 64 blocks: 76, 60, 52, 57, 81; 2 x 30000 x 640,
    // fp32, 80 blocks: 188, 223, 195, 169, 199; 1 x 8192 x 2048, bf16, 128 blocks: 50, 66, 71, 72, 109.)  Wider blocks, which
    // are taken only where they make CTAs enough, are never cut.
    P.cblocks = (P.C + CH - 1) / CH;
    const long long blocks = (long long)B * P.cblocks;
    const int round = kWarps * Sh::RUNS * Sh::SEG, all = (P.N + round - 1) / round;
    int ncta = 1;
    if (Sh::PARTS && blocks < kFew)
        while (ncta < kMaxCluster && blocks * ncta < kEnough && 4 * ncta <= all) ncta *= 2;
    P.rounds = (all + ncta - 1) / ncta;
    if (blocks * ncta >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * ncta));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ncta;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = Sh::PARTS ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, scan_kernel<T, GATE, BACK, CH>, P);
}

// Channels of a CTA: the widest blocks that make three CTAs for two SMs.  Wide rows cost fewer instructions (64 x 1024 x
// 2048, bf16: 148, 161, 195 us for 64, 32, 16 channels), few CTAs leave SMs idle (1 x 65536 x 512, fp32, best parts: 184,
// 174, 129 us).
template <typename T, int GATE, bool BACK> cudaError_t by_width(const Params &P, int B, cudaStream_t s) {
    auto blocks = [&](int ch) { return (long long)B * ((P.C + ch - 1) / ch); };
    if (blocks(64) >= kEnough) return launch<T, GATE, BACK, 64>(P, B, s);
    if (blocks(32) >= kEnough) return launch<T, GATE, BACK, 32>(P, B, s);
    return launch<T, GATE, BACK, 16>(P, B, s);
}

template <bool BACK> cudaError_t by_type(const Params &P, int B, int gate_kind, int dtype, cudaStream_t s) {
    if (dtype == LA_BF16)
        return gate_kind == LA_GATE_LOG ? by_width<__nv_bfloat16, LA_GATE_LOG, BACK>(P, B, s)
                                        : by_width<__nv_bfloat16, LA_GATE_SIGMOID, BACK>(P, B, s);
    return gate_kind == LA_GATE_LOG ? by_width<float, LA_GATE_LOG, BACK>(P, B, s)
                                    : by_width<float, LA_GATE_SIGMOID, BACK>(P, B, s);
}

constexpr int kStepThreads = 256;

// One step: the state is read and written in place, one thread to a channel pair.
template <typename T, int GATE>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const T *x, const T *w, T *h, float *state, long long sx,
                                                        long long sw, long long sh, int C, long long n) {
    const long long i = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    if (i >= n) return;
    const int pairs = (C + 1) / 2;
    const long long b = i / pairs;
    const int c = 2 * (int)(i - b * pairs);
    float *st = state + b * C + c;
    const bool two = c + 1 < C;
    float2 xv, wv;  // a row's last odd channel alone: nothing is read past it
    if (two) {
        xv = load2(x + b * sx + c);
        wv = load2(w + b * sw + c);
    } else {
        xv = make_float2((float)x[b * sx + c], 0.f);
        wv = make_float2((float)w[b * sw + c], 0.f);
    }
    float2 a, g;
    gate<GATE>(wv, a, g);
    if (GATE == LA_GATE_LOG) a = grown(a, wv);
    const float h0 = apply(a.x, gated<GATE>(g.x, xv.x), st[0]);
    st[0] = h0;
    if (!two) {
        store1(h + b * sh + c, h0);
        return;
    }
    const float h1 = apply(a.y, gated<GATE>(g.y, xv.y), st[1]);
    st[1] = h1;
    store2(h + b * sh + c, h0, h1);
}

template <typename T> cudaError_t step(const void *x, const void *w, void *h, float *state, const long long *st, int B, int C, int gate_kind, cudaStream_t s) {
    const long long n = (long long)B * ((C + 1) / 2), blocks = (n + kStepThreads - 1) / kStepThreads;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    auto *k = gate_kind == LA_GATE_LOG ? step_kernel<T, LA_GATE_LOG> : step_kernel<T, LA_GATE_SIGMOID>;
    k<<<(unsigned)blocks, kStepThreads, 0, s>>>((const T *)x, (const T *)w, (T *)h, state, st[0], st[1], st[2], C, n);
    return cudaGetLastError();
}

// Sizes and kinds shared by the entry points; LA_OK with *empty set when there is nothing to do.
int check_kind(int B, int N, int C, int gate_kind, int dtype, bool *empty) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (gate_kind != LA_GATE_LOG && gate_kind != LA_GATE_SIGMOID) return LA_ERR_INVALID_ARG;
    if (B < 0 || N < 0 || N > kMaxRows || C < 0) return LA_ERR_INVALID_ARG;
    if ((long long)B * C >= (1LL << 40) / (N > 0 ? N : 1)) return LA_ERR_INVALID_ARG;
    *empty = B == 0 || C == 0;
    return LA_OK;
}

int check_op(View &v, const void *p, int B, int N, int C, int elem, const long long *strides) {
    if (!p || ((uintptr_t)p & 15)) return LA_ERR_INVALID_ARG;
    v = View{p, {B, N, 1}, {}, C, elem};
    const long long dense[3] = {(long long)N * C, C, C};
    const long long given[3] = {strides ? strides[0] : 0, strides ? strides[1] : 0, C};
    return set_view(v, strides ? given : dense, dense);
}

// No output meets an input or another output.
bool outputs_apart(const View *in, int n_in, const View *out, int n_out, const void *const *fin, int n_fin,
                   void *const *fout, int n_fout, size_t fbytes) {
    for (int o = 0; o < n_out; ++o) {
        for (int k = 0; k < n_in; ++k)
            if (views_meet(out[o], in[k])) return false;
        for (int k = o + 1; k < n_out; ++k)
            if (views_meet(out[o], out[k])) return false;
        for (int k = 0; k < n_fin; ++k)
            if (fin[k] && ranges_meet(out[o].p, view_bytes(out[o]), fin[k], fbytes)) return false;
    }
    for (int o = 0; o < n_fout; ++o) {
        if (!fout[o]) continue;
        for (int k = 0; k < n_in; ++k)
            if (ranges_meet(fout[o], fbytes, in[k].p, view_bytes(in[k]))) return false;
        for (int k = 0; k < n_out; ++k)
            if (ranges_meet(fout[o], fbytes, out[k].p, view_bytes(out[k]))) return false;
        for (int k = 0; k < n_fin; ++k)
            if (fin[k] && ranges_meet(fout[o], fbytes, fin[k], fbytes)) return false;
    }
    return true;
}

int status_of(cudaError_t e) {
    if (e == cudaErrorInvalidConfiguration) return LA_ERR_INVALID_ARG;
    if (e != cudaSuccess) return LA_ERR_CUDA;
    count_launches(1);
    return LA_OK;
}

}  // namespace scan
}  // namespace la

extern "C" {

int la_gated_scan(const void *X, const void *W, const float *h0, void *H, float *h_last, int B, int N, int C, int gate,
                  int dtype, const long long *strides, void *stream) {
    using namespace la;
    using namespace la::scan;
    bool empty;
    int rc = check_kind(B, N, C, gate, dtype, &empty);
    if (rc || empty) return rc;
    const int elem = dtype == LA_BF16 ? 2 : 4;
    const void *ptr[3] = {X, W, H};
    const int ops[3] = {kX, kW, kH};
    View v[3] = {};
    Params P = {};
    for (int k = 0; k < 3 && N > 0; ++k) {  // (X, W, H) x (batch, row)
        if ((rc = check_op(v[k], ptr[k], B, N, C, elem, strides ? strides + 2 * k : nullptr))) return rc;
        P.op[ops[k]] = Op{ptr[k], v[k].st[0], v[k].st[1]};
    }
    if (((uintptr_t)h0 & 3) || ((uintptr_t)h_last & 3)) return LA_ERR_INVALID_ARG;
    const void *fin[1] = {h0};
    void *fout[1] = {h_last};
    const int nv = N > 0 ? 1 : 0;
    if (!outputs_apart(v, 2 * nv, v + 2, nv, fin, 1, fout, 1, (size_t)B * C * 4)) return LA_ERR_INVALID_ARG;
    if (N == 0 && !h_last) return LA_OK;
    P.first = h0;
    P.last = h_last;
    P.N = N;
    P.C = C;
    return status_of(by_type<false>(P, B, gate, dtype, (cudaStream_t)stream));
}

int la_gated_scan_backward(const void *X, const void *W, const void *H, const void *dH, const float *h0,
                           const float *dh_last, void *dX, void *dW, float *dh0, int B, int N, int C, int gate,
                           int dtype, const long long *strides, void *stream) {
    using namespace la;
    using namespace la::scan;
    bool empty;
    int rc = check_kind(B, N, C, gate, dtype, &empty);
    if (rc || empty) return rc;
    const int elem = dtype == LA_BF16 ? 2 : 4;
    const void *ptr[kOps] = {X, W, H, dH, dX, dW};
    View v[kOps] = {};
    Params P = {};
    for (int k = 0; k < kOps && N > 0; ++k) {  // (X, W, H, dH, dX, dW) x (batch, row)
        if ((rc = check_op(v[k], ptr[k], B, N, C, elem, strides ? strides + 2 * k : nullptr))) return rc;
        P.op[k] = Op{ptr[k], v[k].st[0], v[k].st[1]};
    }
    if (((uintptr_t)h0 & 3) || ((uintptr_t)dh_last & 3) || ((uintptr_t)dh0 & 3)) return LA_ERR_INVALID_ARG;
    const void *fin[2] = {h0, dh_last};
    void *fout[1] = {dh0};
    const int nv = N > 0 ? 1 : 0;
    if (!outputs_apart(v, 4 * nv, v + 4, 2 * nv, fin, 2, fout, 1, (size_t)B * C * 4)) return LA_ERR_INVALID_ARG;
    if (N == 0 && !dh0) return LA_OK;
    P.first = dh_last;
    P.last = dh0;
    P.h0 = h0;
    P.N = N;
    P.C = C;
    return status_of(by_type<true>(P, B, gate, dtype, (cudaStream_t)stream));
}

int la_gated_scan_step(const void *x, const void *w, void *h, float *state, int B, int C, int gate, int dtype,
                       const long long *strides, void *stream) {
    using namespace la;
    using namespace la::scan;
    bool empty;
    int rc = check_kind(B, 1, C, gate, dtype, &empty);
    if (rc || empty) return rc;
    const int elem = dtype == LA_BF16 ? 2 : 4;
    const void *ptr[3] = {x, w, h};
    View v[3];
    long long st[3];
    for (int k = 0; k < 3; ++k) {  // (x, w, h): the row stride of [B, C]
        const long long row[2] = {strides ? strides[k] : C, C};
        // (several rows have to be whole 16-byte vectors apart, as everywhere; C itself may be odd)
        if ((rc = check_op(v[k], ptr[k], B, 1, C, elem, row))) return rc;
        st[k] = v[k].st[0];
    }
    if (!state || ((uintptr_t)state & 15)) return LA_ERR_INVALID_ARG;
    const void *fin[1] = {nullptr};
    void *fout[1] = {state};
    if (!outputs_apart(v, 2, v + 2, 1, fin, 0, fout, 1, (size_t)B * C * 4)) return LA_ERR_INVALID_ARG;
    return status_of(dtype == LA_BF16 ? step<__nv_bfloat16>(x, w, h, state, st, B, C, gate, (cudaStream_t)stream)
                                      : step<float>(x, w, h, state, st, B, C, gate, (cudaStream_t)stream));
}

}  // extern "C"
