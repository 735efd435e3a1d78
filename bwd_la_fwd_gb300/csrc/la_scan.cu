// la_scan.cu -- the gated linear recurrence over time, per channel (la_gated_scan), its gradient
// (la_gated_scan_backward) and one step of it (la_gated_scan_step).
//
//   h_t = a_t h_{t-1} + b_t x_t      log gate: a = e^w, b = 1;  sigmoid gate: a = 1 / (1 + e^-w), b = 1 - a
//   G_t = dh_t + a_{t+1} G_{t+1},    dx = b G,  dw = a h_{t-1} G  or  a b (h_{t-1} - x) G,  dh0 = a_0 G_0
//
// A run of steps is an affine map h -> A h + V with A the product of its gates, and maps of neighbouring runs
// compose, so time is cut into runs that are walked side by side.  One warp walks kSeg rows of 64 channels (two to
// a lane) with a and b x in registers; the 8 warps of a CTA and the CTAs of a cluster stand one behind another in
// time and exchange their maps through shared and distributed shared memory; then each warp walks its rows again
// from the value it now knows to enter with.  The cluster goes through the sequence in rounds and every lane keeps
// the running value of its two channels.  Every input is read once and every output written once, which is what
// bounds it (HBM); the rows of the next rounds are on their way (cp.async, each warp its own) meanwhile.
//
// Everything is held in fp32.  A gate is rounded once, to 2^-24: the same gate at every step leaves an error of up to
// 2^-24 / (1 - a) of the value.  A gate of exactly 0 cuts: what came before, infinities and NaN included, has no
// part in what follows.  A product of nonzero gates that underflows is held at the smallest denormal for that.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <string.h>

#include "la_internal.h"
#include "la_views.h"

namespace cg = cooperative_groups;

namespace la {
namespace scan {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCh = 64;          // channels of a CTA
constexpr int kMaxCluster = 16;  // CTAs one behind another in time
constexpr int kTile = 2048;      // bytes of a warp's rows of one operand

template <typename T> constexpr int kSeg = kTile / (kCh * (int)sizeof(T));  // rows of a warp: 16 (bf16), 8 (fp32)

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

// a and b of a gate.  The sigmoid's smaller half comes from e^-|w|, so that neither loses its leading digits.
template <int GATE> __device__ __forceinline__ void gate(float w, float &a, float &b) {
    if (GATE == LA_GATE_LOG) {
        a = expf(w);
        b = 1.f;
    } else {
        const float e = expf(-fabsf(w)), r = __fdividef(1.f, 1.f + e), er = e * r;
        a = w >= 0.f ? r : er;
        b = w >= 0.f ? er : r;
        if (w != w) a = b = w;
    }
}
// b x; an input that the gate shuts out (b = 0) has no part, whatever it is.
template <int GATE> __device__ __forceinline__ float gated(float b, float x) {
    return GATE == LA_GATE_LOG ? x : (b == 0.f ? 0.f : b * x);
}

// h -> a h + v, with a = 0 a cut.
__device__ __forceinline__ float apply(float a, float v, float h) { return a == 0.f ? v : fmaf(a, h, v); }
__device__ __forceinline__ float product(float a, float b) {
    const float p = a * b;
    return p == 0.f && a != 0.f && b != 0.f ? 1.4e-45f : p;
}

// The map of a run of steps on a lane's two channels.
struct Map2 {
    float a0, v0, a1, v1;
};
__device__ __forceinline__ Map2 then(const Map2 &f, const Map2 &g) {  // first f, then g
    return Map2{product(f.a0, g.a0), apply(g.a0, g.v0, f.v0), product(f.a1, g.a1), apply(g.a1, g.v1, f.v1)};
}

template <typename T, int GATE, bool BACK> struct Shape {
    static constexpr int NT = !BACK ? 2 : GATE == LA_GATE_LOG ? 3 : 4;  // operands read
    static constexpr int STAGES = BACK ? 2 : 3;
    static constexpr int SMEM = STAGES * kWarps * NT * kTile;
};

template <typename T, int GATE, bool BACK>
__global__ void __launch_bounds__(kThreads) scan_kernel(const __grid_constant__ Params P) {
    using S = Shape<T, GATE, BACK>;
    constexpr int SEG = kSeg<T>;
    constexpr int VPR = kCh * (int)sizeof(T) / 16;  // 16-byte vectors of a row
    constexpr int E = 16 / (int)sizeof(T);
    extern __shared__ __align__(128) unsigned char stages[];
    __shared__ __align__(16) Map2 of_warp[2][kWarps][32];
    __shared__ __align__(16) Map2 of_cta[2][kMaxCluster][32];
    cg::cluster_group cluster = cg::this_cluster();
    const int ncta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int block = (int)(blockIdx.x / (unsigned)ncta);
    const long long b = block / P.cblocks;
    const int c0 = (block - (int)b * P.cblocks) * kCh, c = c0 + 2 * lane;
    const bool in0 = c < P.C, in1 = c + 1 < P.C;
    // a place in time: the place of this warp's rows among the rows of a round, and the rounds, run backwards in
    // the backward pass
    const int place = rank * kWarps + warp, places = ncta * kWarps;
    const int rounds = (P.N + places * SEG - 1) / (places * SEG);
    auto first_row = [&](int r) {
        const long long run = (long long)r * places + place;
        return (BACK ? (long long)rounds * places - 1 - run : run) * SEG;
    };
    // operand of each slot of a stage; the rows of H are those before the gates'
    constexpr int op_of[4] = {kW, BACK ? kdH : kX, kH, kX};
    unsigned char *mine = stages + warp * (S::NT * kTile);
    auto tile = [&](int r, int k) {
        return (T *)(mine + (r % S::STAGES) * (kWarps * S::NT * kTile) + k * kTile);
    };
    auto fetch = [&](int r) {
        if (r < rounds) {
            const long long t0 = first_row(r);
#pragma unroll
            for (int k = 0; k < S::NT; ++k) {
                const Op &o = P.op[op_of[k]];
                const T *base = (const T *)o.p + b * o.sb + c0;
                const long long shift = op_of[k] == kH ? -1 : 0;
                const uint32_t dst = smem_addr(tile(r, k));
#pragma unroll
                for (int v = 0; v < kTile / 512; ++v) {
                    const int at = v * 32 + lane, row = at / VPR, col = (at % VPR) * E;
                    const long long t = t0 + row + shift;
                    int n = (P.C - c0 - col) * (int)sizeof(T);
                    n = n < 0 || t < 0 || t >= P.N ? 0 : n > 16 ? 16 : n;
                    copy16(dst + at * 16, n ? base + t * o.sn + col : base, n);
                }
            }
        }
        copy_commit();
    };

    float2 carry = make_float2(0.f, 0.f);  // the value that the round starts with
    if (P.first) {
        if (in0) carry.x = P.first[b * P.C + c];
        if (in1) carry.y = P.first[b * P.C + c + 1];
    }
#pragma unroll
    for (int r = 0; r < S::STAGES - 1; ++r) fetch(r);
    for (int r = 0; r < rounds; ++r) {
        __syncwarp();  // every lane is done with the stage that is refilled now
        fetch(r + S::STAGES - 1);
        copy_wait<S::STAGES - 1>();
        __syncwarp();
        const long long t0 = first_row(r);
        const int live = t0 >= P.N ? 0 : (int)(P.N - t0 < SEG ? P.N - t0 : SEG);  // rows there are
        const T *wt = tile(r, 0) + 2 * lane, *ut = tile(r, 1) + 2 * lane;
        float2 a[SEG], u[SEG];  // gates; forward b x, backward dh
        Map2 m{1.f, 0.f, 1.f, 0.f};
        bool cut0 = false, cut1 = false;
#pragma unroll
        for (int i = 0; i < SEG; ++i) {
            const int j = BACK ? SEG - 1 - i : i;
            const float2 w = load2(wt + j * kCh);
            u[j] = load2(ut + j * kCh);
            float2 g;
            gate<GATE>(w.x, a[j].x, g.x);
            gate<GATE>(w.y, a[j].y, g.y);
            if (!BACK) {
                u[j].x = gated<GATE>(g.x, u[j].x);
                u[j].y = gated<GATE>(g.y, u[j].y);
            }
            if (j >= live) {  // no row: nothing happens
                a[j] = make_float2(1.f, 1.f);
                u[j] = make_float2(0.f, 0.f);
            }
            cut0 |= a[j].x == 0.f;
            cut1 |= a[j].y == 0.f;
            m.a0 *= a[j].x;
            m.a1 *= a[j].y;
            if (!BACK) {
                m.v0 = apply(a[j].x, u[j].x, m.v0);
                m.v1 = apply(a[j].y, u[j].y, m.v1);
            } else {  // the value that leaves row j backwards is a_j G_j
                m.v0 = a[j].x == 0.f ? 0.f : a[j].x * (u[j].x + m.v0);
                m.v1 = a[j].y == 0.f ? 0.f : a[j].y * (u[j].y + m.v1);
            }
        }
        if (m.a0 == 0.f && !cut0) m.a0 = 1.4e-45f;
        if (m.a1 == 0.f && !cut1) m.a1 = 1.4e-45f;
        of_warp[r & 1][warp][lane] = m;
        __syncthreads();
        Map2 before{1.f, 0.f, 1.f, 0.f}, all{1.f, 0.f, 1.f, 0.f};
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (k == warp) before = all;
            all = then(all, of_warp[r & 1][k][lane]);
        }
        if (ncta > 1) {
            // the CTA's map to every CTA of the cluster; a buffer is written again two rounds later, behind the next
            // round's barrier, when all have read it
            for (int k = warp; k < ncta; k += kWarps) *cluster.map_shared_rank(&of_cta[r & 1][rank][lane], k) = all;
            cluster.sync();
        }
        float2 h = carry;  // what enters this CTA's rows, then this warp's
        for (int k = 0; k < ncta; ++k) {
            if (k == rank) h = carry;
            const Map2 g = ncta > 1 ? of_cta[r & 1][k][lane] : all;
            carry.x = apply(g.a0, g.v0, carry.x);
            carry.y = apply(g.a1, g.v1, carry.y);
        }
        h.x = apply(before.a0, before.v0, h.x);
        h.y = apply(before.a1, before.v1, h.y);
        if (!BACK) {
            const Op &o = P.op[kH];
            T *out = (T *)o.p + b * o.sb + t0 * o.sn + c;
#pragma unroll
            for (int j = 0; j < SEG; ++j) {
                h.x = apply(a[j].x, u[j].x, h.x);
                h.y = apply(a[j].y, u[j].y, h.y);
                if (j < live) {
                    if (in1) store2(out + j * o.sn, h.x, h.y);
                    else if (in0) store1(out + j * o.sn, h.x);
                }
            }
        } else {
            const Op &ox = P.op[kdX], &ow = P.op[kdW];
            T *dx = (T *)ox.p + b * ox.sb + t0 * ox.sn + c, *dw = (T *)ow.p + b * ow.sb + t0 * ow.sn + c;
            const T *ht = tile(r, 2) + 2 * lane;
#pragma unroll
            for (int i = 0; i < SEG; ++i) {
                const int j = SEG - 1 - i;
                float2 hp = load2(ht + j * kCh);
                if (t0 + j == 0) {
                    hp = make_float2(0.f, 0.f);
                    if (P.h0 && in0) hp.x = P.h0[b * P.C + c];
                    if (P.h0 && in1) hp.y = P.h0[b * P.C + c + 1];
                }
                const float2 G = make_float2(u[j].x + h.x, u[j].y + h.y);
                h.x = a[j].x == 0.f ? 0.f : a[j].x * G.x;
                h.y = a[j].y == 0.f ? 0.f : a[j].y * G.y;
                float2 ex = G, ew;  // gradients of x and w
                if (GATE == LA_GATE_LOG) {
                    ew.x = a[j].x == 0.f ? 0.f : hp.x * h.x;
                    ew.y = a[j].y == 0.f ? 0.f : hp.y * h.y;
                } else {
                    const float2 w = load2(wt + j * kCh), x = load2(tile(r, S::NT - 1) + 2 * lane + j * kCh);
                    float2 t, g;
                    gate<GATE>(w.x, t.x, g.x);
                    gate<GATE>(w.y, t.y, g.y);
                    ex.x = gated<GATE>(g.x, G.x);
                    ex.y = gated<GATE>(g.y, G.y);
                    ew.x = a[j].x == 0.f || g.x == 0.f ? 0.f : (hp.x - x.x) * (a[j].x * ex.x);
                    ew.y = a[j].y == 0.f || g.y == 0.f ? 0.f : (hp.y - x.y) * (a[j].y * ex.y);
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
        }
    }
    if (P.last && place == 0) {
        if (in0) P.last[b * P.C + c] = carry.x;
        if (in1) P.last[b * P.C + c + 1] = carry.y;
    }
    if (ncta > 1) cluster.sync();  // no CTA leaves while another may still write to it
}

template <typename T, int GATE, bool BACK> cudaError_t launch(const Params &P, int B, cudaStream_t s) {
    using Sh = Shape<T, GATE, BACK>;
    static std::atomic<int> attr_state[kMaxDevices];
    if (!once_per_device(attr_state, [] {
            return cudaFuncSetAttribute(scan_kernel<T, GATE, BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        Sh::SMEM) == cudaSuccess &&
                   cudaFuncSetAttribute(scan_kernel<T, GATE, BACK>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                        1) == cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    // CTAs behind one another in time: doubled while there is time for all of them and the GPU is not full.
    const long long blocks = (long long)B * P.cblocks;
    int ncta = 1;
    while (ncta < kMaxCluster && blocks * ncta < 304 && (long long)ncta * kWarps * kSeg<T> < P.N) ncta *= 2;
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scan_kernel<T, GATE, BACK>, P);
}

template <bool BACK> cudaError_t by_type(const Params &P, int B, int gate_kind, int dtype, cudaStream_t s) {
    if (dtype == LA_BF16)
        return gate_kind == LA_GATE_LOG ? launch<__nv_bfloat16, LA_GATE_LOG, BACK>(P, B, s)
                                        : launch<__nv_bfloat16, LA_GATE_SIGMOID, BACK>(P, B, s);
    return gate_kind == LA_GATE_LOG ? launch<float, LA_GATE_LOG, BACK>(P, B, s)
                                    : launch<float, LA_GATE_SIGMOID, BACK>(P, B, s);
}

// One step: the state is read and written in place, one thread to a channel pair.
template <typename T, int GATE>
__global__ void __launch_bounds__(kThreads) step_kernel(const T *x, const T *w, T *h, float *state, long long sx,
                                                        long long sw, long long sh, int C, long long n) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
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
    float a, g;
    gate<GATE>(wv.x, a, g);
    const float h0 = apply(a, gated<GATE>(g, xv.x), st[0]);
    st[0] = h0;
    if (!two) {
        store1(h + b * sh + c, h0);
        return;
    }
    gate<GATE>(wv.y, a, g);
    const float h1 = apply(a, gated<GATE>(g, xv.y), st[1]);
    st[1] = h1;
    store2(h + b * sh + c, h0, h1);
}

template <typename T> cudaError_t step(const void *x, const void *w, void *h, float *state, const long long *st, int B, int C, int gate_kind, cudaStream_t s) {
    const long long n = (long long)B * ((C + 1) / 2), blocks = (n + kThreads - 1) / kThreads;
    if (blocks >= (1LL << 31)) return cudaErrorInvalidConfiguration;
    auto *k = gate_kind == LA_GATE_LOG ? step_kernel<T, LA_GATE_LOG> : step_kernel<T, LA_GATE_SIGMOID>;
    k<<<(unsigned)blocks, kThreads, 0, s>>>((const T *)x, (const T *)w, (T *)h, state, st[0], st[1], st[2], C, n);
    return cudaGetLastError();
}

// Sizes and kinds shared by the entry points; LA_OK with *empty set when there is nothing to do.
int check_kind(int B, int N, int C, int gate_kind, int dtype, bool *empty) {
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (gate_kind != LA_GATE_LOG && gate_kind != LA_GATE_SIGMOID) return LA_ERR_INVALID_ARG;
    if (B < 0 || N < 0 || C < 0) return LA_ERR_INVALID_ARG;
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
    P.cblocks = (C + kCh - 1) / kCh;
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
    P.cblocks = (C + kCh - 1) / kCh;
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
        // a dense [B, C] needs no row of whole vectors: two channels of a row are loaded at a time where C is even
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
