// la_prompt_tc.cu -- tcgen05 / TMA form of la_prompt (bf16, D = 32, 64, 128).
//
// Per key/value head and chunk of 128 rows, with S, z, a, n those of the rows before the chunk, for each query head:
//   T = Q K^T,  P = [j <= i](1 + T) in bf16,  O = (Q Sb + P V + a) / (n + q . z + row sums of P)
// and once per chunk  S += K^T V,  z += K^T 1,  a += V^T 1.  Sb is S rounded to bf16; z goes through the tensor cores
// as two bf16 parts (16 bits).  S itself lives in fp32 registers of the epilogue: a chunk's K^T V is summed by itself in
// TMEM and added there, so that a long sequence's sums are rounded to nearest once a chunk.
//
// Work split.  All (sequence, head, chunk) items are laid end to end in that order and cut into G equal slices, one per
// CTA; the part of a slice in one head is a piece.  A piece that stops short of its head's end is always its CTA's last
// one.  sums_kernel finds the slices (the lengths are on the device) and sums such pieces; carry_kernel turns the sums
// into the state each CTA's first piece starts from; prompt_kernel walks.  Only heads that straddle CTAs have their K
// and V read twice.
//
// Bound by HBM: for r query heads to a key/value head a chunk moves (2 r + 2) tiles of 32 KB (D = 128) and costs 3 r + 1
// products of 128^3, at the measured rates a quarter of the time of its bytes.  Q, K and V come by TMA through rings of
// tiles that different threads fill, and O leaves by TMA from the tile its Q came in.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdlib.h>
#include <string.h>

#include "la_prompt.h"
#include "la_tc_host.h"
#include "la_tc_kern.cuh"

namespace la {
namespace prompt {

using namespace sm100;
using tc::AbortState;
using tc::kBox;
using tc::kC;
using tc::wait_or_abort;

// What a CTA's slice is: its first item, its length, and its last piece where that stops short of its head's end.
struct Slice {
    long long left;      // items; 0: none
    int seq, vh, c;      // the first item's sequence, head and chunk
    int lseq, lvh, la;   // the last piece's sequence, head, first chunk
    int open;            // the last piece stops short of its head's end
    int lchunks;         // its chunks (open only)
};

struct TcArgs {
    CUtensorMap tmQ, tmK, tmV, tmO;  // {D, T, heads}, boxes of 64 columns x 128 rows, 128-byte swizzle
    Args A;
    int gs;              // CTAs a group's query heads are spread over: head vh of Hkv gs, r / gs query heads each
    int r;               // query heads of one vh
    int G;               // slices
    Slice *slices;       // [G]
    float *sums, *carry; // [G] slots
    uint64_t wait_ns;
};

// A slot: S as float4s in (column group, row) order, then z, a (128 each) and n.
template <int NB> constexpr int kSlotS = 128 * 64 * NB;
template <int NB> constexpr int kSlot = kSlotS<NB> + 256 + 64;
// float4 q of half hf of row d
template <int NB> __device__ __forceinline__ int slot_at(int d, int hf, int q) { return (8 * NB * hf + q) * 128 + d; }

__device__ __forceinline__ int chunks_of(int len) { return len > kC ? (len + kC - 1) / kC : 1; }

// The (chunk, query head) units of a slice in order.
struct Units {
    const Args *A;
    int VH, r;
    long long left;      // items from this one on
    int seq, vh, c, j;   // j: query head within vh
    int a, e, nch;       // chunks of the piece, of the head
    int lo, len;         // the sequence's rows
    __device__ __forceinline__ void enter() {
        lo = A->off[seq];
        len = A->off[seq + 1] - lo;
        nch = chunks_of(len);
    }
    __device__ __forceinline__ void piece() {
        a = c;
        e = left < nch - c ? c + (int)left : nch;
    }
    __device__ __forceinline__ Units(const TcArgs &P, const Slice &s)
        : A(&P.A), VH(P.A.Hkv * P.gs), r(P.r), left(s.left), seq(s.seq), vh(s.vh), c(s.c), j(0) {
        if (left > 0) {
            enter();
            piece();
        }
    }
    __device__ __forceinline__ bool valid() const { return left > 0; }
    __device__ __forceinline__ bool last_head() const { return j == r - 1; }
    __device__ __forceinline__ bool last_chunk() const { return c + 1 == e; }
    __device__ __forceinline__ bool ends_head() const { return c + 1 == nch; }
    __device__ __forceinline__ int live() const { return min(kC, len - c * kC); }
    // whether the chunk's sums are needed: by the next chunk, or as the head's final state
    __device__ __forceinline__ bool sums_wanted(int gs) const {
        return !last_chunk() || (ends_head() && A->S != nullptr && vh % gs == 0);
    }
    __device__ __forceinline__ void next() {
        if (++j < r) return;
        j = 0;
        ++c;
        if (--left == 0 || c < e) return;
        c = 0;
        if (++vh == VH) {
            vh = 0;
            ++seq;
            enter();
        }
        piece();
    }
};

// ----------------------------------------------------------------------------------------------------------------
// Slices, and the sums of open pieces.  Warp 0 loads, warp 1 issues MMAs, warps 2-9 keep the sums.
// ----------------------------------------------------------------------------------------------------------------
constexpr int kSumThreads = 320;

// Finds the items x0 and x1 (flat numbers) of CTA blockIdx.x; every thread of the block calls it.
__device__ void find_slice(const TcArgs &P, Slice *out) {
    __shared__ int warp_sum[kSumThreads / 32];
    __shared__ int found[2][3];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int *off = P.A.off;
    const int per = (P.A.nseq + kSumThreads - 1) / kSumThreads;
    const int i0 = min(t * per, P.A.nseq), i1 = min(i0 + per, P.A.nseq);
    int mine = 0;
    for (int i = i0; i < i1; ++i) mine += chunks_of(off[i + 1] - off[i]);
    int upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, x);
        if (lane >= x) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int before = upto - mine, total = 0;
    for (int w = 0; w < kSumThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    const int VH = P.A.Hkv * P.gs;
    const long long X = (long long)total * VH;
    const long long x0 = X * blockIdx.x / P.G, x1 = X * (blockIdx.x + 1) / P.G;
    if (x1 > x0)
        for (int k = 0; k < 2; ++k) {
            long long x = k ? x1 - 1 : x0;
            long long at = (long long)before * VH;
            if (x < at || x >= at + (long long)mine * VH) continue;
            for (int i = i0; i < i1; ++i) {
                const int n = chunks_of(off[i + 1] - off[i]);
                if (x < at + (long long)n * VH) {
                    found[k][0] = i;
                    found[k][1] = (int)((x - at) / n);
                    found[k][2] = (int)((x - at) % n);
                    break;
                }
                at += (long long)n * VH;
            }
        }
    __syncthreads();
    Slice s = {};
    s.left = x1 - x0;
    if (s.left > 0) {
        s.seq = found[0][0], s.vh = found[0][1], s.c = found[0][2];
        s.lseq = found[1][0], s.lvh = found[1][1];
        s.la = s.lseq == s.seq && s.lvh == s.vh ? s.c : 0;
        s.open = found[1][2] + 1 < chunks_of(off[s.lseq + 1] - off[s.lseq]);
        s.lchunks = found[1][2] + 1 - s.la;
    }
    *out = s;
}

template <int NB> constexpr uint32_t kTileB = NB * kBox;  // bytes of a Q, K or V tile
template <int NB> constexpr size_t kSmemSums = 3 * 2 * (size_t)kTileB<NB> + 2048 + 256;

template <int NB>
__global__ void __launch_bounds__(kSumThreads, 1) sums_kernel(const __grid_constant__ TcArgs P) {
    constexpr int NST = 3;
    constexpr uint32_t TILE = kTileB<NB>, STAGE = 2 * TILE;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    bool aligned;
    unsigned char *stages = tc::smem_base(smem_raw, P.A.status, &aligned);
    if (!aligned) return;
    unsigned char *ones = stages + NST * STAGE;  // 8 rows x 128 B of bf16 1.0, read twice for N = 16
    uint64_t *full = (uint64_t *)(ones + 1024);
    uint64_t *empty = full + NST, *sumfull = empty + NST, *sumfree = sumfull + 2, *drain = sumfree + 2;
    uint32_t *tslot = (uint32_t *)(drain + 1);
    AbortState *abst = (AbortState *)(tslot + 2);
    volatile int *abort_flag = &abst->flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch_dependents();
    Slice s = {};
    if (offsets_in_order(P.A)) find_slice(P, &s);
    if (threadIdx.x == 0) P.slices[blockIdx.x] = s;
    if (!s.open) return;  // the same for the whole block

    if (threadIdx.x == 0) {
        for (int k = 0; k < NST; ++k) {
            mbar_init(&full[k], 1);
            mbar_init(&empty[k], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&sumfull[k], 1);
            mbar_init(&sumfree[k], 256);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        abst->limit_ns = P.wait_ns ? P.wait_ns : tc::kWaitNs;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 256; i += blockDim.x) ((uint32_t *)ones)[i] = 0x3F803F80u;
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int row0 = P.A.off[s.lseq] + s.la * kC, n = s.lchunks, h = s.lvh / P.gs;

    if (warp == 0 && lane == 0) {
        int it = 0;
        for (; it < n; ++it) {
            const int k = it % NST;
            if (it >= NST && !wait_or_abort(&empty[k], ((it / NST) - 1) & 1, abort_flag, P.A.status, 0x701)) break;
            mbar_arrive_expect_tx(&full[k], STAGE);
            for (int b = 0; b < NB; ++b) {
                tma_load_3d(stages + k * STAGE + b * kBox, &P.tmK, &full[k], 64 * b, row0 + it * kC, h);
                tma_load_3d(stages + k * STAGE + TILE + b * kBox, &P.tmV, &full[k], 64 * b, row0 + it * kC, h);
            }
        }
        if (*abort_flag)
            for (int k = it > NST ? it - NST : 0; k < it; ++k) mbar_wait(&full[k % NST], (k / NST) & 1, 50000000ull);
    } else if (warp == 1 && lane == 0) {
        const uint32_t idS = idesc_bf16(128, 64 * NB, true, true), idZ = idesc_bf16(128, 16, true, false);
        const uint32_t lbo = NB == 2 ? kBox : 0;  // D <= 64: rows 64-127 of S repeat rows 0-63 and are not read
        const uint32_t on0 = smem_u32(ones);
        for (int it = 0; it < n; ++it) {
            const int k = it % NST, b = it & 1;
            if (!wait_or_abort(&full[k], (it / NST) & 1, abort_flag, P.A.status, 0x702)) break;
            if (it >= 2 && !wait_or_abort(&sumfree[b], ((it >> 1) - 1) & 1, abort_flag, P.A.status, 0x703)) break;
            tc_fence_after();
            const uint32_t kb = smem_u32(stages + k * STAGE), vb = kb + TILE;
            const uint32_t tS = tmem + 128 * b, tZ = tmem + 256 + 32 * b;
#pragma unroll
            for (int x = 0; x < kC / 16; ++x) {
                const uint64_t kt = sdesc_sw128(kb + 2048 * x, lbo, 1024), vt = sdesc_sw128(vb + 2048 * x, lbo, 1024);
                const uint64_t on = sdesc_sw128(on0 + 32 * (x & 3), 16, 0);
                mma_ss(tS, kt, vt, idS, x > 0);
                mma_ss(tZ, kt, on, idZ, x > 0);
                mma_ss(tZ + 16, vt, on, idZ, x > 0);
            }
            mma_commit(&sumfull[b]);
            mma_commit(&empty[k]);
        }
        mma_commit(drain);
        mbar_wait(drain, 0, 50000000ull);
    } else if (warp >= 2) {
        const int q4 = warp & 3, hf = (warp - 2) >> 2, d = 32 * q4 + lane;
        const uint32_t lo = (uint32_t)(32 * q4) << 16;
        float S[32 * NB], za = 0.f;  // row d, columns 32 NB hf ...; z[d] (half 0) or a[d] (half 1)
#pragma unroll
        for (int m = 0; m < 32 * NB; ++m) S[m] = 0.f;
        int it = 0;
        for (; it < n; ++it) {
            const int b = it & 1;
            if (!__all_sync(0xffffffffu, wait_or_abort(&sumfull[b], (it >> 1) & 1, abort_flag, P.A.status, 0x704))) break;
            tc_fence_after();
            uint32_t z0, z1;
            tmem_ld2(tmem + lo + 256 + 32 * b + 16 * hf, z0, z1);
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                uint32_t v[32];
                tmem_ld32(tmem + lo + 128 * b + 32 * NB * hf + 32 * x, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int m = 0; m < 32; ++m) S[32 * x + m] += __uint_as_float(v[m]);
            }
            tmem_wait_ld(z0, z1);
            za += __uint_as_float(z0);
            tc_fence_before();
            mbar_arrive(&sumfree[b]);
        }
        if (it == n) {
            float *slot = P.sums + (long long)blockIdx.x * kSlot<NB>;
#pragma unroll
            for (int q = 0; q < 8 * NB; ++q)
                ((float4 *)slot)[slot_at<NB>(d, hf, q)] = make_float4(S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
            slot[kSlotS<NB> + 128 * hf + d] = za;
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ----------------------------------------------------------------------------------------------------------------
// Carries.  grid = (float4s of a slot / 256, G): the blocks of the CTA b in which a straddling head begins walk that
// head's CTAs in order and leave in each later one's carry the sum of all before it.  b's own sums are replaced by what
// the head starts from (resumed), because the CTA that ends the head writes the state while b may not have read it.
// ----------------------------------------------------------------------------------------------------------------
template <int NB> __global__ void __launch_bounds__(256) carry_kernel(const __grid_constant__ TcArgs P) {
    constexpr int S4 = kSlotS<NB> / 4, N4 = S4 + 64;
    __shared__ int chain[tc::kMaxCtas + 1];  // the head's CTAs after b0, in order
    __shared__ int length;
    griddep_wait();
    griddep_launch_dependents();
    const int b0 = blockIdx.y, x = blockIdx.x * 256 + threadIdx.x;
    const Slice s = P.slices[b0];
    if (!s.open || s.la != 0) return;  // the same for the whole block
    if (threadIdx.x < 32) {  // a CTA carries the head on while its last piece is of that head and open
        int n = 0;
        bool more = true;
        for (int b = b0 + 1; b < P.G && more; b += 32) {
            const int mine = b + threadIdx.x;
            Slice c = {};
            if (mine < P.G) c = P.slices[mine];
            const unsigned any = __ballot_sync(0xffffffffu, c.left > 0);
            const unsigned on = __ballot_sync(0xffffffffu, c.left > 0 && c.open && c.lseq == s.lseq && c.lvh == s.lvh);
            const unsigned stop = any & ~on;                       // the first CTA that does not ends the head
            const unsigned take = stop ? any & (2u * (stop & -stop) - 1u) : any;
            if (take >> threadIdx.x & 1u) chain[n + __popc(take & ((1u << threadIdx.x) - 1u))] = mine;
            n += __popc(take);
            more = !stop;
        }
        if (threadIdx.x == 0) length = n;
    }
    __syncthreads();
    if (x > N4) return;
    const int D = P.A.D, h = s.lvh / P.gs;
    const long long at = (long long)s.lseq * P.A.Hkv + h;
    float *first = P.sums + (long long)b0 * kSlot<NB>;
    const bool resume = P.A.resume;
    if (x == N4) {  // n before the sequence's first row
        const int n0 = resume ? P.A.n[at] : 0;
        *(int *)(first + kSlotS<NB> + 256) = n0;
        for (int k = 0; k < length; ++k) *(int *)(P.carry + (long long)chain[k] * kSlot<NB> + kSlotS<NB> + 256) = n0;
        return;
    }
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (resume) {
        float *r = &run.x;
        for (int m = 0; m < 4; ++m) {
            if (x < S4) {
                const int d = x % 128, e = 4 * (x / 128) + m;
                if (d < D && e < D) r[m] = ((const float *)P.A.S)[(at * D + d) * D + e];
            } else {
                const int i = 4 * (x - S4) + m, d = i % 128;
                if (d < D) r[m] = (i < 128 ? (const float *)P.A.z : (const float *)P.A.a)[at * D + d];
            }
        }
    }
    const float4 start = run;
    for (int k0 = 0; k0 < length; k0 += 8) {  // eight loads in flight
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < length)
                v[k] = ((const float4 *)(P.sums + (long long)(k0 + k ? chain[k0 + k - 1] : b0) * kSlot<NB>))[x];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k0 + k < length) {
                run.x += v[k].x, run.y += v[k].y, run.z += v[k].z, run.w += v[k].w;
                ((float4 *)(P.carry + (long long)chain[k0 + k] * kSlot<NB>))[x] = run;
            }
    }
    ((float4 *)first)[x] = start;
}

// ----------------------------------------------------------------------------------------------------------------
// The walk.  Warp 0 loads K and V, warp 10 loads Q, warp 1 issues MMAs, warps 2-9 (two per TMEM lane quarter, each half
// of the columns) are the epilogue.  A unit u is one query head of one chunk; three epilogue steps
//   A(u)  T -> P (TMEM), row sums              B(u)  O -> out              C  (a chunk's last unit)  S, Sb, z, a
// run as A(u + 1), B(u) [, C]: while A(u + 1) works, the tensor cores form O of u, and while B(u) works, T of u + 2.
// A does not need the state, so the order holds across chunks and across heads.
// TMEM columns: T 0, P 128 (even heads) and 320 (odd), O 192, K^T V 320, z and a sums 448, 464, q . z 480, row sums 496.
// The odd P and K^T V share columns: K^T V is formed behind the last unit's P V and read in C, before the next chunk's
// A(1).
// ----------------------------------------------------------------------------------------------------------------
constexpr int kThreads = 352;
template <int NB> constexpr int kKV = NB == 2 ? 3 : 6;  // K and V tiles, alternating
template <int NB> constexpr int kQ = NB == 2 ? 3 : 5;   // Q tiles
template <int NB> constexpr size_t kSmemWalk = (kKV<NB> + kQ<NB> + 1) * (size_t)kTileB<NB> + 2048 + 512 + 512;
static_assert(kSmemWalk<2> <= 232448, "shared-memory limit");

template <int NB>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ TcArgs P) {
    constexpr uint32_t TILE = kTileB<NB>;
    constexpr int NKV = kKV<NB>, NQ = kQ<NB>, CH = 32 * NB;  // CH: columns of O or S that an epilogue thread has
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    bool aligned;
    unsigned char *kv = tc::smem_base(smem_raw, P.A.status, &aligned);
    if (!aligned) return;
    unsigned char *qt = kv + NKV * TILE;
    unsigned char *Sb = qt + NQ * TILE;   // bf16 S, [d][e]
    unsigned char *zt = Sb + TILE;        // N = 16 operand: rows z (two bf16 parts) and ones
    float *as = (float *)(zt + 2048);     // a
    uint64_t *kvfull = (uint64_t *)(as + 128), *kvempty = kvfull + NKV, *qfull = kvempty + NKV, *qempty = qfull + NQ;
    uint64_t *barT = qempty + NQ, *pready = barT + 1, *barO = pready + 1, *ofree = barO + 1, *barS = ofree + 1;
    uint64_t *sready = barS + 1, *epi = sready + 1, *half = epi + 1, *drain = half + 2;
    uint32_t *tslot = (uint32_t *)(drain + 1);
    AbortState *abst = (AbortState *)(tslot + 2);
    volatile int *abort_flag = &abst->flag;
    uint32_t *status = P.A.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int k = 0; k < NKV; ++k) {
            mbar_init(&kvfull[k], 1);
            mbar_init(&kvempty[k], 1);
        }
        for (int k = 0; k < NQ; ++k) {
            mbar_init(&qfull[k], 1);
            mbar_init(&qempty[k], NB);
        }
        mbar_init(barT, 1);
        mbar_init(pready, 256);
        mbar_init(barO, 1);
        mbar_init(ofree, 256);
        mbar_init(barS, 1);
        mbar_init(sready, 256);
        mbar_init(epi, 256);
        mbar_init(&half[0], 128);
        mbar_init(&half[1], 128);
        mbar_init(drain, 1);
        *abort_flag = 0;
        abst->limit_ns = P.wait_ns ? P.wait_ns : tc::kWaitNs;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 512; i += blockDim.x)  // row 2 of each box ones, the rest zero
        ((uint32_t *)zt)[i] = (i % 256) / 32 == 2 ? 0x3F803F80u : 0u;
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem = *tslot;
    const uint32_t tT = tmem, tO = tmem + 192, tS = tmem + 320, tZA = tmem + 448, tQZ = tmem + 480, tR = tmem + 496;
    const Slice s = P.slices[blockIdx.x];

    if (warp == 0 && lane == 0) {
        // ---- K and V: tile 2 n is K, 2 n + 1 V of the slice's chunk n
        prefetch_tmap(&P.tmK);
        prefetch_tmap(&P.tmV);
        int t = 0;
        bool ok = true;
        Units u(P, s);
        u.r = 1;
        for (; u.valid() && ok; u.next()) {
            const int row = u.lo + u.c * kC, h = u.vh / P.gs;
            for (int k = 0; k < 2; ++k, ++t) {
                const int x = t % NKV;
                if (t >= NKV && !wait_or_abort(&kvempty[x], ((t / NKV) - 1) & 1, abort_flag, status, 0x801)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&kvfull[x], TILE);
                for (int b = 0; b < NB; ++b)
                    tma_load_3d(kv + x * TILE + b * kBox, k ? &P.tmV : &P.tmK, &kvfull[x], 64 * b, row, h);
            }
        }
        if (!ok)  // let the copies already issued land before the CTA exits
            for (int k = t > NKV ? t - NKV : 0; k < t; ++k) mbar_wait(&kvfull[k % NKV], (k / NKV) & 1, 50000000ull);
    } else if (warp == 10 && lane == 0) {
        // ---- Q: one tile a unit
        prefetch_tmap(&P.tmQ);
        int t = 0;
        bool ok = true;
        for (Units u(P, s); u.valid(); u.next(), ++t) {
            const int x = t % NQ;
            if (t >= NQ && !wait_or_abort(&qempty[x], ((t / NQ) - 1) & 1, abort_flag, status, 0x802)) {
                ok = false;
                break;
            }
            mbar_arrive_expect_tx(&qfull[x], TILE);
            for (int b = 0; b < NB; ++b)
                tma_load_3d(qt + x * TILE + b * kBox, &P.tmQ, &qfull[x], 64 * b, u.lo + u.c * kC, u.vh * P.r + u.j);
        }
        if (!ok)
            for (int k = t > NQ ? t - NQ : 0; k < t; ++k) mbar_wait(&qfull[k % NQ], (k / NQ) & 1, 50000000ull);
    } else if (warp == 1 && lane == 0) {
        // ---- MMA
        const uint32_t idT = idesc_bf16(128, 128, false, false), idO = idesc_bf16(128, 64 * NB, false, true);
        const uint32_t idS = idesc_bf16(128, 64 * NB, true, true), idZ = idesc_bf16(128, 16, true, false);
        const uint32_t idQZ = idesc_bf16(128, 16, false, false);
        const uint32_t lbo = NB == 2 ? kBox : 0;
        const uint32_t zb = smem_u32(zt), sb = smem_u32(Sb), kv0 = smem_u32(kv), q0 = smem_u32(qt);
        int n = 0;  // chunk of unit u
        int un = 0;
        // T of unit x (its number) in chunk m
        auto issue_t = [&](const Units &w, int x, int m) {
            if (w.j == 0 && !wait_or_abort(&kvfull[(2 * m) % NKV], ((2 * m) / NKV) & 1, abort_flag, status, 0x803)) return false;
            if (!wait_or_abort(&qfull[x % NQ], (x / NQ) & 1, abort_flag, status, 0x804)) return false;
            tc_fence_after();
            const uint32_t qb = q0 + (x % NQ) * TILE, kb = kv0 + ((2 * m) % NKV) * TILE;
#pragma unroll
            for (int k = 0; k < 4 * NB; ++k)
                mma_ss(tT, sdesc_sw128(qb + (k >> 2) * kBox + 32 * (k & 3), 16, 1024),
                       sdesc_sw128(kb + (k >> 2) * kBox + 32 * (k & 3), 16, 1024), idT, k > 0);
            mma_commit(barT);
            return true;
        };
        Units u(P, s);
        bool ok = u.valid() && issue_t(u, 0, 0);
        while (ok) {
            Units w = u;
            w.next();
            if (!wait_or_abort(pready, un & 1, abort_flag, status, 0x805)) break;  // P(u) is there, T may be overwritten
            tc_fence_after();
            if (w.valid() && !issue_t(w, un + 1, u.last_head() ? n + 1 : n)) break;
            if (un > 0 && !wait_or_abort(ofree, (un - 1) & 1, abort_flag, status, 0x806)) break;
            const int kx = (2 * n) % NKV, vx = (2 * n + 1) % NKV;
            if (u.j == 0) {
                if (!wait_or_abort(&kvfull[vx], ((2 * n + 1) / NKV) & 1, abort_flag, status, 0x807)) break;
                if (!wait_or_abort(sready, n & 1, abort_flag, status, 0x808)) break;
            }
            tc_fence_after();
            const uint32_t qb = q0 + (un % NQ) * TILE, kb = kv0 + kx * TILE, vb = kv0 + vx * TILE;
            const uint32_t tP = tmem + (u.j & 1 ? 320 : 128);
#pragma unroll
            for (int k = 0; k < 4 * NB; ++k) {
                const uint64_t qd = sdesc_sw128(qb + (k >> 2) * kBox + 32 * (k & 3), 16, 1024);
                mma_ss(tO, qd, sdesc_sw128(sb + 2048 * k, lbo, 1024), idO, k > 0);
                mma_ss(tQZ, qd, sdesc_sw128(zb + (k >> 2) * 1024 + 32 * (k & 3), 16, 0), idQZ, k > 0);
            }
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) mma_ts(tO, tP + 8 * k, sdesc_sw128(vb + 2048 * k, lbo, 1024), idO, 1u);
            mma_commit(barO);
            if (u.last_head()) {
                if (u.sums_wanted(P.gs)) {
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {
                        const uint64_t kt = sdesc_sw128(kb + 2048 * k, lbo, 1024), vt = sdesc_sw128(vb + 2048 * k, lbo, 1024);
                        const uint64_t on = sdesc_sw128(zb + (k >> 2) * 1024 + 32 * (k & 3), 16, 0);
                        mma_ss(tS, kt, vt, idS, k > 0);
                        mma_ss(tZA, kt, on, idZ, k > 0);
                        mma_ss(tZA + 16, vt, on, idZ, k > 0);
                    }
                    mma_commit(barS);
                }
                mma_commit(&kvempty[kx]);
                mma_commit(&kvempty[vx]);
                ++n;
            }
            if (!w.valid()) break;
            u = w;
            ++un;
        }
        mma_commit(drain);
        mbar_wait(drain, 0, 50000000ull);
    } else if (warp >= 2 && warp < 10) {
        // ---- epilogue: thread <-> row i of a chunk (of S: row d = i) and half hf of the columns
        const int q4 = warp & 3, hf = (warp - 2) >> 2, i = 32 * q4 + lane;
        const uint32_t lo = (uint32_t)(32 * q4) << 16;
        const int D = P.A.D, col0 = CH * hf;
        const bool has_row = NB == 2 || q4 < 2;          // rows of S there are
        const bool storer = lane == 0 && q4 == 0 && (NB == 2 || hf == 0);
        float S[CH], za = 0.f;                           // S[i][col0 ...]; z[i] (half 0), a[i] (half 1)
        int n0 = 0;                                      // n before the head's first row
        int pending = -1;                                // Q tile whose O is on its way out (storer)
        int epis = 0, halves = 0, ks = 0;
        // A warp gives up together: its TMEM accesses are the whole warp's.
        auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t where) {
            return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, status, where)) != 0;
        };

        // The state a piece starts from, into registers, Sb, z and a (shared).
        auto put_state = [&]() {
            if (has_row) {
                unsigned char *tile = Sb + (NB == 2 ? hf * kBox : 0);
#pragma unroll
                for (int g = 0; g < CH / 8; ++g) {
                    uint4 w;
                    w.x = pack_bf16(S[8 * g], S[8 * g + 1]);
                    w.y = pack_bf16(S[8 * g + 2], S[8 * g + 3]);
                    w.z = pack_bf16(S[8 * g + 4], S[8 * g + 5]);
                    w.w = pack_bf16(S[8 * g + 6], S[8 * g + 7]);
                    *(uint4 *)(tile + tc::sw128_off(i, (NB == 2 ? 0 : 4 * hf) + g)) = w;
                }
                if (hf == 0) tc::split_tile_put(zt, i, za);
                else as[i] = za;
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(sready);
        };
        auto load_state = [&](const Units &u) {
            const long long at = (long long)u.seq * P.A.Hkv + u.vh / P.gs;
            const bool carried = u.a > 0, open = u.e < u.nch;
            const bool slot = carried || (open && P.A.resume);
            n0 = 0;
            za = 0.f;
#pragma unroll
            for (int m = 0; m < CH; ++m) S[m] = 0.f;
            if (slot) {
                const float *f = (carried ? P.carry : P.sums) + (long long)blockIdx.x * kSlot<NB>;
                if (has_row) {
#pragma unroll
                    for (int q = 0; q < 8 * NB; ++q) {
                        const float4 v = ((const float4 *)f)[slot_at<NB>(i, hf, q)];
                        S[4 * q] = v.x, S[4 * q + 1] = v.y, S[4 * q + 2] = v.z, S[4 * q + 3] = v.w;
                    }
                    za = f[kSlotS<NB> + 128 * hf + i];
                }
                n0 = *(const int *)(f + kSlotS<NB> + 256);
            } else if (P.A.resume) {
                if (i < D && col0 < D) {
                    const float4 *src = (const float4 *)((const float *)P.A.S + (at * D + i) * D + col0);
#pragma unroll
                    for (int q = 0; q < CH / 4; ++q) {
                        const float4 v = src[q];
                        S[4 * q] = v.x, S[4 * q + 1] = v.y, S[4 * q + 2] = v.z, S[4 * q + 3] = v.w;
                    }
                }
                if (i < D) za = (hf == 0 ? (const float *)P.A.z : (const float *)P.A.a)[at * D + i];
                n0 = P.A.n[at];
            }
        };
        auto save_state = [&](const Units &u) {
            const long long at = (long long)u.seq * P.A.Hkv + u.vh / P.gs;
            if (i < D && col0 < D) {
                float4 *dst = (float4 *)((float *)P.A.S + (at * D + i) * D + col0);
#pragma unroll
                for (int q = 0; q < CH / 4; ++q) dst[q] = make_float4(S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
            }
            if (i < D) (hf == 0 ? (float *)P.A.z : (float *)P.A.a)[at * D + i] = za;
            if (hf == 0 && i == 0) P.A.n[at] = n0 + u.len;
        };
        // A: P and row sums of unit x in chunk m
        auto step_a = [&](const Units &u, int x, int m) {
            if (!wait(barT, x & 1, 0x810)) return false;
            tc_fence_after();
            uint32_t pk[2][16];
            float sum = 0.f;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int j0 = 64 * hf + 32 * b, blk = 2 * hf + b;
                if (blk > q4) {  // above the diagonal
#pragma unroll
                    for (int k = 0; k < 16; ++k) pk[b][k] = 0u;
                } else {
                    uint32_t v[32];
                    tmem_ld32(tT + lo + j0, v);
                    tmem_wait_ld(v);
                    if (blk < q4) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float p0 = 1.f + __uint_as_float(v[2 * k]), p1 = 1.f + __uint_as_float(v[2 * k + 1]);
                            pk[b][k] = pack_bf16(p0, p1);
                            sum += p0 + p1;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float p0 = 2 * k <= lane ? 1.f + __uint_as_float(v[2 * k]) : 0.f;
                            const float p1 = 2 * k + 1 <= lane ? 1.f + __uint_as_float(v[2 * k + 1]) : 0.f;
                            pk[b][k] = pack_bf16(p0, p1);
                            sum += p0 + p1;
                        }
                    }
                }
            }
            if (u.j == 0 && x > 0 && (u.r & 1)) {  // the unit before has its P in the same columns
                if (!wait(barO, (x - 1) & 1, 0x811)) return false;
                tc_fence_after();
            }
            if (u.j == 1 && !wait(sready, m & 1, 0x818)) return false;  // all have read K^T V
            const uint32_t tP = tmem + (u.j & 1 ? 320 : 128) + lo + 32 * hf;
            tmem_st16(tP, pk[0]);
            tmem_st16(tP + 16, pk[1]);
            tmem_st1(tR + lo + 2 * (x & 1) + hf, __float_as_uint(sum));
            tmem_st_wait();
            if (u.j == 0 && u.live() < kC) {
                // the chunk reaches past its sequence: rows that are not its own must not enter P V and K^T V, where
                // a zero weight would not keep an infinity out
                for (int k = 0; k < 2; ++k) {
                    const int t = 2 * m + k;
                    if (!wait(&kvfull[t % NKV], (t / NKV) & 1, 0x812)) return false;
                    unsigned char *tile = kv + (t % NKV) * TILE;
                    const int first = u.live() > 0 ? u.live() : 0, e = threadIdx.x - 64;
                    for (int y = e; y < (kC - first) * 8 * NB; y += 256) {
                        const int row = first + y / (8 * NB), g = y % (8 * NB);
                        *(uint4 *)(tile + (g >> 3) * kBox + row * 128 + (g & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
            }
            tc_fence_before();
            mbar_arrive(pready);
            return true;
        };
        auto release = [&]() {
            if (pending >= 0) {
                bulk_wait_read0();
                mbar_arrive(&qempty[pending]);
                pending = -1;
            }
        };
        // B: output of unit x
        auto step_b = [&](const Units &u, int x) {
            if (!wait(barO, x & 1, 0x813)) return false;
            tc_fence_after();
            uint32_t z0, z1, r0, r1;
            tmem_ld2(tQZ + lo, z0, z1);
            tmem_ld2(tR + lo + 2 * (x & 1), r0, r1);
            tmem_wait_ld(z0, z1);
            tmem_wait_ld(r0, r1);
            const float g = (float)(n0 + u.c * kC) + (__uint_as_float(z0) + __uint_as_float(z1)) +
                            (__uint_as_float(r0) + __uint_as_float(r1));
            const float inv = 1.f / g;
            const int live = u.live(), hq = u.vh * P.r + u.j;
            unsigned char *tile = qt + (x % NQ) * TILE + (NB == 2 ? hf * kBox : 0);
            __nv_bfloat16 *out = (__nv_bfloat16 *)P.A.o + hq * P.A.oh + (long long)(u.lo + u.c * kC + i) * P.A.on + col0;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t v[32];
                tmem_ld32(tO + lo + col0 + 32 * b, v);
                tmem_wait_ld(v);
                const float4 *a4 = (const float4 *)(as + col0 + 32 * b);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float4 c0 = a4[2 * y], c1 = a4[2 * y + 1];
                    uint4 w;
                    w.x = pack_bf16((__uint_as_float(v[8 * y]) + c0.x) * inv, (__uint_as_float(v[8 * y + 1]) + c0.y) * inv);
                    w.y = pack_bf16((__uint_as_float(v[8 * y + 2]) + c0.z) * inv, (__uint_as_float(v[8 * y + 3]) + c0.w) * inv);
                    w.z = pack_bf16((__uint_as_float(v[8 * y + 4]) + c1.x) * inv, (__uint_as_float(v[8 * y + 5]) + c1.y) * inv);
                    w.w = pack_bf16((__uint_as_float(v[8 * y + 6]) + c1.z) * inv, (__uint_as_float(v[8 * y + 7]) + c1.w) * inv);
                    const int e = 32 * b + 8 * y;  // column within the thread's
                    if (live == kC) *(uint4 *)(tile + tc::sw128_off(i, (NB == 2 ? 0 : 4 * hf) + (e >> 3))) = w;
                    else if (i < live && col0 + e < D) *(uint4 *)(out + e) = w;  // rows of others stay as they are
                }
            }
            tc_fence_before();
            mbar_arrive(ofree);
            if (live == kC) {
                fence_proxy_async_smem();
                uint64_t *bar = NB == 2 ? &half[hf] : &half[0];
                if (NB == 2 || hf == 0) mbar_arrive(bar);
                else mbar_arrive(&half[1]);
                if (storer && wait_or_abort(bar, halves & 1, abort_flag, status, 0x814) &&
                    (NB == 2 || wait_or_abort(&half[1], halves & 1, abort_flag, status, 0x815))) {
                    tma_store_3d(&P.tmO, tile, NB == 2 ? col0 : 0, u.lo + u.c * kC, hq);
                    bulk_commit();
                    pending = x % NQ;
                }
                __syncwarp();
                ++halves;
            } else if (storer) {
                mbar_arrive(&qempty[x % NQ]);
            }
            return true;
        };
        // C: the state after unit x's chunk; then what the next chunk (w) starts from
        auto step_c = [&](const Units &u, const Units &w) {
            // everyone has read a
            mbar_arrive(epi);
            if (!wait(epi, epis & 1, 0x816)) return false;
            ++epis;
            if (u.sums_wanted(P.gs)) {
                if (!wait(barS, ks & 1, 0x817)) return false;
                ++ks;
                tc_fence_after();
                if (has_row) {
                    uint32_t z0, z1;
                    tmem_ld2(tZA + lo + 16 * hf + 2, z0, z1);  // column 2: the ones
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t v[32];
                        tmem_ld32(tS + lo + col0 + 32 * b, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int m = 0; m < 32; ++m) S[32 * b + m] += __uint_as_float(v[m]);
                    }
                    tmem_wait_ld(z0, z1);
                    za += __uint_as_float(z0);
                }
                tc_fence_before();
            }
            if (u.last_chunk()) {
                if (u.ends_head() && P.A.S && u.vh % P.gs == 0) save_state(u);
                if (w.valid()) load_state(w);
            }
            if (w.valid()) put_state();
            return true;
        };

        Units u(P, s);
        int x = 0, m = 0;
        bool ok = u.valid();
        if (ok) {
            load_state(u);
            put_state();
            ok = step_a(u, 0, 0);
        }
        while (ok) {
            Units w = u;
            w.next();
            if (w.valid() && !step_a(w, x + 1, u.last_head() ? m + 1 : m)) break;
            release();
            if (!step_b(u, x)) break;
            if (u.last_head()) {
                if (!step_c(u, w)) break;
                ++m;
            }
            if (!w.valid()) break;
            u = w;
            ++x;
        }
        if (storer) bulk_wait0();  // output stores complete before the CTA exits
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------------------------------------------------ host

bool tc_supported(int D, int dtype) { return dtype == 1 && (D == 32 || D == 64 || D == 128); }

// Upper bound of (sequence, head, chunk) items for heads of which there are VH.
static long long max_items(int T, int nseq, int VH) { return ((long long)T / kC + nseq) * VH; }

size_t tc_workspace_bytes(int T, int nseq, int Hkv, int r, int D) {
    const int NB = D > 64 ? 2 : 1;
    long long G = max_items(T, nseq, Hkv * r);
    if (G > tc::kMaxCtas) G = tc::kMaxCtas;
    const size_t slot = (size_t)(NB == 2 ? kSlot<2> : kSlot<1>) * sizeof(float);
    return 256 + tc::kMaxCtas * 64 + 2 * (size_t)G * slot;
}
static_assert(sizeof(Slice) <= 64, "a slice's record");

static bool head_map(CUtensorMap *m, PFN_cuTensorMapEncodeTiled_v12000 enc, const void *p, int D, int T, int H,
                     long long sh, long long sn) {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)H};
    cuuint64_t st[2] = {(cuuint64_t)sn * 2, (cuuint64_t)sh * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)kC, 1}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, st, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static cudaError_t launch(void (*kernel)(const TcArgs), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                          const TcArgs &P) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <int NB> static cudaError_t run(TcArgs &P, unsigned char *ws, cudaStream_t s) {
    static std::atomic<int> state[kMaxDevices];
    if (!once_per_device(state, [] {
            const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
            return cudaFuncSetAttribute(sums_kernel<NB>, a, (int)kSmemSums<NB>) == cudaSuccess &&
                   cudaFuncSetAttribute(prompt_kernel<NB>, a, (int)kSmemWalk<NB>) == cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    P.slices = (Slice *)(ws + 256);
    P.sums = (float *)(ws + 256 + tc::kMaxCtas * 64);
    P.carry = P.sums + (size_t)P.G * kSlot<NB>;
    cudaError_t e = launch(sums_kernel<NB>, dim3(P.G), kSumThreads, kSmemSums<NB>, s, P);
    if (e == cudaSuccess && P.G > 1)
        e = launch(carry_kernel<NB>, dim3((kSlotS<NB> / 4 + 64 + 256) / 256, P.G), 256, 0, s, P);
    if (e == cudaSuccess) e = launch(prompt_kernel<NB>, dim3(P.G), kThreads, kSmemWalk<NB>, s, P);
    return e;
}

cudaError_t tensor_cores(const Args &A, unsigned char *ws, cudaStream_t s) {
    const int nsm = tc_host::sm_count();
    auto enc = tc_host::encode_fn();
    if (nsm <= 0 || !enc) return cudaErrorInvalidDevice;
    TcArgs P;
    memset(&P, 0, sizeof(P));
    P.A = A;
    P.r = A.r;
    P.gs = 1;
    // Few items: a group's query heads are spread over CTAs, which each walk K and V.  Not for resumed sequences, whose
    // state one of those CTAs would replace while another has yet to read it.
    while (!A.resume && P.r % 2 == 0 && 2 * max_items(A.T, A.nseq, A.Hkv * P.gs) <= nsm) {
        P.r /= 2;
        P.gs *= 2;
    }
    long long G = max_items(A.T, A.nseq, A.Hkv * P.gs);
    if (G > nsm) G = nsm;
    if (G > tc::kMaxCtas) G = tc::kMaxCtas;
    if (const char *env = getenv("LA_TC_MAX_CTAS")) {  // test hook: slices of several pieces on small problems
        const long long cap = atoll(env);
        if (cap >= 1 && cap < G) G = cap;
    }
    P.G = (int)G;
    if (const char *env = getenv("LA_TEST_WAIT_NS")) {
        const long long ns = atoll(env);
        if (ns >= 1000000) P.wait_ns = (uint64_t)ns;
    }
    if (A.T > 0 && (!head_map(&P.tmQ, enc, A.q, A.D, A.T, A.Hq, A.qh, A.qn) ||
                    !head_map(&P.tmK, enc, A.k, A.D, A.T, A.Hkv, A.kh, A.kn) ||
                    !head_map(&P.tmV, enc, A.v, A.D, A.T, A.Hkv, A.vh, A.vn) ||
                    !head_map(&P.tmO, enc, A.o, A.D, A.T, A.Hq, A.oh, A.on)))
        return cudaErrorInvalidValue;
    return A.D > 64 ? run<2>(P, ws, s) : run<1>(P, ws, s);
}

}  // namespace prompt
}  // namespace la
