// la_prompt_tc.cu -- tcgen05 / TMA form of la_prompt (bf16, D = 32, 64, 128).
//
// Per key/value head and chunk of 128 rows, with S, z, a, n those of the rows before the chunk, for each query head:
//   T = Q K^T,  P = [j <= i](1 + T),  O = (Q Sb + P V + a) / (n + q . z + row sums of P)
// and once per chunk  S += K^T V,  z += K^T 1,  a += V^T 1.  The tensor cores take S rounded to bf16 (Sb) and P as bf16,
// in two parts (16 bits) where P's rounding would show beside the output's.  S itself lives in fp32 registers of the
// epilogue: a chunk's K^T V is summed by itself in TMEM and added there, so that a long sequence's sums are rounded to
// nearest once a chunk.
//
// Work split.  All (sequence, head, chunk) items are laid end to end in that order and cut into G equal slices, one per
// CTA; the part of a slice in one head is a piece.  A piece that stops short of its head's end is always its CTA's last
// one.  sums_kernel finds the slices (the lengths are on the device) and sums such pieces; carry_kernel turns the sums
// into the state each CTA's first piece starts from; prompt_kernel walks.  Only heads that straddle CTAs have their K
// and V read twice.
//
// For r query heads to a key/value head a chunk has to move (2 r + 2) tiles of 32 KB (D = 128).  65,536 tokens, 16 query
// and 4 key/value heads of 128 (671 MB): 171 us, about 30 for the sums (which read K and V once more), 10 for the carries
// and 124 for the walk (5.4 TB/s).  12 prompts of 12,000 tokens together: 57 us; a CTA has three chunks there, and what
// it waits for at each kernel's and each piece's beginning counts for as much as they do.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdlib.h>
#include <string.h>

#include "la_f32x2.cuh"
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
    int drop;            // test hook: the unit whose Q CTA 0 of the walk does not load; -1: none
};

// A slot: S as float4s in (column group, row) order, then z, a (128 each) and n.
template <int NB> constexpr int kSlotS = 128 * 64 * NB;
template <int NB> constexpr int kSlot = kSlotS<NB> + 256 + 64;
// float4 q of half hf of row d
template <int NB> __device__ __forceinline__ int slot_at(int d, int hf, int q) { return (8 * NB * hf + q) * 128 + d; }

__device__ __forceinline__ int chunks_of(int len) { return len > kC ? (len + kC - 1) / kC : 1; }

// The (chunk, query head) units of CTA blockIdx.x's slice in order.
struct Units {
    int left;               // items from this one on
    int seq, vh, c, j;      // j: query head within vh
    int nch, lo, len;       // the head's chunks, the sequence's rows
    __device__ __forceinline__ void enter(const TcArgs &P) {
        lo = __ldcg(P.A.off + seq);
        len = __ldcg(P.A.off + seq + 1) - lo;
        nch = chunks_of(len);
    }
    __device__ __forceinline__ explicit Units(const TcArgs &P) {
        const Slice *s = P.slices + blockIdx.x;
        left = (int)__ldcg(&s->left), seq = __ldcg(&s->seq), vh = __ldcg(&s->vh), c = __ldcg(&s->c), j = 0;
        nch = lo = len = 0;
        if (left > 0) enter(P);
    }
    __device__ __forceinline__ bool valid() const { return left > 0; }
    // of the piece in this slice; the head's
    __device__ __forceinline__ bool last_chunk() const { return left == 1 || c + 1 == nch; }
    __device__ __forceinline__ bool ends_head() const { return c + 1 == nch; }
    __device__ __forceinline__ int live() const { return min(kC, len - c * kC); }
    // whether the CTA writes the head's state behind this chunk
    __device__ __forceinline__ bool saves(const TcArgs &P) const { return ends_head() && P.A.S && vh % P.gs == 0; }
    // whether the chunk's sums are needed: by the next chunk, or for the head's state
    __device__ __forceinline__ bool sums_wanted(const TcArgs &P) const { return !last_chunk() || saves(P); }
    // the unit after this one, for r query heads of each of VH heads
    __device__ __forceinline__ void next(const TcArgs &P, int r, int VH) {
        if (++j < r) return;
        j = 0;
        ++c;
        if (--left == 0 || c < nch) return;
        c = 0;
        if (++vh == VH) {
            vh = 0;
            ++seq;
            enter(P);
        }
    }
    // At the first unit of a piece: the slot that holds what it starts from, null if that is the caller's state (or
    // nothing); where the head's state is; the rows before the first of this call.
    template <int NB> __device__ __forceinline__ const float *slot(const TcArgs &P) const {
        if (c > 0) return P.carry + (long long)blockIdx.x * kSlot<NB>;                       // carried on from others
        if (P.A.resume && left < nch) return P.sums + (long long)blockIdx.x * kSlot<NB>;     // others carry it on
        return nullptr;
    }
    __device__ __forceinline__ long long state(const TcArgs &P) const { return (long long)seq * P.A.Hkv + vh / P.gs; }
    template <int NB> __device__ __forceinline__ int rows_before(const TcArgs &P) const {
        const float *f = slot<NB>(P);
        if (f) return *(const int *)(f + kSlotS<NB> + 256);
        return P.A.resume ? P.A.n[state(P)] : 0;
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
// Carries.  A chain is the CTAs of one head that straddles CTAs: b0, whose last piece is the head's first and open, those
// that only have a piece of the same head's middle, and the one that ends it.  Every later CTA's carry is the sum of all
// pieces before it.  b0's own sums are replaced by what the head starts from (resumed), because the CTA that ends the
// head writes the state while b0 may not have read it.
// A float4 of the slots goes along a chain in up to 32 segments of at most 5 CTAs, one thread each, which first add up
// their own: with one thread to a whole chain of 38 CTAs (65,536 tokens, 4 heads) the loads came in five rounds of 3 us.
// A chain in m segments is the work of m blocks for each kCarryThreads float4s, so that all chains together keep about as
// many blocks busy whether they are few and long or many and short.
// ----------------------------------------------------------------------------------------------------------------
constexpr int kCarryThreads = 256, kCarryBlocks = 44;  // 17 x 44 blocks, five on an SM, are all there at once
constexpr int kSegment = 5, kWords = tc::kMaxCtas / 32;
static_assert(tc::kMaxCtas <= kCarryThreads && tc::kMaxCtas % 32 == 0 && tc::kMaxCtas <= 32 * kSegment, "slices in a chain");
__device__ __forceinline__ int segments(int length) {
    int m = 1;
    while (m < 32 && length > kSegment * m) m *= 2;
    return m;
}

template <int NB> __global__ void __launch_bounds__(kCarryThreads, 5) carry_kernel(const __grid_constant__ TcArgs P) {
    constexpr int S4 = kSlotS<NB> / 4, N4 = S4 + 64;
    __shared__ uint32_t any[kWords], ends[kWords];     // CTAs with items; of those, the ones that no chain passes through
    __shared__ int before[kWords + 1];                 // blocks' worth of the chains that begin in the words before
    __shared__ int begin, length, share, chain[tc::kMaxCtas];
    __shared__ float4 total[kCarryThreads];
    griddep_wait();
    griddep_launch_dependents();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    Slice s = {};
    if (t < P.G) s = P.slices[t];
    const uint32_t on = __ballot_sync(0xffffffffu, s.left > 0);
    const uint32_t stop = __ballot_sync(0xffffffffu, s.left > 0 && !(s.open && s.la > 0));
    if (lane == 0 && warp < kWords) any[warp] = on, ends[warp] = stop;
    __syncthreads();
    // of a chain that begins at CTA t: its last CTA and its length
    int last = t, len = 0;
    if (s.left > 0 && s.open && s.la == 0) {
        for (int w = warp; w < kWords; ++w) {
            const uint32_t from = w == warp ? ~1u << lane : ~0u, e = ends[w] & from;  // (lane 31: none left of this word)
            const uint32_t to = e ? 2u * (e & -e) - 1u : ~0u;
            len += __popc(any[w] & from & to);
            if (e) {
                last = 32 * w + __ffs(e) - 1;
                break;
            }
        }
    }
    const int blocks = len > 0 ? segments(len) : 0;
    int upto = blocks;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, x);
        if (lane >= x) upto += v;
    }
    if (lane == 31 && warp < kWords) before[warp + 1] = upto;
    __syncthreads();
    if (t == 0) {
        before[0] = 0;
        for (int w = 0; w < kWords; ++w) before[w + 1] += before[w];
    }
    __syncthreads();
    for (int y = blockIdx.y; y < before[kWords]; y += gridDim.y) {
        if (warp < kWords && y >= before[warp] + upto - blocks && y < before[warp] + upto) {
            begin = t;
            length = len;
            share = y - (before[warp] + upto - blocks);
            int n = 0;
            for (int w = warp; w <= last >> 5; ++w)
                for (uint32_t m = any[w] & (w == warp ? ~1u << lane : ~0u) & (w == last >> 5 ? 2u * (1u << (last & 31)) - 1u : ~0u); m; m &= m - 1)
                    chain[n++] = 32 * w + __ffs(m) - 1;
        }
        __syncthreads();
        const int L = length, b0 = begin, m = segments(L), wide = kCarryThreads / m, seg = t / wide, col = t % wide;
        const int x = blockIdx.x * kCarryThreads + share * wide + col;
        const int k0 = L * seg / m, count = L * (seg + 1) / m - k0;  // <= kSegment
        const Slice h = P.slices[b0];
        const long long at = (long long)h.lseq * P.A.Hkv + h.lvh / P.gs;
        float *first = P.sums + (long long)b0 * kSlot<NB>;
        float4 v[kSegment];
        if (x < N4) {
#pragma unroll
            for (int k = 0; k < kSegment; ++k)
                if (k < count) {
                    const int from = k0 + k ? chain[k0 + k - 1] : b0;
                    v[k] = ((const float4 *)(P.sums + (long long)from * kSlot<NB>))[x];
                }
        }
        float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < N4 && P.A.resume) {
            float *r = &run.x;
            for (int k = 0; k < 4; ++k) {
                const int D = P.A.D;
                if (x < S4) {
                    const int d = x % 128, e = 4 * (x / 128) + k;
                    if (d < D && e < D) r[k] = ((const float *)P.A.S)[(at * D + d) * D + e];
                } else {
                    const int i = 4 * (x - S4) + k, d = i % 128;
                    if (d < D) r[k] = (i < 128 ? (const float *)P.A.z : (const float *)P.A.a)[at * D + d];
                }
            }
        }
        const float4 start = run;
        auto add = [](float4 &r, const float4 &y) { r.x += y.x, r.y += y.y, r.z += y.z, r.w += y.w; };
        if (m > 1) {
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kSegment; ++k)
                if (x < N4 && k < count) add(sum, v[k]);
            total[t] = sum;
            __syncthreads();
            for (int y2 = 0; y2 < seg; ++y2) add(run, total[y2 * wide + col]);
        }
        if (x < N4) {
#pragma unroll
            for (int k = 0; k < kSegment; ++k)
                if (k < count) {
                    add(run, v[k]);
                    ((float4 *)(P.carry + (long long)chain[k0 + k] * kSlot<NB>))[x] = run;
                }
            if (seg == 0) ((float4 *)first)[x] = start;
        } else if (x == N4 && seg == 0) {  // n before the sequence's first row
            const int n0 = P.A.resume ? P.A.n[at] : 0;
            *(int *)(first + kSlotS<NB> + 256) = n0;
            for (int k = 0; k < L; ++k) *(int *)(P.carry + (long long)chain[k] * kSlot<NB> + kSlotS<NB> + 256) = n0;
        }
        __syncthreads();  // chain and total have been read
    }
}

// ----------------------------------------------------------------------------------------------------------------
// The walk.  A unit u is one query head of one chunk.  Warp 0 loads K and V, warp 2 loads Q, warp 1 issues MMAs; the
// epilogue is two groups of eight warps (two per TMEM lane quarter, each half of the columns):
//   A(u)  T -> P (TMEM), row sums; after a chunk's last unit  C  S, Sb, z, a        B(u)  O -> out
// The tensor cores form Q S of u + 1 and A works on u + 1 while B writes u: O has two buffers, and K^T V is formed in
// the one that the next unit will take.  O is staged in the tile its Q came in and leaves by TMA.
// K and V have one tile each: K is free behind the last T and K^T V, V behind the last P V; four Q tiles, because one is
// held from its load to its O's store, some 2 units and a load's latency.  (With two K, V tiles and three Q tiles every
// unit waited for its Q.)
// What bounds it are the MMAs of a CTA, one behind another: T 0.7 k clocks, Q S and P V 0.7 k each (8 of 128 x 128 x 16,
// 64 clocks of shared memory each at best), once a chunk K^T V with the sums of K and V 1.7 k; HBM would take 3.4 k for a
// unit's bytes (D = 128, r = 4).  An N = 16 MMA takes more than an N = 128 one: z stands behind K's rows, so that T
// brings q . z along (N = 144), and only a chunk's first unit, whose T is formed before the chunk's z is known, has
// products of its own for it.  (Such products in each unit: 204 us for the first case where this took 191.)  The sums of
// K and V on the CUDA cores took twice the epilogue's time.  Two threads that issue MMAs side by side (T, and the rest):
// 191 us where one takes 182.  K^T V formed a unit earlier, so that K is filled again in time: 176 where this takes 171.
// Two things cost the epilogue more than its arithmetic: code that does not come round again within a unit (the warps
// then wait for instructions), hence loops that are not unrolled and one group per step; and spilled registers, which
// with this much shared memory are L2 accesses, hence 32-bit shared addresses and registers split by role.
// P's low part: with n rows before the chunk, P's rounding enters a row's O as sqrt(rows / n) of the output's own, so it
// is kept for a sequence's first kLowChunks chunks, beyond which it adds less than a tenth to the output's rounding.  It
// stands in the columns of the T it comes from.
// TMEM columns: O 0 and 128 (K^T V), T 256, its q . z 384, P 400, sums of K and V 464 and 480, a first unit's q . z 496.
// ----------------------------------------------------------------------------------------------------------------

// Shared memory by 32-bit address.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts_f4(uint32_t a, float4 v) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void sts_f(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
// (No suspend time: with one of 20 us the waiting threads wake later, 65,536 tokens taking 176 us where they take 171.)
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int row, int head) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(m), "r"(bar), "r"(x), "r"(row), "r"(head)
        : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap *m, uint32_t src, int x, int row, int head) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m), "r"(src),
                 "r"(x), "r"(row), "r"(head)
                 : "memory");
}
// As tc::wait_or_abort: bounded in time, and over early once a role has given up.  `ab`: the CTA's AbortState.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, uint32_t ab, uint32_t *status, uint32_t where) {
    if (try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (try_wait(bar, parity)) return true;
        uint32_t gone;
        uint64_t limit;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gone) : "r"(ab) : "memory");
        if (gone) return false;
        asm volatile("ld.volatile.shared.u64 %0, [%1];" : "=l"(limit) : "r"(ab + 8) : "memory");
        if (globaltimer_ns() - t0 > limit) {
            asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(ab) : "memory");
            tc::report(status, kDevTimeout, where);
            return false;
        }
    }
}
// A last wait for something that is on its way, in a CTA that gives up.
__device__ __forceinline__ void wait_briefly(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!try_wait(bar, parity) && globaltimer_ns() - t0 < 50000000ull) {
    }
}

// As sdesc_sw128, at `off` bytes behind 16-byte unit s4 of shared memory: one addition.
__device__ __forceinline__ uint64_t desc_at(uint32_t s4, uint32_t off, uint32_t lbo, uint32_t sbo) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(s4 + (off >> 4) + (lbo >> 4 << 16)), "r"((sbo >> 4) | 1u << 14 | 2u << 29));
    return d;
}

constexpr int kThreads = 640;
// Registers: 640 threads start with 96 each; A, which holds S, takes what the others leave.
constexpr int kRegsFew = 72, kRegsA = 128, kRegsB = 72;
static_assert(128 * kRegsFew + 256 * kRegsA + 256 * kRegsB <= 640 * 96, "more registers than the block is launched with");
constexpr int kLowChunks = 4;

// Shared memory of the walk, from its base.
template <int NB> struct Walk {
    static constexpr uint32_t TILE = kTileB<NB>;
    static constexpr int NQ = NB == 2 ? 4 : 6;      // Q tiles
    // K's boxes, each followed by 8 rows of 128 bytes: rows z (two bf16 parts) and ones.  As rows 128 and 129 of K they
    // give T two columns of q . z; by themselves they are an N = 16 operand.  The products with the other rows are not
    // used, so rows 3-6 hold a (first box) and the first half's row sums (second box).
    static constexpr uint32_t KBOX = NB == 2 ? kBox + 1024 : kBox, ZT = kBox, ZBOX = NB == 2 ? KBOX : 1024;
    static constexpr uint32_t K = 0, V = TILE + 2048, Q = V + TILE;
    static constexpr uint32_t SB = Q + NQ * TILE;   // bf16 S, [d][e]
    static constexpr uint32_t A = ZT + 384, R0 = ZT + ZBOX + 384;
    static constexpr uint32_t R1 = SB + TILE;       // the second half's row sums
    static constexpr uint32_t BARS = R1 + 512;
    // barriers, 8 bytes each
    static constexpr uint32_t KFULL = BARS, KEMPTY = KFULL + 8, VFULL = KEMPTY + 8, VEMPTY = VFULL + 8;
    static constexpr uint32_t QFULL = VEMPTY + 8, QEMPTY = QFULL + 8 * NQ, T = QEMPTY + 8 * NQ, PREADY = T + 8;
    static constexpr uint32_t O = PREADY + 8, OFREE = O + 8, RFREE = OFREE + 16, S = RFREE + 8, SREADY = S + 8, ADONE = SREADY + 8;
    static constexpr uint32_t HALF = ADONE + 8, DRAIN = HALF + 16, TSLOT = DRAIN + 8, ABORT = TSLOT + 8;
    static constexpr size_t BYTES = ABORT + 16;
    static_assert(BYTES <= 232448, "shared-memory limit");
};

template <int NB>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ TcArgs P) {
    using W = Walk<NB>;
    constexpr uint32_t TILE = W::TILE;
    constexpr int NQ = W::NQ, CH = 32 * NB;  // CH: columns of O or S that an epilogue thread has
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    bool aligned;
    const uint32_t sm = smem_u32(tc::smem_base(smem_raw, P.A.status, &aligned)), ab = sm + W::ABORT;
    if (!aligned) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        auto init = [&](uint32_t at, uint32_t count) { mbar_init((uint64_t *)(smem_raw + at), count); };
        init(W::KFULL, 1);
        init(W::KEMPTY, 1);
        init(W::VFULL, 1);
        init(W::VEMPTY, 1);
        for (int k = 0; k < NQ; ++k) {
            init(W::QFULL + 8 * k, 1);
            init(W::QEMPTY + 8 * k, NB);
        }
        init(W::T, 1);
        init(W::PREADY, 256);
        init(W::O, 1);
        init(W::OFREE, 256);
        init(W::OFREE + 8, 256);
        init(W::RFREE, 256);
        init(W::S, 1);
        init(W::SREADY, 256);
        init(W::ADONE, 256);
        init(W::HALF, 128);
        init(W::HALF + 8, 128);
        init(W::DRAIN, 1);
        AbortState *st = (AbortState *)(smem_raw + W::ABORT);
        st->flag = 0;
        st->limit_ns = P.wait_ns ? P.wait_ns : tc::kWaitNs;
        fence_mbar_init();
    }
    for (int k = threadIdx.x; k < 512; k += kThreads)
        ((uint32_t *)(smem_raw + W::ZT + k / 256 * W::ZBOX))[k % 256] = (k % 256) / 32 == 2 ? 0x3F803F80u : 0u;
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc((uint32_t *)(smem_raw + W::TSLOT), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Before the carries are there: a kernel that waits for the sums has let this one start, so that the slices, and all
    // that was there before the sums, are.  Only A and B wait for it, A for its state and B before it writes.
    if (P.G == 1) griddep_wait();  // no carries: this one follows the sums
    griddep_launch_dependents();
    const uint32_t tmem = *(const uint32_t *)(smem_raw + W::TSLOT);
    const uint32_t tO = tmem, tT = tmem + 256, tX = tmem + 384, tP = tmem + 400, tZA = tmem + 464;
    // q . z of a chunk's first unit x
    auto tQZ = [&](int x) { return P.r == 1 && (x & 1) ? tX : tmem + 496; };
    uint32_t *status = P.A.status;
    const int VH = P.A.Hkv * P.gs;
    auto wait1 = [&](uint32_t bar, uint32_t parity, uint32_t where) { return wait_for(sm + bar, parity & 1, ab, status, where); };
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t where) {  // a warp gives up together
        return __all_sync(0xffffffffu, wait_for(sm + bar, parity & 1, ab, status, where)) != 0;
    };
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        if (warp == 0 && lane == 0) {
            // ---- K and V of the slice's chunk n
            prefetch_tmap(&P.tmK);
            prefetch_tmap(&P.tmV);
            int n = 0, kn = 0, vn = 0;  // chunks whose K, V have been asked for
            for (Units u(P); u.valid(); u.next(P, 1, VH), ++n) {
                const int row = u.lo + u.c * kC, h = u.vh / P.gs;
                if (n > 0 && !wait1(W::KEMPTY, n - 1, 0x801)) break;
                expect_bytes(sm + W::KFULL, TILE);
                for (int b = 0; b < NB; ++b) load_box(sm + W::K + b * W::KBOX, &P.tmK, sm + W::KFULL, 64 * b, row, h);
                ++kn;
                if (n > 0 && !wait1(W::VEMPTY, n - 1, 0x802)) break;
                expect_bytes(sm + W::VFULL, TILE);
                for (int b = 0; b < NB; ++b) load_box(sm + W::V + b * kBox, &P.tmV, sm + W::VFULL, 64 * b, row, h);
                ++vn;
            }
            // copies already issued land before the CTA exits
            if (kn > 0) wait_briefly(sm + W::KFULL, (kn - 1) & 1);
            if (vn > 0) wait_briefly(sm + W::VFULL, (vn - 1) & 1);
        } else if (warp == 2 && lane == 0) {
            // ---- Q: one tile a unit
            prefetch_tmap(&P.tmQ);
            int t = 0;
            for (Units u(P); u.valid(); u.next(P, P.r, VH), ++t) {
                const uint32_t x = t % NQ;
                if (t >= NQ && !wait1(W::QEMPTY + 8 * x, t / NQ - 1, 0x803)) break;
                if (t == P.drop && blockIdx.x == 0) continue;
                expect_bytes(sm + W::QFULL + 8 * x, TILE);
                for (int b = 0; b < NB; ++b)
                    load_box(sm + W::Q + x * TILE + b * kBox, &P.tmQ, sm + W::QFULL + 8 * x, 64 * b, u.lo + u.c * kC,
                             u.vh * P.r + u.j);
            }
            for (int k = t > NQ ? t - NQ : 0; k < t; ++k) wait_briefly(sm + W::QFULL + 8 * (k % NQ), (k / NQ) & 1);
        } else if (warp == 1 && lane == 0) {
            // ---- MMA
            constexpr uint32_t idT = idesc_bf16(128, 128, false, false), idTX = idesc_bf16(128, 144, false, false);
            constexpr uint32_t idO = idesc_bf16(128, 64 * NB, false, true), idS = idesc_bf16(128, 64 * NB, true, true);
            constexpr uint32_t idZ = idesc_bf16(128, 16, true, false), idQZ = idesc_bf16(128, 16, false, false);
            // D <= 64: rows 64-127 of S repeat rows 0-63 and are not read
            constexpr uint32_t lbo = NB == 2 ? kBox : 0, lboK = NB == 2 ? W::KBOX : 0;
            int n = 0, un = 0;                            // chunk and number of unit u
            uint32_t sx = sm >> 4;
            // T of unit x in chunk m
            auto issue_t = [&](bool fresh, int x, int m) {
                if (fresh && !wait1(W::KFULL, m, 0x804)) return false;
                if (!wait1(W::QFULL + 8 * (x % NQ), x / NQ, 0x805)) return false;
                tc_fence_after();
                const uint32_t qb = sx + (x % NQ) * (TILE >> 4), id = fresh ? idT : idTX;
#pragma unroll
                for (int k = 0; k < 4 * NB; ++k)
                    mma_ss(tT, desc_at(qb, W::Q + (k >> 2) * kBox + 32 * (k & 3), 16, 1024),
                           desc_at(sx, W::K + (k >> 2) * W::KBOX + 32 * (k & 3), 16, 1024), id, k > 0);
                commit(sm + W::T);
                return true;
            };
            // the chunk's K^T V, at its last unit x, where O of x + 1 is going to be; K is then done with
            auto issue_s = [&](bool wanted, int x) {
                if (wanted) {
                    if (x > 0 && !wait1(W::OFREE + 8 * ((x - 1) & 1), (x - 1) >> 1, 0x80a)) return false;
                    tc_fence_after();
                    const uint32_t tS = tO + 128 * ((x + 1) & 1);
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k) {
                        const uint64_t kd = desc_at(sx, W::K + 2048 * k, lboK, 1024);
                        const uint64_t vd = desc_at(sx, W::V + 2048 * k, lbo, 1024);
                        const uint64_t on = desc_at(sx, W::ZT + (k >> 2) * W::ZBOX + 32 * (k & 3), 16, 0);
                        mma_ss(tS, kd, vd, idS, k > 0);
                        mma_ss(tZA, kd, on, idZ, k > 0);
                        mma_ss(tZA + 16, vd, on, idZ, k > 0);
                    }
                    commit(sm + W::S);
                }
                commit(sm + W::KEMPTY);
                return true;
            };
            Units u(P);
            bool ok = u.valid() && issue_t(true, 0, 0), parts = false;
            while (ok) {
                asm volatile("" : "+r"(sx));  // descriptors are formed where they are used, not kept in registers
                const bool last = u.j == P.r - 1, first = u.j == 0, wanted = last && u.sums_wanted(P);
                const uint32_t ob = un & 1, tOu = tO + 128 * ob;
                if (first) {
                    parts = u.c < kLowChunks;
                    if (!wait1(W::SREADY, n, 0x807)) break;  // Sb is there, K^T V has been read
                }
                if (last && !first && !issue_s(wanted, un)) break;  // early, so that K is filled again in time
                if (un > 1 && !wait1(W::OFREE + 8 * ob, (un >> 1) - 1, 0x809)) break;
                tc_fence_after();
                const uint32_t qb = sx + (un % NQ) * (TILE >> 4);
#pragma unroll
                for (int k = 0; k < 4 * NB; ++k)
                    mma_ss(tOu, desc_at(qb, W::Q + (k >> 2) * kBox + 32 * (k & 3), 16, 1024),
                           desc_at(sx, W::SB + 2048 * k, lbo, 1024), idO, k > 0);
                if (first) {
                    const uint32_t tQ = tQZ(un);
#pragma unroll
                    for (int k = 0; k < 4 * NB; ++k)
                        mma_ss(tQ, desc_at(qb, W::Q + (k >> 2) * kBox + 32 * (k & 3), 16, 1024),
                               desc_at(sx, W::ZT + (k >> 2) * W::ZBOX + 32 * (k & 3), 16, 0), idQZ, k > 0);
                }
                u.next(P, P.r, VH);
                if (first && !wait1(W::VFULL, n, 0x806)) break;
                if (!wait1(W::PREADY, un, 0x808)) break;  // P is there, T may be overwritten
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kC / 16; ++k)
                    mma_ts(tOu, tP + 8 * k, desc_at(sx, W::V + 2048 * k, lbo, 1024), idO, 1u);
                if (parts) {
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        mma_ts(tOu, tT + 32 * (k >> 1) + 8 * (k & 1), desc_at(sx, W::V + 2048 * k, lbo, 1024), idO, 1u);
                }
                commit(sm + W::O);
                // behind A, which clears rows that are not the sequence's
                if (last && first && !issue_s(wanted, un)) break;
                if (!last && !issue_t(false, un + 1, n)) break;
                if (last) {
                    commit(sm + W::VEMPTY);
                    ++n;
                    if (u.valid() && !issue_t(true, un + 1, n)) break;
                }
                if (!u.valid()) break;
                ++un;
            }
            commit(sm + W::DRAIN);
            wait_briefly(sm + W::DRAIN, 0);
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsA));
        // ---- A: P and row sums, and C: the state.  Thread <-> row i of a chunk (of S: row d = i) and half hf of the
        // columns.
        const int q4 = warp & 3, hf = (warp - 4) >> 2, i = 32 * q4 + lane;
        const uint32_t lo = (uint32_t)(32 * q4) << 16;
        const int D = P.A.D, col0 = CH * hf;
        const bool has_row = NB == 2 || q4 < 2;          // rows of S there are
        float2 S[CH / 2];                                // S[i][col0 ...]
        float za = 0.f;                                  // z[i] (first half) or a[i] (second half)
        int ks = 0, m = 0, x = 0;                        // K^T V read, chunk, unit
        // The caller's S is loaded and stored by way of the warp's own part of Sb, half of its columns at a time, so
        // that neighbouring lanes have neighbouring columns.  (A lane to a row took 6 k clocks.)
        constexpr int GP = 4 * NB;                       // float4s of a row in a half
        auto staged = [&](int r, int g) {
            return sm + W::SB + (NB == 2 ? hf * kBox : 0) + tc::sw128_off(32 * q4 + r, (NB == 2 ? 0 : 4 * hf) + g);
        };
        Units u(P);
        griddep_wait();
        for (; u.valid(); ++x) {
            const bool parts = u.c < kLowChunks;
            if (x > 0 && !wait(W::O, x - 1, 0x812)) break;  // Q S and P V of the unit before have read Sb and P
            if (u.j == 0 && (x == 0 || u.c == 0)) {  // the state a piece starts from
#pragma unroll
                for (int k = 0; k < CH / 2; ++k) S[k] = make_float2(0.f, 0.f);
                const float *f = u.slot<NB>(P);
                za = 0.f;
                if (f) za = f[kSlotS<NB> + 128 * hf + i];
                else if (P.A.resume && i < D) za = (hf ? (const float *)P.A.a : (const float *)P.A.z)[u.state(P) * D + i];
                if (f && has_row) {
#pragma unroll
                    for (int q = 0; q < 8 * NB; ++q) {
                        const float4 v = ((const float4 *)f)[slot_at<NB>(i, hf, q)];
                        S[2 * q] = make_float2(v.x, v.y), S[2 * q + 1] = make_float2(v.z, v.w);
                    }
                } else if (!f && P.A.resume && has_row) {
                    const float *src = (const float *)P.A.S + (u.state(P) * D + 32 * q4) * D + col0;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
#pragma unroll
                        for (int y = lane; y < 32 * GP; y += 32) {
                            const int r = y / GP, g = y % GP, e = 4 * (GP * b + g);
                            if (32 * q4 + r < D && col0 + e < D) sts128(staged(r, g), *(const uint4 *)(src + r * D + e));
                        }
                        __syncwarp();
                        if (i < D && col0 + 4 * GP * b < D) {
#pragma unroll
                            for (int g = 0; g < GP; ++g) {
                                const float4 v = lds_f4(staged(lane, g));
                                S[2 * (GP * b + g)] = make_float2(v.x, v.y), S[2 * (GP * b + g) + 1] = make_float2(v.z, v.w);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (u.j == 0) {
                if (has_row) {
                    const uint32_t tile = sm + W::SB + (NB == 2 ? hf * kBox : 0);
#pragma unroll
                    for (int g = 0; g < CH / 8; ++g)
                        sts128(tile + tc::sw128_off(i, (NB == 2 ? 0 : 4 * hf) + g),
                               make_uint4(pack_bf16(S[4 * g].x, S[4 * g].y), pack_bf16(S[4 * g + 1].x, S[4 * g + 1].y),
                                          pack_bf16(S[4 * g + 2].x, S[4 * g + 2].y), pack_bf16(S[4 * g + 3].x, S[4 * g + 3].y)));
                }
                if (has_row && hf == 0) tc::split_tile_put(smem_raw + W::ZT + (i >> 6) * W::ZBOX, i & 63, za);
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(sm + W::SREADY);
                ++m;
            }
            if (!wait(W::T, x, 0x811)) break;
            tc_fence_after();
            float2 sum = make_float2(0.f, 0.f);
            uint32_t qz0 = 0u, qz1 = 0u;  // q . z, but for the first unit, whose T was formed before z was known
            if (u.j > 0 && hf == 0) {
                tmem_ld2(tX + lo, qz0, qz1);
                tmem_wait_ld(qz0, qz1);
            }
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                const int blk = 2 * hf + b;
                uint32_t hi[16];
                if (blk > q4) {  // above the diagonal
#pragma unroll
                    for (int k = 0; k < 16; ++k) hi[k] = 0u;
                    tmem_st16(tP + lo + 16 * blk, hi);
                    if (parts) tmem_st16(tT + lo + 32 * blk, hi);
                    continue;
                }
                uint32_t v[32];
                tmem_ld32(tT + lo + 32 * blk, v);
                tmem_wait_ld(v);
                if (blk == q4) {  // -1 where P is to be 0
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = k <= lane ? v[k] : 0xbf800000u;
                }
                float2 p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    p[k] = add2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), make_float2(1.f, 1.f));
                    hi[k] = pack_bf16(p[k].x, p[k].y);
                    sum = add2(sum, p[k]);
                }
                tmem_st16(tP + lo + 16 * blk, hi);
                if (parts) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) hi[k] = pack_bf16(p[k].x - tc::bf16lo(hi[k]), p[k].y - tc::bf16hi(hi[k]));
                    tmem_st16(tT + lo + 32 * blk, hi);  // over the T it came from
                }
            }
            if (u.j == 0 && u.live() < kC) {
                // the chunk reaches past its sequence: rows that are not its own must not enter P V and K^T V, where
                // a zero weight would not keep an infinity out
                if (!wait(W::VFULL, m - 1, 0x815)) break;
                if (!wait(W::KFULL, m - 1, 0x816)) break;
                const int none = u.live() > 0 ? u.live() : 0;
                for (int y = threadIdx.x - 128; y < (kC - none) * 8 * NB; y += 256) {
                    const int row = none + y / (8 * NB), g = y % (8 * NB);
                    const uint32_t at = sm + row * 128 + (g & 7) * 16;
                    sts128(at + W::K + (g >> 3) * W::KBOX, make_uint4(0u, 0u, 0u, 0u));
                    sts128(at + W::V + (g >> 3) * kBox, make_uint4(0u, 0u, 0u, 0u));
                }
                fence_proxy_async_smem();
            }
            if (x > 0 && !wait(W::RFREE, x - 1, 0x817)) break;  // B has read the row sums of the unit before
            if (u.j == 0) {
                if (m > 1 && !wait(W::ADONE, m - 2, 0x825)) break;  // and a of the chunk before
                if (hf && has_row) sts_f(sm + W::A + 4 * i, za);
            }
            sts_f(sm + (hf ? W::R1 : W::R0) + 4 * i, (sum.x + sum.y) + (__uint_as_float(qz0) + __uint_as_float(qz1)));
            tmem_st_wait();
            tc_fence_before();
            arrive(sm + W::PREADY);
            if (u.j == P.r - 1) {
                // C: the state after the chunk
                if (u.sums_wanted(P)) {
                    if (!wait(W::S, ks, 0x824)) break;
                    ++ks;
                    tc_fence_after();
                    if (has_row) {
                        uint32_t s0, s1;
                        tmem_ld2(tZA + lo + 16 * hf + 2, s0, s1);  // column 2: the ones
                        tmem_wait_ld(s0, s1);
                        za += __uint_as_float(s0);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            uint32_t v[32];
                            tmem_ld32(tO + 128 * ((x + 1) & 1) + lo + col0 + 32 * b, v);
                            tmem_wait_ld(v);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                S[16 * b + k] = add2(S[16 * b + k], make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])));
                        }
                    }
                    tc_fence_before();
                }
                if (u.saves(P)) {
                    if (i < D) (hf ? (float *)P.A.a : (float *)P.A.z)[u.state(P) * D + i] = za;
                    if (!wait(W::O, x, 0x826)) break;  // Q S has read Sb
                    float *dst = (float *)P.A.S + (u.state(P) * D + 32 * q4) * D + col0;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        if (!has_row) break;
#pragma unroll
                        for (int g = 0; g < GP; ++g) {
                            const float2 s0 = S[2 * (GP * b + g)], s1 = S[2 * (GP * b + g) + 1];
                            sts128(staged(lane, g), make_uint4(__float_as_uint(s0.x), __float_as_uint(s0.y), __float_as_uint(s1.x),
                                                               __float_as_uint(s1.y)));
                        }
                        __syncwarp();
#pragma unroll 1
                        for (int y = lane; y < 32 * GP; y += 32) {
                            const int r = y / GP, g = y % GP, e = 4 * (GP * b + g);
                            if (32 * q4 + r < D && col0 + e < D) *(uint4 *)(dst + r * D + e) = lds128(staged(r, g));
                        }
                        __syncwarp();
                    }
                }
            }
            u.next(P, P.r, VH);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsB));
        // ---- B: O -> out.  Thread <-> row i of a chunk and half hf of the columns.
        const int q4 = warp & 3, hf = (warp - 12) >> 2, i = 32 * q4 + lane;
        const uint32_t lo = (uint32_t)(32 * q4) << 16;
        const int D = P.A.D, col0 = CH * hf;
        const bool storer = lane == 0 && q4 == 0 && (NB == 2 || hf == 0);
        int n0 = 0;                                      // rows of the sequence before the first of this call
        int pending = -1;                                // Q tile whose O is on its way out (storer)
        int halves = 0, m = 0, x = 0;                    // m: chunk
        Units u(P);
        griddep_wait();
        for (; u.valid(); ++x) {
            if (u.j == 0 && (x == 0 || u.c == 0)) n0 = u.rows_before<NB>(P);
            if (pending >= 0) {  // the last unit's O has been read out of its Q tile, which may be filled again
                bulk_wait_read0();
                arrive(sm + W::QEMPTY + 8 * pending);
                pending = -1;
            }
            __syncwarp();
            if (!wait(W::O, x, 0x821)) break;
            tc_fence_after();
            uint32_t qz0 = 0u, qz1 = 0u;
            if (u.j == 0) {
                tmem_ld2(tQZ(x) + lo, qz0, qz1);
                tmem_wait_ld(qz0, qz1);
            }
            const float sc = 1.f / ((float)(n0 + u.c * kC) + (__uint_as_float(qz0) + __uint_as_float(qz1)) +
                                    (lds_f(sm + W::R0 + 4 * i) + lds_f(sm + W::R1 + 4 * i)));
            arrive(sm + W::RFREE);
            const int live = u.live();
            const uint32_t tile = sm + W::Q + (x % NQ) * TILE + (NB == 2 ? hf * kBox : 0);
#pragma unroll 1
            for (int b = 0; b < NB; ++b) {
                uint32_t v[32];
                tmem_ld32(tO + 128 * (x & 1) + lo + col0 + 32 * b, v);
                tmem_wait_ld(v);
                if (b == NB - 1) {  // O and q . z have been read
                    tc_fence_before();
                    arrive(sm + W::OFREE + 8 * (x & 1));
                }
                const uint32_t acol = sm + W::A + 4 * (col0 + 32 * b);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    uint32_t w[4];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float4 a = lds_f4(acol + 32 * y + 16 * c);
                        const uint32_t *o = v + 8 * y + 4 * c;
                        const float2 s0 = mul2(add2(make_float2(__uint_as_float(o[0]), __uint_as_float(o[1])), make_float2(a.x, a.y)),
                                               make_float2(sc, sc));
                        const float2 s1 = mul2(add2(make_float2(__uint_as_float(o[2]), __uint_as_float(o[3])), make_float2(a.z, a.w)),
                                               make_float2(sc, sc));
                        w[2 * c] = pack_bf16(s0.x, s0.y);
                        w[2 * c + 1] = pack_bf16(s1.x, s1.y);
                    }
                    const uint4 w4 = make_uint4(w[0], w[1], w[2], w[3]);
                    const int e = 32 * b + 8 * y;  // column within the thread's
                    sts128(tile + tc::sw128_off(i, (NB == 2 ? 0 : 4 * hf) + (e >> 3)), w4);
                }
            }
            const bool last = u.j == P.r - 1;
            if (last) arrive(sm + W::ADONE);  // a of this chunk has been read
            if (live < kC) {
                // rows of others stay as they are: the warp copies its own, a row's columns by neighbouring lanes
                constexpr int PER = CH / 8;
                __nv_bfloat16 *out = (__nv_bfloat16 *)P.A.o + (u.vh * P.r + u.j) * P.A.oh + (long long)(u.lo + u.c * kC) * P.A.on + col0;
                __syncwarp();
#pragma unroll 1
                for (int y = lane; y < 32 * PER; y += 32) {
                    const int row = 32 * q4 + y / PER, g = y % PER;
                    if (row < live && col0 + 8 * g < D)
                        *(uint4 *)(out + (long long)row * P.A.on + 8 * g) = lds128(tile + tc::sw128_off(row, (NB == 2 ? 0 : 4 * hf) + g));
                }
            }
            fence_proxy_async_smem();
            arrive(sm + W::HALF + 8 * hf);
            if (storer && wait1(W::HALF + 8 * hf, halves, 0x822) && (NB == 2 || wait1(W::HALF + 8, halves, 0x823))) {
                if (live == kC) {
                    store_box(&P.tmO, tile, NB == 2 ? col0 : 0, u.lo + u.c * kC, u.vh * P.r + u.j);
                    bulk_commit();
                    pending = x % NQ;
                } else {
                    arrive(sm + W::QEMPTY + 8 * (x % NQ));
                }
            }
            __syncwarp();
            ++halves;
            if (last) {
                // the head's n, which every thread of B has read
                if (u.saves(P)) {
                    if (!wait(W::ADONE, m, 0x825)) break;
                    if (hf == 0 && i == 0) P.A.n[u.state(P)] = n0 + u.len;
                }
                ++m;
            }
            u.next(P, P.r, VH);
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
                   cudaFuncSetAttribute(prompt_kernel<NB>, a, (int)Walk<NB>::BYTES) == cudaSuccess;
        }))
        return cudaErrorInvalidValue;
    P.slices = (Slice *)(ws + 256);
    P.sums = (float *)(ws + 256 + tc::kMaxCtas * 64);
    P.carry = P.sums + (size_t)P.G * kSlot<NB>;
    cudaError_t e = launch(sums_kernel<NB>, dim3(P.G), kSumThreads, kSmemSums<NB>, s, P);
    if (e == cudaSuccess && P.G > 1)
        e = launch(carry_kernel<NB>, dim3((kSlotS<NB> / 4 + 64 + kCarryThreads) / kCarryThreads, P.G < kCarryBlocks ? P.G : kCarryBlocks),
                   kCarryThreads, 0, s, P);
    if (e == cudaSuccess) e = launch(prompt_kernel<NB>, dim3(P.G), kThreads, Walk<NB>::BYTES, s, P);
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
    P.drop = -1;
    if (const char *env = getenv("LA_TEST_DROP_LOAD")) P.drop = atoi(env);
    if (A.T > 0 && (!head_map(&P.tmQ, enc, A.q, A.D, A.T, A.Hq, A.qh, A.qn) ||
                    !head_map(&P.tmK, enc, A.k, A.D, A.T, A.Hkv, A.kh, A.kn) ||
                    !head_map(&P.tmV, enc, A.v, A.D, A.T, A.Hkv, A.vh, A.vn) ||
                    !head_map(&P.tmO, enc, A.o, A.D, A.T, A.Hq, A.oh, A.on)))
        return cudaErrorInvalidValue;
    return A.D > 64 ? run<2>(P, ws, s) : run<1>(P, ws, s);
}

}  // namespace prompt
}  // namespace la
