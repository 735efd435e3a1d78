// la_prompt.h -- what the two forms of la_prompt share: parameters, the check of the offsets.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace prompt {

struct Args {
    const void *q, *k, *v;
    void *o;
    const int *off;                     // [nseq + 1], device
    void *S, *z, *a;                    // [nseq, Hkv, ...] of the accumulator type, or null
    int *n;                             // [nseq, Hkv]
    int resume;
    int T, nseq, Hq, Hkv, r, D;
    long long qh, qn, kh, kn, vh, vn, oh, on;  // head and row strides in elements
    uint32_t *status;                   // workspace status word
};

// Whether the offsets run in order within [0, T]; the same answer for every thread of a block, which all call it.
// Sequences out of order would read and write rows that are not there or that others write.
__device__ __forceinline__ bool offsets_in_order(const Args &A) {
    int bad = 0;
    for (int i = threadIdx.x; i < A.nseq; i += blockDim.x) {
        const int lo = A.off[i], hi = A.off[i + 1];
        bad |= lo < 0 || hi < lo || hi > A.T;
    }
    bad = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0)
        tc::report(A.status, kDevBounds, 0x0FF5u);
    return !bad;
}

bool tc_supported(int D, int dtype);  // the tensor-core form: bf16, D = 32, 64, 128
size_t tc_workspace_bytes(int T, int nseq, int Hkv, int r, int D);
cudaError_t tensor_cores(const Args &A, unsigned char *ws, cudaStream_t s);  // T > 0
cudaError_t simt(const Args &A, int dtype, cudaStream_t s);  // T > 0, what tensor_cores() does not do

}  // namespace prompt
}  // namespace la
