// tb_layernorm.cuh -- what the layer norm's forward and backward kernels
// share: a row's threads, their sums and barrier.
#pragma once

#include "tb_elem.cuh"

namespace tb {

// Threads per CTA: a row's threads, at least eight warps.
__host__ __device__ constexpr int ln_block(int tpr) { return tpr < 256 ? 256 : tpr; }
// Threads of the one CTA that takes a row too long for registers.
constexpr int LONG_BLOCK = 1024;

// Waits for the TPR threads of one row (row group rl of the CTA).
template <int TPR, int BLOCK>
__device__ __forceinline__ void row_barrier(int rl) {
    if constexpr (TPR == BLOCK) {
        __syncthreads();
    } else {
        asm volatile("bar.sync %0, %1;" ::"r"(rl + 1), "n"(TPR) : "memory");
    }
}

// Sum over the TPR threads of a row; every thread gets the result.  `slots`
// (one float per warp of the CTA) must not be reused before another barrier.
template <int TPR, int BLOCK>
__device__ __forceinline__ float row_sum(float v, float* slots, int rl) {
    constexpr int HOLD = TPR < 32 ? TPR : 32;  // lanes of a warp in one row
#pragma unroll
    for (int d = HOLD / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
        row_barrier<TPR, BLOCK>(rl);
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) v += slots[rl * (TPR / 32) + w];
    }
    return v;
}

}  // namespace tb
