// scan.cuh -- exclusive scan over the threads of one CTA, for the kernels that turn counts into
// places (page lists, work lists).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pha {

// Exclusive prefix of v over the NT threads of the CTA (in thread order) and the total. sums: NT /
// 32 values of shared scratch, free again on return. Every thread of the CTA calls it.
template <int NT, typename T>
__device__ __forceinline__ T cta_exclusive_scan(T v, T* sums, T& total) {
    static_assert(NT % 32 == 0 && NT <= 1024, "whole warps, one warp of warp sums");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const T s = sums[w];
        before += w < warp ? s : 0;
        all += s;
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

}  // namespace pha
