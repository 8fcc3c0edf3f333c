// Exclusive scan of one int per thread over a CTA of 1024 threads.
#pragma once

#include <cuda_runtime.h>

constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;    // one warp's lanes scan the warps' sums

// `warp_sum` is shared scratch of kScanWarps ints; `total` receives the CTA's sum.
__device__ __forceinline__ int cta_scan(int x, int* warp_sum, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    __syncthreads();                       // the previous scan's readers are done
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int w = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp > 0 ? before : 0) + incl - x;
}
