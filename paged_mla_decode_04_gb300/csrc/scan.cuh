// Prefix sums over a block, several 64-bit values at a time.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mla {

// Exclusive prefix sums over the block of kN 64-bit values; total[] receives the
// block's sums. `sh`: 32 * kN values of shared memory. Two barriers.
template <int kN>
__device__ __forceinline__ void block_scan(int64_t (&v)[kN], int64_t (&total)[kN], int64_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t own[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) own[i] = v[i];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v[i], d);
      if (lane >= d) v[i] += u;
    }
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < kN; ++i) sh[32 * i + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {  // every warp scans the warps' sums
    int64_t w = lane < warps ? sh[32 * i + lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += u;
    }
    total[i] = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    v[i] += (warp > 0 ? before : 0) - own[i];
  }
  __syncthreads();
}

}  // namespace mla
