// Prefix sums over a block, several 64-bit values at a time.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mla {

// Exclusive prefix sums over the block of kN 64-bit values; total[] receives the
// block's sums. `sh`: 32 * kN values of shared memory. Three barriers. (Shuffles pass
// one a cycle, so the warps' sums are scanned by one warp a value, not by all.)
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
  for (int i = warp; i < kN; i += warps) {
    int64_t w = lane < warps ? sh[32 * i + lane] : 0;
    for (int d = 1; d < warps; d <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += u;
    }
    sh[32 * i + lane] = w;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    total[i] = sh[32 * i + warps - 1];
    v[i] += (warp > 0 ? sh[32 * i + warp - 1] : 0) - own[i];
  }
  __syncthreads();
}

}  // namespace mla
