// Small requests of a chunk-attention call, before and after the decode kernel
// that attends them in the latent space:
//   q_latent[slot][h] = (q_nope W_UK[h], q_rope)      [512 + 64], rounded to bf16,
//   out[row][h]       = latent[slot][h] W_UV[h]       [128].
// A slot is a token's place in its group (group g holds slots g t .. g t + t - 1,
// t tokens a full group); slots without a token are left out. Per head these are
// products over all slots, [slots x 128] x [128 x 512] and [slots x 512] x
// [512 x 128], bound by reading the weights (256 KB a head) for the few hundred
// slots of a step: one block per (head, 128 slots), one pass over the weights. With
// about 600 slots of 16 heads they take 11 and 7.6 us beside 40 us of the decode; in a
// call that turns out to have no small request, the path's four launches cost 10 to 13.
#include <cuda_bf16.h>

#include "../../include/mla_decode.h"
#include "ptx_prefill.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = 128 * 128;  // [128 rows][64 columns] of bf16, swizzled

// The token of a slot, or false.
__device__ __forceinline__ bool slot_token(const PrefillArgs& a, int slot, int num_groups, int* row) {
  const int t = a.lay.group_tokens, g = slot / t, i = slot - g * t;
  if (g >= num_groups) return false;
  const PfGroup& group = reinterpret_cast<const PfGroup*>(a.ws + a.lay.groups)[g];
  *row = group.q_row + i;
  return i < group.tokens;
}

constexpr int kQOffB = 2 * kChunk;             // A: 128 slots x 128 dims; B: W_UK[h], 8 chunks of 64 columns
constexpr int kQOffBar = kQOffB + 8 * kChunk;
constexpr int kQSmem = kQOffBar + 64 + 1024;

__global__ void __launch_bounds__(kThreads, 1)
    prefill_q_latent_kernel(const __grid_constant__ CUtensorMap w_uk, const __grid_constant__ PrefillArgs a,
                            const uint4* __restrict__ q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem), full = sbase + kQOffBar, done = full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kQOffBar + 16);
  const int tid = threadIdx.x, warp = tid >> 5;
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const int h = blockIdx.x, slot = blockIdx.y * 128 + tid, heads = a.num_heads;
  pdl_launch_dependents();
  pdl_wait();
  const int num_groups = hd->num_groups;
  {  // page lists of the groups, for the decode kernel: their rows lie one after the other
    const PfGroup* groups = reinterpret_cast<const PfGroup*>(a.ws + a.lay.groups);
    int32_t* pages = reinterpret_cast<int32_t*>(a.ws + a.lay.group_pages);
    const int warps = kThreads / 32, first = blockIdx.y * gridDim.x + blockIdx.x;
    for (int g = first * warps + warp; g < num_groups; g += gridDim.x * gridDim.y * warps) {
      const PfGroup p = groups[g];
      for (int j = tid & 31; j < p.pages; j += 32) pages[p.page0 + j] = p.base / kBlockTokens + j;
    }
  }
  if (blockIdx.y * 128 >= num_groups * a.lay.group_tokens) return;
  if (tid == 0) {
    mbar_init(full, 1);
    mbar_init(done, 1);
    fence_mbar_init_cluster();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) {
    mbar_arrive_expect_tx(full, 8 * kChunk);
    for (int c = 0; c < 8; ++c)
      for (int k = 0; k < 2; ++k)
        tma_load_2d(sbase + kQOffB + c * kChunk + k * (kChunk / 2), &w_uk, full, 64 * c, h * kDimNope + 64 * k);
  }
  // A row a thread: 256 bytes into the swizzled layout.
  int row = 0;
  const bool valid = slot_token(a, slot, num_groups, &row);
  const uint4* src = q + (static_cast<int64_t>(row) * heads + h) * (kDimQk * 2 / 16);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (valid) v = src[j];
    st_shared_v4(sbase + (j >> 3) * kChunk + tid * 128 + (((j & 7) ^ (tid & 7)) << 4), v.x, v.y, v.z, v.w);
  }
  fence_proxy_async_smem();
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  if (tid == 0) {
    constexpr uint32_t idesc = idesc_bf16(128, 256, false, true);
    if (mbar_wait(full, 0, nullptr)) {
      tc_fence_after();
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ss(tmem + 256 * half, sdesc_sw128(sbase + (k >> 2) * kChunk + (k & 3) * 32, 16, 1024),
                      sdesc_sw128(sbase + kQOffB + 4 * half * kChunk + k * 2048, kChunk, 1024), idesc, k != 0);
      mma_commit(done);
    }
  }
  __syncwarp();
  const bool ready = __all_sync(0xffffffffu, mbar_wait(done, 0, nullptr));
  tc_fence_after();
  if (!ready && (tid & 31) == 0) atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  if (ready) {
    uint8_t* dst = a.ws + a.lay.q_latent + (static_cast<int64_t>(slot) * heads + h) * (kDimRow * 2);
#pragma unroll 1
    for (int c = 0; c < 16; ++c) {
      uint32_t r[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 32 * c, r);
      tmem_wait_ld();
      if (valid) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(r[16 * v + 2 * i]), __uint_as_float(r[16 * v + 2 * i + 1]));
          st_global_v8(dst + 64 * c + 32 * v, pk);
        }
      }
    }
    if (valid)
      for (int j = 0; j < 8; ++j) reinterpret_cast<uint4*>(dst + kDimCkv * 2)[j] = src[16 + j];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

constexpr int kStages = 6;
constexpr int kVStage = 2 * kChunk;  // 64 of the 512 dims: [128 slots][64], W_UV [64][2 x 64]
constexpr int kVOffBar = kStages * kVStage;
constexpr int kVSmem = kVOffBar + 256 + 1024;

__global__ void __launch_bounds__(kThreads, 1)
    prefill_v_latent_kernel(const __grid_constant__ CUtensorMap latent, const __grid_constant__ CUtensorMap w_uv,
                            const __grid_constant__ PrefillArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem), bar0 = sbase + kVOffBar;
  auto full = [&](int s) -> uint32_t { return bar0 + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return bar0 + 8u * (kStages + s); };
  const uint32_t done = bar0 + 8u * (2 * kStages);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kVOffBar + 8 * (2 * kStages + 1));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const int h = blockIdx.x, slot0 = blockIdx.y * 128, heads = a.num_heads;
  pdl_launch_dependents();
  pdl_wait();
  const int num_groups = hd->num_groups;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    const int bits = reinterpret_cast<const WsHeader*>(a.ws + a.lay.decode)->status;  // (of the decode kernel)
    if (bits) atomicOr(&hd->status, bits);
  }
  if (slot0 >= num_groups * a.lay.group_tokens) return;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr int kSteps = kDimCkv / 64;
  // A wait that runs out stops its loop; the epilogue's own wait reports it.
  if (warp == 0 && lane == 0) {
    for (int k = 0; k < kSteps; ++k) {
      const int s = k % kStages;
      if (k >= kStages && !mbar_wait(empty(s), ((k / kStages) & 1) ^ 1, nullptr)) break;
      const uint32_t dst = sbase + s * kVStage;
      mbar_arrive_expect_tx(full(s), kVStage);
      tma_load_3d(dst, &latent, full(s), 64 * k, h, slot0);
      tma_load_2d(dst + kChunk, &w_uv, full(s), 0, h * kDimCkv + 64 * k);
      tma_load_2d(dst + kChunk + kChunk / 2, &w_uv, full(s), 64, h * kDimCkv + 64 * k);
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_bf16(128, 128, false, true);
    for (int k = 0; k < kSteps; ++k) {
      const int s = k % kStages;
      if (!mbar_wait(full(s), (k / kStages) & 1, nullptr)) break;
      tc_fence_after();
      const uint32_t st = sbase + s * kVStage;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_bf16_ss(tmem, sdesc_sw128(st + i * 32, 16, 1024), sdesc_sw128(st + kChunk + i * 2048, kChunk / 2, 1024), idesc,
                    (k | i) != 0);
      mma_commit(empty(s));
      if (k == kSteps - 1) mma_commit(done);
    }
  }
  __syncwarp();
  const bool ready = __all_sync(0xffffffffu, mbar_wait(done, 0, nullptr));
  tc_fence_after();
  if (!ready && lane == 0) atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  int row = 0;
  const bool valid = slot_token(a, slot0 + tid, num_groups, &row);
  const int64_t out_row = static_cast<int64_t>(row) * heads + h;
  if (ready) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t r[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 32 * c, r);
      tmem_wait_ld();
      if (valid) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(r[16 * v + 2 * i]), __uint_as_float(r[16 * v + 2 * i + 1]));
          st_global_v8(static_cast<uint8_t*>(a.out) + out_row * (kDimV * 2) + 64 * c + 32 * v, pk);
        }
      }
    }
    if (a.lse && valid)
      a.lse[out_row] = reinterpret_cast<const float*>(a.ws + a.lay.latent_lse)[static_cast<int64_t>(slot0 + tid) * heads + h];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 128);
}

dim3 slots_grid(const PrefillArgs& a) {
  return dim3(a.num_heads, (a.lay.max_groups * a.lay.group_tokens + 127) / 128);
}

}  // namespace

cudaError_t launch_prefill_q_latent(const CUtensorMap& w_uk, const PrefillArgs& a, const void* q, cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(prefill_q_latent_kernel, kQSmem, attr_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_q_latent_kernel, slots_grid(a), dim3(kThreads), kQSmem, stream, w_uk, a,
                    static_cast<const uint4*>(q));
}

cudaError_t launch_prefill_v_latent(const CUtensorMap& latent, const CUtensorMap& w_uv, const PrefillArgs& a,
                                    cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(prefill_v_latent_kernel, kVSmem, attr_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_v_latent_kernel, slots_grid(a), dim3(kThreads), kVSmem, stream, latent, w_uv, a);
}

}  // namespace mla
