// Small requests of a chunk-attention call, before and after the decode kernel
// that attends them in the latent space:
//   q_latent[slot][h] = (q_nope W_UK[h], q_rope)      [512 + 64], rounded to bf16,
//   out[row][h]       = latent[slot][h] W_UV[h]       [128].
// The decode leaves every item's sums in fp32 (one rounding of the result to bf16, not
// two), which a kernel between joins, weighed by their lse, into a pair of bf16 rows,
// the value and what rounding took from it: both are multiplied.
// A slot is a token's place in its pair of groups (pair g holds slots g t .. g t + t - 1,
// t tokens a full group); slots without a token are left out. The query is stored
// twice, rounded one way and the other (see PfGroup). Per head these are
// products over all slots, [slots x 128] x [128 x 512] and [slots x 512] x
// [512 x 128], bound by reading the weights (256 KB a head) for the few hundred
// slots of a step: one or two blocks per (head, 128 slots), one pass over the weights.
// For the small requests of a step of 24 mixed ones, 16 heads, they take 11 and 9 us, the
// join 7, the decode between 60; in a call that turns out to have no small request, the
// path's four launches cost 10 to 13.
#include <cuda_bf16.h>
#include <math_constants.h>

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
  if (2 * g >= num_groups) return false;
  const PfGroup& group = reinterpret_cast<const PfGroup*>(a.ws + a.lay.groups)[2 * g];
  *row = group.q_row + i;
  return i < group.tokens;
}

constexpr int kQOffB = 2 * kChunk;             // A: 128 slots x 128 dims; B: half of W_UK[h], 4 chunks of 64 columns
constexpr int kQOffBar = kQOffB + 4 * kChunk;
constexpr int kQSmem = kQOffBar + 64 + 1024;

// Half of the 512 columns a block: a step's slots are too few to fill the GPU.
__global__ void __launch_bounds__(kThreads, 1)
    prefill_q_latent_kernel(const __grid_constant__ CUtensorMap w_uk, const __grid_constant__ PrefillArgs a,
                            const uint4* __restrict__ q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem), full = sbase + kQOffBar, done = full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kQOffBar + 16);
  const int tid = threadIdx.x, warp = tid >> 5;
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const int h = blockIdx.x >> 1, half = blockIdx.x & 1, slot = blockIdx.y * 128 + tid, heads = a.num_heads;
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
  if (blockIdx.y * 128 >= num_groups / 2 * a.lay.group_tokens) return;
  if (tid == 0) {
    mbar_init(full, 1);
    mbar_init(done, 1);
    fence_mbar_init_cluster();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(tmem_slot), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) {
    mbar_arrive_expect_tx(full, 4 * kChunk);
    for (int c = 0; c < 4; ++c)
      for (int k = 0; k < 2; ++k)
        tma_load_2d(sbase + kQOffB + c * kChunk + k * (kChunk / 2), &w_uk, full, 256 * half + 64 * c, h * kDimNope + 64 * k);
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
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_bf16_ss(tmem, sdesc_sw128(sbase + (k >> 2) * kChunk + (k & 3) * 32, 16, 1024),
                    sdesc_sw128(sbase + kQOffB + k * 2048, kChunk, 1024), idesc, k != 0);
      mma_commit(done);
    }
  }
  __syncwarp();
  const bool ready = __all_sync(0xffffffffu, mbar_wait(done, 0, nullptr));
  tc_fence_after();
  if (!ready && (tid & 31) == 0) atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  if (ready) {
    const int t = a.lay.group_tokens, first = slot + slot / t * t;  // the slot's place in the pair's first group
    uint8_t* dst = a.ws + a.lay.q_latent + (static_cast<int64_t>(first) * heads + h) * (kDimRow * 2) + 512 * half;
    uint8_t* dst2 = dst + static_cast<int64_t>(t) * heads * (kDimRow * 2);
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      uint32_t r[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 32 * c, r);
      tmem_wait_ld();
      if (valid) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint32_t pk[8], other[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = __uint_as_float(r[16 * v + 2 * i]), y = __uint_as_float(r[16 * v + 2 * i + 1]);
            pk[i] = pack_bf16x2(x, y);
            other[i] = pack_bf16x2(2.f * x - __uint_as_float(pk[i] << 16), 2.f * y - __uint_as_float(pk[i] & 0xffff0000u));
          }
          st_global_v8(dst + 64 * c + 32 * v, pk);
          st_global_v8(dst2 + 64 * c + 32 * v, other);
        }
      }
    }
    if (valid && half)
      for (int j = 0; j < 8; ++j)
        reinterpret_cast<uint4*>(dst + 512)[j] = reinterpret_cast<uint4*>(dst2 + 512)[j] = src[16 + j];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 256);
}

// A warp joins the partial sums of one (slot, head), 16 dims a lane.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(32 * kJoinWarps) prefill_latent_kernel(const PrefillArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const PfHeader* hd = reinterpret_cast<const PfHeader*>(a.ws);
  const int lane = threadIdx.x & 31, heads = a.num_heads;
  const PfGroup* groups = reinterpret_cast<const PfGroup*>(a.ws + a.lay.groups);
  const float* lses = reinterpret_cast<const float*>(a.ws + a.lay.decode + a.lay.decode_lay.partial_lse);
  const float4* sums = reinterpret_cast<const float4*>(a.ws + a.lay.decode + a.lay.decode_lay.partial_o);
  uint2* out = reinterpret_cast<uint2*>(a.ws + a.lay.latent);
  const int64_t rest = static_cast<int64_t>(a.lay.max_pairs) * kGroupRows * (kDimCkv / 4);  // of a row's remainder, in uint2
  const int rows = hd->num_groups / 2 * kGroupRows;
  for (int r = blockIdx.x * kJoinWarps + (threadIdx.x >> 5); r < rows; r += gridDim.x * kJoinWarps) {
    const int row = r % kGroupRows, token = row / heads;  // of the group
    const PfGroup g = groups[2 * (r / kGroupRows)];
    if (token >= g.tokens) continue;
    const int items = g.items + groups[2 * (r / kGroupRows) + 1].items;  // (the pair's lie one after the other)
    const int64_t first = static_cast<int64_t>(g.first_item) * kGroupRows + row;
    float m = -3e38f;
    for (int p = 0; p < items; ++p) m = fmaxf(m, lses[first + static_cast<int64_t>(p) * kGroupRows]);
    float4 o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int p = 0; p < items; ++p) {
      const int64_t at = first + static_cast<int64_t>(p) * kGroupRows;
      const float lse = lses[at];
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = sums[at * (kDimCkv / 4) + lane + 32 * j];
      const float w = exp2f(lse - m);  // 0 (of zeros) where the row has no position in the item; NaN sums stay NaN
      l += w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j].x = fmaf(w, v[j].x, o[j].x);
        o[j].y = fmaf(w, v[j].y, o[j].y);
        o[j].z = fmaf(w, v[j].z, o[j].z);
        o[j].w = fmaf(w, v[j].w, o[j].w);
      }
    }
    const float inv = 1.f / l;
    auto rounded = [](float x) { return __bfloat162float(__float2bfloat16_rn(x)); };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x[4] = {o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv};
      const int64_t at = static_cast<int64_t>(r) * (kDimCkv / 4) + lane + 32 * j;
      out[at] = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      out[rest + at] = make_uint2(pack_bf16x2(x[0] - rounded(x[0]), x[1] - rounded(x[1])),
                                  pack_bf16x2(x[2] - rounded(x[2]), x[3] - rounded(x[3])));
    }
    if (a.lse && lane == 0)  // (a row without a NaN attends itself: l > 0)
      a.lse[(static_cast<int64_t>(g.q_row) + token) * heads + row % heads] =
          l > 0.f && o[0].x == o[0].x ? (m + log2f(l) - 1.f) * 0.69314718055994531f : CUDART_NAN_F;
  }
}

constexpr int kStages = 4;
constexpr int kVStage = 3 * kChunk;  // 64 of the 512 dims: [128 slots][64] twice, W_UV [64][2 x 64]
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
  if (slot0 >= num_groups / 2 * a.lay.group_tokens) return;
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
      tma_load_3d(dst + kChunk, &latent, full(s), 64 * k, h, a.lay.max_pairs * a.lay.group_tokens + slot0);
      tma_load_2d(dst + 2 * kChunk, &w_uv, full(s), 0, h * kDimCkv + 64 * k);
      tma_load_2d(dst + 2 * kChunk + kChunk / 2, &w_uv, full(s), 64, h * kDimCkv + 64 * k);
    }
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = idesc_bf16(128, 128, false, true);
    for (int k = 0; k < kSteps; ++k) {
      const int s = k % kStages;
      if (!mbar_wait(full(s), (k / kStages) & 1, nullptr)) break;
      tc_fence_after();
      const uint32_t st = sbase + s * kVStage;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        mma_bf16_ss(tmem, sdesc_sw128(st + (i >> 2) * kChunk + (i & 3) * 32, 16, 1024),
                    sdesc_sw128(st + 2 * kChunk + (i & 3) * 2048, kChunk / 2, 1024), idesc, (k | i) != 0);
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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 128);
}

dim3 slots_grid(const PrefillArgs& a, int blocks_a_head) {
  return dim3(a.num_heads * blocks_a_head, (a.lay.max_pairs * a.lay.group_tokens + 127) / 128);
}

}  // namespace

cudaError_t launch_prefill_q_latent(const CUtensorMap& w_uk, const PrefillArgs& a, const void* q, cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(prefill_q_latent_kernel, kQSmem, attr_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_q_latent_kernel, slots_grid(a, 2), dim3(kThreads), kQSmem, stream, w_uk, a,
                    static_cast<const uint4*>(q));
}

cudaError_t launch_prefill_latent(const PrefillArgs& a, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(a.lay.max_pairs) * (kGroupRows / kJoinWarps);
  return launch_pdl(prefill_latent_kernel, dim3(static_cast<unsigned>(most < 152 * 4 ? most : 152 * 4)), dim3(32 * kJoinWarps),
                    0, stream, a);
}

cudaError_t launch_prefill_v_latent(const CUtensorMap& latent, const CUtensorMap& w_uv, const PrefillArgs& a,
                                    cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(prefill_v_latent_kernel, kVSmem, attr_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_v_latent_kernel, slots_grid(a, 1), dim3(kThreads), kVSmem, stream, latent, w_uv, a);
}

}  // namespace mla
