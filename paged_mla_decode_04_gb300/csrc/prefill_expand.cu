// Keys and values of the gathered rows, for every head h of a pass:
//   K[h][t][0:128] = c_kv[t] W_UK[h]^T,   V[h][t][0:128] = c_kv[t] W_UV[h],
// a product of [rows x 512] with [512 x 256] per head, rounded to bf16 (the
// precision at which models keep K and V; attention multiplies them in bf16).
//
// A persistent block per SM takes tiles of 128 rows x one head: both halves
// accumulate side by side in 256 TMEM columns (K in the first 128, V in the
// others), two such accumulators alternate, so the epilogue of one tile runs
// under the products of the next. Operands come by TMA in chunks of 64 of the
// 512 dims: rows (K-major), W_UK (K-major) and W_UV (MN-major), 48 KB a stage.
// Heads vary fastest over the blocks: a row block is then read by neighbours
// at the same time and the weights stay in L2.
#include <cuda_bf16.h>

#include "../../include/mla_decode.h"
#include "ptx_prefill.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kStages = 4;
constexpr int kChunk = 64;
constexpr int kChunks = kDimCkv / kChunk;          // 8
constexpr int kABytes = 128 * kChunk * 2;          // [128 rows][64 dims]
constexpr int kUkBytes = kDimNope * kChunk * 2;    // [128 key dims][64 dims]
constexpr int kUvBytes = kChunk * 64 * 2;          // [64 dims][64 value dims], two of them
constexpr int kStageBytes = kABytes + kUkBytes + 2 * kUvBytes;
constexpr int kOffBar = kStages * kStageBytes;
constexpr int kSmemBytes = kOffBar + 256 + 1024;
constexpr int kThreads = 192;  // producer, issuer, four epilogue warps

enum { kBarFull = 0, kBarEmpty = kStages, kBarAccFull = 2 * kStages, kBarAccFree = kBarAccFull + 2, kBarDrain = kBarAccFree + 2, kNumBars };

__global__ void __launch_bounds__(kThreads, 1)
    prefill_expand_kernel(const __grid_constant__ PrefillMaps m, const __grid_constant__ PrefillArgs a, int head0, int heads) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 8 * kNumBars + 4);
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kBarAccFull + s), 1);
      mbar_init(bar(kBarAccFree + s), 128);
    }
    mbar_init(bar(kBarDrain), 1);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) hd->next_item = 0;  // for the attention that follows
  const int row_blocks = (hd->kv_rows + 127) / 128;
  const int64_t tiles = static_cast<int64_t>(row_blocks) * heads;
  auto fail = [&] {
    *abort_flag = 1;
    atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t k = 0;  // chunks issued
      bool ok = true;
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const int head = head0 + static_cast<int>(t % heads), row = static_cast<int>(t / heads) * 128;
        for (int c = 0; c < kChunks; ++c, ++k) {
          const uint32_t s = k % kStages, use = k / kStages;
          if (!(ok = mbar_wait(bar(kBarEmpty + s), (use & 1u) ^ 1u, abort_flag))) break;
          const uint32_t dst = sbase + s * kStageBytes, fb = bar(kBarFull + s);
          mbar_arrive_expect_tx(fb, kStageBytes);
          tma_load_2d(dst, &m.rows, fb, c * kChunk, row);
          tma_load_2d(dst + kABytes, &m.w_uk, fb, c * kChunk, head * kDimNope);
          tma_load_2d(dst + kABytes + kUkBytes, &m.w_uv, fb, 0, head * kDimCkv + c * kChunk);
          tma_load_2d(dst + kABytes + kUkBytes + kUvBytes, &m.w_uv, fb, 64, head * kDimCkv + c * kChunk);
        }
      }
      if (!ok) fail();
      if (*abort_flag)  // let the copies in flight land (each wait bounded)
        for (uint32_t i = k > kStages ? k - kStages : 0; i < k; ++i)
          mbar_wait(bar(kBarFull + i % kStages), (i / kStages) & 1u, nullptr);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc_k = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_v = idesc_bf16(128, 128, false, true);
      uint32_t k = 0, n = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++n) {
        const uint32_t acc = n & 1u;
        if (!(ok = mbar_wait(bar(kBarAccFree + acc), ((n >> 1) & 1u) ^ 1u, abort_flag))) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * 256;
        for (int c = 0; c < kChunks; ++c, ++k) {
          const uint32_t s = k % kStages;
          if (!(ok = mbar_wait(bar(kBarFull + s), (k / kStages) & 1u, abort_flag))) break;
          tc_fence_after();
          const uint32_t st = sbase + s * kStageBytes;
#pragma unroll
          for (int i = 0; i < kChunk / 16; ++i) {
            const uint64_t ad = sdesc_sw128(st + i * 32, 16, 1024);
            mma_bf16_ss(d, ad, sdesc_sw128(st + kABytes + i * 32, 16, 1024), idesc_k, (c | i) != 0);
            mma_bf16_ss(d + 128, ad, sdesc_sw128(st + kABytes + kUkBytes + i * 16 * 128, kUvBytes, 1024), idesc_v,
                        (c | i) != 0);
          }
          mma_commit(bar(kBarEmpty + s));
        }
        if (ok) mma_commit(bar(kBarAccFull + acc));
      }
      if (!ok) fail();
      mma_commit(bar(kBarDrain));
      mbar_wait(bar(kBarDrain), 0, nullptr);
    }
  } else {
    const int quarter = warp & 3;
    const int row_in = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t n = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
      const uint32_t acc = n & 1u;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarAccFull + acc), (n >> 1) & 1u, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const int64_t row = (t / heads) * 128 + row_in;
      const int64_t out_row = (t % heads) * a.lay.kv_capacity + row;
      // Rows of the buffer are a multiple of 128: every row of a tile has its place.
#pragma unroll
      for (int c = 0; c < 4; ++c) {  // 64 columns each: K, K, V, V
        uint32_t r[64];
        tmem_ld32(tmem + lane_base + acc * 256 + c * 64, r);
        tmem_ld32(tmem + lane_base + acc * 256 + c * 64 + 32, r + 32);
        tmem_wait_ld();
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.ws + (c < 2 ? a.lay.keys : a.lay.values)) +
                             out_row * 128 + (c & 1) * 64;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(r[16 * v + 2 * i]), __uint_as_float(r[16 * v + 2 * i + 1]));
          st_global_v8(dst + v * 16, pk);
        }
      }
      tc_fence_before();
      mbar_arrive(bar(kBarAccFree + acc));
    }
    if (!ok) fail();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_prefill_expand(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(prefill_expand_kernel, kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t most = a.lay.kv_capacity / 128 * heads;
  return launch_pdl(prefill_expand_kernel, dim3(static_cast<unsigned>(most < sms ? most : sms)), dim3(kThreads), kSmemBytes,
                    stream, m, a, head0, heads);
}

}  // namespace mla
