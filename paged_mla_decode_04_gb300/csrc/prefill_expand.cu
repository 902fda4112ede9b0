// Keys and values of the gathered rows, for every head h of a pass:
//   K[h][t][0:128] = c_kv[t] W_UK[h]^T,   V[h][t][0:128] = c_kv[t] W_UV[h],
// a product of [rows x 512] with [512 x 256] per head. Keys are rounded to bf16, as
// models keep them: their errors reach the result through the scores alone, damped
// by the softmax scale, and they may be as large as the queries. Values and softmax
// weights are errors of the result itself, so they are f16, three bits more: with bf16
// the result was off by 2.9e-3 (2-norm) where its own rounding to bf16 is 1.7e-3, with
// f16 by 2.1e-3. f16 has few exponents: a row's 128 values of a head are stored times
// 2^(-20 k), k being the bin of the largest (0 for values of usual sizes), and k beside
// them for the attention, which takes it into the row's score (the header says whether
// any row has another k than 0).
//
// Bound by the tensor core once the operands arrive: per tile of 128 rows x one
// head an SM would read 128 KB of rows and 256 KB of weights in the 4,096 cycles of
// its products, more than L2 gives it. So pairs of SMs multiply M = 256 rows
// (each block holds 128 of them and one half of the weights' N), a block keeps its
// 128 rows of all 512 dims in shared memory (128 KB) over the heads of its run,
// and only its half of the weights streams: 128 KB a tile.
//
// A cluster takes a run of (256 rows, head) units, heads fastest. Both halves of
// a unit accumulate side by side in 256 TMEM columns (K in the first 128, V in
// the others); two such accumulators alternate, so that the epilogue of one unit
// runs under the products of the next. Weights come by TMA in chunks of 64 of the
// 512 dims, W_UK K-major and W_UV MN-major, 16 KB a stage and block.
//
// 16,384 rows for 128 heads: 334 us, 1.65 PFLOP/s (85 % of the library product's burst
// rate, 95 % of what it sustains); 19,799 rows for 16 heads: 55 us, 1.50, where a
// cluster's last run is short and each run's rows arrive before its first product. Of
// the rest the tensor core waits 26 % (active 74 %): at a run's start, and for power.
// Stores through shared memory and TMA instead of 32 bytes a thread: no gain, or 10 %
// lost where they took two of the five stages.
#include <cuda_bf16.h>

#include "../../include/mla_decode.h"
#include "ptx_prefill.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kStages = 5;
constexpr int kChunk = 64;
constexpr int kChunks = kDimCkv / kChunk;          // 8
constexpr int kABytes = 128 * kChunk * 2;          // a chunk of this block's rows
constexpr int kWBytes = 64 * kChunk * 2;           // [64 key dims][64 dims], or [64 dims][64 value dims]
constexpr int kStageBytes = 2 * kWBytes;
constexpr int kOffRing = kChunks * kABytes;
constexpr int kOffBar = kOffRing + kStages * kStageBytes;
constexpr int kSmemBytes = kOffBar + 256 + 1024;
constexpr int kThreads = 192;  // producer, issuer, four epilogue warps
static_assert(kSmemBytes <= 232448, "shared memory");

enum {
  // In the even block: copies of both blocks landed, accumulator read by both.
  kBarFull = 0,                       // [stages]
  kBarRows = kBarFull + kStages,      // [chunks]
  kBarAccFree = kBarRows + kChunks,   // [2]
  kBarDrain = kBarAccFree + 2,
  // In both blocks: products complete.
  kBarEmpty = kBarDrain + 1,          // [stages]
  kBarRowsFree = kBarEmpty + kStages,
  kBarAccFull,                        // [2]
  kNumBars = kBarAccFull + 2
};
static_assert(8 * kNumBars + 8 <= 256, "barrier area");

// Bin of a row whose largest value has this size.
__device__ __forceinline__ int bin_of(float most) {
  if (most == 0.f) return kZeroBin;
  const int e = (__float_as_int(most) >> 23) - 127;  // -127 .. 128
  return min(max((e - kBinLow + 10 * kBinBits) / kBinBits - 10, -kMostBin), kMostBin);
}

// halves == 2: so few units that half the clusters would do, and keys and values are
// units of their own, at most one a cluster (the smallest call, 95 rows of 16 heads, became
// 1.5 us shorter by it, of 21; in larger ones the choice would sit in the loops of
// all, which costs 1 to 2 %, hence the template).
template <int halves>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
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
  const uint32_t cta = cluster_rank();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), i >= kBarAccFree && i < kBarAccFree + 2 ? 8 : 1);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 1) {
    tmem_alloc2(smem_addr(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lead0 = mapa(bar0, 0);
  auto lead = [&](int i) -> uint32_t { return lead0 + 8u * i; };
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == kThreads - 1) {  // for the attention that follows (by a thread that has time)
    hd->next_item = 0;
    if (hd->zero_rows) hd->odd_bins = 1;
    hd->zero_rows = 0;
  }
  const int kv_rows = hd->kv_rows, row_blocks = (kv_rows + 255) / 256;
  const int64_t clusters = gridDim.x / 2, mine = blockIdx.x / 2;
  const int64_t units = static_cast<int64_t>(row_blocks) * heads * halves;
  const int64_t u0 = units * mine / clusters, u1 = units * (mine + 1) / clusters;
  auto fail = [&] {
    *abort_flag = 1;
    atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t k = 0, loads = 0;  // weight chunks, row blocks
      int row_block = -1;
      bool ok = true;
      for (int64_t u = u0; u < u1 && ok; ++u) {
        const int head = head0 + static_cast<int>(u / halves % heads), rb = static_cast<int>(u / halves / heads);
        const bool with_k = halves == 1 || !(u & 1), with_v = halves == 1 || (u & 1);
        const bool fresh = rb != row_block;
        if (fresh) {
          if (!(ok = mbar_spin(bar(kBarRowsFree), (loads & 1u) ^ 1u, abort_flag))) break;
          row_block = rb;
          ++loads;
        }
        for (int c = 0; c < kChunks; ++c, ++k) {
          if (fresh) {
            if (cta == 0) mbar_arrive_expect_tx(bar(kBarRows + c), 2 * kABytes);
            tma2_load_2d(sbase + c * kABytes, &m.rows, lead(kBarRows + c), c * kChunk, rb * 256 + 128 * cta);
          }
          const uint32_t s = k % kStages;
          if (!(ok = mbar_spin(bar(kBarEmpty + s), ((k / kStages) & 1u) ^ 1u, abort_flag))) break;
          const uint32_t dst = sbase + kOffRing + s * kStageBytes;
          if (cta == 0) mbar_arrive_expect_tx(bar(kBarFull + s), 2 * kStageBytes / halves);
          if (with_k) tma2_load_2d(dst, &m.w_uk, lead(kBarFull + s), c * kChunk, head * kDimNope + 64 * cta);
          if (with_v) tma2_load_2d(dst + kWBytes, &m.w_uv, lead(kBarFull + s), 64 * cta, head * kDimCkv + c * kChunk);
        }
      }
      if (!ok) fail();
      if (*abort_flag && cta == 0) {  // let the copies in flight land (each wait bounded)
        for (uint32_t i = k > kStages ? k - kStages : 0; i < k; ++i)
          mbar_wait(bar(kBarFull + i % kStages), (i / kStages) & 1u, nullptr);
        if (loads)
          for (int c = 0; c < kChunks; ++c) mbar_wait(bar(kBarRows + c), (loads - 1) & 1u, nullptr);
      }
    }
  } else if (warp == 1) {
    if (cta == 0 && elect_one()) {
      constexpr uint32_t idesc_k = idesc_bf16(256, 128, false, false);
      constexpr uint32_t idesc_v = idesc_bf16(256, 128, false, true);
      const uint32_t a_lo = desc_lo(sbase), ring_lo = desc_lo(sbase + kOffRing);
      uint32_t stage = 0, par = 0, n = 0, loads = 0;
      int row_block = -1;
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && mbar_spin(b, parity, abort_flag); };
      int64_t left = heads - u0 % heads;  // units until the next row block (with halves a cluster has one unit)
      for (int64_t u = u0; u < u1 && ok; ++u, ++n) {
        const int rb = static_cast<int>(u / halves / heads);
        const bool with_k = halves == 1 || !(u & 1), with_v = halves == 1 || (u & 1);
        const bool fresh = rb != row_block;
        if (fresh) {
          row_block = rb;
          ++loads;
        }
        const uint32_t acc = n & 1u, d = tmem + acc * 256;
        wait(bar(kBarAccFree + acc), ((n >> 1) & 1u) ^ 1u);
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          if (fresh) wait(bar(kBarRows + c), (loads - 1) & 1u);
          wait(bar(kBarFull + stage), par);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ad = a_lo + c * (kABytes >> 4), wd = ring_lo + stage * (kStageBytes >> 4);
#pragma unroll
          for (int i = 0; i < kChunk / 16; ++i) {
            if (with_k) mma2_bf16_ss(d, ad + 2 * i, wd + 2 * i, idesc_k, (c | i) != 0);
            if (with_v) mma2_bf16_ss(d + 128, ad + 2 * i, wd + (kWBytes >> 4) + 128 * i, idesc_v, (c | i) != 0);
          }
          mma2_commit(bar(kBarEmpty + stage));
          stage = stage == kStages - 1 ? 0 : stage + 1;
          par ^= stage == 0 ? 1u : 0u;
        }
        if (!ok) break;
        mma2_commit(bar(kBarAccFull + acc));
        if (--left == 0) {
          mma2_commit(bar(kBarRowsFree));
          left = heads;
        }
      }
      if (!ok) fail();
      mma2_commit(bar(kBarDrain));
      mbar_wait(bar(kBarDrain), 0, nullptr);
    }
  } else {
    const int quarter = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t n = 0;
    bool ok = true, told = false;
    for (int64_t u = u0; u < u1; ++u, ++n) {
      const uint32_t acc = n & 1u;
      if (!(ok = mbar_spin_warp(bar(kBarAccFull + acc), (n >> 1) & 1u, abort_flag))) break;
      tc_fence_after();
      const int64_t row = (u / halves / heads) * 256 + 128 * cta + quarter * 32 + lane;
      const bool keep = row < a.lay.kv_capacity;  // (a multiple of 128: whole blocks)
      const int64_t out_row = (u / halves % heads) * a.lay.kv_capacity + row;
      const bool with_k = halves == 1 || !(u & 1), with_v = halves == 1 || (u & 1);
      const uint32_t acc_k = tmem + lane_base + acc * 256, acc_v = acc_k + 128;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!with_k) break;
        uint32_t r[64];
        tmem_ld32(acc_k + c * 64, r);
        tmem_ld32(acc_k + c * 64 + 32, r + 32);
        tmem_wait_ld();
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.ws + a.lay.keys) + out_row * 128 + c * 64;
        if (keep) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              pk[i] = pack_bf16x2(__uint_as_float(r[16 * v + 2 * i]), __uint_as_float(r[16 * v + 2 * i + 1]));
            st_global_v8(dst + v * 16, pk);
          }
        }
      }
      uint32_t r[128];
      if (with_v) {
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(acc_v + c * 32, r + 32 * c);
        tmem_wait_ld();
      }
      tc_fence_before();  // all read: the products may go on
      if (lane == 0) mbar_arrive_cluster(lead(kBarAccFree + acc));
      if (with_v && keep) {
        float most[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 128; i += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            most[e] = fmax3(most[e], fabsf(__uint_as_float(r[i + 2 * e])), fabsf(__uint_as_float(r[i + 2 * e + 1])));
        const int k = bin_of(fmaxf(most[0], most[1]));
        const float f = __int_as_float((127 - kBinBits * k) << 23);
        a.ws[a.lay.bins + out_row] = static_cast<uint8_t>(k);
        if (!told && k != 0 && row < kv_rows && (most[0] > 0.f || most[1] > 0.f)) {
          hd->odd_bins = 1;
          told = true;  // (a store a unit and thread to the one address cost 30 % of the time)
        }
        uint16_t* dst = reinterpret_cast<uint16_t*>(a.ws + a.lay.values) + out_row * 128;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          uint32_t pk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float x, y;
            f2_split(f2_mul(f2_make(__uint_as_float(r[16 * v + 2 * i]), __uint_as_float(r[16 * v + 2 * i + 1])), f2_make(f, f)), x, y);
            pk[i] = pack_f16x2(x, y);
          }
          st_global_v8(dst + v * 16, pk);
        }
      }
    }
    if (!ok) fail();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // no block ends while the other's products or arrivals reach into it
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, 512);
}

}  // namespace

cudaError_t launch_prefill_expand(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream) {
  static bool attr_set[2][kMaxDevices] = {};
  const int pairs = sm_count() / 2;
  if (pairs <= 0) return cudaErrorInvalidDevice;
  const int64_t most = (a.lay.kv_capacity + 255) / 256 * heads;
  const bool halves = 2 * most <= pairs;
  const auto kernel = halves ? prefill_expand_kernel<2> : prefill_expand_kernel<1>;
  const cudaError_t e = set_smem_once(kernel, kSmemBytes, attr_set[halves]);
  if (e != cudaSuccess) return e;
  const int64_t blocks = halves ? 4 * most : 2 * (most < pairs ? most : pairs);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), kSmemBytes, stream, m, a, head0, heads);
}

}  // namespace mla
