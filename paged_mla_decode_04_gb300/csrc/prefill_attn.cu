// Attention of the new tokens over the expanded keys and values, in the
// 192/128 multi-head form: for query row r and head h
//   S_t = scale (q_nope . K[h][t] + q_rope . k_rope[t]) over the positions t
//   that r may see (causal, windowed),  out = sum_t softmax(S)_t V[h][t].
//
// Per key: 2 * 192 + 2 * 128 flops a row, so it is bound by the tensor core.
// A persistent block per SM takes (256 query rows, head) tiles. The two blocks of
// 128 rows run as two streams over the same 128-key steps: while the softmax
// warps of one stream turn S into P, the tensor core works for the other.
//   TMEM (512 columns): S0 [0, 128) S1 [128, 256) O0 [256, 384) O1 [384, 512);
//   a stream's P (bf16 pairs, 64 columns) overwrites its S.
//   Shared memory: Q (2 x 48 KB) and a ring of eight 16 KB slots: a step's
//   keys take three (64 of the 192 dims each, K-major), its values two (64
//   keys each, MN-major).
// The issuing thread runs QK0(j), PV1(j-1), QK1(j), PV0(j): each stream's softmax
// has the other stream's two products to hide under. All products are issued
// by one thread and complete in order, so S(j) being complete implies that
// P V (j-1) of that stream is: softmax warps may rescale O without asking.
// Softmax: one thread a row, base 2, the reference maximum moves only when
// the running one exceeds it by 2^8 (the final division makes it exact); P is
// rounded to bf16 for the product, its sum is kept in fp32.
// Positions beyond a row's range are masked by selection, never by adding, so
// NaN in them stays out; the last step multiplies only up to the last 16 keys
// with a valid one, beyond which the buffer may hold another request's rows.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "../../include/mla_decode.h"
#include "ptx_prefill.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kSlots = 8;
constexpr int kSlotBytes = 128 * 128;       // 128 rows of 64 bf16, or two 64-row halves
constexpr int kQBytes = 3 * kSlotBytes;     // one stream's 128 rows of 192
constexpr int kOffRing = 2 * kQBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
constexpr int kSmemBytes = kOffBar + 512 + 1024;
constexpr int kThreads = 384;               // two softmax warpgroups; producer, issuer and two idle warps
// Registers a thread after setmaxnreg: a softmax row keeps 128 scores. They
// add up to the launch's 3 x 168.
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
static_assert(2 * kRegsSoftmax + kRegsOther == 3 * 168, "register split");
constexpr int kProducerWarp = 8, kIssueWarp = 9;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per stream
constexpr float kRescaleThreshold = 8.0f;   // log2 units
static_assert(kSmemBytes <= 232448, "shared memory");

enum {
  kBarFull = 0,                    // [slots] copy landed
  kBarEmpty = kBarFull + kSlots,   // [slots] products that read it are complete
  kBarQFull = kBarEmpty + kSlots,  // [streams]
  kBarQEmpty = kBarQFull + 2,
  kBarS = kBarQEmpty + 2,          // S complete
  kBarP = kBarS + 2,               // P stored, O rescaled
  kBarO = kBarP + 2,               // the tile's last P V complete
  kBarDrain = kBarO + 2,
  kNumBars
};
static_assert(8 * kNumBars + 8 <= 512, "barrier area");

__device__ __forceinline__ int steps_of(int begin, int end) { return end > begin ? (end - begin + kPfKvTile - 1) / kPfKvTile : 0; }

// What the roles need of a tile: steps of each stream (0: no rows).
struct Work {
  PfTile t;
  int n0, n1, n;
  int end0;  // end of stream 0's last row
};

__device__ __forceinline__ Work work_of(const PfTile* tiles, int i) {
  Work w;
  w.t = tiles[i];
  w.end0 = w.t.first_end + min(w.t.rows, 128) - 1;
  w.n0 = w.t.refused ? 0 : steps_of(w.t.kv_begin, w.end0);
  w.n1 = w.t.refused || w.t.rows <= 128 ? 0 : steps_of(w.t.kv_begin, w.t.kv_end);
  w.n = max(w.n0, w.n1);
  return w;
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_attn_kernel(const __grid_constant__ PrefillMaps m, const __grid_constant__ PrefillArgs a, int head0, int heads) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 8 * kNumBars + 4);
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const PfTile* tiles = reinterpret_cast<const PfTile*>(a.ws + a.lay.tiles);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), (i >= kBarP && i < kBarP + 2) ? 128 : 1);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int num_tiles = hd->num_tiles;
  const int64_t items = static_cast<int64_t>(num_tiles) * heads;
  auto fail = [&] {
    *abort_flag = 1;
    atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  };

  if (warp >= kProducerWarp) setmaxnreg_dec<kRegsOther>();
  if (warp == kProducerWarp) {
    if (lane == 0) {
      uint32_t k = 0;             // ring slots issued
      uint32_t q_use[2] = {0, 0};
      bool ok = true;
      auto slot = [&](uint32_t bytes) -> uint32_t {  // waits for the next slot; its number, or kSlots on failure
        const uint32_t s = k % kSlots;
        if (!mbar_wait(bar(kBarEmpty + s), ((k / kSlots) & 1u) ^ 1u, abort_flag)) {
          ok = false;
          return kSlots;
        }
        mbar_arrive_expect_tx(bar(kBarFull + s), bytes);
        ++k;
        return s;
      };
      for (int64_t it = blockIdx.x; it < items && ok; it += gridDim.x) {
        const Work w = work_of(tiles, static_cast<int>(it % num_tiles));
        const int hl = static_cast<int>(it / num_tiles);  // head within the pass
        for (int j = 0; j < w.n && ok; ++j) {
          const int row = w.t.base + w.t.kv_begin + j * kPfKvTile;
          for (int c = 0; c < 3; ++c) {
            const uint32_t s = slot(kSlotBytes);
            if (!ok) break;
            const uint32_t dst = sbase + kOffRing + s * kSlotBytes;
            if (c < 2) tma_load_3d(dst, &m.keys, bar(kBarFull + s), 64 * c, row, hl);
            else tma_load_2d(dst, &m.rows, bar(kBarFull + s), kDimCkv, row);
          }
          if (j == 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || (x ? w.n1 : w.n0) == 0) continue;
              if (!(ok = mbar_wait(bar(kBarQEmpty + x), (q_use[x] & 1u) ^ 1u, abort_flag))) continue;
              ++q_use[x];
              mbar_arrive_expect_tx(bar(kBarQFull + x), kQBytes);
              for (int c = 0; c < 3; ++c)
                tma_load_3d(sbase + x * kQBytes + c * kSlotBytes, &m.q, bar(kBarQFull + x), 64 * c, head0 + hl,
                            w.t.q_row + 128 * x);
            }
          }
          for (int half = 0; half < 2 && ok; ++half) {
            const uint32_t s = slot(kSlotBytes);
            if (!ok) break;
            const uint32_t dst = sbase + kOffRing + s * kSlotBytes;
            for (int c = 0; c < 2; ++c)
              tma_load_3d(dst + c * (kSlotBytes / 2), &m.values, bar(kBarFull + s), 64 * c, row + 64 * half, hl);
          }
        }
      }
      if (!ok) fail();
      if (*abort_flag) {  // let the copies in flight land (each wait bounded)
        for (uint32_t i = k > kSlots ? k - kSlots : 0; i < k; ++i)
          mbar_wait(bar(kBarFull + i % kSlots), (i / kSlots) & 1u, nullptr);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (q_use[x]) mbar_wait(bar(kBarQFull + x), (q_use[x] - 1) & 1u, nullptr);
      }
    }
  } else if (warp == kIssueWarp) {
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16(128, 128, false, true);
      uint32_t k = 0;               // first ring slot of the current step
      uint32_t p_use[2] = {0, 0}, q_use[2] = {0, 0};
      bool ok = true;
      auto full = [&](uint32_t i) {  // waits for ring slot number i
        if (ok && !mbar_wait(bar(kBarFull + i % kSlots), (i / kSlots) & 1u, abort_flag)) ok = false;
      };
      auto release = [&](uint32_t i) { mma_commit(bar(kBarEmpty + i % kSlots)); };
      auto slot_addr = [&](uint32_t i) { return sbase + kOffRing + (i % kSlots) * kSlotBytes; };
      auto qk = [&](int x) {  // S_x = Q_x K^T of the step at ring slots k .. k + 2
        for (int c = 0; c < 3; ++c) {
          const uint64_t ad = sdesc_sw128(sbase + x * kQBytes + c * kSlotBytes, 16, 1024);
          const uint64_t bd = sdesc_sw128(slot_addr(k + c), 16, 1024);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_bf16_ss(tmem + kColS + 128 * x, ad + 2 * i, bd + 2 * i, idesc_qk, (c | i) != 0);
        }
        mma_commit(bar(kBarS + x));
      };
      // O_x += P_x V for the step whose values sit at slots v, v + 1.
      auto pv = [&](int x, uint32_t v, int ksteps, bool first) {
        for (int i = 0; i < ksteps; ++i) {
          const uint64_t bd = sdesc_sw128(slot_addr(v + (i >> 2)) + (i & 3) * 2048, kSlotBytes / 2, 1024);
          mma_bf16_ts(tmem + kColO + 128 * x, tmem + kColS + 128 * x + 8 * i, bd, idesc_pv, !first || i != 0);
        }
      };
      auto ksteps_of = [&](const Work& w, int end, int j) {
        const int left = end - (w.t.kv_begin + j * kPfKvTile);
        return min(8, (left + 15) / 16);
      };
      auto wait_p = [&](int x) {
        if (ok && !mbar_wait(bar(kBarP + x), p_use[x] & 1u, abort_flag)) ok = false;
        ++p_use[x];
        tc_fence_after();
      };
      auto pv1 = [&](const Work& w, int j, uint32_t v) {  // stream 1's product and the values' release
        wait_p(1);
        full(v);
        full(v + 1);
        if (!ok) return;
        pv(1, v, ksteps_of(w, w.t.kv_end, j), j == 0);
        release(v);
        release(v + 1);
        if (j == w.n1 - 1) mma_commit(bar(kBarO + 1));
      };
      for (int64_t it = blockIdx.x; it < items && ok; it += gridDim.x) {
        const Work w = work_of(tiles, static_cast<int>(it % num_tiles));
        for (int j = 0; j < w.n && ok; ++j, k += 5) {
          for (int c = 0; c < 3; ++c) full(k + c);
          if (!ok) break;
          tc_fence_after();
          if (j < w.n0) {
            if (j == 0 && !(ok = mbar_wait(bar(kBarQFull), q_use[0]++ & 1u, abort_flag))) break;
            qk(0);
            if (j == w.n0 - 1) mma_commit(bar(kBarQEmpty));
          }
          if (w.n1) {
            if (j > 0) pv1(w, j - 1, k - 2);
            if (!ok) break;
            if (j == 0 && !(ok = mbar_wait(bar(kBarQFull + 1), q_use[1]++ & 1u, abort_flag))) break;
            qk(1);
            if (j == w.n1 - 1) mma_commit(bar(kBarQEmpty + 1));
          }
          for (int c = 0; c < 3; ++c) release(k + c);
          if (j < w.n0) {
            wait_p(0);
            full(k + 3);
            full(k + 4);
            if (!ok) break;
            pv(0, k + 3, ksteps_of(w, w.end0, j), j == 0);
            if (j == w.n0 - 1) mma_commit(bar(kBarO));
          }
          if (!w.n1) {
            release(k + 3);
            release(k + 4);
          }
        }
        if (ok && w.n1) pv1(w, w.n - 1, k - 2);
      }
      if (!ok) fail();
      mma_commit(bar(kBarDrain));
      mbar_wait(bar(kBarDrain), 0, nullptr);
    }
  } else if (warp < kProducerWarp) {
    setmaxnreg_inc<kRegsSoftmax>();
    const int x = warp >> 2, quarter = warp & 3;
    const int r = x * 128 + quarter * 32 + lane;  // row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + kColS + 128 * x, tO = tmem + lane_base + kColO + 128 * x;
    const float scale = a.scale_log2;
    const uint64_t scale2 = f2_make(scale, scale);
    const float threshold = kRescaleThreshold / scale;  // in units of S
    uint32_t s_use = 0, o_use = 0;
    bool ok = true;
    for (int64_t it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const Work w = work_of(tiles, static_cast<int>(it % num_tiles));
      const int head = head0 + static_cast<int>(it / num_tiles);
      if (w.t.rows <= 128 * x) continue;
      const bool valid = r < w.t.rows;
      const int64_t out_row = (static_cast<int64_t>(w.t.q_row) + r) * a.num_heads + head;
      uint8_t* dst = static_cast<uint8_t*>(a.out) + out_row * (kDimV * 2);
      if (w.t.refused) {
        if (valid) {
          const uint32_t nan8[8] = {0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u,
                                    0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
          for (int i = 0; i < kDimV * 2 / 32; ++i) st_global_v8(dst + 32 * i, nan8);
          if (a.lse) a.lse[out_row] = CUDART_NAN_F;
        }
        continue;
      }
      const int n = x ? w.n1 : w.n0;
      const int end = min(w.t.first_end + r, x ? w.t.kv_end : w.end0);
      const int begin = a.window > 0 ? max(0, w.t.first_end + r - a.window) : 0;
      float mx_ref = -CUDART_INF_F, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int pos0 = w.t.kv_begin + j * kPfKvTile;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarS + x), s_use & 1u, abort_flag));
        if (!ok) break;
        ++s_use;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
        tmem_wait_ld();
        if (begin > pos0 || end < pos0 + kPfKvTile) {
          const int b0 = begin - pos0, e0 = end - pos0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i < b0 || i >= e0) s[i] = 0xff800000u;
        }
        float mxa = -CUDART_INF_F, mxb = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < 128; i += 4) {
          mxa = fmax3(mxa, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          mxb = fmax3(mxb, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
        }
        const float mx = fmaxf(mxa, mxb);
        float alpha = 1.f;
        if (mx > mx_ref + threshold) {
          alpha = exp2_approx((mx_ref - mx) * scale);  // 0 on the first step with a key
          l *= alpha;
          mx_ref = mx;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(tO + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(tO + 16 * c, o);
          }
        }
        const float neg = mx_ref == -CUDART_INF_F ? 0.f : -mx_ref * scale;
        const uint64_t neg2 = f2_make(neg, neg);
        uint64_t sum2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float t0, t1;
          f2_split(f2_fma(f2_make(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, neg2), t0, t1);
          const float p0 = exp2_approx(t0), p1 = exp2_approx(t1);
          sum2[i & 1] = f2_add(sum2[i & 1], f2_make(p0, p1));
          s[i] = pack_bf16x2(p0, p1);
        }
        tmem_st32(tS, s);
        tmem_st32(tS + 32, s + 32);
        float s0, s1, s2, s3;
        f2_split(sum2[0], s0, s1);
        f2_split(sum2[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarP + x));
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarO + x), o_use & 1u, abort_flag));
      if (!ok) break;
      ++o_use;
      tc_fence_after();
      const float inv = a.out_scale / l;  // every valid row attends itself: l > 0
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t o[64];
        tmem_ld32(tO + 64 * c, o);
        tmem_ld32(tO + 64 * c + 32, o + 32);
        tmem_wait_ld();
        if (valid) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              pk[i] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * i]) * inv, __uint_as_float(o[16 * v + 2 * i + 1]) * inv);
            st_global_v8(dst + 128 * c + 32 * v, pk);
          }
        }
      }
      if (a.lse && valid) a.lse[out_row] = (mx_ref * scale + log2f(l)) * 0.69314718055994531f;
      tc_fence_before();
    }
    if (!ok) fail();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_prefill_attn(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(prefill_attn_kernel, kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t most = a.lay.max_tiles * heads;
  return launch_pdl(prefill_attn_kernel, dim3(static_cast<unsigned>(most < sms ? most : sms)), dim3(kThreads), kSmemBytes,
                    stream, m, a, head0, heads);
}

}  // namespace mla
