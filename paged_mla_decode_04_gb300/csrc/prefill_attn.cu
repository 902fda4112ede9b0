// Attention of the new tokens over the expanded keys and values, in the
// 192/128 multi-head form: for query row r and head h
//   S_t = scale (q_nope . K[h][t] + q_rope . k_rope[t]) over the positions t
//   that r may see (causal, windowed),  out = sum_t softmax(S)_t V[h][t].
//
// Per key: 2 * 192 + 2 * 128 flops a row, so it is bound by the tensor core.
// A persistent block per SM draws items, (256 query rows, head), from a counter,
// the expensive ones of a group of heads first. The two blocks of 128 rows run as two streams over the same 128-key steps: while the softmax
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
// Softmax: two threads of a warp share a row (64 keys of a step each; eight warps
// a stream keep the chain from S to P short), base 2, the reference maximum moves only when
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
constexpr int kSoftmaxWarps = 16;           // eight a stream
constexpr int kProducerWarp = 16, kIssueWarp = 17;
constexpr int kThreads = 640;               // (the last two warps idle)
// Registers a thread after setmaxnreg; they add up to the launch's 5 x 96.
constexpr int kRegsSoftmax = 104, kRegsOther = 64;
static_assert(4 * kRegsSoftmax + kRegsOther == 5 * 96, "register split");
constexpr int kSched = 2;                   // items announced ahead
// Items that a group of heads should have for each block: within a group the
// costly tiles of all its heads come first, groups follow each other so that
// their keys and values stay in L2.
constexpr int kGroupItems = 3;
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
  kBarItem = kBarO + 2,            // [kSched] item announced
  kBarItemFree = kBarItem + kSched,  // [kSched] read by every role
  kBarDrain = kBarItemFree + kSched,
  kNumBars
};
constexpr int kOffItems = 8 * kNumBars + 8;  // after TMEM address and abort flag

// What the roles need of an item: a tile, its head within the pass and the steps of
// each stream (0: no rows).
struct Item {
  PfTile t;
  int head;  // -1: no further items
  int n0, n1, n;
  int end0;  // end of stream 0's last row
};
static_assert(kOffItems + kSched * sizeof(Item) <= 512, "barrier area");

__device__ __forceinline__ Item item_of(const PfTile& t, int head) {
  Item w;
  w.t = t;
  w.head = head;
  w.end0 = t.first_end + min(t.rows, 128) - 1;
  w.n0 = t.refused ? 0 : pf_steps(t.kv_begin, w.end0);
  w.n1 = t.refused || t.rows <= 128 ? 0 : pf_steps(t.kv_begin, t.kv_end);
  w.n = max(w.n0, w.n1);
  return w;
}

// Tile rank and head of item `it`: groups of heads one after the other, within
// a group all heads' tiles of one rank before the next rank's.
__device__ __forceinline__ void split_item(int64_t it, int num_tiles, int heads, int groups, int* rank, int* head) {
  int g = static_cast<int>(it * groups / (static_cast<int64_t>(num_tiles) * heads));
  int h0 = heads * g / groups, h1 = heads * (g + 1) / groups;
  if (it < static_cast<int64_t>(h0) * num_tiles) {
    --g;
    h1 = h0;
    h0 = heads * g / groups;
  } else if (it >= static_cast<int64_t>(h1) * num_tiles) {
    ++g;
    h0 = h1;
    h1 = heads * (g + 1) / groups;
  }
  const int64_t in = it - static_cast<int64_t>(h0) * num_tiles;
  *rank = static_cast<int>(in / (h1 - h0));
  *head = h0 + static_cast<int>(in % (h1 - h0));
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
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bar(i), (i >= kBarP && i < kBarP + 2) ? kSoftmaxWarps / 2
                        : (i >= kBarItemFree && i < kBarItemFree + kSched) ? kSoftmaxWarps + 1 : 1);
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
  Item* board = reinterpret_cast<Item*>(smem + kOffBar + kOffItems);
  // The i-th item of this block, as every role but the producer reads it.
  auto read_item = [&](uint32_t i, Item& w) -> bool {
    if (!__all_sync(0xffffffffu, mbar_wait(bar(kBarItem + i % kSched), (i / kSched) & 1u, abort_flag))) return false;
    w = board[i % kSched];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarItemFree + i % kSched));
    return true;
  };
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
      const int* order = reinterpret_cast<const int*>(a.ws + a.lay.order);
      const int64_t group_items = static_cast<int64_t>(kGroupItems) * gridDim.x;
      const int group_heads = static_cast<int>(min(static_cast<int64_t>(heads), (group_items + num_tiles - 1) / max(num_tiles, 1)));
      const int groups = max(1, heads / max(group_heads, 1));
      auto load_item = [&](int64_t it) {
        int rank, head;
        if (it >= items) return item_of(PfTile{0, 0, 0, 0, 0, 0, 1, 0}, -1);
        split_item(it, num_tiles, heads, groups, &rank, &head);
        return item_of(tiles[order[rank]], head);
      };
      Item w = load_item(blockIdx.x);
      for (uint32_t i = 0; ok; ++i) {
        // Announce the item, draw the next one (its number comes while this
        // item's copies are issued).
        if (!(ok = mbar_wait(bar(kBarItemFree + i % kSched), ((i / kSched) & 1u) ^ 1u, abort_flag))) break;
        board[i % kSched] = w;
        mbar_arrive(bar(kBarItem + i % kSched));
        if (w.head < 0) break;
        const int64_t next = static_cast<int64_t>(gridDim.x) + atomicAdd(&hd->next_item, 1);
        const int hl = w.head;
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
        w = load_item(next);
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
    constexpr uint32_t idesc_qk = idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16(128, 128, false, true);
    // Descriptors differ in their address field only (units of 16 bytes).
    const uint64_t q_desc = sdesc_sw128(sbase, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(sbase + kOffRing, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sbase + kOffRing, kSlotBytes / 2, 1024);
    uint32_t k = 0;  // first ring slot of the current step
    uint32_t p_use0 = 0, p_use1 = 0, q_use0 = 0, q_use1 = 0;
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag)); };
    auto full = [&](uint32_t i) { wait(bar(kBarFull + i % kSlots), (i / kSlots) & 1u); };
    // S_x = Q_x K^T of the step at ring slots k .. k + 2.
    auto qk = [&](int x) {
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const uint64_t ad = q_desc + ((x * kQBytes + c * kSlotBytes) >> 4);
        const uint64_t bd = k_desc + ((k + c) % kSlots) * (kSlotBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_bf16_ss(tmem + kColS + 128 * x, ad + 2 * i, bd + 2 * i, idesc_qk, (c | i) != 0);
          if (c == 2) mma_commit(bar(kBarS + x));
        }
      }
    };
    // O_x += P_x V for the step whose values sit at slots v, v + 1: up to the
    // last 16 keys below `end`.
    auto pv = [&](int x, uint32_t v, int left, bool first) {
      const int ksteps = min(8, (left + 15) / 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t bd = v_desc + ((v + h) % kSlots) * (kSlotBytes >> 4);
        const uint32_t td = tmem + kColO + 128 * x, ta = tmem + kColS + 128 * x + 32 * h;
        if (ksteps >= 4 * h + 4) {
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16_ts(td, ta + 8 * i, bd + i * (2048 >> 4), idesc_pv, !first || (h | i) != 0);
          }
        } else {
          for (int i = 0; i < ksteps - 4 * h; ++i)
            if (elect_one()) mma_bf16_ts(td, ta + 8 * i, bd + i * (2048 >> 4), idesc_pv, !first || (h | i) != 0);
        }
      }
    };
    // Stream 1's product and the values' release.
    auto pv1 = [&](const Item& w, int j, uint32_t v) {
      wait(bar(kBarP + 1), p_use1++ & 1u);
      full(v);
      full(v + 1);
      if (!ok) return;
      tc_fence_after();
      pv(1, v, w.t.kv_end - w.t.kv_begin - j * kPfKvTile, j == 0);
      if (elect_one()) {
        mma_commit(bar(kBarEmpty + v % kSlots));
        mma_commit(bar(kBarEmpty + (v + 1) % kSlots));
        if (j == w.n1 - 1) mma_commit(bar(kBarO + 1));
      }
    };
    Item w;
    for (uint32_t i = 0; ok; ++i) {
      ok = read_item(i, w);
      if (!ok || w.head < 0) break;
      for (int j = 0; j < w.n && ok; ++j, k += 5) {
        full(k);
        full(k + 1);
        full(k + 2);
        if (j < w.n0) {
          if (j == 0) wait(bar(kBarQFull), q_use0++ & 1u);
          if (!ok) break;
          tc_fence_after();
          qk(0);
          if (j == w.n0 - 1 && elect_one()) mma_commit(bar(kBarQEmpty));
        }
        if (w.n1) {
          if (j > 0) pv1(w, j - 1, k - 2);
          if (j == 0) wait(bar(kBarQFull + 1), q_use1++ & 1u);
          if (!ok) break;
          tc_fence_after();
          qk(1);
          if (j == w.n1 - 1 && elect_one()) mma_commit(bar(kBarQEmpty + 1));
        }
        if (!ok) break;
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 3; ++c) mma_commit(bar(kBarEmpty + (k + c) % kSlots));
        }
        if (j < w.n0) {
          wait(bar(kBarP), p_use0++ & 1u);
          full(k + 3);
          full(k + 4);
          if (!ok) break;
          tc_fence_after();
          pv(0, k + 3, w.end0 - w.t.kv_begin - j * kPfKvTile, j == 0);
          if (j == w.n0 - 1 && elect_one()) mma_commit(bar(kBarO));
        }
        if (!w.n1 && elect_one()) {
          mma_commit(bar(kBarEmpty + (k + 3) % kSlots));
          mma_commit(bar(kBarEmpty + (k + 4) % kSlots));
        }
      }
      if (ok && w.n1) pv1(w, w.n - 1, k - 2);
    }
    if (!ok && lane == 0) fail();
    __syncwarp();
    if (elect_one()) mma_commit(bar(kBarDrain));
    mbar_wait(bar(kBarDrain), 0, nullptr);
  } else if (warp < kProducerWarp) {
    setmaxnreg_inc<kRegsSoftmax>();
    // Warp w works for stream w >> 3 on 16 lanes of TMEM lane quarter w & 3. A
    // row belongs to threads t and t + 16: keys [0, 64) and [64, 128) of every
    // step, value dims [0, 64) and [64, 128) of O.
    const int x = warp >> 3, quarter = warp & 3, th = lane >> 4;
    const int lane0 = quarter * 32 + ((warp >> 2) & 1) * 16;
    const int r = x * 128 + lane0 + (lane & 15);  // row of the tile
    const uint32_t tbase = tmem + (static_cast<uint32_t>(lane0) << 16) + 128 * x;
    const uint32_t tS = tbase + kColS, tO = tbase + kColO;
    const float scale = a.scale_log2;
    const uint64_t scale2 = f2_make(scale, scale);
    const float threshold = kRescaleThreshold / scale;  // in units of S
    uint32_t s_use = 0, o_use = 0;
    bool ok = true;
    Item w;
    for (uint32_t i = 0; ok; ++i) {
      ok = read_item(i, w);
      if (!ok || w.head < 0) break;
      if (w.t.rows <= 128 * x) continue;
      const bool valid = r < w.t.rows;
      const int64_t out_row = (static_cast<int64_t>(w.t.q_row) + r) * a.num_heads + head0 + w.head;
      uint8_t* dst = static_cast<uint8_t*>(a.out) + out_row * (kDimV * 2) + th * kDimV;
      if (w.t.refused) {
        if (valid) {
          const uint32_t nan8[8] = {0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u,
                                    0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
          for (int v = 0; v < kDimV / 32; ++v) st_global_v8(dst + 32 * v, nan8);
          if (a.lse && th == 0) a.lse[out_row] = CUDART_NAN_F;
        }
        continue;
      }
      const int n = x ? w.n1 : w.n0;
      // The row's range, relative to this thread's first key of step 0.
      const int off = w.t.kv_begin + 64 * th;
      const int end = min(w.t.first_end + r, x ? w.t.kv_end : w.end0) - off;
      const int begin = a.window > 0 ? max(0, w.t.first_end + r - a.window) - off : -off;
      float mx_ref = -CUDART_INF_F, l = 0.f;  // l: this thread's keys only
      for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarS + x), s_use & 1u, abort_flag));
        if (!ok) break;
        ++s_use;
        tc_fence_after();
        uint32_t s[64];
        tmem_ld_h32<64>(tS, s);
        tmem_ld_h32<64>(tS + 32, s + 32);
        tmem_wait_ld();
        const int b0 = begin - j * kPfKvTile, e0 = end - j * kPfKvTile;
        if (b0 > 0 || e0 < 64) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < b0 || c >= e0) s[c] = 0xff800000u;
        }
        float mxa = -CUDART_INF_F, mxb = -CUDART_INF_F;
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          mxa = fmax3(mxa, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          mxb = fmax3(mxb, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        }
        float mx = fmaxf(mxa, mxb);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        float alpha = 1.f;
        if (mx > mx_ref + threshold) {
          alpha = exp2_approx((mx_ref - mx) * scale);  // 0 on the first step with a key
          l *= alpha;
          mx_ref = mx;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[16];
            tmem_ld_h16<64>(tO + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int v = 0; v < 16; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * alpha);
            tmem_st_h16<64>(tO + 16 * c, o);
          }
        }
        const float neg = mx_ref == -CUDART_INF_F ? 0.f : -mx_ref * scale;
        const uint64_t neg2 = f2_make(neg, neg);
        uint64_t sum2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float t0, t1;
          f2_split(f2_fma(f2_make(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, neg2), t0, t1);
          const float p0 = exp2_approx(t0), p1 = exp2_approx(t1);
          sum2[c & 1] = f2_add(sum2[c & 1], f2_make(p0, p1));
          s[c] = pack_bf16x2(p0, p1);
        }
        tmem_st_h32<32>(tS, s);
        float s0, s1, s2, s3;
        f2_split(sum2[0], s0, s1);
        f2_split(sum2[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + x));
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarO + x), o_use & 1u, abort_flag));
      if (!ok) break;
      ++o_use;
      tc_fence_after();
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const float inv = a.out_scale / l;  // every valid row attends itself: l > 0
      uint32_t o[64];
      tmem_ld_h32<64>(tO, o);
      tmem_ld_h32<64>(tO + 32, o + 32);
      tmem_wait_ld();
      if (valid) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t pk[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            pk[c] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * c]) * inv, __uint_as_float(o[16 * v + 2 * c + 1]) * inv);
          st_global_v8(dst + 32 * v, pk);
        }
        if (a.lse && th == 0) a.lse[out_row] = (mx_ref * scale + log2f(l)) * 0.69314718055994531f;
      }
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
