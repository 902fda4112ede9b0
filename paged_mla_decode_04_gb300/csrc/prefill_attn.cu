// Attention of the new tokens over the expanded keys and values, in the
// 192/128 multi-head form: for query row r and head h
//   S_t = scale (q_nope . K[h][t] + q_rope . k_rope[t]) over the positions t
//   that r may see (causal, windowed),  out = sum_t softmax(S)_t V[h][t].
//
// Per key: 2 * 192 + 2 * 128 flops a row, so it is bound by the tensor core, and
// next to it by shared memory: a 128-row product with both operands there
// reads 128 bytes a cycle, all that an SM has, and copies and barriers then wait.
// Hence pairs of SMs: a cluster of two blocks multiplies M = 256 rows by tiles of
// which each block holds and reads one half (64 of a step's 128 keys; 64 of the 128
// value dims), and the copies of keys and values halve as well.
//
// A persistent cluster per SM pair draws items, (up to 512 query rows, head), from a
// counter, the expensive ones of a group of heads first. An item runs as two
// streams: while the softmax warps of one turn S into P, the tensor core works for
// the other. With more than 256 rows the streams are row blocks: rows [0, 256)
// and [256, 512), both over every 128-key step. With fewer they share the rows and
// take the even and the odd steps; their two results are merged at the end.
//   TMEM of a block (512 columns): S0 [0, 128) S1 [128, 256) O0 [256, 384)
//   O1 [384, 512), 128 rows each; a stream's P (f16 pairs, 64 columns)
//   overwrites its S.
//   Shared memory of a block: its 128 rows of each stream's Q (2 x 48 KB) and three
//   stages of a step: keys [64][192] (K-major, 24 KB), values [128][64]
//   (MN-major, 16 KB).
// The issuing thread (of the even block) runs QK of a unit (stream, step), then PV
// of the unit before: each stream's softmax has the other stream's two products
// to hide under. All products are issued by one thread and complete in order, so S
// of a stream being complete implies that its previous P V is: softmax warps may
// rescale O without asking.
// Softmax: one thread a row (with 128 scores in registers the exponentials of a
// step overlap; two threads a row in twice the warps took as long, short of
// registers), base 2. The reference maximum moves
// only when a score exceeds it by 8 (the final division makes it exact), so a step
// takes its exponentials against the reference as it stands and looks at the
// largest afterwards: above 2^8 the warp does the step again, with a maximum taken
// first. P is rounded to f16 for the product, as V is (see the expansion); its sum is
// kept in fp32. P is taken 2^7 times as large as against the reference, so that with
// the 2^8 of above it fills f16's range: weights keep all eleven bits down to 2^-21 of
// the row's largest (2^-14 without), some down to 2^-31. The result's division takes the
// factor out again.
// V of a key t is stored times 2^(-e_t), e_t = 20 k_t by the size of its row (see the
// expansion), so P holds weights times 2^(e_t): what a key adds to O, whose largest sets
// the reference, not the weight alone. The row's sum takes 2^(-e_t) again:
//   P_t = 2^(S_t + e_t - m),  O = sum P_t V_t 2^(-e_t),  l = sum P_t 2^(-e_t).
// Nearly always e is 0 throughout, which the workspace's header says. Else steps take a
// loop of their own, 32 keys at a time in two passes, for little code: the long chunk
// below takes 3.1 ms where all rows have one other e, 4.3 where each step's differ, and
// 1.9 with e = 0, within a percent of what it took without any of this (6 % more with
// both kinds of step in one loop, unrolled over the 128 keys).
// 2,048 new tokens behind 14,336 cached, 128 heads: 1,510 us alone, 1.70 PFLOP/s (88 % of
// the library product's burst rate); calls in a row run into the power limit (1,790 us).
// Three prompts of 4,500 to 8,192 tokens, 16 heads: 465 us, 1.52 (the diagonal's masked
// halves, and each item's start and end, about five units of (stream, step)). A window of
// 4,096 and chunks of 300 to 1,024 tokens, 128 heads: 741 us, 1.20 (86 % of the rows of
// its tiles are real, and a tile's rows span 511 keys more than each attends).
// Positions beyond a row's range are masked by selection, never by adding, so
// NaN in them stays out; the last step multiplies only up to the last 16 keys
// with a valid one, beyond which the buffer may hold another request's rows.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <type_traits>

#include "../../include/mla_decode.h"
#include "ptx_prefill.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kStages = 3;
constexpr int kQChunk = 128 * 128;          // [128 rows][64 dims]
constexpr int kQBytes = 3 * kQChunk;        // one stream's rows of this block
constexpr int kKChunk = 64 * 128;           // [64 keys][64 dims]
constexpr int kKBytes = 3 * kKChunk;
constexpr int kVBytes = 128 * 128;          // [128 keys][64 value dims]
constexpr int kStageBytes = kKBytes + kVBytes;
constexpr int kOffRing = 2 * kQBytes;
constexpr int kOffBar = kOffRing + kStages * kStageBytes;
constexpr int kSoftmaxWarps = 8;            // four a stream
constexpr int kProducerWarp = 8, kIssueWarp = 9;
constexpr int kThreads = 384;               // (the last two warps idle)
// Registers a thread after setmaxnreg; they add up to the launch's 3 x 168.
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
static_assert(2 * kRegsSoftmax + kRegsOther == 3 * 168, "register split");
constexpr int kSched = 2;                   // items announced ahead
// Items are drawn head after head, so that the clusters at work share few heads' keys
// and values in L2 (2,048 new tokens over 16,384, 128 heads: 2,060 us a call; 2,160 with
// the tiles of 57 heads interleaved). Where tiles differ in cost, the last heads, with
// this many items for each cluster, go together, costly tiles first, so that the last
// items are short (three prompts, 16 heads: 577 us; 618 to 627 without).
constexpr int kTailItems = 3;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 per stream
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr float kBinSteps = kBinBits / kRescaleThreshold;
constexpr float kMostWeight = 32768.0f;     // 2^(kRescaleThreshold + kWeightShift)
// The reference of a row that has seen no key: below every score, and finite so
// that a score of -inf against it is a weight of zero and any other infinite.
constexpr float kNoMax = -1e30f;

enum {
  // In the even block: a step's copies of both blocks landed.
  kBarKFull = 0,                     // [stages]
  kBarVFull = kBarKFull + kStages,   // [stages]
  kBarQFull = kBarVFull + kStages,   // [streams]
  kBarP = kBarQFull + 2,             // [streams] P stored and O rescaled, both blocks
  kBarItemFree = kBarP + 2,          // [kSched] read by every role of both blocks
  kBarDrain = kBarItemFree + kSched,
  // In both blocks: products complete, items announced.
  kBarKFree = kBarDrain + 1,         // [stages]
  kBarVFree = kBarKFree + kStages,   // [stages]
  kBarQFree = kBarVFree + kStages,   // [streams]
  kBarS = kBarQFree + 2,             // [streams] S complete
  kBarO = kBarS + 2,                 // [streams] the item's last P V complete
  kBarItem = kBarO + 2,              // [kSched]
  // Within a block: stream 1's statistics of a shared row are there / read.
  kBarStats = kBarItem + kSched,
  kBarStatsFree,
  kNumBars
};

// What the roles need of an item. Sent to both blocks as four 16-byte words.
struct alignas(16) Item {
  PfTile t;
  int head;    // head within the pass; -1: no further items
  int n0, n1;  // steps of each stream (0: none)
  int shared;  // the streams share the rows and alternate over the steps
};
static_assert(sizeof(Item) == 64, "four 16-byte words");

constexpr int kOffItems = (8 * kNumBars + 8 + 15) / 16 * 16;  // after TMEM address and abort flag
constexpr int kOffStats = kOffItems + kSched * 64;            // float2 [128]: stream 1's maximum and sum
constexpr int kSmemBytes = kOffBar + kOffStats + 1024 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");

__device__ __forceinline__ Item item_of(const PfTile& t, int head) {
  Item w;
  w.t = t;
  w.head = head;
  w.shared = t.rows <= 256;
  if (t.refused) {
    w.n0 = w.n1 = w.shared = 0;
  } else if (w.shared) {
    const int n = pf_steps(t.kv_begin, t.kv_end);
    w.n0 = (n + 1) / 2;
    w.n1 = n / 2;
  } else {
    w.n0 = pf_steps(t.kv_begin, min(t.first_end + 255, t.kv_end));
    w.n1 = pf_steps(t.kv_begin, t.kv_end);
  }
  return w;
}

// End of the positions that a stream's rows attend.
__device__ __forceinline__ int end_of(const Item& w, int x) {
  return x == 0 && !w.shared ? min(w.t.first_end + 255, w.t.kv_end) : w.t.kv_end;
}

// Tile rank and head of item `it`: head by head up to head `tail`, from there all
// heads' tiles of one rank before the next rank's.
__device__ __forceinline__ void split_item(int64_t it, int num_tiles, int heads, int tail, int* rank, int* head) {
  const int64_t in = it - static_cast<int64_t>(tail) * num_tiles;
  if (in < 0) {
    *head = static_cast<int>(it / num_tiles);
    *rank = static_cast<int>(it % num_tiles);
  } else {
    *rank = static_cast<int>(in / (heads - tail));
    *head = tail + static_cast<int>(in % (heads - tail));
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefill_attn_kernel(const __grid_constant__ PrefillMaps m, const __grid_constant__ PrefillArgs a, int head0, int heads) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 8 * kNumBars + 4);
  Item* board = reinterpret_cast<Item*>(smem + kOffBar + kOffItems);
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t cta = cluster_rank();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int count = 1;
      if (i >= kBarP && i < kBarP + 2) count = kSoftmaxWarps;                            // four of each block
      if (i >= kBarItemFree && i < kBarItemFree + kSched) count = 2 * (kSoftmaxWarps + 1);  // + issuer, + odd producer
      if (i == kBarStats || i == kBarStatsFree) count = kSoftmaxWarps / 2;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == kIssueWarp) {
    tmem_alloc2(smem_addr(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();  // barriers of both blocks are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lead0 = mapa(bar0, 0);  // the even block's barriers
  auto lead = [&](int i) -> uint32_t { return lead0 + 8u * i; };
  pdl_wait();
  auto fail = [&] {
    *abort_flag = 1;
    atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  };
  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool { return mbar_spin_warp(b, parity, abort_flag); };
  // The announced item comes from the even block: once its barrier is seen
  // complete (polls have the block's scope), acquire at the cluster's.
  auto acquire_item = [&](uint32_t i) { mbar_test_wait_cluster(bar(kBarItem + i % kSched), (i / kSched) & 1u); };

  if (warp >= kProducerWarp) setmaxnreg_dec<kRegsOther>();
  if (warp == kProducerWarp) {
    if (lane == 0) {
      const int num_tiles = hd->num_tiles;
      const int64_t items = static_cast<int64_t>(num_tiles) * heads;
      const int clusters = gridDim.x / 2;
      const PfTile* tiles = reinterpret_cast<const PfTile*>(a.ws + a.lay.sorted);
      const int tail_heads = (kTailItems * clusters + num_tiles - 1) / max(num_tiles, 1);
      const int tail = hd->even ? heads : max(0, heads - tail_heads);
      uint32_t k_steps = 0, v_steps = 0;  // steps whose copies are issued
      uint32_t q_use[2] = {0, 0};
      bool ok = true;
      auto load_item = [&](int64_t it) {
        int rank, head;
        if (it >= items) return item_of(PfTile{0, 0, 0, 0, 0, 0, 1, -1, {}}, -1);
        split_item(it, num_tiles, heads, tail, &rank, &head);
        return item_of(tiles[rank], head);
      };
      // The even block announces an item to both.
      auto announce = [&](uint32_t i, const Item& w) {
        if (!(ok = mbar_spin(bar(kBarItemFree + i % kSched), ((i / kSched) & 1u) ^ 1u, abort_flag))) return;
        const int* v = reinterpret_cast<const int*>(&w);
#pragma unroll
        for (uint32_t r = 0; r < 2; ++r) {
          const uint32_t rb = mapa(bar(kBarItem + i % kSched), r), dst = mapa(smem_addr(&board[i % kSched]), r);
          mbar_arrive_expect_tx_cluster(rb, sizeof(Item));
#pragma unroll
          for (int c = 0; c < 4; ++c) st_async_v4(dst + 16 * c, v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3], rb);
        }
      };
      Item w, w_next;
      if (cta == 0) {
        w_next = load_item(blockIdx.x >> 1);
        announce(0, w_next);
      }
      for (uint32_t i = 0; ok; ++i) {
        int64_t next = 0;
        if (cta == 0) {
          w = w_next;
        } else {
          if (!(ok = mbar_spin(bar(kBarItem + i % kSched), (i / kSched) & 1u, abort_flag))) break;
          acquire_item(i);
          w = board[i % kSched];
          mbar_arrive_cluster(lead(kBarItemFree + i % kSched));
        }
        if (w.head < 0) break;
        // The next item is drawn now, looked up and announced once this one's
        // first copies are under way.
        if (cta == 0) next = (gridDim.x >> 1) + static_cast<int64_t>(atomicAdd(&hd->next_item, 1));
        bool drawn = cta != 0;
        const int n = w.shared ? w.n0 + w.n1 : max(w.n0, w.n1);
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t s = k_steps % kStages, par = (k_steps / kStages) & 1u;
          const uint32_t dst = sbase + kOffRing + s * kStageBytes;
          const int row = w.t.base + w.t.kv_begin + j * kPfKvTile;
          if (!(ok = mbar_spin(bar(kBarKFree + s), par ^ 1u, abort_flag))) break;
          ++k_steps;
          if (cta == 0) mbar_arrive_expect_tx(bar(kBarKFull + s), 2 * kKBytes);
          tma2_load_3d(dst, &m.keys, lead(kBarKFull + s), 0, row + 64 * cta, w.head);
          tma2_load_3d(dst + kKChunk, &m.keys, lead(kBarKFull + s), 64, row + 64 * cta, w.head);
          tma2_load_2d(dst + 2 * kKChunk, &m.ropes, lead(kBarKFull + s), kDimCkv, row + 64 * cta);
          if (j == 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!ok || (x == 1 ? w.shared || w.n1 == 0 : w.n0 == 0)) continue;
              if (!(ok = mbar_spin(bar(kBarQFree + x), (q_use[x] & 1u) ^ 1u, abort_flag))) continue;
              ++q_use[x];
              if (cta == 0) mbar_arrive_expect_tx(bar(kBarQFull + x), 2 * kQBytes);
              for (int c = 0; c < 3; ++c)
                tma2_load_3d(sbase + x * kQBytes + c * kQChunk, &m.q, lead(kBarQFull + x), 64 * c, head0 + w.head,
                             w.t.q_row + 256 * x + 128 * cta);
            }
          }
          if (!ok || !(ok = mbar_spin(bar(kBarVFree + s), par ^ 1u, abort_flag))) break;
          ++v_steps;
          if (cta == 0) mbar_arrive_expect_tx(bar(kBarVFull + s), 2 * kVBytes);
          tma2_load_3d(dst + kKBytes, &m.values, lead(kBarVFull + s), 64 * cta, row, w.head);
          if (!drawn && j == 1) {
            w_next = load_item(next);
            announce(i + 1, w_next);
            drawn = true;
          }
        }
        if (!drawn && ok) {
          w_next = load_item(next);
          announce(i + 1, w_next);
        }
      }
      if (!ok) fail();
      if (*abort_flag && cta == 0) {  // let the copies in flight land (each wait bounded)
        for (uint32_t i = k_steps > kStages ? k_steps - kStages : 0; i < k_steps; ++i) {
          mbar_wait(bar(kBarKFull + i % kStages), (i / kStages) & 1u, nullptr);
          if (i < v_steps) mbar_wait(bar(kBarVFull + i % kStages), (i / kStages) & 1u, nullptr);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (q_use[x]) mbar_wait(bar(kBarQFull + x), (q_use[x] - 1) & 1u, nullptr);
      }
    }
  } else if (warp == kIssueWarp) {
    // One elected lane of the even block runs the whole role. Between two products
    // of the chain it does as little as it can: the next unit is worked out, and its
    // copies are waited for, while the tensor core is busy with the last one's.
    if (cta == 0 && elect_one()) {
      constexpr uint32_t idesc_qk = idesc_bf16(256, 128, false, false);
      constexpr uint32_t idesc_pv = idesc_f16(256, 128, false, true);  // P and V are f16
      const uint32_t q_lo = desc_lo(sbase), ring_lo = desc_lo(sbase + kOffRing);
      constexpr uint32_t kStageUnits = kStageBytes >> 4, kVUnits = kKBytes >> 4;
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && mbar_spin(b, parity, abort_flag); };
      // Generator of units: stream, step and item, with what the products need.
      uint32_t item_no = 0, stage = kStages - 1, par = 1, q_par = 0;  // (the first step turns to stage 0, parity 0)
      int j = 0, n = 0, n0 = 0, n1 = 0, left0 = 0, left1 = 0, ux = -1;
      bool shared = false;
      auto advance = [&]() -> bool {  // false: no further units
        if (ux == 0 && !shared && n1 > 0) {
          ux = 1;  // the same step's second stream
          return true;
        }
        if (ux >= 0) ++j;
        while (ux < 0 || j >= n) {
          wait(bar(kBarItem + (item_no & 1u)), (item_no >> 1) & 1u);
          if (!ok) return false;
          acquire_item(item_no);
          const Item& w = board[item_no & 1u];
          const int head = w.head;
          n0 = w.n0;
          n1 = w.n1;
          shared = w.shared != 0;
          left0 = end_of(w, 0) - w.t.kv_begin;
          left1 = end_of(w, 1) - w.t.kv_begin;
          mbar_arrive_cluster(lead(kBarItemFree + (item_no & 1u)));
          ++item_no;
          if (head < 0) return false;
          n = shared ? n0 + n1 : max(n0, n1);
          j = 0;
          ux = 0;
        }
        ux = shared ? (j & 1) : (j < n0 ? 0 : 1);
        stage = stage == kStages - 1 ? 0 : stage + 1;
        par ^= stage == 0 ? 1u : 0u;
        return true;
      };
      static_assert(kSched == 2, "item_no & 1");
      // A unit's P V, kept until its softmax is done.
      int p_x = -1, p_left = 0;
      uint32_t p_par = 0, p_v = 0, p_vfull = 0, p_vpar = 0, p_vfree = 0, p_o = 0;  // barriers: 0 is none
      bool p_acc = false;
      auto flush = [&] {
        if (p_x < 0 || !ok) return;
        if (p_vfull) wait(p_vfull, p_vpar);
        wait(bar(kBarP + p_x), (p_par >> p_x) & 1u);
        if (!ok) return;
        tc_fence_after();
        const uint32_t d = tmem + kColO + 128 * p_x, p = tmem + kColS + 128 * p_x;
        if (p_left > 112) {
          mma2_bf16_ts(d, p, p_v, idesc_pv, p_acc);
#pragma unroll
          for (int i = 1; i < 8; ++i) mma2_bf16_ts(d, p + 8 * i, p_v + 128 * i, idesc_pv, 1);
        } else {
#pragma unroll 1
          for (int i = 0; 16 * i < p_left; ++i) mma2_bf16_ts(d, p + 8 * i, p_v + 128 * i, idesc_pv, p_acc || i > 0);
        }
        if (p_vfree) mma2_commit(p_vfree);
        if (p_o) mma2_commit(p_o);
        p_par ^= 1u << p_x;
        p_x = -1;
      };
      bool have = advance();
      while (have && ok) {
        // The unit: constants of its products and its place in the item.
        const int x = ux;
        const bool first_of_step = shared || x == 0 || j >= n0, last_of_step = shared || x == 1 || n1 == 0;
        const int step_in = shared ? j >> 1 : j;
        const uint32_t d = tmem + kColS + 128 * x, q = q_lo + (shared ? 0 : x) * (kQBytes >> 4), k = ring_lo + stage * kStageUnits;
        const bool q_last = shared ? j == n - 1 : j == (x ? n1 : n0) - 1;
        const uint32_t u_stage = stage, u_par = par;
        const int u_left = (x ? left1 : left0) - j * kPfKvTile;
        const bool o_last = step_in == (x ? n1 : n0) - 1;
        const int q_buf = shared ? 0 : x;
        const bool q_first = shared ? j == 0 : j == 0;
        // S_x still holds P of this stream's previous unit where no other came between.
        if (p_x == x) flush();
        if (first_of_step) wait(bar(kBarKFull + u_stage), u_par);
        if (q_first) {
          wait(bar(kBarQFull + q_buf), (q_par >> q_buf) & 1u);
          q_par ^= 1u << q_buf;
        }
        if (!ok) break;
        // (the unit before, if its softmax is done by now or else later)
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 3; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma2_bf16_ss(d, q + c * (kQChunk >> 4) + 2 * e, k + c * (kKChunk >> 4) + 2 * e, idesc_qk, (c | e) != 0);
        mma2_commit(bar(kBarS + x));
        if (last_of_step) mma2_commit(bar(kBarKFree + u_stage));
        if (q_last) mma2_commit(bar(kBarQFree + q_buf));
        have = advance();  // works out the next unit before the wait
        flush();
        p_x = x;
        p_left = u_left;
        p_v = ring_lo + kVUnits + u_stage * kStageUnits;
        p_vfull = first_of_step ? bar(kBarVFull + u_stage) : 0;
        p_vpar = u_par;
        p_vfree = last_of_step ? bar(kBarVFree + u_stage) : 0;
        p_o = o_last ? bar(kBarO + x) : 0;
        p_acc = step_in != 0;
      }
      flush();
      if (!ok) fail();
      mma2_commit(bar(kBarDrain));
      mbar_wait(bar(kBarDrain), 0, nullptr);
    }
  } else if (warp < kSoftmaxWarps) {
    setmaxnreg_inc<kRegsSoftmax>();
    // Warp w works for stream w >> 2 on TMEM lane quarter w & 3, a row a thread.
    const int x = warp >> 2;
    const int lrow = (warp & 3) * 32 + lane;  // row of this block
    const uint32_t tbase = tmem + (static_cast<uint32_t>(lrow & ~31) << 16);
    const uint32_t tS = tbase + kColS + 128 * x, tO = tbase + kColO + 128 * x;
    float2* stats = reinterpret_cast<float2*>(smem + kOffBar + kOffStats);
    const float scale = a.scale_log2;
    const uint64_t scale2 = f2_make(scale, scale);
    const float threshold = kRescaleThreshold / scale;  // in units of S
    const bool odd_bins = hd->odd_bins != 0;
    uint32_t s_use = 0, o_use = 0, o1_use = 0, stats_use = 0;
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      if (!(ok = warp_wait(bar(kBarItem + i % kSched), (i / kSched) & 1u))) break;
      acquire_item(i);
      const Item w = board[i % kSched];
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead(kBarItemFree + i % kSched));
      if (w.head < 0) break;
      const int r = 128 * cta + lrow + (w.shared ? 0 : 256 * x);  // row of the tile
      const bool valid = r < w.t.rows;
      const bool any = r - lane < w.t.rows;  // any row of this warp
      const int q_row = w.t.q_row, head = head0 + w.head;
      auto out_row = [&] { return (static_cast<int64_t>(q_row) + r) * a.num_heads + head; };
      auto out_ptr = [&] { return static_cast<uint8_t*>(a.out) + out_row() * (kDimV * 2); };
      if (w.t.refused) {
        if (valid) {
          const uint32_t nan8[8] = {0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u,
                                    0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
          for (int v = 0; v < kDimV * 2 / 32; ++v) st_global_v8(out_ptr() + 32 * v, nan8);
          if (a.lse) a.lse[out_row()] = CUDART_NAN_F;
        }
        continue;
      }
      const int n = x ? w.n1 : w.n0, n1 = w.n1;
      const bool shared = w.shared != 0;
      // Where the row's sums go if this is a piece of a split tile.
      const int part_row = w.t.part_row;
      auto part = [&] { return static_cast<int64_t>(head - head0) * a.lay.part_rows + part_row + r; };
      const bool split = part_row >= 0;
      if (n == 0) {
        if (x == 0 && n1 > 0) ++o1_use;
        if (split && valid && !(x == 1 && shared))
          reinterpret_cast<float2*>(a.ws + a.lay.part_stats)[part()] = make_float2(kNoMax, 0.f);
        continue;
      }
      // The row's range, relative to the first key of the stream's first step.
      const int stride = w.shared ? 2 * kPfKvTile : kPfKvTile;
      const int off = w.t.kv_begin + (w.shared ? kPfKvTile * x : 0);
      const int end = min(w.t.first_end + r, end_of(w, x)) - off;
      const int begin = a.window > 0 ? max(0, w.t.first_end + r - a.window) - off : -off;
      // Steps [full0, full1) have no position to mask in any row of the warp.
      const int full0 = __reduce_max_sync(0xffffffffu, begin > 0 ? (begin + stride - 1) / stride : 0);
      const int full1 = __reduce_min_sync(0xffffffffu, end >= kPfKvTile ? (end - kPfKvTile) / stride + 1 : 0);
      float mx_ref = kNoMax, l = 0.f;
      // The kept positions among keys [32 g, 32 g + 32) of step j, a bit each.
      auto kept = [&](int j, int g) {
        const int b0 = begin - j * stride, e0 = end - j * stride;
        const uint32_t above = e0 >= 32 * g + 32 ? ~0u : (1u << max(e0 - 32 * g, 0)) - 1u;
        const uint32_t below = b0 >= 32 * g + 32 ? ~0u : (1u << max(b0 - 32 * g, 0)) - 1u;
        return above & ~below;
      };
      // Takes mx as the reference if it exceeds the one of now by the threshold.
      auto move_reference = [&](int j, float mx) {
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
            for (int v = 0; v < 16; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * alpha);
            tmem_st16(tO + 16 * c, o);
          }
        }
      };
      // (uniform: all keys of the step have the bin k0)
      auto weights_of_odd_bins = [&](int j, uint32_t bins, int k0, auto uniform) {
        constexpr bool kUniform = uniform.value;
        auto bin_at = [&](int key) {
          if constexpr (kUniform) return k0;
          else return static_cast<int>(static_cast<int8_t>(__shfl_sync(0xffffffffu, bins, key >> 2) >> (8 * (key & 3))));
        };
        const float per_bin = fminf(threshold * kBinSteps, 1e38f);  // kBinBits in units of S
        uint32_t s[32];
        auto scores = [&](int g) {  // with their keys' e
          tmem_ld32(tS + 32 * g, s);
          tmem_wait_ld();
          const uint32_t keep = kept(j, g);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float e = fmaf(static_cast<float>(bin_at(32 * g + c)), per_bin, __uint_as_float(s[c]));
            s[c] = keep & (1u << c) ? __float_as_uint(e) : 0xff800000u;
          }
        };
        float mx = -CUDART_INF_F;
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          scores(g);
#pragma unroll
          for (int c = 0; c < 32; c += 2) mx = fmax3(mx, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        }
        move_reference(j, mx);
        const float neg = kWeightShift - mx_ref * scale;
        const uint64_t neg2 = f2_make(neg, neg);
        uint64_t sum2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
        auto unit = [](int k) { return __int_as_float((127 - kBinBits * k) << 23); };  // 2^(-e)
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          scores(g);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float t0, t1;
            f2_split(f2_fma(f2_make(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, neg2), t0, t1);
            const float p0 = exp2_approx(t0), p1 = exp2_approx(t1);
            const uint64_t units = f2_make(unit(bin_at(32 * g + 2 * c)), unit(bin_at(32 * g + 2 * c + 1)));
            sum2[c & 1] = f2_fma(f2_make(p0, p1), units, sum2[c & 1]);
            s[c] = pack_f16x2(p0, p1);
          }
          tmem_st16(tS + 16 * g, s);  // (over scores that are read already)
        }
        float s0, s1, s2, s3;
        f2_split(sum2[0], s0, s1);
        f2_split(sum2[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
      };
      auto step_of_odd_bins = [&](int j) {
        // The bins of keys 4 lane .. 4 lane + 3. (Keys behind the request's have any byte; they are masked.)
        // (rows x heads x 513 bytes lie in the workspace: 32 bits are enough)
        const uint32_t at = static_cast<uint32_t>(w.head * a.lay.kv_capacity) + w.t.base + off + j * stride + 4 * lane;
        const uint32_t bytes = *reinterpret_cast<const uint32_t*>(a.ws + a.lay.bins + at);
        uint32_t bins = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          bins |= (min(max(static_cast<int8_t>(bytes >> (8 * i)), -kMostBin), kMostBin) & 0xff) << (8 * i);
        const int k0 = static_cast<int8_t>(__shfl_sync(0xffffffffu, bins, 0));
        if (__all_sync(0xffffffffu, bins == (k0 & 0xff) * 0x01010101u)) weights_of_odd_bins(j, bins, k0, std::true_type{});
        else weights_of_odd_bins(j, bins, k0, std::false_type{});
      };
      if (odd_bins) {
        for (int j = 0; j < n; ++j) {
          if (!(ok = warp_wait(bar(kBarS + x), s_use & 1u))) break;
          ++s_use;
          if (any) {
            tc_fence_after();
            step_of_odd_bins(j);
            tmem_wait_st();
            tc_fence_before();
          }
          if (lane == 0) mbar_arrive_cluster(lead(kBarP + x));
        }
      }
      for (int j = odd_bins ? n : 0; j < n; ++j) {
        if (!(ok = warp_wait(bar(kBarS + x), s_use & 1u))) break;
        ++s_use;
        if (any) {
          tc_fence_after();
          uint32_t s[128];
          // P against the reference maximum as it stands, the sum and maximum of
          // P beside it: no pass over S before the exponentials.
          float neg = kWeightShift - mx_ref * scale;
          uint64_t sum2[2];
          float top;
          auto weights = [&] {
            const uint64_t neg2 = f2_make(neg, neg);
            float top1 = 0.f;
            top = 0.f;
            sum2[0] = sum2[1] = f2_make(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              float t0, t1;
              f2_split(f2_fma(f2_make(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, neg2), t0, t1);
              const float p0 = exp2_approx(t0), p1 = exp2_approx(t1);
              sum2[c & 1] = f2_add(sum2[c & 1], f2_make(p0, p1));
              if (c & 1) top1 = fmax3(top1, p0, p1);
              else top = fmax3(top, p0, p1);
              s[c] = pack_f16x2(p0, p1);
            }
            top = fmaxf(top, top1);
          };
          const bool full = j >= full0 && j < full1;
          for (bool anew = j == 0;; anew = true) {
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
            tmem_wait_ld();
            if (!full) {
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const uint32_t keep = kept(j, g);
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!(keep & (1u << c))) s[32 * g + c] = 0xff800000u;
              }
            }
            if (anew) {
              // The stream's first step, or scores that outgrow the reference: take
              // the maximum, rescale what there is.
              float mx = -CUDART_INF_F, mx1 = -CUDART_INF_F;
#pragma unroll
              for (int c = 0; c < 128; c += 4) {
                mx = fmax3(mx, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                mx1 = fmax3(mx1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
              }
              move_reference(j, fmaxf(mx, mx1));
              neg = kWeightShift - mx_ref * scale;
            }
            weights();
            if (anew || !__any_sync(0xffffffffu, top > kMostWeight)) break;
          }
          tmem_st32(tS, s);
          tmem_st32(tS + 32, s + 32);
          float s0, s1, s2, s3;
          f2_split(sum2[0], s0, s1);
          f2_split(sum2[1], s2, s3);
          l += (s0 + s1) + (s2 + s3);
          tmem_wait_st();  // (of the whole warp: one lane may announce it)
          tc_fence_before();
        }
        if (lane == 0) mbar_arrive_cluster(lead(kBarP + x));
      }
      if (!ok) break;
      if (x == 1 && shared) {
        // Stream 0 stores the row: hand over its maximum and sum, keep O until read.
        stats[lrow] = make_float2(mx_ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarStats));
        if (!(ok = warp_wait(bar(kBarStatsFree), stats_use++ & 1u))) break;
        if (!(ok = warp_wait(bar(kBarO + 1), o_use++ & 1u))) break;
        continue;
      }
      if (!(ok = warp_wait(bar(kBarO + x), o_use++ & 1u))) break;
      float f0 = 1.f, f1 = 0.f;  // factors of the streams' O
      const bool merge = shared && n1 > 0;
      if (merge) {
        if (!(ok = warp_wait(bar(kBarStats), stats_use++ & 1u))) break;
        if (!(ok = warp_wait(bar(kBarO + 1), o1_use & 1u))) break;
        mbar_test_wait(bar(kBarStats), (stats_use - 1) & 1u);  // (every lane acquires what it reads next)
        const float2 other = stats[lrow];
        const float both = fmaxf(mx_ref, other.x);
        f0 = exp2_approx((mx_ref - both) * scale);
        f1 = exp2_approx((other.x - both) * scale);
        l = l * f0 + other.y * f1;  // (a NaN of either stays: 0 * NaN)
        mx_ref = both;
      }
      if (x == 0 && n1 > 0) ++o1_use;  // (phases of stream 1's barrier, waited for or not)
      tc_fence_after();
      if (any) {
        // (every valid row attends itself: l > 0; a piece is scaled when joined)
        const float inv = split ? 1.f : a.out_scale / l;
        f0 *= inv;
        f1 *= inv;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int v = 0; v < 32; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * f0);
          if (merge) {
            uint32_t o1[32];
            tmem_ld32(tO + 128 + 32 * c, o1);
            tmem_wait_ld();
#pragma unroll
            for (int v = 0; v < 32; ++v) o[v] = __float_as_uint(fmaf(__uint_as_float(o1[v]), f1, __uint_as_float(o[v])));
          }
          if (valid && split) {
#pragma unroll
            for (int v = 0; v < 4; ++v) st_global_v8(reinterpret_cast<float*>(a.ws + a.lay.part_o) + part() * kDimV + 32 * c + 8 * v, o + 8 * v);
          } else if (valid) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t pk[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                pk[e] = pack_bf16x2(__uint_as_float(o[16 * v + 2 * e]), __uint_as_float(o[16 * v + 2 * e + 1]));
              st_global_v8(out_ptr() + 64 * c + 32 * v, pk);
            }
          }
        }
        if (split && valid) reinterpret_cast<float2*>(a.ws + a.lay.part_stats)[part()] = make_float2(mx_ref, l);
        else if (a.lse && valid) a.lse[out_row()] = (mx_ref * scale + log2f(l * kWeightUnit)) * 0.69314718055994531f;
      }
      tc_fence_before();
      if (merge) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarStatsFree));
      }
    }
    if (!ok) fail();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // no block ends while the other's products or arrivals reach into it
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc2(tmem, 512);
}

}  // namespace

cudaError_t launch_prefill_attn(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(prefill_attn_kernel, kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  const int pairs = sm_count() / 2;
  if (pairs <= 0) return cudaErrorInvalidDevice;
  const int64_t most = (a.lay.max_tiles + (pf_may_split(a.max_kv) ? kPfMostPieces : 0)) * heads;
  return launch_pdl(prefill_attn_kernel, dim3(2 * static_cast<unsigned>(most < pairs ? most : pairs)), dim3(kThreads),
                    kSmemBytes, stream, m, a, head0, heads);
}

}  // namespace mla
