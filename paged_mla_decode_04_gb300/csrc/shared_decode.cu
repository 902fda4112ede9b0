// Attention of a decode over shared prefixes, on the tensor core: rows of queries (of all
// requests and heads of a tile) against positions that they share, 576 dims a key, the
// first 512 of which are the value.
//   S_t = scale q . K_t,  out = sum_t softmax(S)_t K_t[0:512]
//
// 2 * (576 + 512) flops a row and position: with 256 rows to a position it is the tensor
// core that bounds it, and the accumulator that shapes it. 256 rows of 512 values in fp32
// fill two SMs' tensor memory, with nothing left for scores. So a cluster of four blocks
// works as two pairs (products of M = 256 over two SMs, each with half of the columns'
// operand in its shared memory):
//   blocks 0, 1  S = Q K^T and its softmax. Tensor memory: Q's 512 dims (256 columns of
//                16-bit pairs), two buffers of S (128 columns each); the rope dims of Q and a
//                ring of K's pieces in shared memory.
//   blocks 2, 3  O += P V. Tensor memory: O (512 columns). Shared memory: three buffers of
//                P, a ring of V's pieces.
// The two products are 576 and 512 dims long, so both pairs are busy, and neither waits
// for the other within a block of positions: weights P go one way, from the softmax
// warps' registers by way of their own shared memory into the other pair's (32 KB a block's
// 128 positions and 2,304 cycles of products), with a factor for each row by which O is
// rescaled where the running maximum moved. The first pair is up to five blocks of
// positions ahead.
//
// A cluster works through its items (see shared_internal.h): blocks of a tile's
// positions, those that all its rows share and then each request's own. In the latter only
// the request's rows take part: other rows' scores are not looked at, and the product's
// row mask leaves their accumulators alone, so that one request's cache never touches
// another's result. Positions outside a segment are masked by selection in S; their rows of
// V are made zero, or left out 16 at a time.
//
// What bounds it: the tensor core, at 2,690 cycles a block of 256 rows and 128 positions (the
// scores' products take 2,304 of them at the full rate, the values' 2,048; 8 of 152 SMs have no
// cluster; long calls meet the power limit) where blocks are many: 1.38 PFLOP/s of 16,384 rows at
// 8,450 positions, 1.36 of 1,024 rows at 65,700, 108 us: 71 % of a library product's rate in
// short, 79 % of its sustained one. A tile with few rows, and a request's own positions, take the
// same products. Where blocks are few, what a call cannot overlap: 2 us until queries are in
// place, 4 from the first scores to the first product of values, 4 to 6 for an item's results
// (they go out at L2's rate, of all SMs at once) and 3 for the join of its pieces, so that 4
// tiles of 100 blocks take 41 us. e4m3 pools: four warps widen a block's codes in 2,800
// cycles, about as long as the products, and queries become f16; 1,024 rows at 65,700 positions
// take 127 us. (Of the roles' code 108 bytes of registers are spilled, 276 for e4m3 pools.)
#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "../../include/mla_decode.h"
#include "ptx_shared.cuh"
#include "shared_internal.h"

namespace mla {
namespace {

constexpr int kWorkers = 8;                 // warps of softmax or accumulators, two groups of four
constexpr int kProducerWarp = kWorkers, kIssueWarp = kWorkers + 1, kSendWarp = kWorkers + 2, kProducerWarp2 = kWorkers + 3;
constexpr int kConvertWarp = kWorkers + 4;  // (fp8 pools) four that widen the codes
// Registers a thread after setmaxnreg; they add up to the launch's 3 x 168 (bf16 pools) or
// 4 x 128.
template <bool kFp8>
struct Regs {
  static constexpr int kThreads = kFp8 ? 512 : 384;
  static constexpr int kWorker = kFp8 ? 176 : 208, kOther = kFp8 ? 64 : 88, kConvert = 96;
};
static_assert(2 * Regs<false>::kWorker + Regs<false>::kOther == 3 * 168, "register split");
static_assert(2 * Regs<true>::kWorker + Regs<true>::kOther + Regs<true>::kConvert == 4 * 128, "register split");
constexpr int kChunk = 64 * 128;            // [64 positions][64 dims]
// Scores' pair: K in stages of three chunks (192 dims), three stages a block.
constexpr int kKStages = 5, kKStageBytes = 3 * kChunk, kKParts = 3;
constexpr int kOffQRope = kKStages * kKStageBytes;  // [128 rows][64 dims]
// Accumulators' pair: P of 128 rows, two chunks of 64 positions; V in stages of 64
// positions, four chunks (256 dims).
constexpr int kPChunk = 128 * 128, kPBytes = 2 * kPChunk, kPBuffers = 3;
constexpr int kOffV = kPBuffers * kPBytes;
constexpr int kVStages = 4, kVStageBytes = 4 * kChunk;
constexpr int kOffAlpha = kOffV + kVStages * kVStageBytes;  // float [kPBuffers][128]
constexpr int kOffStats = kOffAlpha + kPBuffers * 128 * 4;  // float2 [128]
// Scores' pair: P on its way to the other; each row's reference maximum, as the block
// before left it; the sum and reference of the group that an item's last block is not of.
constexpr int kOffPOut = kOffQRope + 128 * 128;
constexpr int kOffRef = kOffPOut + 2 * kPBytes;             // float [128]
constexpr int kOffSum = kOffRef + 128 * 4;                  // float2 [2 items][128]
constexpr int kOffAlphaOut = kOffSum + 2 * 128 * 8;         // float [2 groups][128]
constexpr int kOffBar = kOffStats + 128 * 8;
constexpr int kOffNotes = kOffAlphaOut + 2 * 512;            // Block [kNotes]
constexpr int kNotes = 4;  // (the copies run less than four blocks ahead of the softmax)
static_assert(kOffNotes + kNotes * 32 <= kOffBar, "both pairs' buffers end before the barriers");

enum {
  // In the scores' pair. (Of its first block: K landed, Q in place, S read.)
  kBarKFull = 0,                       // [kKStages]
  kBarKFree = kBarKFull + kKStages,    // [kKStages]
  kBarQ = kBarKFree + kKStages,
  kBarS = kBarQ + 1,                   // [2] scores complete
  kBarSFree = kBarS + 2,               // [2]
  kBarStaged = kBarSFree + 2,          // [2 groups] P is ready to leave
  kBarOutFree = kBarStaged + 2,        // [2 groups] P has left
  kBarPFree = kBarOutFree + 2,         // [kPBuffers] P multiplied (in both pairs)
  kBarStatsFree = kBarPFree + kPBuffers,
  kBarRef = kBarStatsFree + 1,         // [2 groups][4 warps] the reference is there
  kBarSum = kBarRef + 8,               // [2 items][4 warps] the other group's sum is
  // In the accumulators' pair. (Of its first block: P ready, O read.)
  kBarVFull = kBarSum + 8,       // [kVStages]
  kBarVFree = kBarVFull + kVStages,    // [kVStages]
  kBarNote = kBarVFree,                // [kNotes] (scores' pair) the block is described
  kBarP = kBarVFree + kVStages,        // [kPBuffers] weights have arrived
  kBarQIn = kBarP,                     // [8 warps] (scores' pair) queries have landed
  kBarPReady = kBarP + kPBuffers,      // [kPBuffers] and O is rescaled, V landed
  kBarO = kBarPReady + kPBuffers,      // an item's last product complete
  kBarStats = kBarO + 1,               // an item's maxima and sums have arrived
  kBarOFree = kBarStats + 1,           // (from kBarP on: enough for the queries' eight)
  // (fp8 pools) In either pair: codes have landed; every warp that widens has read its share.
  kBarRaw = kBarOFree + 1,             // [most stages]
  kBarMeet = kBarRaw + (kKStages > kVStages ? kKStages : kVStages),
  kNumBars = kBarMeet + 1
};

// (all that a block may have: its start has to be at a multiple of 1,024, see the kernel)
constexpr int kSmemBytes = kOffBar + 8 * kNumBars + 8;
static_assert(kSmemBytes <= 232448, "shared memory");
static_assert(kBarQIn + kWorkers <= kBarRaw, "barriers that the other pair alone uses");
constexpr uint32_t kColS = 256;             // + 128 a buffer; Q from 0
constexpr float kRescaleThreshold = 8.0f;   // log2 units
// The reference of a row that has seen no position: below every score, and finite, so that
// a score of -inf against it is a weight of zero.
constexpr float kNoMax = -1e30f;
// Weights are this many powers of two larger than 2^(score - reference), in P, O and l alike (the
// maximum that stands for them is smaller by as much), so that those of f16 use its range: with
// the reference's lag they reach 2^15, and only weights below 2^-21 of a row's largest lose bits,
// to 2^-32 of it. (Without, 65,536 positions of 2^-25 each were lost beside one of 1. bf16 has
// fp32's range.)
template <bool kFp8>
constexpr float kWeightShift = kFp8 ? 7.0f : 0.0f;
constexpr uint16_t kScorePair = 0x3, kAccPair = 0xc;  // blocks of the cluster

// A block of positions, as every role sees it.
struct alignas(16) Block {
  int owner;
  int t0;              // first position
  int v0, v1;          // those of the segment: [t0 + v0, t0 + v1)
  int row_lo, row_hi;  // rows that attend it
  int end;             // row of query position i: below t0 + end + i
  int add;             // to what these rows have already
};
static_assert(sizeof(Block) == 32 && kNotes <= kVStages, "two 16-byte words");

// Walks an item's blocks, a segment ahead in what it has loaded.
struct Walk {
  const ShSegment* segs;
  ShSegment s, next;
  int k, last, x, end, begin;
  bool with_prefix;  // the item has blocks of the prefix
  __device__ __forceinline__ void start(const ShDecodeArgs& a, const ShItem& it) {
    segs = reinterpret_cast<const ShSegment*>(a.ws + a.lay.segs);
    k = it.seg;
    last = it.seg_last;
    x = begin = it.begin;
    end = it.end;
    with_prefix = it.begin < it.prefix_end;
    s = it.first;
    next = segs[min(k + 1, last)];
  }
  __device__ __forceinline__ bool more() const { return x < end; }
  __device__ __forceinline__ Block get() {
    if (k < last && x >= next.block0) {
      s = next;
      ++k;
      next = segs[min(k + 1, last)];
    }
    Block b;
    b.owner = s.owner;
    b.t0 = s.tok0 + (x - s.block0) * kShTokens;
    b.v0 = max(s.tok_lo - b.t0, 0);
    b.v1 = min(s.tok_hi - b.t0, kShTokens);
    b.row_lo = s.row_lo;
    b.row_hi = s.row_hi;
    b.end = s.base + 1 - b.t0;
    // (rows of a request's own blocks have the prefix's before them, where the item has)
    b.add = x > max(s.block0, begin) || (with_prefix && s.base != s.tok_hi);
    ++x;
    return b;
  }
};

// Four lanes' 128 bytes each, as four pieces of 32, transposed: piece j of lane i becomes
// piece i of lane j. A lane that has 128 bytes of its own row writes them by way of this, so
// that a store covers eight whole lines (as the rows lie it is 32 pieces of 32 bytes, and
// an item's results took 2 us longer to go out).
__device__ __forceinline__ void turn(uint32_t* o, int lane) {
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      const int lo = d == 1 ? 16 * pair : 8 * pair, hi = lo + 8 * d;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? o[lo + e] : o[hi + e], d);
        if (up) o[lo + e] = got;
        else o[hi + e] = got;
      }
    }
  }
}

struct Params {
  // bf16 pools: as [rows][576], box {64, positions of a copy}; where a copy brings 64 positions
  // as [chunk][rows][64], boxes of three and four chunks. fp8 pools: (none), boxes of 192 and
  // of 256 codes. Queries as [rows][576], boxes of 32 rows and 64 dims.
  CUtensorMap rows, chunks3, chunks4, q;
  ShDecodeArgs a;
};

template <bool kFp8>
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(Regs<kFp8>::kThreads, 1)
    shared_decode_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const ShDecodeArgs& a = p.a;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 8 * kNumBars + 4);
  ShHeader* hd = reinterpret_cast<ShHeader*>(a.ws);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), half = rank & 1;
  const bool scores = rank < 2;  // which pair
  const int unit = sh_copy_tokens(a.page_size), page_shift = 31 - __clz(a.page_size);
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int count = 1;
      if (i == kBarQ) count = 2 * kWorkers;
      if (i >= kBarSFree && i < kBarSFree + 2) count = 8;                       // a group of both blocks
      if (i >= kBarStaged && i < kBarStaged + 2) count = 4;                     // a group of one
      if (i == kBarStats) count = 4;
      if (kFp8 && i >= kBarKFull && i < kBarKFull + kKStages) count = 8;        // warps that widen, of both blocks
      if (kFp8 && i >= kBarVFull && i < kBarVFull + kVStages) count = 4;        // those of one
      if (i == kBarMeet) count = 4;
      if (i >= kBarPReady && i < kBarPReady + kPBuffers) count = 2 * kWorkers;
      if (i == kBarOFree) count = 2 * kWorkers;
      if (i == kBarStatsFree) count = kWorkers;
      if (scores && i >= kBarQIn && i < kBarQIn + kWorkers) count = 1;
      mbar_init(bar(i), count);
    }
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 0 && lane == 0 && scores) tma_prefetch_map(&p.q);
  if (warp == kProducerWarp && lane == 0) tma_prefetch_map(unit != 64 && !kFp8 ? &p.rows : scores ? &p.chunks3 : &p.chunks4);
  if (warp == kIssueWarp) {
    tmem_alloc2(smem_addr(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();  // all blocks' barriers are initialised before any arrival from another
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // This pair's first block's barriers; the block that this one's rows are shared with.
  const uint32_t lead0 = mapa(bar0, rank & 2), peer0 = mapa(bar0, rank ^ 2);
  auto lead = [&](int i) -> uint32_t { return lead0 + 8u * i; };
  auto peer = [&](int i) -> uint32_t { return peer0 + 8u * i; };
  pdl_wait();
  auto fail = [&] {
    *abort_flag = 1;
    atomicOr(&hd->status, MLA_STATUS_TIMEOUT);
  };
  // Waits of a thread and of a warp. What the first two are for is ordered by tcgen05 and
  // proxy fences before the arrival, or by the copy's own completion (an acquire at the
  // cluster's scope takes 2,000 cycles beside products in flight); the others acquire what
  // this block's or the cluster's threads wrote to shared memory, for the whole warp.
  auto spin = [&](uint32_t b, uint32_t parity) -> bool { return mbar_spin(b, parity, abort_flag); };
  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool { return mbar_spin_warp(b, parity, abort_flag); };
  auto warp_wait_block = [&](uint32_t b, uint32_t parity) -> bool {
    if (!mbar_spin_warp(b, parity, abort_flag)) return false;
    __syncwarp();
    return true;
  };
  auto warp_wait_cluster = [&](uint32_t b, uint32_t parity) -> bool {
    if (!mbar_spin_warp(b, parity, abort_flag)) return false;
    if (lane == 0) mbar_test_wait_cluster(b, parity);
    __syncwarp();
    return true;
  };
  const int cluster = blockIdx.x >> 2;
  Block* notes = reinterpret_cast<Block*>(smem + kOffNotes);
  // (Buffers at another start than the tensor core's patterns ask for: never seen; nothing is
  // computed then, and the status tells.)
  const ShCluster* record = reinterpret_cast<const ShCluster*>(a.ws + a.lay.clusters) + cluster;
  const ShItem* items = reinterpret_cast<const ShItem*>(a.ws + a.lay.items);
  int item0 = record->item0, item1 = record->item1;  // (asked for with the header)
  auto item = [&](int k) -> const ShItem& { return k == item0 ? record->first : items[k]; };
  const bool planned = sh_planned(hd, a) && (sbase & 1023u) == 0;
  if (!planned && threadIdx.x == 0 && rank == 0) atomicOr(&hd->status, MLA_STATUS_PLAN_MISMATCH);
  if (!planned || cluster >= hd->num_clusters) item0 = item1 = 0;

  if (warp >= kConvertWarp) {
    if (kFp8) setmaxnreg_dec<Regs<kFp8>::kConvert>();
  } else if (warp >= kWorkers) {
    setmaxnreg_dec<Regs<kFp8>::kOther>();
  }
  if (warp == kProducerWarp || warp == kProducerWarp2) {
    // Each block of the scores' pair brings its 64 of a block's positions, all dims; each of
    // the accumulators' pair all positions, its 256 value dims. A lane has a copy's page id,
    // asked for a block ahead; a stage's copies are one instruction of several lanes, or one copy.
    // Two warps take the even and the odd blocks: one needs 2,300 cycles for a block, as long
    // as the products. (With ids looked up as they were needed, and a copy for each 64 dims
    // one after the other, it was 6,100.)
    const uint32_t mine = warp == kProducerWarp ? 0 : 1;
    const int subs = (scores ? 64 : 128) / unit;  // copies along the positions
    const int offset = (scores ? 64 * static_cast<int>(half) : 0) + unit * lane;
    const int layer_row0 = static_cast<int>(static_cast<int64_t>(a.layer) * a.num_pages * a.page_size);
    const int no_row = static_cast<int>(static_cast<int64_t>(a.num_layers) * a.num_pages * a.page_size);  // reads as zeros
    bool ok = true;
    uint32_t issued = 0;  // stages, of blocks up to this warp's last
    struct Page {
      int id;  // kNone: no position of the segment
      int t;
    };
    constexpr int kNone = INT_MIN;
    int owner = -1, list_pages = a.max_blocks;
    const int32_t* list = nullptr;
    auto ask = [&](const Block& b) {
      if (b.owner != owner) {
        owner = b.owner;
        if (a.page_indptr) {
          list = a.page_ids + a.page_indptr[owner];
          list_pages = a.page_indptr[owner + 1] - a.page_indptr[owner];
        } else {
          list = a.page_ids + static_cast<int64_t>(owner) * a.max_blocks;
        }
      }
      const int t = b.t0 + offset, j = t >> page_shift;
      const bool in = lane < subs && t < b.t0 + b.v1 && t + unit > b.t0 + b.v0;
      return Page{!in ? kNone : j < list_pages ? list[j] : -1, t};
    };
    auto row_of = [&](const Page& g) -> int {
      if (g.id >= 0 && g.id < a.num_pages) return layer_row0 + (g.id << page_shift) + (g.t & (a.page_size - 1));
      if (g.id != kNone && scores) atomicOr(&hd->status, MLA_STATUS_BAD_PAGE);
      return no_row;
    };
    constexpr uint32_t kStages = kKStages;
    uint32_t n0 = 0;  // blocks of the items before
    for (int k = item0; k < item1 && ok; ++k) {
      const ShItem it = item(k);
      Walk w;
      w.start(a, it);
      const uint32_t blocks = it.end - it.begin;
      uint32_t at = (n0 ^ mine) & 1u;  // this warp's first block of the item
      Block now = {}, next = {};
      Page page = {kNone, 0}, next_page = {kNone, 0};
      auto take = [&] {  // a block of this warp's; the next is the other's
        const Block b = w.get();
        if (w.more()) w.get();
        return b;
      };
      if (at == 1 && w.more()) w.get();
      if (at < blocks) {
        now = take();
        page = ask(now);
      }
      if (scores && mine == 0 && lane == 0 && k + 1 < item1) {  // the next item's queries (each block its rows) on their way to L2
        const int row0 = item(k + 1).row0 + 128 * static_cast<int>(half);
        const int rows = min(item(k + 1).rows - 128 * static_cast<int>(half), 128);
        if (rows > 0)
          prefetch_l2(static_cast<const uint8_t*>(a.q) + static_cast<int64_t>(row0) * (kDimRow * 2), rows * (kDimRow * 2));
      }
      for (; at < blocks && ok; at += 2) {
        if (w.more()) {
          next = take();
          next_page = ask(next);
        }
        const int row = row_of(page);
        const uint32_t n = n0 + at;
        if (scores) {
          const int i = unit == 64 ? 0 : lane / 3, c = lane % 3;
          const int copied = __shfl_sync(0xffffffffu, row, i & 31);
#pragma unroll 1
          for (uint32_t part = 0; part < kKParts; ++part) {
            const uint32_t use = kKParts * n + part, stage = use % kStages;
            // (This wait is the longest: as one that lets other warps issue, 54.0 us instead of 54.9
            // a decode of an fp8 pool. Its lanes wait one by one, so they vote: all go on or none.)
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarKFree + stage), (use / kStages & 1u) ^ 1u, abort_flag)))) break;
            issued = use + 1;
            if (part == 0 && lane == 0) {
              // What the softmax warps need of the block. (Now that block n - 2 is multiplied in
              // part, its buffer of scores was free: block n - 4's note has been read.)
              notes[n % kNotes] = now;
              mbar_arrive(bar(kBarNote + n % kNotes));
            }
            const uint32_t dst = sbase + stage * kKStageBytes, full = lead(kBarKFull + stage);
            if (kFp8) {  // codes, behind the room that they will take when widened
              if (lane == 0) mbar_arrive_expect_tx(bar(kBarRaw + stage), kKStageBytes / 2);
              if (lane < subs)
                tma_load_2d(dst + kKStageBytes / 2 + lane * unit * 192, &p.chunks3, bar(kBarRaw + stage), 192 * part, row);
            } else {
              if (half == 0 && lane == 0) mbar_arrive_expect_tx(bar(kBarKFull + stage), 2 * kKStageBytes);
              if (unit == 64) {
                if (lane == 0) tma2_load_3d(dst, &p.chunks3, full, 0, copied, 3 * part);
              } else if (lane < 3 * subs) {
                tma2_load_2d(dst + c * kChunk + i * unit * 128, &p.rows, full, 64 * (3 * part + c), copied);
              }
            }
          }
        } else {
#pragma unroll 1
          for (uint32_t part = 0; part < 2; ++part) {
            const uint32_t use = 2 * n + part, stage = use % kVStages;
            if (!(ok = warp_wait(bar(kBarVFree + stage), (use / kVStages & 1u) ^ 1u))) break;
            issued = use + 1;
            const uint32_t dst = sbase + kOffV + stage * kVStageBytes;
            const uint32_t full = bar((kFp8 ? kBarRaw : kBarVFull) + stage);
            const int j = lane - static_cast<int>(part) * (subs / 2);
            if (lane == 0) mbar_arrive_expect_tx(full, kFp8 ? kVStageBytes / 2 : kVStageBytes);
            if (j >= 0 && j < subs / 2) {
              if (kFp8) tma_load_2d(dst + kVStageBytes / 2 + j * unit * 256, &p.chunks4, full, 256 * static_cast<int>(half), row);
              else tma_load_3d(dst + j * unit * 512, &p.chunks4, full, 0, row, 4 * static_cast<int>(half));
            }
          }
        }
        now = next;
        page = next_page;
      }
      n0 += blocks;
    }
    if (lane == 0) {
      if (!ok) fail();
      if (*abort_flag && (kFp8 || !scores || half == 0)) {  // let the copies in flight land (each wait bounded)
        const uint32_t stages = scores ? kKStages : kVStages;
        for (uint32_t i = issued > stages ? issued - stages : 0; i < issued; ++i)
          mbar_wait(bar((kFp8 ? kBarRaw : scores ? kBarKFull : kBarVFull) + i % stages), (i / stages) & 1u, nullptr, 100000000ull);
      }
    }
  } else if (kFp8 && warp >= kConvertWarp) {
    // Codes, 64 positions of `width` each, widened to f16 where they lie: read by all four
    // warps before any of them writes. (e4m3 values are exact in f16.)
    int blocks = 0;
    for (int k = item0; k < item1; ++k) blocks += item(k).end - item(k).begin;
    bool ok = true;
    auto widen = [&](auto width, auto stages, auto parts, uint32_t ring, auto tell) {
      constexpr int kWidth = decltype(width)::value, kStages = decltype(stages)::value, kParts = decltype(parts)::value;
      constexpr int kChunks = kWidth / 64, kBytes = 64 * kWidth * 2;
      // A thread has 16 codes of each chunk of rows t / 4 and t / 4 + 32: whatever eight threads
      // write at a time lies in eight different banks, and all offsets are constants.
      const int t = threadIdx.x - 32 * kConvertWarp, row = t >> 2, piece = t & 3;
      const uint32_t from = ring + kBytes / 2 + row * kWidth + 16 * piece, to = ring + row * 128 + 16 * (2 * piece ^ (row & 7));
      uint32_t use = 0, meet = 0;
      int stage = 0;
      for (int n = 0; n < kParts * blocks; ++n) {
        if (!(ok = warp_wait_block(bar(kBarRaw + stage), use))) break;
        uint32_t v[2 * kChunks][4];
#pragma unroll
        for (int i = 0; i < 2 * kChunks; ++i)
          ld_shared_v4(from + stage * kBytes + (i & 1) * 32 * kWidth + (i >> 1) * 64, v[i][0], v[i][1], v[i][2], v[i][3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarMeet));
        if (!(ok = warp_wait(bar(kBarMeet), meet))) break;
        meet ^= 1u;
#pragma unroll
        for (int i = 0; i < 2 * kChunks; ++i) {
          uint32_t f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = e4m3x2_to_f16x2(static_cast<uint16_t>(v[i][e >> 1] >> (16 * (e & 1))));
          const uint32_t at = to + stage * kBytes + (i >> 1) * kChunk + (i & 1) * 32 * 128;
          st_shared_v4(at, f[0], f[1], f[2], f[3]);
          st_shared_v4(at ^ 16, f[4], f[5], f[6], f[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tell(stage);
        if (++stage == kStages) {
          stage = 0;
          use ^= 1u;
        }
      }
    };
    using std::integral_constant;
    if (scores)
      widen(integral_constant<int, 192>{}, integral_constant<int, kKStages>{}, integral_constant<int, kKParts>{}, sbase,
            [&](int stage) { mbar_arrive_cluster(lead(kBarKFull + stage)); });
    else
      widen(integral_constant<int, 256>{}, integral_constant<int, kVStages>{}, integral_constant<int, 2>{}, sbase + kOffV,
            [&](int stage) { mbar_arrive(bar(kBarVFull + stage)); });
    if (!ok) fail();
  } else if (warp == kSendWarp) {
    // One lane sends P to the other pair, rows that attend the block alone, so that no softmax
    // warp waits for a buffer there. (Stored row by row into the peer's memory by the softmax
    // warps it took them 4,600 cycles a block.)
    if (scores && lane == 0) {
      const uint32_t there = mapa(sbase, rank ^ 2);
      uint32_t n = 0;
      bool ok = true;
      for (int k = item0; k < item1 && ok; ++k) {
        const ShItem it = item(k);
        Walk w;
        w.start(a, it);
        for (; w.more(); ++n) {
          const Block b = w.get();
          const int lo = max(b.row_lo - 128 * static_cast<int>(half), 0), hi = min(b.row_hi - 128 * static_cast<int>(half), 128);
          const uint32_t group = n & 1u, buf = n % kPBuffers, rb = peer(kBarP + buf);
          if (!(ok = spin(bar(kBarStaged + group), (n >> 1) & 1u))) break;
          if (!(ok = spin(bar(kBarPFree + buf), ((n / kPBuffers) & 1u) ^ 1u))) break;
          mbar_arrive_expect_tx_relaxed(rb, hi > lo ? (hi - lo) * 256 + 512 : 0);
          if (hi > lo) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              bulk_copy_to(there + buf * kPBytes + c * kPChunk + lo * 128, sbase + kOffPOut + group * kPBytes + c * kPChunk + lo * 128,
                           (hi - lo) * 128, rb);
            bulk_copy_to(there + kOffAlpha + 512 * buf, sbase + kOffAlphaOut + 512 * group, 512, rb);
          }
        }
      }
      if (!ok) fail();
    } else if (!scores && lane == 0) {
      // P has landed: its room in the other pair is free. (Told by the accumulators' warps,
      // which wait for V as well, it took long enough to bound the whole.)
      int blocks = 0;
      for (int k = item0; k < item1; ++k) blocks += item(k).end - item(k).begin;
      bool ok = true;
      for (int n = 0; n < blocks && ok; ++n) {
        ok = spin(bar(kBarP + n % kPBuffers), (n / kPBuffers) & 1u);
        if (ok) mbar_arrive_remote_relaxed(peer(kBarOutFree + (n & 1)));
      }
      if (!ok) fail();
    }
  } else if (warp == kIssueWarp) {
    if (scores && half == 0 && elect_one()) {
      constexpr uint32_t idesc = kFp8 ? idesc_f16(256, kShTokens, false, false) : idesc_bf16(256, kShTokens, false, false);
      const uint32_t ring = desc_lo(sbase), rope = desc_lo(sbase + kOffQRope);
      uint32_t n = 0, stage = 0, use = 0;
      bool ok = true;
      for (int k = item0; k < item1 && ok; ++k) {
        const int blocks = item(k).end - item(k).begin;
        ok = spin(bar(kBarQ), (k - item0) & 1u);
        for (int x = 0; x < blocks && ok; ++x, ++n) {
          const uint32_t buf = n & 1u;
          if (!(ok = spin(bar(kBarSFree + buf), ((n >> 1) & 1u) ^ 1u))) break;
          const uint32_t d = tmem + kColS + 128 * buf;
#pragma unroll
          for (int part = 0; part < kKParts; ++part) {
            if (!ok || !(ok = spin(bar(kBarKFull + stage), use))) break;
            tc_fence_after();
            const uint32_t kb = ring + stage * (kKStageBytes >> 4);
#pragma unroll
            for (int c = 0; c < 3; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int step = 4 * (3 * part + c) + e;  // dims 16 step ...
                if (step < 32) mma2_bf16_ts(d, tmem + 8 * step, kb + c * (kChunk >> 4) + 2 * e, idesc, step != 0);
                else mma2_bf16_ss(d, rope + 2 * e, kb + c * (kChunk >> 4) + 2 * e, idesc, 1);
              }
            mma2_commit_to(bar(kBarKFree + stage), kScorePair);
            if (++stage == kKStages) {
              stage = 0;
              use ^= 1u;
            }
          }
          if (ok) mma2_commit_to(bar(kBarS + buf), kScorePair);
        }
      }
      if (!ok) fail();
    } else if (!scores && half == 0 && elect_one()) {
      constexpr uint32_t idesc = kFp8 ? idesc_f16(256, 256, false, true) : idesc_bf16(256, 256, false, true);
      uint32_t n = 0, stage = 0;
      bool ok = true;
      for (int k = item0; k < item1 && ok; ++k) {
        const ShItem it = item(k);
        Walk w;
        w.start(a, it);
        ok = spin(bar(kBarOFree), ((k - item0) & 1u) ^ 1u);
        for (; w.more() && ok; ++n) {
          const Block b = w.get();
          const uint32_t buf = n % kPBuffers;
          const bool all = b.row_lo == 0 && b.row_hi == it.rows;
          uint32_t off[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int lo = min(max(b.row_lo - 32 * i, 0), 32), hi = min(max(b.row_hi - 32 * i, 0), 32);
            const uint32_t below_hi = hi == 32 ? ~0u : (1u << hi) - 1u, below_lo = lo == 32 ? ~0u : (1u << lo) - 1u;
            off[i] = ~(below_hi & ~below_lo);
          }
          if (!(ok = spin(bar(kBarPReady + buf), (n / kPBuffers) & 1u))) break;
          tc_fence_after();
          const uint32_t pa = desc_lo(sbase + buf * kPBytes);
          // V lies as it was copied: `span` positions of four chunks, then the next
          const uint32_t span = kFp8 ? 64 : unit;
          const int k0 = b.v0 >> 4, k1 = (b.v1 + 15) >> 4;  // steps of 16 positions
          bool add = b.add;
          for (int h = 0; h < 2; ++h) {
            const uint32_t vb = desc_lo_mn(sbase + kOffV + stage * kVStageBytes, span * 128);
            for (int e = max(k0, 4 * h); e < min(k1, 4 * h + 4); ++e) {
              const uint32_t pe = pa + h * (kPChunk >> 4) + 2 * (e & 3), t16 = 16 * (e & 3);
              const uint32_t ve = vb + (t16 / span * 512 * span + t16 % span * 128 >> 4);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (all) mma2_bf16_ss(tmem + 256 * c, pe, ve + c * 16 * span, idesc, add);
                else mma2_bf16_ss_rows(tmem + 256 * c, pe, ve + c * 16 * span, idesc, off, add);
              }
              add = true;
            }
            mma2_commit_to(bar(kBarVFree + stage), kAccPair);
            if (++stage == kVStages) stage = 0;
          }
          mma2_commit_to(bar(kBarPFree + buf), kScorePair | kAccPair);
          if (!w.more()) mma2_commit_to(bar(kBarO), kAccPair);
        }
      }
      if (!ok) fail();
    }
  } else if (scores && warp < kWorkers) {
    setmaxnreg_inc<Regs<kFp8>::kWorker>();
    // Softmax: a row a thread. The two groups of four warps take the even and the odd
    // blocks, of their own buffers of S and P, so that one group's loads
    // and waits hide behind the other's exponentials. A row's reference maximum goes from block to block through
    // shared memory; each group has a sum of its own.
    const int group = warp >> 2, quarter = warp & 3;
    const int lrow = 32 * quarter + lane, r = 128 * static_cast<int>(half) + lrow;
    const int w0 = r - lane;  // this warp's first row
    const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const float scale = a.scale_log2, threshold = kRescaleThreshold / scale;
    const uint64_t scale2 = f2_make(scale, scale);
    const uint32_t sw = lrow & 7, tS = tbase + kColS + 128 * group;
    const uint32_t p_here = sbase + kOffPOut + group * kPBytes + lrow * 128;  // this row of P
    float* alpha_here = reinterpret_cast<float*>(smem + kOffAlphaOut) + 128 * group + lrow;
    const uint32_t stats_at = mapa(sbase + kOffStats, rank ^ 2) + 8 * lrow;
    float* refs = reinterpret_cast<float*>(smem + kOffRef);
    float2* sums = reinterpret_cast<float2*>(smem + kOffSum);
    const uint32_t ref_mine = bar(kBarRef + 4 * group + quarter), ref_other = bar(kBarRef + 4 * (group ^ 1) + quarter);
    uint32_t n = 0, last = 0;
    float ref = kNoMax, sum_ref = kNoMax, l = 0.f;
    bool ok = true;
    for (int k = item0 - 1; ok; ++k) {
      // The next item's queries, into place once the scores of this one are complete (which a
      // group's last block tells, or a wait for the other's): half a row's c_kv dims a thread.
      const bool mine_last = (last & 1u) == static_cast<uint32_t>(group);
      if (k >= item0 && !mine_last) {
        if (!(ok = warp_wait(bar(kBarS + (last & 1u)), (last >> 1) & 1u))) break;
        tc_fence_after();
      }
      if (k + 1 < item1) {
        // A warp's rows of 64 dims a copy, by way of where it puts P when that has left; the rope
        // dims to where they stay. (Rows that attend nothing of the item may hold anything. Loaded
        // by the rows' threads, 32 bytes a time, the queries of 20 tiles took 6 us to come in.)
        const int row0 = item(k + 1).row0;
        if (w0 < item(k + 1).row_hi && w0 + 32 > item(k + 1).row_lo) {
          const uint32_t before = k < item0 ? 0 : (last + 2 - group) >> 1;  // this group's blocks so far
          if (!(ok = warp_wait(bar(kBarOutFree + group), (before & 1u) ^ 1u))) break;
          const uint32_t landed = bar(kBarQIn + warp), room = p_here - 128 * lane;
          const uint32_t rope = sbase + kOffQRope + 32 * quarter * 128;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const bool with_rope = h == 0 && group == 0;
            if (lane == 0) {
              mbar_arrive_expect_tx(landed, with_rope ? 3 * 4096 : 2 * 4096);
              tma_load_2d(room, &p.q, landed, 256 * group + 128 * h, row0 + w0);
              tma_load_2d(room + kPChunk, &p.q, landed, 256 * group + 128 * h + 64, row0 + w0);
              if (with_rope) tma_load_2d(rope, &p.q, landed, kDimCkv, row0 + w0);
            }
            __syncwarp();
            if (!(ok = warp_wait_block(landed, h))) {
              if (lane == 0) mbar_wait(landed, h, nullptr, 100000000ull);  // (nothing may land in a block that has ended)
              break;
            }
            uint32_t x[64];
#pragma unroll
            for (int c = 0; c < 16; ++c)
              ld_shared_v4(p_here + (c >> 3) * kPChunk + 16 * ((c & 7) ^ sw), x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            if (kFp8) {
#pragma unroll
              for (int c = 0; c < 64; ++c) x[c] = bf16x2_to_f16x2(x[c]);
            }
            __syncwarp();
            tmem_st32(tbase + 128 * group + 64 * h, x);
            tmem_st32(tbase + 128 * group + 64 * h + 32, x + 32);
            if (kFp8 && with_rope) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint32_t v[4];
                const uint32_t at = rope + 128 * lane + 16 * c;
                ld_shared_v4(at, v[0], v[1], v[2], v[3]);
                st_shared_v4(at, bf16x2_to_f16x2(v[0]), bf16x2_to_f16x2(v[1]), bf16x2_to_f16x2(v[2]), bf16x2_to_f16x2(v[3]));
              }
            }
          }
          if (!ok) break;
        }
        fence_proxy_async_smem();
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(kBarQ));
      }
      if (k >= item0) {
        // The row's maximum and sum, from the group of the last block. First every warp waits until
        // the item before's have been read: the last block's group needs the other's sum before it can
        // send, so no warp's wait for that phase can come after the next one. One group may be done
        // with the next item's blocks before the other reads this one's sum, but no further: the
        // next item's end waits for this one's maxima and sums.
        if (!(ok = warp_wait(bar(kBarStatsFree), ((k - item0) & 1u) ^ 1u))) break;
        const int odd = (k - item0) & 1;
        float2* sum = sums + 128 * odd + lrow;
        const uint32_t sum_bar = bar(kBarSum + 4 * odd + quarter);
        if (!mine_last) {
          *sum = make_float2(sum_ref, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(sum_bar);
        }
        if (mine_last) {
          if (!(ok = warp_wait_block(sum_bar, ((k - item0) >> 1) & 1u))) break;
          const float2 other = *sum;
          if (sum_ref != ref) l *= exp2_approx((sum_ref - ref) * scale);
          if (other.x != ref) l = fmaf(other.y, exp2_approx((other.x - ref) * scale), l);
          else l += other.y;
          st_async_v2(stats_at, __float_as_uint(-fmaf(-ref, scale, kWeightShift<kFp8>)), __float_as_uint(l), peer(kBarStats));
          if (lane == 0) mbar_arrive_expect_tx_relaxed(peer(kBarStats), 32 * 8);
        }
      }
      if (k + 1 >= item1) break;
      const ShItem it = item(k + 1);
      const int i = static_cast<int>((static_cast<int64_t>(it.row0) + r) / a.num_heads) % a.q_len;
      ref = sum_ref = kNoMax;
      l = 0.f;
      const uint32_t first = k + 1 == item0 ? 0 : last + 1;
      n = first;
      last = first + (it.end - it.begin) - 1;
      n += (n ^ group) & 1u;  // (the other group's block first)
      for (; n <= last; n += 2) {
        if (!(ok = warp_wait_block(bar(kBarNote + n % kNotes), (n / kNotes) & 1u))) break;
        const Block b = notes[n % kNotes];
        const bool here = b.row_lo < w0 + 32 && b.row_hi > w0;
        const bool mine = r >= b.row_lo && r < b.row_hi;
        if (!(ok = warp_wait(bar(kBarS + group), (n >> 1) & 1u))) break;
        tc_fence_after();
        // A row's maximum first, then its weights: 64 columns at a time, of which the second are
        // still there when the first are fetched once more. (All 128 at once do not fit the
        // registers.)
        float alpha = 1.f, mx = -CUDART_INF_F;
        uint32_t s[64];
        const int b0 = mine ? b.v0 : kShTokens, e0 = mine ? min(b.v1, b.end + i) : 0;
        const bool all = __all_sync(0xffffffffu, b0 == 0 && e0 == kShTokens);
        auto fetch = [&](int h) {
          tmem_ld32(tS + 64 * h, s);
          tmem_ld32(tS + 64 * h + 32, s + 32);
          tmem_wait_ld();
          if (all) return;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int c0 = 64 * h + 32 * g;
            const uint32_t above = e0 >= c0 + 32 ? ~0u : (1u << max(e0 - c0, 0)) - 1u;
            const uint32_t below = b0 >= c0 + 32 ? ~0u : (1u << max(b0 - c0, 0)) - 1u;
            const uint32_t keep = above & ~below;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(keep & (1u << c))) s[32 * g + c] = 0xff800000u;
          }
        };
        if (here) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            fetch(h);
            float mx1 = -CUDART_INF_F;
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              mx = fmax3(mx, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
              mx1 = fmax3(mx1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
            }
            mx = fmaxf(mx, mx1);
          }
        }
        // The reference from the block before, and on to the next.
        if (n > 0 && !(ok = warp_wait_block(ref_other, ((n - 1) >> 1) & 1u))) break;
        ref = n == first ? kNoMax : refs[lrow];
        if (mx > ref + threshold) {
          if (b.add) alpha = exp2_approx((ref - mx) * scale);  // (else nothing is there to rescale)
          ref = mx;
        }
        refs[lrow] = ref;
        __syncwarp();
        if (lane == 0) mbar_arrive(ref_mine);
        // P leaves by way of this block's memory, with the factor of each row.
        if (!(ok = warp_wait(bar(kBarOutFree + group), ((n >> 1) & 1u) ^ 1u))) break;
        if (here) {
          if (sum_ref != ref) l *= exp2_approx((sum_ref - ref) * scale);
          sum_ref = ref;
          const float neg = fmaf(-ref, scale, kWeightShift<kFp8>);
          const uint64_t neg2 = f2_make(neg, neg);
          uint64_t sum2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll
          for (int h = 1; h >= 0; --h) {
            if (h == 0) fetch(0);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float t0, t1;
              f2_split(f2_fma(f2_make(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), scale2, neg2), t0, t1);
              const float p0 = exp2_approx(t0), p1 = exp2_approx(t1);
              sum2[c & 1] = f2_add(sum2[c & 1], f2_make(p0, p1));
              s[c] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)
              st_shared_v4(p_here + h * kPChunk + 16 * (c ^ sw), s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]);
          }
          float s0, s1, s2, s3;
          f2_split(sum2[0], s0, s1);
          f2_split(sum2[1], s2, s3);
          l += (s0 + s1) + (s2 + s3);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(kBarSFree + group));
        *alpha_here = alpha;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarStaged + group));
      }
    }
    if (!ok) fail();
  } else if (!scores && warp < kWorkers) {
    setmaxnreg_inc<Regs<kFp8>::kWorker>();
    // Accumulators: the warps of a quarter of the lanes have half of the columns each.
    const int lrow = 32 * (warp & 3) + lane, r = 128 * static_cast<int>(half) + lrow, side = warp >> 2;
    const uint32_t tO = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 256 * side;
    const float* alphas = reinterpret_cast<const float*>(smem + kOffAlpha);
    const float2* stats = reinterpret_cast<const float2*>(smem + kOffStats);
    uint32_t n = 0, stage = 0, use = 0;
    bool ok = true;
    for (int k = item0; k < item1 && ok; ++k) {
      const ShItem it = item(k);
      Walk w;
      w.start(a, it);
      for (; w.more(); ++n) {
        const Block b = w.get();
        const uint32_t buf = n % kPBuffers;
        const int w0 = r - lane;
        const bool here = b.row_lo < w0 + 32 && b.row_hi > w0;
        // Rows of V outside the segment, among the 16 at its ends that are multiplied, and
        // positions that only later queries of a request see: an infinity or NaN there would
        // reach the others through a weight of zero. (Those that see it have it in their
        // scores.)
        constexpr uint32_t kExponent = kFp8 ? 0x7c00u : 0x7f80u;
        bool wrote = false;
        for (int h = 0; h < 2 && ok; ++h) {
          if (!(ok = warp_wait_block(bar(kBarVFull + stage), use))) break;
          const uint32_t v = sbase + kOffV + stage * kVStageBytes;
          const int lo0 = (b.v0 & ~15) - 64 * h, lo1 = b.v0 - 64 * h, hi0 = b.v1 - 64 * h, hi1 = ((b.v1 + 15) & ~15) - 64 * h;
          const int span = kFp8 ? 64 : unit;
          auto at_row = [&](int t) { return v + t / span * 512 * span + ((lane >> 3) * span + t % span) * 128 + 16 * (lane & 7); };
          auto zero = [&](int from, int to) {  // 512 bytes a row: a warp each
            for (int t = max(from, 0) + warp; t < min(to, 64); t += kWorkers) {
              st_shared_v4(at_row(t), 0, 0, 0, 0);
              wrote = true;
            }
          };
          if (b.v0 & 15) zero(lo0, lo1);
          if (b.v1 & 15) zero(hi0, hi1);
          for (int t = max(b.end - 64 * h, 0) + warp; t < min(hi0, 64); t += kWorkers) {
            const uint32_t at = at_row(t);
            uint32_t x[4];
            ld_shared_v4(at, x[0], x[1], x[2], x[3]);
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) odd |= (x[i] & kExponent) == kExponent || (x[i] & (kExponent << 16)) == kExponent << 16;
            if (__any_sync(0xffffffffu, odd)) {
              st_shared_v4(at, 0, 0, 0, 0);
              wrote = true;
            }
          }
          if (++stage == kVStages) {
            stage = 0;
            use ^= 1u;
          }
        }
        if (!ok) break;
        if (wrote) fence_proxy_async_smem();
        if (!(ok = warp_wait_cluster(bar(kBarP + buf), (n / kPBuffers) & 1u))) break;
        const float alpha = here ? alphas[128 * buf + lrow] : 1.f;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
          if (!(ok = warp_wait(bar(kBarPFree + (n - 1) % kPBuffers), ((n - 1) / kPBuffers) & 1u))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int v = 0; v < 32; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * alpha);
            tmem_st32(tO + 32 * c, o);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        // (What was written to V is in this block's memory since the proxy fence, and read there
        // by its own tensor core: no release at the cluster's scope, which takes 1,700 cycles.)
        if (lane == 0) mbar_arrive_cluster(lead(kBarPReady + buf));
      }
      if (!ok) break;
      if (!(ok = warp_wait_cluster(bar(kBarStats), (k - item0) & 1u))) break;
      const float2 ml = stats[lrow];
      if (!(ok = warp_wait(bar(kBarO), (k - item0) & 1u))) break;
      tc_fence_after();
      const bool real = r < it.rows;
      const int64_t out_row = static_cast<int64_t>(it.row0) + r;
      const int64_t part_row = static_cast<int64_t>(it.part) * kShRows + r;
      const bool part = it.part >= 0;
      // (a piece without a position of the row: its accumulator was never begun)
      const bool store = real && !(part && ml.y == 0.f);
      const uint32_t stores = __ballot_sync(0xffffffffu, store);
      // columns [0, 128) of a side are the first block's dims, the others the second's
      auto dim_of = [&](int col) { return 128 * side + (col & 127) + (col >= 128 ? 256 : 0); };
      if (stores == 0) {
      } else if (part) {
        // [dims / 8][rows][8 dims]: a warp's rows are next to each other
        float* dst = reinterpret_cast<float*>(a.ws + a.lay.partial) + it.part * static_cast<int64_t>(kShRows * kDimCkv) + 8 * r;
        uint32_t o[2][32];  // (the next columns are asked for while these go out)
        tmem_ld32(tO, o[0]);
        tmem_wait_ld();
#pragma unroll 1
        for (int c = 0; c < 8; c += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (c + h < 7) tmem_ld32(tO + 32 * (c + h + 1), o[h ^ 1]);
            if (store) {
#pragma unroll
              for (int i = 0; i < 4; ++i) st_global_v8(dst + (dim_of(32 * (c + h)) + 8 * i) * kShRows, o[h] + 8 * i);
            }
            __syncwarp();
            tmem_wait_ld();
          }
        }
      } else {
        uint8_t* dst = static_cast<uint8_t*>(a.out) + (out_row - (lane & 3)) * (kDimCkv * 2) + 32 * (lane & 3);
        const float inv = a.out_scale / ml.y;
        uint32_t o[64];
        tmem_ld32(tO, o);
        tmem_ld32(tO + 32, o + 32);
        tmem_wait_ld();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          if (c < 3) {
            tmem_ld32(tO + 64 * c + 64, o);
            tmem_ld32(tO + 64 * c + 96, o + 32);
          }
          turn(pk, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (stores >> ((lane & 28) + i) & 1u) st_global_v8(dst + i * kDimCkv * 2 + dim_of(64 * c) * 2, pk + 8 * i);
          __syncwarp();
          tmem_wait_ld();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(lead(kBarOFree));
        mbar_arrive_cluster(peer(kBarStatsFree));
      }
      if (side == 0 && real) {
        if (part) reinterpret_cast<float2*>(a.ws + a.lay.stats)[part_row] = ml;
        else if (a.lse) a.lse[out_row] = (ml.x + log2f(ml.y)) * 0.69314718055994531f;
      }
    }
    if (!ok) fail();
  }
  __syncwarp();
  __syncthreads();
  if (*abort_flag) {  // stores from other blocks may be on their way here
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 100000ull) {}
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // no block ends while another's products, stores or arrivals reach into it
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc2(tmem, 512);
}

template <bool kFp8>
int max_active_clusters() {
  if (cudaFuncSetAttribute(shared_decode_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
    return -1;
  int sms = 0, n = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kShClusterBlocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(sms / kShClusterBlocks * kShClusterBlocks);
  cfg.blockDim = dim3(Regs<kFp8>::kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, shared_decode_kernel<kFp8>, &cfg) != cudaSuccess || n <= 0) return -1;
  return n;
}

template <bool kFp8>
cudaError_t launch_variant(const Params& p, cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  const cudaError_t e = set_smem_once(shared_decode_kernel<kFp8>, kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(shared_decode_kernel<kFp8>, dim3(kShClusterBlocks * p.a.clusters), dim3(Regs<kFp8>::kThreads), kSmemBytes,
                    stream, p);
}

}  // namespace

// Clusters of the kernel that run at once on the current device (cached), or -1: the smaller
// of the variants' counts, so that a plan serves either. (36 on a GB300.)
int shared_max_active_clusters() {
  static int cached[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return -1;
  if (cached[dev] > 0) return cached[dev];
  const int a = max_active_clusters<false>(), b = max_active_clusters<true>();
  if (a <= 0 || b <= 0) return -1;
  return cached[dev] = std::min({a, b, kShMostClusters});
}

cudaError_t launch_shared_decode(const CUtensorMap (&maps)[4], const ShDecodeArgs& a, cudaStream_t stream) {
  Params p;
  p.rows = maps[0];
  p.chunks3 = maps[1];
  p.chunks4 = maps[2];
  p.q = maps[3];
  p.a = a;
  return a.dtype == MLA_DTYPE_FP8_E4M3 ? launch_variant<true>(p, stream) : launch_variant<false>(p, stream);
}

}  // namespace mla
