// First half of the chunk attention's preparation: which query tiles there
// are, and the cache rows that they attend, gathered from their pages.
//
// plan: one block, bound by the latency of its scans (12,000 cycles for three prompts,
// 16,500 for 24 mixed requests; with 512 threads and two passes always it was 24,000 to
// 35,000). The gather runs beside it where every block can place the requests itself. Request b has n = q_indptr[b + 1] - q_indptr[b] new tokens
// at positions L .. L + n - 1; its rows attend positions [lo, L + n) with
// lo = max(0, L + 1 - window), the first row's start. Those rows are packed
// request after request into a buffer, every request starting at a multiple of
// 16 rows and followed by zero rows up to the next, so that the last 16-row
// step of a P V product reads only this request's rows and zeros.
//
// gather: a warp per row copies (bf16) or widens (e4m3 codes, exact in bf16;
// kv_scale multiplies the scores and the output) the 576 values; bound by memory:
// 55,492 rows, read and written, 128 MB in 23 us, 5.6 TB/s. A row whose
// c_kv holds an infinity or NaN would poison, as 0 * inf, rows that do not
// attend it once it is multiplied by their zero weights. It is stored with
// c_kv = 0 and a NaN rope part: its scores are then NaN for the rows that do
// attend it, which makes their output NaN as it should be, and masked for the
// others.
#include <cuda_bf16.h>

#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "scan.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kPlanThreads = 512;  // in a launch of its own (kGatherThreads beside the gather)
constexpr int kCostBins = 128;     // (no more than threads)
constexpr int kRowVecs = kDimRow * 2 / 16;  // 72

__device__ __forceinline__ int64_t block_exclusive(int64_t x, int64_t* sh, int64_t* total) {
  int64_t v[1] = {x}, t[1];
  block_scan(v, t, sh);
  *total = t[0];
  return v[0];
}

// Few items: cut tiles along the keys so that every cluster has work. With N(P)
// pieces of at most P steps a head, all heads' pieces run in w waves if N(P) x
// heads <= w x clusters, and take about w (P + kPieceSteps), kPieceSteps being what
// an item costs beyond its steps. The best of up to four waves is taken if it beats
// the uncut tiles by a tenth. Returns the number of tiles; all threads call it.
// Cut against whole, us a call: 1 request of 100 new tokens over 12,000, 8 heads: 75 / 126;
// 2 of 300 over 8,000 (e4m3), 16 heads: 147 / 192; 512 over 4,000, 16 heads: 75 / 101.
constexpr int kPieceSteps = 6;   // measured: start-up, partial rows and joining, in steps
constexpr int kLeastPiece = 3;   // steps
constexpr int kMostWaves = 4;    // pieces a head fit in kPfMostPieces entries: heads >= 2, or waves <= 2

__device__ int split_tiles(const PrefillArgs& a, PfTile* tiles, int nt, int64_t* sh) {
  constexpr int kFew = kMostWaves * kPfPairs;
  __shared__ int steps[kFew], found[kMostWaves];
  const int heads = a.lay.heads;
  int per = 0;
  if (pf_may_split(a.max_kv) && static_cast<int64_t>(nt) * heads < kFew) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (static_cast<int>(threadIdx.x) < nt) steps[threadIdx.x] = pf_steps(tiles[threadIdx.x].kv_begin, tiles[threadIdx.x].kv_end);
    __syncthreads();
    int longest = 0, all = 0;
    for (int i = lane; i < nt; i += 32) {
      longest = max(longest, steps[i]);
      all += steps[i] + kPieceSteps;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    all = __reduce_add_sync(0xffffffffu, all);
    if (warp < kMostWaves) {  // a warp per number of waves: the least P that fits, 32 candidates at a time
      const int room = min((warp + 1) * kPfPairs / heads, kPfMostPieces);  // pieces a head
      int lo = kLeastPiece, hi = max(longest, kLeastPiece);
      while (lo < hi && room > nt) {
        const int gap = (hi - lo + 31) / 32, p = min(lo + lane * gap, hi);
        int count = 0;
        for (int i = 0; i < nt; ++i) count += max(1, (steps[i] + p - 1) / p);
        const unsigned ok = __ballot_sync(0xffffffffu, count <= room);
        const int first = ok ? __ffs(ok) - 1 : 32;
        const int new_hi = min(lo + first * gap, hi);
        lo = first > 0 ? min(lo + (first - 1) * gap + 1, new_hi) : lo;
        hi = new_hi;
      }
      if (lane == 0) found[warp] = room > nt ? hi : longest;
    }
    __syncthreads();
    const float whole = max(static_cast<float>(longest + kPieceSteps), 1.1f * all * heads / kPfPairs);
    float least = 0.9f * whole;
    for (int w = 0; w < kMostWaves; ++w) {
      const int p = found[w];
      const float t = static_cast<float>(w + 1) * (p + kPieceSteps);
      if (t < least && p < longest) {
        least = t;
        per = p;
      }
    }
  }
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  if (threadIdx.x == 0) hd->num_split = hd->merge_rows = 0;
  if (per == 0) return nt;
  // (fewer than kMostWaves x kPfPairs tiles: one round of threads)
  const int i = threadIdx.x;
  PfTile t = {};
  int n = 0, pieces = 1;
  if (i < nt) {
    t = tiles[i];
    n = pf_steps(t.kv_begin, t.kv_end);
    pieces = max(1, (n + per - 1) / per);
  }
  // Partial rows that would not fit leave their tiles whole.
  int64_t rows = pieces > 1 ? static_cast<int64_t>(pieces) * t.rows : 0, total;
  const int64_t row0 = block_exclusive(rows, sh, &total);
  const bool cut = pieces > 1 && row0 + rows <= a.lay.part_rows;
  // (room for the entries: pieces a head fit in kMostWaves waves of clusters, or
  // in kPfMostPieces entries beyond the first of each)
  int64_t v[3] = {cut ? pieces - 1 : 0, cut ? 1 : 0, cut ? t.rows : 0}, sums[3];  // further entries, split tiles, their rows
  block_scan(v, sums, sh);
  const int64_t to = nt + v[0], at = v[1], merge_row = v[2];
  if (cut) {
    t.part_row = static_cast<int>(row0);
    const int begin = t.kv_begin, end = t.kv_end;
    for (int p = 0; p < pieces; ++p) {
      t.kv_begin = begin + static_cast<int>(static_cast<int64_t>(n) * p / pieces) * kPfKvTile;
      t.kv_end = p == pieces - 1 ? end : begin + static_cast<int>(static_cast<int64_t>(n) * (p + 1) / pieces) * kPfKvTile;
      tiles[p == 0 ? i : to + p - 1] = t;
      t.part_row += t.rows;
    }
    PfSplit& s = reinterpret_cast<PfSplit*>(a.ws + a.lay.splits)[at];
    s.q_row = t.q_row;
    s.rows = t.rows;
    s.part_row = static_cast<int>(row0);
    s.pieces = pieces;
    s.merge_row = static_cast<int>(merge_row);
  }
  if (threadIdx.x == 0) {
    hd->num_split = static_cast<int>(sums[1]);
    hd->merge_rows = static_cast<int>(sums[2]);
  }
  __syncthreads();
  return nt + static_cast<int>(sums[0]);
}

// Decode blocks of a group of a small request.
__device__ __forceinline__ int group_first(const PfGroup& g, int window) { return window > 0 ? max(0, g.first + 1 - window) : 0; }
__device__ __forceinline__ int group_blocks(const PfGroup& g, int window) {
  return (g.first + g.tokens - 1) / kBlockTokens - group_first(g, window) / kBlockTokens + 1;
}

// The decode kernel's schedule for the groups of small requests: their 64-row
// blocks, each group weighing kGroupCost more for its start and end, `total` in all,
// laid out in a row and cut into equal ranges, one a cluster; a group across a cut has
// several items. All threads call it.
constexpr int kGroupCost = 4;
constexpr int kMostItems = kPfSmallRows / kGroupRows + kPfPairs;

__device__ void schedule_groups(const PrefillArgs& a, int groups, int64_t total, int64_t* sh) {
  __shared__ uint8_t cluster_of_item[kMostItems];
  const PfLayout& lay = a.lay;
  PfGroup* gs = reinterpret_cast<PfGroup*>(a.ws + lay.groups);
  uint8_t* ws = a.ws + lay.decode;
  WsHeader* hd = reinterpret_cast<WsHeader*>(ws);
  WorkItem* items = reinterpret_cast<WorkItem*>(ws + lay.decode_lay.items);
  int* cstart = reinterpret_cast<int*>(ws + lay.decode_lay.cluster_start);
  const int tid = threadIdx.x, step = blockDim.x;
  const int64_t per = max(static_cast<int64_t>(1), (total + a.clusters - 1) / a.clusters);  // units of a cluster
  int64_t carry[2] = {0, 0};  // units, items
  for (int i0 = 0; i0 < groups; i0 += step) {
    const int i = i0 + tid;
    PfGroup g = {};
    int n = 0;
    if (i < groups) {
      g = gs[i];
      n = group_blocks(g, a.window);
    }
    int64_t units, round;
    const int64_t off = carry[0] + block_exclusive(n ? n + kGroupCost : 0, sh, &units) + kGroupCost;
    const int cf = n ? static_cast<int>(off / per) : 0, cl = n ? static_cast<int>((off + n - 1) / per) : -1;
    const int pieces = cl - cf + 1;
    const int item0 = static_cast<int>(carry[1] + block_exclusive(pieces, sh, &round));
    for (int k = 0; k < pieces; ++k) {
      WorkItem w;
      const int64_t lo = max(off, (cf + k) * per), hi = min(off + n, (cf + k + 1) * per);
      const int first = group_first(g, a.window), blk0 = first / kBlockTokens;
      w.b = i;
      w.blk_begin = blk0 + static_cast<int>(lo - off);
      w.blk_end = blk0 + static_cast<int>(hi - off);
      w.slot = item0 + k;  // (even a whole group's sums stay in fp32)
      w.tok_lo = first;
      w.tok_hi = g.first + lay.group_tokens;  // (as if the group were full: its rows count from here)
      w.cluster = cf + k;
      w.row0 = 0;
      items[item0 + k] = w;
      cluster_of_item[item0 + k] = static_cast<uint8_t>(cf + k);
    }
    if (i < groups) {
      gs[i].first_item = item0;
      gs[i].items = pieces;
    }
    carry[0] += units;
    carry[1] += round;
  }
  __syncthreads();
  const int num_items = static_cast<int>(carry[1]);
  for (int c = tid; c <= a.clusters; c += step) {
    int lo = 0, hi = num_items;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cluster_of_item[mid] < c) lo = mid + 1;
      else hi = mid;
    }
    cstart[c] = lo;
  }
  if (tid == 0) {
    hd->status = 0;
    hd->batch = 2 * lay.max_pairs;
    hd->num_heads = a.num_heads;
    hd->q_len = lay.group_tokens;
    hd->page_size = kBlockTokens;
    hd->window = a.window;
    hd->num_clusters = static_cast<int>(max(static_cast<int64_t>(1), (total + per - 1) / per));
    hd->total_blocks = static_cast<int>(min(total, static_cast<int64_t>(INT32_MAX)));
    hd->num_items = num_items;
    hd->num_partials = num_items;
    hd->num_split = 0;
    hd->schedule = kScheduleCut;
    hd->planned = 1;
  }
}
static_assert(kPfPairs < 256, "clusters in a byte");

// Request b (a thread's) of one round. Carries what earlier rounds wished for and
// spanned. All threads call it.
struct Request {
  int64_t len, n, q0, lo, want, groups, span;
  bool small, good;
};

__device__ __forceinline__ Request request_of(const PrefillArgs& a, int b, int64_t* wished, int64_t* spanned, int64_t* sh) {
  Request r = {};
  const bool absorb = a.lay.absorb != 0;
  bool ok = true;
  if (b < a.batch) {
    r.len = a.context_lens[b];
    r.q0 = a.q_indptr[b];
    r.n = a.q_indptr[b + 1] - r.q0;
    // Row pointers outside q leave nothing that could be written.
    if (r.q0 < 0 || r.n < 0 || r.q0 + r.n > a.q_rows) {
      r.n = 0;
      ok = false;
    }
    // (no ids at all: every list is empty)
    const int64_t nb = !a.page_ids ? 0 : a.page_indptr ? a.page_indptr[b + 1] - a.page_indptr[b] : a.max_blocks;
    if (r.len < 0 || r.len + r.n > nb * a.page_size || r.len + r.n > INT32_MAX) ok = ok && r.n == 0;
    r.lo = a.window > 0 ? max(static_cast<int64_t>(0), r.len + 1 - a.window) : 0;
  }
  r.want = ok && r.n > 0 ? r.len + r.n - r.lo : 0;
  int64_t round;
  if (absorb) {
    const int per_group = a.lay.group_tokens;  // (a power of two)
    const int most = r.want >= kPfSmallSpan ? kPfSmallTokens : kPfSmallTokensShort;
    r.groups = r.want > 0 && r.n <= most ? (r.n + per_group - 1) >> (31 - __clz(per_group)) << 1 : 0;
    const int64_t before = *wished + block_exclusive(r.groups, sh, &round);
    r.small = r.groups > 0 && before + r.groups <= 2 * a.lay.max_pairs;
    *wished += round;
  }
  const int align = r.small ? kBlockTokens : kPfKvAlign;
  r.span = (r.want + align - 1) & -static_cast<int64_t>(align);
  const int64_t upto = *spanned + block_exclusive(r.span, sh, &round) + r.span;
  *spanned += round;
  r.good = ok && upto + (absorb ? 256 : 0) <= a.lay.kv_capacity;
  r.small = r.small && r.good;
  return r;
}

// Where small requests' rows start, behind `rows` of the expanded ones.
__device__ __forceinline__ int64_t small_rows_start(int64_t rows) { return (rows + 255) / 256 * 256; }

// The plan, by one block.
__device__ __forceinline__ void plan(const PrefillArgs& a, int64_t* sh) {
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  PfRequest* reqs = reinterpret_cast<PfRequest*>(a.ws + a.lay.requests);
  PfTile* tiles = reinterpret_cast<PfTile*>(a.ws + a.lay.tiles);
  PfGroup* groups = reinterpret_cast<PfGroup*>(a.ws + a.lay.groups);
  const bool absorb = a.lay.absorb != 0;
  const int per_group = a.lay.group_tokens;
  // Sums over the requests so far: rows of the expanded ones, rows of the small ones,
  // requests that are not small, tiles, groups. With small requests a first pass
  // finds where their rows start, after all others'
  // (unless one round of threads serves all requests: its own sums tell).
  int64_t sum[5] = {0, 0, 0, 0, 0}, small_start = 0, small_first = 0;
  const int threads = blockDim.x;
  const bool one_round = a.batch <= threads;
  for (int pass = absorb && !one_round ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1) {
      small_start = small_rows_start(sum[0]);
      small_first = sum[2];
    }
    int64_t wished = 0, spanned = 0;
#pragma unroll
    for (int k = 0; k < 5; ++k) sum[k] = 0;
    for (int b0 = 0; b0 < a.batch; b0 += threads) {
      const int b = b0 + threadIdx.x;
      const Request r = request_of(a, b, &wished, &spanned, sh);
      const bool small = r.small, good = r.good;
      const int64_t len = r.len, n = r.n, q0 = r.q0, lo = r.lo, span = r.span, ng = r.groups;
      const int64_t nt = small ? 0 : (n + kPfRows - 1) / kPfRows;
      int64_t v[5] = {small || !good ? 0 : span, small ? span : 0, b < a.batch && !small ? 1 : 0, nt, small ? ng : 0}, total[5];
      block_scan(v, total, sh);
      if (one_round) {
        small_start = small_rows_start(total[0]);
        small_first = total[2];
      }
      if (pass == 1 && b < a.batch) {
        if (!good) atomicOr(&hd->status, MLA_STATUS_BAD_LENGTH);
        PfRequest p;
        p.base = static_cast<int>(small ? small_start + sum[1] + v[1] : sum[0] + v[0]);
        p.rows = good ? static_cast<int>(r.want) : 0;
        p.lo = static_cast<int>(lo);
        p.b = b;
        // (v[2] counts the others before this one: the rest before it are small)
        reqs[small ? small_first + b - (sum[2] + v[2]) : sum[2] + v[2]] = p;
        const int64_t tile0 = sum[3] + v[3];
        for (int64_t k = 0; k < nt && tile0 + k < a.lay.max_tiles; ++k) {
          PfTile t;
          const int64_t i0 = k * kPfRows;
          t.q_row = static_cast<int>(q0 + i0);
          t.rows = static_cast<int>(min(n - i0, static_cast<int64_t>(kPfRows)));
          t.base = p.base;
          t.first_end = good ? static_cast<int>(len + i0 + 1 - lo) : 0;
          t.kv_end = good ? t.first_end + t.rows - 1 : 0;
          t.kv_begin = good && a.window > 0 ? max(0, t.first_end - a.window) / kPfKvAlign * kPfKvAlign : 0;
          t.refused = good ? 0 : 1;
          t.part_row = -1;
          t.pad[0] = t.pad[1] = t.pad[2] = t.pad[3] = 0;
          tiles[tile0 + k] = t;
        }
        if (small)
          for (int64_t k = 0; 2 * k < ng; ++k) {
            PfGroup g = {};
            g.base = p.base;
            g.first = static_cast<int>(len + k * per_group - lo);
            g.q_row = static_cast<int>(q0 + k * per_group);
            g.tokens = static_cast<int>(min(n - k * per_group, static_cast<int64_t>(per_group)));
            g.pages = (g.first + g.tokens - 1) / kBlockTokens + 1;
            groups[sum[4] + v[4] + 2 * k] = g;
            groups[sum[4] + v[4] + 2 * k + 1] = g;
          }
      }
#pragma unroll
      for (int k = 0; k < 5; ++k) sum[k] += total[k];
    }
  }
  const int64_t tiles_before = sum[3];
  if (absorb) {
    __syncthreads();  // groups are written
    const int count = static_cast<int>(sum[4]);
    int32_t* indptr = reinterpret_cast<int32_t*>(a.ws + a.lay.group_indptr);
    int64_t pages = 0, units = 0;
    for (int i0 = 0; i0 < count; i0 += threads) {
      const int i = i0 + threadIdx.x;
      PfGroup g = {};
      if (i < count) g = groups[i];
      int64_t v[2] = {g.pages, i < count ? group_blocks(g, a.window) + kGroupCost : 0}, total[2];
      block_scan(v, total, sh);
      if (i < count) {
        groups[i].page0 = static_cast<int>(pages + v[0]);
        indptr[i] = static_cast<int>(pages + v[0]);
      }
      pages += total[0];
      units += total[1];
    }
    if (threadIdx.x == 0) {
      indptr[count] = static_cast<int>(pages);
      hd->num_groups = count;
    }
    schedule_groups(a, count, units, sh);
  }
  // Tiles by falling cost (key steps, in kCostBins classes of the most expensive
  // one's): blocks draw them in this order, so that what is drawn last is
  // short. The order within a class varies from call to call and changes nothing
  // but who computes a tile.
  __shared__ int most, least, bins[kCostBins];
  int nt = static_cast<int>(min(tiles_before, a.lay.max_tiles));
  PfTile* sorted = reinterpret_cast<PfTile*>(a.ws + a.lay.sorted);
  if (threadIdx.x < kCostBins) bins[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    most = 1;
    least = INT32_MAX;
  }
  __syncthreads();  // (also: tiles are written)
  auto cost = [&](int i) { return pf_steps(tiles[i].kv_begin, tiles[i].kv_end); };
  nt = split_tiles(a, tiles, nt, sh);
  // (a thread's first tile's cost is read once)
  const int mine = threadIdx.x < nt ? cost(threadIdx.x) : 0;
  auto cost_of = [&](int i) { return i == static_cast<int>(threadIdx.x) ? mine : cost(i); };
  int top = mine, low = threadIdx.x < nt ? mine : INT32_MAX;
  for (int i = threadIdx.x + threads; i < nt; i += threads) {
    top = max(top, cost(i));
    low = min(low, cost(i));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  low = __reduce_min_sync(0xffffffffu, low);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&most, top);
    atomicMin(&least, low);
  }
  __syncthreads();
  const uint32_t scale = most;  // (steps are fewer than 2^24)
  auto bin = [&](int i) { return kCostBins - 1 - static_cast<int>(static_cast<uint32_t>(cost_of(i)) * (kCostBins - 1) / scale); };
  for (int i = threadIdx.x; i < nt; i += threads) atomicAdd(&bins[bin(i)], 1);
  __syncthreads();
  int64_t first = threadIdx.x < kCostBins ? bins[threadIdx.x] : 0, ignored;
  first = block_exclusive(first, sh, &ignored);
  if (threadIdx.x < kCostBins) bins[threadIdx.x] = static_cast<int>(first);
  __syncthreads();
  for (int i = threadIdx.x; i < nt; i += threads) sorted[atomicAdd(&bins[bin(i)], 1)] = tiles[i];
  if (threadIdx.x == 0) {
    hd->odd_bins = 0;
    hd->kv_rows = static_cast<int>(sum[0]);
    hd->all_rows = static_cast<int>(absorb && sum[1] > 0 ? small_start + sum[1] : sum[0]);
    hd->num_tiles = nt;
    hd->even = least >= most - least;
    if (tiles_before > a.lay.max_tiles) atomicOr(&hd->status, MLA_STATUS_BAD_LENGTH);
  }
}

__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const PrefillArgs a) {
  __shared__ int64_t sh[32 * 5];
  pdl_launch_dependents();
  pdl_wait();
  plan(a, sh);
}

// Two e4m3 codes to a bf16 pair (exact: bf16 has e4m3's values).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t v) {
  const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(v));
  float lo, hi;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint4 widen(uint2 c) {
  return make_uint4(e4m3x2_to_bf16x2(c.x & 0xffffu), e4m3x2_to_bf16x2(c.x >> 16), e4m3x2_to_bf16x2(c.y & 0xffffu),
                    e4m3x2_to_bf16x2(c.y >> 16));
}

// The largest sizes among the low and among the high halves of bf16 pairs, as their bits.
__device__ __forceinline__ uint32_t sizes(uint32_t w) { return w & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t sizes(const uint4& v) {
  return __vmaxu2(__vmaxu2(sizes(v.x), sizes(v.y)), __vmaxu2(sizes(v.z), sizes(v.w)));
}
__device__ __forceinline__ bool reach(uint32_t sizes, uint32_t bits) { return (sizes & 0xffffu) >= bits || sizes >> 16 >= bits; }

constexpr int kGatherWarps = 8, kGatherThreads = 32 * kGatherWarps;

// A block takes runs of kPfKvAlign rows (all of one request), two a warp. kFused: up to
// kGatherThreads requests, whose places every block works out for itself while one
// more block, the first, makes the plan.
template <int kDtype, bool kFused>
__global__ void __launch_bounds__(kGatherThreads, 4) prefill_gather_kernel(const PrefillArgs a) {
  __shared__ PfRequest placed[kFused ? kGatherThreads : 1];
  pdl_launch_dependents();
  pdl_wait();
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const PfRequest* reqs = reinterpret_cast<const PfRequest*>(a.ws + a.lay.requests);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int used;
  if (kFused) {
    __shared__ int64_t sh[32 * 5];
    if (blockIdx.x == 0) {
      plan(a, sh);
      return;
    }
    const int b = threadIdx.x;
    int64_t wished = 0, spanned = 0;
    const Request r = request_of(a, b, &wished, &spanned, sh);
    int64_t v[3] = {r.small || !r.good ? 0 : r.span, r.small ? r.span : 0, b < a.batch && !r.small ? 1 : 0}, total[3];
    block_scan(v, total, sh);
    const int64_t start = small_rows_start(total[0]);
    if (b < a.batch)
      placed[r.small ? total[2] + b - v[2] : v[2]] = {static_cast<int>(r.small ? start + v[1] : v[0]),
                                                      r.good ? static_cast<int>(r.want) : 0, static_cast<int>(r.lo), b};
    used = static_cast<int>(total[1] > 0 ? start + total[1] : total[0]);
    reqs = placed;
    __syncthreads();
  } else {
    used = hd->all_rows;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int first = blockIdx.x - (kFused ? 1 : 0), step = gridDim.x - (kFused ? 1 : 0);
  for (int64_t run = first; run * kPfKvAlign < used; run += step) {
    const int row0 = static_cast<int>(run) * kPfKvAlign;
    int lo = 0, hi = a.batch;  // the last request with base <= row0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (reqs[mid].base <= row0) lo = mid;
      else hi = mid;
    }
    const PfRequest r = reqs[lo];
    const int b = r.b;
    const int nb = a.page_indptr ? a.page_indptr[b + 1] - a.page_indptr[b] : a.max_blocks;
    const int32_t* ids = a.page_indptr ? a.page_ids + a.page_indptr[b] : a.page_ids + static_cast<int64_t>(b) * a.max_blocks;
#pragma unroll
    for (int k = 0; k < kPfKvAlign / kGatherWarps; ++k) {
      const int row = row0 + warp + k * kGatherWarps;
      const int rel = row - r.base;
      uint4 v[3] = {zero, zero, zero};
      if (rel < r.rows) {
        bool zeros = true;
        const int pos = r.lo + rel, j = pos / a.page_size;
        const int id = j < nb ? ids[j] : -1;
        if (id < 0 || id >= a.num_pages) {
          if (lane == 0) atomicOr(&hd->status, MLA_STATUS_BAD_PAGE);
        } else {
          const int64_t src = (static_cast<int64_t>(a.layer) * a.num_pages + id) * a.page_size + pos % a.page_size;
          if (kDtype == MLA_DTYPE_BF16) {
            const uint4* s = static_cast<const uint4*>(a.pool) + src * kRowVecs;
            v[0] = s[lane];
            v[1] = s[lane + 32];
            if (lane < 8) v[2] = s[lane + 64];
          } else {
            const uint2* s = reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.pool) + src * kDimRow);
            v[0] = widen(s[lane]);
            v[1] = widen(s[lane + 32]);
            if (lane < 8) v[2] = widen(s[lane + 64]);
          }
          const uint32_t ckv = __vmaxu2(sizes(v[0]), sizes(v[1]));
          zeros = !__any_sync(0xffffffffu, ckv);
          if (__any_sync(0xffffffffu, reach(ckv, 0x7f80u))) {
            zeros = true;
            v[0] = v[1] = zero;
            v[2] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
          }
        }
        if (zeros && lane == 0) hd->zero_rows = 1;
      }
      uint4* dst = reinterpret_cast<uint4*>(a.ws + a.lay.rows) + static_cast<int64_t>(row) * kRowVecs;
      dst[lane] = v[0];
      dst[lane + 32] = v[1];
      if (lane < 8) dst[lane + 64] = v[2];
    }
  }
}

// Joins the pieces of split tiles: a warp per (row, head), four value dims a
// lane. Each piece left its sums O and l, 2^kWeightShift of what they are relative to
// its own maximum m. 2.3 us where
// nothing or little was cut, most of it the launch.
__global__ void __launch_bounds__(256) prefill_merge_kernel(const PrefillArgs a, int head0, int heads) {
  pdl_launch_dependents();
  pdl_wait();
  const PfHeader* hd = reinterpret_cast<const PfHeader*>(a.ws);
  const PfSplit* splits = reinterpret_cast<const PfSplit*>(a.ws + a.lay.splits);
  const int lane = threadIdx.x & 31;
  const int64_t units = static_cast<int64_t>(hd->merge_rows) * heads, step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units; u += step) {
    const int row = static_cast<int>(u / heads), head = static_cast<int>(u % heads);
    int lo = 0, hi = hd->num_split;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (splits[mid].merge_row <= row) lo = mid;
      else hi = mid;
    }
    const PfSplit s = splits[lo];
    const int r = row - s.merge_row;
    const int64_t first = static_cast<int64_t>(head) * a.lay.part_rows + s.part_row + r;
    const float2* stats = reinterpret_cast<const float2*>(a.ws + a.lay.part_stats) + first;
    const float4* part = reinterpret_cast<const float4*>(a.ws + a.lay.part_o) + first * (kDimV / 4) + lane;
    float m = -3e38f;
    for (int p = 0; p < s.pieces; ++p) m = fmaxf(m, stats[static_cast<int64_t>(p) * s.rows].x);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < s.pieces; ++p) {
      const float2 st = stats[static_cast<int64_t>(p) * s.rows];
      const float4 v = part[static_cast<int64_t>(p) * s.rows * (kDimV / 4)];
      if (st.y == 0.f) continue;  // no key of this row (its sums are not written)
      const float w = exp2f((st.x - m) * a.scale_log2);
      l = fmaf(w, st.y, l);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    const float inv = a.out_scale / l;
    const int64_t out_row = (static_cast<int64_t>(s.q_row) + r) * a.num_heads + head0 + head;
    reinterpret_cast<uint2*>(a.out)[out_row * (kDimV / 4) + lane] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (a.lse && lane == 0) a.lse[out_row] = (m * a.scale_log2 + log2f(l * kWeightUnit)) * 0.69314718055994531f;
  }
}

}  // namespace

int sm_count() {
  static int count[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return 0;
  if (!count[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    count[dev] = n;
  }
  return count[dev];
}

cudaError_t launch_prefill_merge(const PrefillArgs& a, int head0, int heads, cudaStream_t stream) {
  return launch_pdl(prefill_merge_kernel, dim3(152 * 4), dim3(256), 0, stream, a, head0, heads);
}

// One launch for both where a block's threads are enough for the requests and tiles,
// else two. The smallest call takes 21.3 us so, 24.9 with two launches; a mixed step of
// 24 requests 195 and 202 (210 with 2 blocks an SM instead of 4, 198 with 6).
cudaError_t launch_prefill_gather(const PrefillArgs& a, cudaStream_t stream) {
  const bool bf16 = a.dtype == MLA_DTYPE_BF16;
  const int64_t runs = a.lay.kv_capacity / kPfKvAlign, most = max(static_cast<int64_t>(a.batch), a.lay.max_tiles);
  const int64_t blocks = 152 * 4;
  if (most <= kGatherThreads) {
    const dim3 grid(static_cast<unsigned>(1 + min(runs, blocks)));
    return launch_pdl(bf16 ? prefill_gather_kernel<MLA_DTYPE_BF16, true> : prefill_gather_kernel<MLA_DTYPE_FP8_E4M3, true>, grid,
                      dim3(kGatherThreads), 0, stream, a);
  }
  const cudaError_t e = launch_pdl(prefill_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(bf16 ? prefill_gather_kernel<MLA_DTYPE_BF16, false> : prefill_gather_kernel<MLA_DTYPE_FP8_E4M3, false>,
                    dim3(static_cast<unsigned>(min(runs, blocks))), dim3(kGatherThreads), 0, stream, a);
}

}  // namespace mla
