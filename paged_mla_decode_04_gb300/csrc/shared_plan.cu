// Schedule of a decode over shared prefixes, and the join of its partial sums.
//
// The plan reads only lengths: group g's requests [prefix_indptr[g], [g + 1]) share
// their first P positions, P the least of prefix_lens[g] and its requests' cached
// lengths, as far as these are in range. A tile of the group's rows attends the P positions once and then each of its
// requests' own ones (see shared_internal.h). One block of threads, a launch a step; its
// time is that of a few passes over the requests, one after the other.
#include <cuda_bf16.h>
#include <limits.h>
#include <math_constants.h>

#include "../../include/mla_decode.h"
#include "ptx_shared.cuh"
#include "scan.cuh"
#include "shared_internal.h"

namespace mla {
namespace {

constexpr int kPlanThreads = 1024;

// The first of n ascending values' index whose successor exceeds x: the last i with
// start(i) <= x.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, int64_t x, F start) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Pieces of a tile of so many blocks (the prefix's among them), of a weight of `most` each:
// no more than blocks.
__device__ __forceinline__ int pieces_of(int blocks, int shared, int most) {
  const int64_t weight = static_cast<int64_t>(blocks) * most + static_cast<int64_t>(shared) * kShRowsCost;  // (times most)
  const int64_t unit = static_cast<int64_t>(most) * most;
  return static_cast<int>(min((weight + unit - 1) / unit, static_cast<int64_t>(blocks)));
}

__device__ __forceinline__ int64_t tiles_of(int64_t rows, int tile_rows) { return (rows + tile_rows - 1) / tile_rows; }

// Rows of a group's tiles: whole requests, or as many as there is room for, whichever is
// fewer blocks. The latter has fewer tiles, so fewer of the prefix's blocks; requests across
// two tiles have their own positions in both. (40 requests of 96 rows and 550 positions each
// behind 3,001 shared ones, e4m3: 55 us a decode in 15 full tiles, 59 in 20 of two requests.)
__device__ __forceinline__ int tile_rows_of(int64_t r, int count, int prefix, int64_t cached) {
  const int whole = sh_whole_rows(r);
  if (whole == kShRows || count == 0) return whole;
  const int64_t fewer = tiles_of(count * r, kShRows), saved = tiles_of(count * r, whole) - fewer;
  int64_t period = r;  // tiles after which one ends with a request: r / gcd(r, kShRows)
  while (period % 2 == 0) period /= 2;
  const int64_t across = fewer - 1 - (fewer - 1) / period;
  const int64_t shared_blocks = (prefix + kShTokens - 1) / kShTokens;
  const int64_t own_blocks = max(cached / count - prefix, static_cast<int64_t>(0)) / kShTokens + 1;  // (of a request, about)
  return saved * (shared_blocks + kShItemCost) > across * own_blocks ? kShRows : whole;
}

// A request's cached positions, or a prefix's: none for a length out of range.
__device__ __forceinline__ int length_of(int l) { return l < 0 || l >= kShMostLength ? 0 : l; }

__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const ShPlanArgs a) {
  __shared__ int64_t sh[64];
  __shared__ int bad, apart;
  pdl_launch_dependents();
  pdl_wait();
  ShHeader* hd = reinterpret_cast<ShHeader*>(a.ws);
  ShGroup* groups = reinterpret_cast<ShGroup*>(a.ws + a.lay.groups);
  ShTile* tiles = reinterpret_cast<ShTile*>(a.ws + a.lay.tiles);
  ShSegment* segs = reinterpret_cast<ShSegment*>(a.ws + a.lay.segs);
  ShItem* items = reinterpret_cast<ShItem*>(a.ws + a.lay.items);
  ShCluster* clusters = reinterpret_cast<ShCluster*>(a.ws + a.lay.clusters);
  ShSplit* splits = reinterpret_cast<ShSplit*>(a.ws + a.lay.splits);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  if (tid == 0) bad = 0;
  __syncthreads();

  // Groups in ascending order within the batch; else nothing is planned.
  int wrong = 0;
  for (int g = tid; g <= a.num_prefixes; g += blockDim.x) {
    const int p = a.prefix_indptr[g];
    if (p < 0 || p > a.batch || (g > 0 && p < a.prefix_indptr[g - 1])) wrong = 1;
  }
  const bool refused = __syncthreads_or(wrong) != 0;
  if (refused && tid == 0) bad = 1;

  // Shared positions and tiles of each group.
  const int64_t r = static_cast<int64_t>(a.q_len) * a.num_heads;
  for (int g = warp; g < a.num_prefixes && !refused; g += warps) {
    const int first = a.prefix_indptr[g], count = a.prefix_indptr[g + 1] - first;
    int p = a.prefix_lens[g];
    int least = INT_MAX, any_bad = p != length_of(p);
    p = length_of(p);
    int64_t cached = 0;
    for (int b = lane; b < count; b += 32) {
      const int l = a.context_lens[first + b];
      if (l == length_of(l)) {
        least = min(least, l);
        cached += l;
      } else {
        any_bad = 1;
      }
    }
    for (int d = 16; d > 0; d >>= 1) cached += __shfl_xor_sync(0xffffffffu, cached, d);
    least = __reduce_min_sync(0xffffffffu, least);
    any_bad = __any_sync(0xffffffffu, any_bad);
    if (lane == 0) {
      if (any_bad && count > 0) bad = 1;
      // (a request by itself has its positions in one segment; nor is anything shared where no
      // length is in range)
      p = count > 1 && least < kShMostLength ? min(p, least) : 0;
      groups[g] = ShGroup{first, count, p, 0, tile_rows_of(r, count, p, cached)};
    }
  }
  __syncthreads();
  int64_t before = 0;
  for (int g0 = 0; g0 < a.num_prefixes && !refused; g0 += blockDim.x) {
    const int g = g0 + tid;
    int64_t v[1] = {0}, total[1];
    if (g < a.num_prefixes) v[0] = tiles_of(static_cast<int64_t>(groups[g].count) * r, groups[g].tile_rows);
    block_scan<1>(v, total, sh);
    if (g < a.num_prefixes) groups[g].tile0 = static_cast<int>(before + v[0]);
    before += total[0];
  }
  const int num_tiles = refused ? 0 : static_cast<int>(before);
  __syncthreads();

  // A warp a tile: its segments, a lane a request.
  const int unit = sh_copy_tokens(a.page_size);
  for (int t = warp; t < num_tiles; t += warps) {
    const int g = last_at_most(a.num_prefixes, t, [&](int i) { return groups[i].tile0; });
    const ShGroup gr = groups[g];
    const int64_t from = static_cast<int64_t>(t - gr.tile0) * gr.tile_rows;  // within the group's rows
    const int rows = static_cast<int>(min(static_cast<int64_t>(gr.count) * r - from, static_cast<int64_t>(gr.tile_rows)));
    const int64_t row0 = static_cast<int64_t>(gr.first) * r + from;
    ShSegment* out = segs + static_cast<int64_t>(t) * a.lay.segs_per_tile;
    const int shared_blocks = (gr.prefix + kShTokens - 1) / kShTokens;
    if (lane == 0) out[0] = ShSegment{gr.first, 0, rows, 0, 0, 0, gr.prefix, gr.prefix};
    const int b0 = static_cast<int>(from / r), b1 = static_cast<int>((from + rows - 1) / r);  // requests of the group
    int done = shared_blocks;
    for (int j0 = b0; j0 <= b1; j0 += 32) {
      const int j = j0 + lane;
      int n = 0;
      ShSegment s = {};
      if (j <= b1) {
        const int64_t first_row = static_cast<int64_t>(j) * r;  // of the request, within the group
        s.owner = gr.first + j;
        s.row_lo = static_cast<int>(max(first_row - from, static_cast<int64_t>(0)));
        s.row_hi = static_cast<int>(min(first_row + r - from, static_cast<int64_t>(rows)));
        const int last_i = static_cast<int>((from + s.row_hi - 1 - first_row) / a.num_heads);
        s.base = max(length_of(a.context_lens[s.owner]), gr.prefix);  // (of a length out of range: the prefix)
        s.tok_lo = gr.prefix;
        s.tok0 = gr.prefix / unit * unit;
        s.tok_hi = s.base + last_i + 1;
        n = (s.tok_hi - s.tok0 + kShTokens - 1) / kShTokens;
      }
      int upto = n;
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += u;
      }
      s.block0 = done + upto - n;
      if (j <= b1) out[1 + j - b0] = s;
      done += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) {
      ShTile w = {};
      w.row0 = static_cast<int>(row0);
      w.rows = rows;
      w.seg0 = t * a.lay.segs_per_tile + (shared_blocks == 0 ? 1 : 0);
      w.segs = b1 - b0 + 1 + (shared_blocks == 0 ? 0 : 1);
      w.blocks = done;
      w.shared = shared_blocks;
      tiles[t] = w;
    }
  }
  __syncthreads();

  // The blocks of all tiles dealt to the clusters, in one of two ways:
  //  - cut: all tiles' weights (their blocks and an item's cost, which comes first) as one
  //    sequence, cut into equal ranges. Most clusters then have an item more than they need;
  //  - apart, where there are no more tiles than clusters: each tile in pieces of at most
  //    `most` blocks, a cluster each, with the least `most` for which the clusters suffice.
  //    A piece of the prefix counts kShRowsCost blocks more: all rows' queries come in and
  //    all rows' sums go out, where a piece of requests' own positions has theirs only. So a
  //    prefix's blocks weigh 1 + kShRowsCost / most.
  // (4 tiles of about 100 blocks, 36 clusters: 44 us a decode cut, 42 apart; 20 tiles of about
  // 32 blocks: 69 cut, 79 apart, where a piece has as much as a whole tile.)
  int64_t weight = 0;
  for (int t0 = 0; t0 < num_tiles; t0 += blockDim.x) {
    int64_t v[1] = {t0 + tid < num_tiles ? tiles[t0 + tid].blocks + kShItemCost : 0}, total[1];
    block_scan<1>(v, total, sh);
    weight += total[0];
  }
  // No more clusters than have some blocks each: pieces have to be joined.
  const int64_t all = weight - static_cast<int64_t>(kShItemCost) * num_tiles;
  const int64_t c = max(static_cast<int64_t>(1), min(all / kShLeastBlocks, static_cast<int64_t>(a.clusters)));
  if (tid == 0) apart = 0;
  __syncthreads();
  if (warp == 0 && num_tiles > 0 && num_tiles <= a.clusters && all < 1 << 30) {
    constexpr int kEach = kShMostClusters / 32;
    int mine[kEach], shared[kEach];  // blocks of tiles lane, lane + 32, ...; of their prefixes
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const ShTile t = lane + 32 * j < num_tiles ? tiles[lane + 32 * j] : ShTile{};
      mine[j] = t.blocks;
      shared[j] = t.shared;
    }
    int lo = kShLeastBlocks, hi = max(kShLeastBlocks, static_cast<int>(all) + kShRowsCost);  // (one piece a tile: always)
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      int pieces = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) pieces += pieces_of(mine[j], shared[j], mid);
      pieces = __reduce_add_sync(0xffffffffu, pieces);
      if (pieces <= a.clusters) hi = mid;
      else lo = mid + 1;
    }
    if (lane == 0 && lo <= all / c + kShItemCost / 2) apart = lo;
  }
  __syncthreads();
  const int most = apart;
  auto range_begin = [&](int64_t k) { return k * weight / c; };
  auto cluster_of = [&](int64_t x) { return static_cast<int>(((x + 1) * c + weight - 1) / weight - 1); };
  int64_t at = 0, num_items = 0, num_parts = 0, num_split = 0;
  for (int t0 = 0; t0 < num_tiles; t0 += blockDim.x) {
    const int t = t0 + tid;
    const int blocks = t < num_tiles ? tiles[t].blocks : 0, shared = t < num_tiles ? tiles[t].shared : 0;
    int64_t v[1] = {t < num_tiles ? blocks + kShItemCost : 0}, total[1];
    block_scan<1>(v, total, sh);
    const int64_t off = at + v[0] + kShItemCost;  // the tile's first block
    at += total[0];
    int c0 = 0, pieces = 0;
    if (t < num_tiles) {
      c0 = cluster_of(off);
      pieces = most > 0 ? pieces_of(blocks, shared, most) : cluster_of(off + blocks - 1) - c0 + 1;
    }
    // items, partial sums and split tiles before this one's
    int64_t w[2] = {pieces, pieces > 1 ? pieces | (1ll << 40) : 0}, sums[2];
    block_scan<2>(w, sums, sh);
    const int item0 = static_cast<int>(num_items + w[0]);
    const int part0 = static_cast<int>(num_parts + (w[1] & ((1ll << 40) - 1)));
    ShTile tile = {};
    if (pieces > 0) tile = tiles[t];
    int end = 0;
    for (int k = 0; k < pieces; ++k) {
      ShItem i = {};
      if (most > 0) {
        // equal weights (times most), a block at least
        const int64_t heavy = static_cast<int64_t>(shared) * (most + kShRowsCost);
        const int64_t to = (heavy + static_cast<int64_t>(blocks - shared) * most) * (k + 1) / pieces;
        const int64_t upto = to <= heavy ? to / (most + kShRowsCost) : shared + (to - heavy) / most;
        i.begin = end;
        i.end = end = static_cast<int>(min(max(upto, static_cast<int64_t>(end + 1)), static_cast<int64_t>(blocks - (pieces - 1 - k))));
        i.cluster = item0 + k;
      } else {
        i.begin = static_cast<int>(max(range_begin(c0 + k), off) - off);
        i.end = static_cast<int>(min(range_begin(c0 + k + 1), off + blocks) - off);
        i.cluster = c0 + k;
      }
      i.part = pieces > 1 ? part0 + k : -1;
      i.row0 = tile.row0;
      i.rows = tile.rows;
      i.seg = tile.seg0 + last_at_most(tile.segs, i.begin, [&](int j) { return segs[tile.seg0 + j].block0; });
      i.seg_last = tile.seg0 + tile.segs - 1;
      i.prefix_end = shared;
      i.first = segs[i.seg];
      i.row_lo = i.first.row_lo;
      i.row_hi = i.begin < shared
                     ? tile.rows
                     : segs[tile.seg0 + last_at_most(tile.segs, i.end - 1, [&](int j) { return segs[tile.seg0 + j].block0; })].row_hi;
      items[item0 + k] = i;
    }
    if (pieces > 1) splits[num_split + (w[1] >> 40)] = ShSplit{tile.row0, tile.rows, pieces, part0};
    num_items += sums[0];
    num_parts += sums[1] & ((1ll << 40) - 1);
    num_split += sums[1] >> 40;
  }
  __syncthreads();
  for (int k = tid; k < a.clusters; k += blockDim.x) {  // (items are in the clusters' order)
    auto first_of = [&](int c) {
      int lo = 0, hi = static_cast<int>(num_items);
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (items[mid].cluster < c) lo = mid + 1;
        else hi = mid;
      }
      return lo;
    };
    ShCluster r = {};
    r.item0 = first_of(k);
    r.item1 = first_of(k + 1);
    if (r.item0 < r.item1) r.first = items[r.item0];
    clusters[k] = r;
  }
  if (tid == 0) {
    if (bad) atomicOr(&hd->status, MLA_STATUS_BAD_LENGTH);
    hd->batch = a.batch;
    hd->q_len = a.q_len;
    hd->num_heads = a.num_heads;
    hd->num_prefixes = a.num_prefixes;
    hd->page_size = a.page_size;
    hd->num_clusters = most > 0 ? static_cast<int>(num_items) : static_cast<int>(c);
    hd->num_tiles = num_tiles;
    hd->num_items = static_cast<int>(num_items);
    hd->num_split = static_cast<int>(num_split);
    hd->none = 0;
    hd->planned = kShPlanned;
  }
}

constexpr int kMergeWarps = 8;  // of a block
// Pieces whose loads are issued together, and blocks of the grid an SM that the decode uses.
// (6 pieces and 3 blocks, of more registers: 40.0 us instead of 41.3 a decode whose tiles are in
// 9 pieces, but 56.5 instead of 54.5 and 219 instead of 216.5 where they are in 2 or 3; over 28
// calls of other sizes as fast in the mean, 0.92 to 1.08 of the time.)
constexpr int kMergeBatch = 4, kMergeBlocks = 4;

// out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k over a split tile's pieces k, M the
// largest m_k of those seen so far. Pieces without a position of the row have l_k = 0 and
// whatever their O_k hold. A warp has eight rows of 32 dims at a time, a lane eight dims of a
// row; a batch's maxima, sums and accumulators come in together. Bound by the latency of its
// loads and by L2: about 3 us of a decode of 5 to 40 MB of partial sums, besides a launch.
__global__ void __launch_bounds__(32 * kMergeWarps) shared_merge_kernel(const ShDecodeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const ShHeader* hd = reinterpret_cast<const ShHeader*>(a.ws);
  if (!sh_planned(hd, a)) return;
  constexpr int kAcross = kDimCkv / 32, kUnits = kShRows / 8 * kAcross;  // of a tile
  const int lane = threadIdx.x & 31, units = hd->num_split * kUnits;
  for (int u = blockIdx.x * kMergeWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kMergeWarps) {
    const ShSplit sp = reinterpret_cast<const ShSplit*>(a.ws + a.lay.splits)[u / kUnits];
    const int row = u % kUnits / kAcross * 8 + (lane & 7), dim = u % kAcross * 32 + 8 * (lane >> 3);
    if (row >= sp.rows) continue;
    const float2* stats = reinterpret_cast<const float2*>(a.ws + a.lay.stats) + static_cast<int64_t>(sp.part0) * kShRows + row;
    const float* part = reinterpret_cast<const float*>(a.ws + a.lay.partial) +
                        static_cast<int64_t>(sp.part0) * (kShRows * kDimCkv) + dim * kShRows + 8 * row;
    float acc[8] = {}, sum = 0.f, top = -CUDART_INF_F;
    for (int k0 = 0; k0 < sp.pieces; k0 += kMergeBatch) {
      float2 ml[kMergeBatch];
      float x[kMergeBatch][8];
      float most = top;
#pragma unroll
      for (int k = 0; k < kMergeBatch; ++k) {
        ml[k] = make_float2(0.f, 0.f);
        if (k0 + k < sp.pieces) {
          ml[k] = stats[static_cast<int64_t>(k0 + k) * kShRows];
          ld_global_v8(part + static_cast<int64_t>(k0 + k) * (kShRows * kDimCkv), x[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kMergeBatch; ++k)
        if (ml[k].y != 0.f) most = fmaxf(most, ml[k].x);
      if (most != top) {
        const float w = exp2f(top - most);  // (0 at first)
        sum *= w;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= w;
        top = most;
      }
#pragma unroll
      for (int k = 0; k < kMergeBatch; ++k) {
        if (ml[k].y != 0.f) {
          const float w = exp2f(ml[k].x - top);
          sum = fmaf(w, ml[k].y, sum);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, x[k][e], acc[e]);
        }
      }
    }
    const float inv = a.out_scale / sum;
    const int64_t out_row = static_cast<int64_t>(sp.row0) + row;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + out_row * kDimCkv + dim) =
        make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                   pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    if (a.lse && dim == 0) a.lse[out_row] = (top + log2f(sum)) * 0.69314718055994531f;
  }
}

}  // namespace

cudaError_t launch_shared_plan(const ShPlanArgs& a, cudaStream_t stream) {
  return launch_pdl(shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
}

cudaError_t launch_shared_merge(const ShDecodeArgs& a, cudaStream_t stream) {
  return launch_pdl(shared_merge_kernel, dim3(kMergeBlocks * kShClusterBlocks * a.clusters), dim3(32 * kMergeWarps), 0, stream, a);
}

}  // namespace mla
