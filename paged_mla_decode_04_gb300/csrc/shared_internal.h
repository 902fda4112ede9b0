// Workspace layout, records and launchers of the decode over shared prefixes, and
// of the compact latent store.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mla_internal.h"

namespace mla {

// The batch's rows are numbered through: row r = (b * q_len + i) * num_heads + h, as q
// and out have them. A tile is up to kShRows rows of one group of requests (those with
// the same prefix), in order. What its rows attend is a sequence of segments: the
// group's prefix, which all of them attend, then each request's own positions, which
// only that request's rows attend. A segment is worked off in blocks of kShTokens
// positions, dealt to the clusters of the attention kernel; a tile that several clusters
// share is joined afterwards.
constexpr int kShRows = 256;
constexpr int kShTokens = 128;
constexpr int kShClusterBlocks = 4;  // thread blocks of a cluster
constexpr int kShMostClusters = 128; // that a plan deals to
// A tile's first block costs a cluster this many more (queries into place, the
// pipeline's start, the result's way out, in part behind the item before). 2, 3, 4 and 6 took
// 56.5, 55.0, 54.7 and 55.6 us a decode of 15 tiles of 37 blocks. Over 28 calls of 2 to 215
// requests, 8 to 256 rows each, behind 17 to 50,000 positions, 2 and 3 are 0.3 % slower in the
// mean (0.97 to 1.07 of the time) and 6 is 0.5 % slower (0.98 to 1.05) but for one call of theirs:
// 69 requests of 128 rows behind 202 positions, 35 tiles for 36 clusters, 20.5 us instead of 33.1.
constexpr int kShItemCost = 4;
// A piece of a prefix's blocks costs this many more than one of requests' own (see the plan).
// Within 2 % from 3 to 7 but for small batches: 18 to 29 us, by turns one or the other. (Those 28
// calls: 2 is 0.2 % slower in the mean but for the same one, 7 is 0.3 % faster, 0.93 to 1.04.)
constexpr int kShRowsCost = 4;
// Clusters are used as far as each has this many blocks. 2 instead of 3: 15.2 us instead of
// 16.6, 18.9 instead of 20.1, 24.5 instead of 26.2; at worst 19.6 instead of 18.6. (Those 28
// calls: 3 is 1.5 % slower in the mean, 0.93 to 1.13; 1 is as fast, 0.93 to 1.13.)
constexpr int kShLeastBlocks = 2;

// Cached positions of a request are fewer (a tile's blocks then count in 32 bits).
constexpr int kShMostLength = 1 << 29;

struct ShTile {
  int row0;  // first row
  int rows;
  int seg0, segs;  // its segments
  int blocks;      // of all of them
  int shared;      // those of the prefix
  int pad[2];
};

// Positions [tok_lo, tok_hi) of request `owner`'s pages, which rows [row_lo, row_hi) of
// the tile attend: row r = (b, i, h) up to position base + i. Its blocks start at tok0,
// a multiple of what one copy brings (no more than a page), so tok0 <= tok_lo.
struct ShSegment {
  int owner;
  int row_lo, row_hi;
  int block0;  // the tile's blocks before it
  int tok0, tok_lo, tok_hi;
  int base;
};

// Blocks [begin, end) of a tile, with what the kernel's roles start from (each load that
// waits for another costs them half a microsecond).
struct ShItem {
  int begin, end;
  int part;            // -1: the whole tile; else the partial sums' number
  int cluster;
  int row0, rows;      // the tile's
  int seg, seg_last;   // segment of the first block; the tile's last one
  int prefix_end;      // blocks of the prefix
  int row_lo, row_hi;  // rows of the tile that attend any of the blocks
  int pad[5];
  ShSegment first;     // segment `seg`
};

// A cluster's items [item0, item1), and the first of them.
struct ShCluster {
  int item0, item1;
  int pad[6];
  ShItem first;
};

// A split tile.
struct ShSplit {
  int row0, rows, pieces, part0;
};

// A group as the plan sees it.
struct ShGroup {
  int first, count;  // requests
  int prefix;        // positions shared
  int tile0;         // tiles of the groups before it
  int tile_rows;     // of a full tile
  int pad[3];
};

static_assert(sizeof(ShTile) == 32 && sizeof(ShSegment) == 32 && sizeof(ShItem) == 96 && sizeof(ShCluster) == 128, "16-byte words");

struct ShHeader {
  int status;  // sticky MLA_STATUS_* bits
  int batch, q_len, num_heads, num_prefixes, page_size;
  int planned;  // kShPlanned
  int num_clusters, num_tiles, num_items, num_split;
  int none;  // 0: where mla_decode's plan has its q_len
  int pad[52];
};
// (no count that another plan has there: a workspace may serve several kinds of calls by turns, and
// a plan one of them only)
constexpr int kShPlanned = 0x53684c6e;
static_assert(sizeof(ShHeader) == 256, "one header of 256 bytes");

struct ShLayout {
  size_t groups, tiles, segs, items, clusters, splits, stats, partial, total;
  int max_tiles;
  int segs_per_tile;  // at most
};

// Rows of a tile that has whole requests, where one fits: no request's own positions are
// attended by two tiles then. (The plan fills tiles up where that is less work.)
__host__ __device__ inline int sh_whole_rows(int64_t r) { return r <= kShRows ? static_cast<int>(kShRows / r * r) : kShRows; }

__host__ __device__ inline ShLayout sh_layout(int batch, int q_len, int heads, int prefixes, int clusters) {
  ShLayout L = {};
  const int64_t r = static_cast<int64_t>(q_len) * heads;
  // the prefix; of a full tile's rows the first one's request and those that the others begin
  L.segs_per_tile = 2 + static_cast<int>((kShRows - 2 + r) / r);
  const int64_t tiles = batch * r / sh_whole_rows(r) + (prefixes < batch ? prefixes : batch);
  L.max_tiles = static_cast<int>(tiles);
  size_t off = sizeof(ShHeader);
  L.groups = off;
  off = align_up(off + sizeof(ShGroup) * static_cast<size_t>(prefixes), 256);
  L.tiles = off;
  off = align_up(off + sizeof(ShTile) * static_cast<size_t>(tiles), 256);
  L.segs = off;
  off = align_up(off + sizeof(ShSegment) * static_cast<size_t>(tiles) * L.segs_per_tile, 256);
  L.items = off;
  off = align_up(off + sizeof(ShItem) * static_cast<size_t>(tiles + clusters), 256);
  L.clusters = off;
  off = align_up(off + sizeof(ShCluster) * static_cast<size_t>(clusters), 256);
  L.splits = off;
  off = align_up(off + sizeof(ShSplit) * static_cast<size_t>(clusters), 256);
  const size_t parts = 2 * static_cast<size_t>(clusters);
  L.stats = off;
  off = align_up(off + sizeof(float2) * parts * kShRows, 1024);
  L.partial = off;
  off = align_up(off + sizeof(float) * parts * kShRows * kDimCkv, 1024);
  L.total = off;
  return L;
}

// Positions that one copy brings: of one page, and at most half a block.
__host__ __device__ inline int sh_copy_tokens(int page_size) { return page_size < 64 ? page_size : 64; }

struct ShPlanArgs {
  const int32_t* context_lens;
  const int32_t* prefix_indptr;
  const int32_t* prefix_lens;
  uint8_t* ws;
  ShLayout lay;
  int batch, q_len, num_heads, num_prefixes, page_size;
  int clusters;  // to cut for
};

struct ShDecodeArgs {
  const void* pool;
  const void* q;
  const int32_t* page_indptr;
  const int32_t* page_ids;
  void* out;   // bf16 [rows][512]
  float* lse;  // [rows] or null
  uint8_t* ws;
  ShLayout lay;
  int max_blocks;
  int batch, q_len, num_heads, num_prefixes;
  int page_size, num_pages, num_layers, layer, dtype;
  int clusters;      // of the grid
  float scale_log2;  // softmax_scale * log2(e) (* kv_scale for fp8 pools)
  float out_scale;   // 1, or kv_scale for fp8 pools
};

// Whether the workspace holds a plan for this call. (Clusters beyond the grid's would go
// unserved.)
__device__ __forceinline__ bool sh_planned(const ShHeader* hd, const ShDecodeArgs& a) {
  return hd->planned == kShPlanned && hd->batch == a.batch && hd->q_len == a.q_len && hd->num_heads == a.num_heads &&
         hd->num_prefixes == a.num_prefixes && hd->page_size == a.page_size && hd->num_clusters <= a.clusters;
}

// shared_plan.cu
cudaError_t launch_shared_plan(const ShPlanArgs& a, cudaStream_t stream);
cudaError_t launch_shared_merge(const ShDecodeArgs& a, cudaStream_t stream);
// shared_decode.cu
// maps: bf16 pools as [rows][576], box {64, sh_copy_tokens}; where that is 64, as
// [chunk][rows][64 dims] with boxes of three and of four chunks. fp8 pools: none, boxes
// {192, sh_copy_tokens} and {256, sh_copy_tokens}, unswizzled. Then q as [rows][576], box
// {64, 32}.
cudaError_t launch_shared_decode(const CUtensorMap (&maps)[4], const ShDecodeArgs& a, cudaStream_t stream);
int shared_max_active_clusters();

// ---------------------------------------------------------------- compact latent store
// Rows of codes, their groups' scales and the rope dims in bf16:
//   e4m3: 512 codes, 4 fp32 scales (128 dims each), 64 bf16        656 bytes
//   e2m1: 256 bytes of two codes, 16 bf16 scales (32 dims each), 64 bf16   416 bytes
constexpr int kStoreE4m3Row = 656, kStoreE2m1Row = 416;

struct StoreWriteArgs {
  uint8_t* layer_base;
  int64_t layer_rows;
  const uint4* rows;
  const int64_t* slots;
  int* status;
  int n;
};

struct StoreReadArgs {
  const uint8_t* layer_base;
  int64_t layer_rows;
  const int64_t* slots;
  uint8_t* out;          // rows in order, or the pool layer's first row
  const int64_t* out_slots;  // null: rows in order
  int64_t out_rows;
  float kv_scale;
  int* status;
  int n;
};

// quant_store.cu
cudaError_t launch_store_write(const StoreWriteArgs& a, int format, cudaStream_t stream);
// (out_dtype: MLA_DTYPE_*)
cudaError_t launch_store_read(const StoreReadArgs& a, int format, int out_dtype, cudaStream_t stream);

}  // namespace mla
