// Launcher prototypes and workspace layout of the prefill-step kernels: page
// tables, the rotary latent write and the chunk attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mla_internal.h"

namespace mla {

struct TablesArgs {
  const int32_t* context_lens;
  const int32_t* new_lens;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* block_table;
  int64_t* slot_mapping;
  int32_t* positions;    // or null
  int32_t* q_indptr;
  int32_t* page_indptr;  // or null (then page_ids is null too)
  int32_t* page_ids;
  int32_t* state;
  int* status;           // or null
  int batch;
  int page_size;
  int page_shift;  // log2 of it
  int num_pages;
  int free_capacity;
  int max_blocks;
  int max_tokens;
  int max_page_ids;
};

constexpr int kRopePairs = kDimRope / 2;
constexpr int kMaxAxes = 4;

struct RopeArgs {
  uint8_t* layer_base;   // first row of the layer, or null: no latent rows
  int64_t layer_rows;
  const uint4* rows;
  const int64_t* slots;  // or null: no row is a pad row by its slot
  const int32_t* positions;  // [num_axes][n]
  const float* cos_sin;      // [max_position][64]: 32 cosines, 32 sines
  const void* norm_weight;   // bf16 [512] or null
  const uint16_t* q;         // first rope element of (token 0, head 0), or null
  uint16_t* q_out;
  int64_t q_pitch;           // elements between the heads' rows (token t, head h at row t * heads + h)
  int64_t q_out_pitch;
  int* status;
  uint64_t pair_axis;        // two bits for each of the 32 pairs
  float norm_eps;
  float kv_scale;
  int n;
  int num_axes;
  int max_position;
  int num_heads;
  int interleaved;
};

// ---------------------------------------------------------------- chunk attention (prefill)
constexpr int kDimNope = 128;
constexpr int kDimQk = 192;
constexpr int kPfRows = 512;      // query rows of one tile: two streams of two blocks' 128
constexpr int kPfKvAlign = 16;    // a request's gathered rows start at a multiple of this (one K step of an MMA)
constexpr int kPfKvTile = 128;    // key rows per step

// Request b as the plan sees it. Gathered positions are [lo, lo + rows); they
// sit at rows base .. of the workspace's row buffer, followed by zero rows up
// to a multiple of kPfKvAlign.
struct PfRequest {
  int base, rows, lo, pad;
};

// One query tile of one request, the same for every head. Positions below are
// relative to the request's first gathered position: row r attends
// [max(0, first_end + r - window), first_end + r).
struct PfTile {
  int q_row;      // first row of q and out
  int rows;       // 1 .. kPfRows
  int base;       // workspace row of relative position 0
  int kv_begin;   // first relative position any row attends, rounded down to kPfKvAlign
  int kv_end;     // end of the last row's range
  int first_end;  // end of row 0's range
  int refused;    // the request's lengths are bad: its rows are written as NaN
  // Where items are few, a tile runs as several over consecutive key steps, each
  // of which leaves its rows' sums in the partial buffers.
  int part_row;   // partial row (per head) of row 0, or -1: not split
  int pad[4];
};

static_assert(sizeof(PfTile) == 48, "three 16-byte words");

constexpr int kPfPairs = 76;         // SM pairs of the GPU: the clusters that run at once
constexpr int kPfMostPieces = 2 * kPfPairs;  // pieces of all split tiles of a head beyond the first of each

// A split tile: its pieces' partial rows follow each other, `rows` each. Row r of
// it is row merge_row + r of all split tiles' rows.
struct PfSplit {
  int q_row, rows, part_row, pieces, merge_row, pad[3];
};

struct PfHeader {
  int status;  // sticky MLA_STATUS_* bits
  int kv_rows;     // rows of the row buffer in use
  int num_tiles;
  int next_item;   // items of the current pass handed out beyond the first of each block
  int num_split;   // split tiles
  int merge_rows;  // their rows
  int pad[58];
};

// Key steps of a tile whose rows attend relative positions [begin, end).
__host__ __device__ inline int pf_steps(int begin, int end) {
  return end > begin ? (end - begin + kPfKvTile - 1) / kPfKvTile : 0;
}

struct PfLayout {
  size_t requests, tiles, order, splits, part_stats, part_o, rows, keys, values, total;
  int64_t part_rows;    // partial rows of each head
  int64_t kv_capacity;  // rows of the row buffer
  int64_t max_tiles;
  int heads;            // heads whose keys and values fit
};

// Workspace regions for `heads` heads at a time.
inline PfLayout pf_layout(int batch, int64_t q_rows, int64_t max_kv, int heads) {
  PfLayout L;
  L.heads = heads;
  L.kv_capacity = (max_kv + static_cast<int64_t>(batch) * kPfKvAlign + kPfKvTile - 1) / kPfKvTile * kPfKvTile;
  L.max_tiles = q_rows / kPfRows + batch;
  // Partial rows: two tiles' rows for each pair of SMs, no more than the pieces of every row.
  L.part_rows = 2ll * kPfPairs * kPfRows / heads;
  if (L.part_rows > kPfMostPieces * q_rows) L.part_rows = kPfMostPieces * q_rows;
  const int64_t entries = L.max_tiles + kPfMostPieces;
  size_t off = sizeof(PfHeader);
  L.requests = off;
  off = align_up(off + sizeof(PfRequest) * (static_cast<size_t>(batch) + 1), 256);
  L.tiles = off;
  off = align_up(off + sizeof(PfTile) * static_cast<size_t>(entries), 256);
  L.order = off;
  off = align_up(off + sizeof(int) * static_cast<size_t>(entries), 256);
  L.splits = off;
  off = align_up(off + sizeof(PfSplit) * kPfMostPieces, 256);
  L.part_stats = off;
  off = align_up(off + 8 * static_cast<size_t>(L.part_rows) * heads, 1024);
  L.part_o = off;
  off = align_up(off + 4 * kDimV * static_cast<size_t>(L.part_rows) * heads, 1024);
  L.rows = off;
  off = align_up(off + static_cast<size_t>(L.kv_capacity) * kDimRow * 2, 1024);
  L.keys = off;
  off = align_up(off + static_cast<size_t>(L.kv_capacity) * kDimNope * 2 * heads, 1024);
  L.values = off;
  off = align_up(off + static_cast<size_t>(L.kv_capacity) * kDimV * 2 * heads, 1024);
  L.total = off;
  return L;
}

struct PrefillArgs {
  const void* pool;
  const int32_t* page_indptr;
  const int32_t* page_ids;
  const int32_t* context_lens;
  const int32_t* q_indptr;
  void* out;
  float* lse;
  uint8_t* ws;
  PfLayout lay;
  int64_t max_kv;
  int max_blocks;
  int batch;
  int q_rows;
  int num_heads;
  int page_size;
  int num_pages;
  int layer;
  int dtype;
  int window;
  float scale_log2;  // softmax_scale * log2(e) (* kv_scale for fp8 pools)
  float out_scale;   // 1, or kv_scale for fp8 pools
};

struct PrefillMaps {
  CUtensorMap q;        // [T][H][192] as {192, H, T}, box {64, 1, 128}
  CUtensorMap rows;     // gathered rows [kv][576], box {64, 128}
  CUtensorMap ropes;    // same, box {64, 64}
  CUtensorMap keys;     // [heads][kv][128] as {128, kv, heads}, box {64, 64, 1}
  CUtensorMap values;   // same, box {64, 128, 1}
  CUtensorMap w_uk;     // [H * 128][512], box {64, 64}
  CUtensorMap w_uv;     // [H * 512][128], box {64, 64}
};

// step_tables.cu
cudaError_t launch_extend_tables(const TablesArgs& a, cudaStream_t stream);
// rope_write.cu
cudaError_t launch_rope_write(const RopeArgs& a, int dtype, cudaStream_t stream);
// prefill_gather.cu: tiles and row numbers, then the rows themselves
cudaError_t launch_prefill_plan(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_gather(const PrefillArgs& a, cudaStream_t stream);
// prefill_expand.cu: keys and values of heads [head0, head0 + heads)
cudaError_t launch_prefill_expand(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream);
// prefill_attn.cu
cudaError_t launch_prefill_attn(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream);
// prefill_gather.cu: split tiles' partial sums joined
cudaError_t launch_prefill_merge(const PrefillArgs& a, int head0, int heads, cudaStream_t stream);
// Whether any tile may be split (its plan decides): too few keys for two pieces otherwise.
__host__ __device__ inline bool pf_may_split(int64_t max_kv) { return max_kv > 6 * kPfKvTile; }
// Streaming multiprocessors of the current device (0 on failure).
int sm_count();

}  // namespace mla
