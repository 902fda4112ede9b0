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
// The expanded path's softmax weights and their sums are 2^7 of what they are against
// the reference maximum (see the attention kernel).
constexpr float kWeightShift = 7.f, kWeightUnit = 1.f / 128;
// Values are kept in f16 with a power of two of their own for each row and head,
// 2^(kBinBits k): bin k is that of the row's largest value, from 2^(kBinBits k + kBinLow)
// up, with no bins beyond +-kMostBin. Wide bins, so that the rows of a key step hardly
// ever differ; values between 2^-8 and 2^12 have bin 0 and are kept as they are. Rows of
// zeros may have any; kZeroBin leaves room for weights 2^40 times the others'. (A score
// takes its key's power, which rounds it to 2^-24 of that: a log of the sum is off by up
// to 2e-6 with 40, 4e-6 with 60.)
constexpr int kBinBits = 20, kBinLow = -8, kMostBin = 3, kZeroBin = -2;

// Request b as the plan sees it. Gathered positions are [lo, lo + rows); they
// sit at rows base .. of the workspace's row buffer, followed by zero rows up
// to a multiple of kPfKvAlign.
// Requests lie in the order of their rows: expanded ones first, then small ones.
struct PfRequest {
  int base, rows, lo, b;
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

// Requests with few new tokens are attended in the latent space (the absorbed
// form: 2,176 flops a pair and head instead of 640, but no keys and values to
// make) by the decode kernel, in row groups of up to kGroupRows (token, head)
// rows that are requests of their own to it. Their rows start at multiples of its
// 64-token blocks, so that the row buffer is its pool, with pages of 64 rows.
// Latent / expanded, us a call, 8 requests of n new tokens over 4,000: 128 heads, n = 1
// 86 / 1089, 16 350 / 1093, 56 1114 / 1300, 64 1273 / 1301; 32 heads, 56 313 / 327, 64
// 349 / 328; 16 heads, 16 105 / 184, 48 173 / 187, 56 191 / 187. Where there are few
// positions the expanded form starts no later: 4 requests over 1,000, 128 heads, 32
// 169 / 190, 40 206 / 195; one over 1,600, 32 87 / 100, 48 109 / 102.
constexpr int kPfSmallTokens = 56;       // at most, from kPfSmallSpan attended positions on
constexpr int kPfSmallSpan = 3000;
constexpr int kPfSmallTokensShort = 32;  // with fewer
constexpr int kPfSmallRows = 1 << 18;  // rows of all groups at most: 1,024 tokens of 128 heads, 1.1 GB of workspace

// Groups come in pairs of the same tokens: rounding the latent query to bf16 alone
// would cost 1.5e-3 of the result, nearly as much as the result's own rounding. The
// second group's query is what is left of twice the exact one, rounded: their mean
// is on a grid twice as fine, and their sums are joined into one, which averages the
// softmax weights' roundings as well. The result is off by about 2.0e-3 (2-norm); with
// single groups it was 2.6e-3, and with a rounded latent result 3.0e-3.
struct PfGroup {
  int base;      // workspace row of the request's relative position 0
  int first;     // relative position of the group's first token
  int q_row;     // its row of q and out
  int tokens;    // 1 .. tokens a full group has
  int page0;     // first entry of its page list
  int pages;
  int first_item, items;  // its work items of the decode, each of which leaves partial sums
};

struct PfHeader {
  int status;  // sticky MLA_STATUS_* bits
  int kv_rows;     // rows of the row buffer whose keys and values are made
  int num_tiles;
  int next_item;   // items of the current pass handed out beyond the first of each block
  int num_split;   // split tiles
  int merge_rows;  // their rows
  int all_rows;    // rows of the row buffer in use
  int num_groups;
  int even;        // no tile costs more than twice what another does
  int zero_rows;   // (gather) a row that is attended has c_kv zero; taken over by the expansion
  int odd_bins;    // any value row attended may have another bin than 0
  int pad[53];
};

// Key steps of a tile whose rows attend relative positions [begin, end).
__host__ __device__ inline int pf_steps(int begin, int end) {
  return end > begin ? (end - begin + kPfKvTile - 1) / kPfKvTile : 0;
}

struct PfLayout {
  size_t requests, tiles, sorted, splits, part_stats, part_o, rows, keys, values, bins, total;
  int64_t part_rows;    // partial rows of each head
  // Small requests in the latent space (absorb: whether the call may have any).
  size_t groups, group_indptr, group_pages, q_latent, latent, decode;
  int absorb;
  int group_tokens;     // tokens of a full group
  int max_pairs;        // groups come in pairs (see PfGroup)
  WsLayout decode_lay;
  int64_t kv_capacity;  // rows of the row buffer
  int64_t max_tiles;
  int heads;            // heads whose keys and values fit
};

// Calls look for small requests if the keys and values of all heads would take more than
// about 30 us to make: the four launches of that path cost 10 to 13 us where there are
// none (404 / 392 us with and without). Calls of few tokens a request (8 on average) from
// half of that on, or with so many (request, head) items that their starts count. Latent
// / expanded, us a call: 14 requests of one token over 60, 64 heads, 43 / 73; 4 of 4 over
// 200, 128 heads, 48 / 72; 30 of one over 50, 16 heads, 45 / 48; one of 8 over 1,000, 128
// heads, 52 / 63; below, 16 of one over 100, 16 heads, 45 / 41; 7 of one over 200 45 / 32;
// one of 16 over 2,000, 32 heads, 55 / 43. With more tokens: 2 of 20 over 400, 64 heads,
// 53 / 41.
inline bool pf_may_absorb(int64_t batch, int64_t q_rows, int64_t max_kv, int64_t num_heads) {
  if (num_heads != 16 && num_heads != 32 && num_heads != 64 && num_heads != 128) return false;
  if (max_kv * num_heads >= 200000) return true;
  return q_rows <= 8 * batch && (max_kv * num_heads >= 100000 || batch * num_heads >= 400);
}

// Workspace regions for `heads` of num_heads heads at a time, with or without the latent
// path. Every region grows with each of the arguments.
inline PfLayout pf_layout(int batch, int64_t q_rows, int64_t max_kv, int num_heads, int heads, bool absorb) {
  PfLayout L = {};
  L.heads = heads;
  L.absorb = absorb;
  const int64_t slack = static_cast<int64_t>(batch) * (L.absorb ? kBlockTokens : kPfKvAlign) + (L.absorb ? 256 : 0);
  L.kv_capacity = (max_kv + slack + kPfKvTile - 1) / kPfKvTile * kPfKvTile;
  L.max_tiles = q_rows / kPfRows + batch;
  if (L.max_tiles > q_rows) L.max_tiles = q_rows;  // (a tile has a row)
  // Partial rows of all heads: two tiles' rows for each pair of SMs, no more than the
  // pieces of every row. (The remainder of the division is kept, so that fewer heads
  // never take more room: a call cuts its heads into equal passes after it has found
  // how many fit.)
  int64_t part_rows = 2ll * kPfPairs * kPfRows;
  if (part_rows > kPfMostPieces * q_rows * heads) part_rows = kPfMostPieces * q_rows * heads;
  L.part_rows = part_rows / heads;
  const int64_t entries = L.max_tiles + kPfMostPieces;
  size_t off = sizeof(PfHeader);
  L.requests = off;
  off = align_up(off + sizeof(PfRequest) * (static_cast<size_t>(batch) + 1), 256);
  L.tiles = off;
  off = align_up(off + sizeof(PfTile) * static_cast<size_t>(entries), 256);
  L.sorted = off;
  off = align_up(off + sizeof(PfTile) * static_cast<size_t>(entries), 256);
  L.splits = off;
  off = align_up(off + sizeof(PfSplit) * kPfMostPieces, 256);
  L.part_stats = off;
  off = align_up(off + 8 * static_cast<size_t>(part_rows), 1024);
  L.part_o = off;
  off = align_up(off + 4 * kDimV * static_cast<size_t>(part_rows), 1024);
  L.rows = off;
  off = align_up(off + static_cast<size_t>(L.kv_capacity) * kDimRow * 2, 1024);
  L.keys = off;
  off = align_up(off + static_cast<size_t>(L.kv_capacity) * kDimNope * 2 * heads, 1024);
  L.values = off;
  off = align_up(off + static_cast<size_t>(L.kv_capacity) * kDimV * 2 * heads, 1024);
  L.bins = off;  // a byte a row and head; steps read whole, past the last row
  off = align_up(off + static_cast<size_t>(L.kv_capacity) * heads + kPfKvTile, 1024);
  if (L.absorb) {
    L.group_tokens = kGroupRows / num_heads;
    const int64_t per_request = (kPfSmallTokens + L.group_tokens - 1) / L.group_tokens;
    int64_t g = (q_rows + L.group_tokens - 1) / L.group_tokens + batch;
    if (g > per_request * batch) g = per_request * batch;
    if (g > kPfSmallRows / kGroupRows / 2) g = kPfSmallRows / kGroupRows / 2;
    L.max_pairs = static_cast<int>(g);
    const int groups = 2 * L.max_pairs;
    const size_t rows = static_cast<size_t>(g) * kGroupRows;
    L.groups = off;
    off = align_up(off + sizeof(PfGroup) * groups, 256);
    L.group_indptr = off;
    off = align_up(off + sizeof(int32_t) * (groups + 1), 256);
    L.group_pages = off;
    off = align_up(off + sizeof(int32_t) * (static_cast<size_t>(L.kv_capacity / kBlockTokens) * 2 * per_request + groups), 1024);
    L.q_latent = off;
    off = align_up(off + 2 * rows * kDimRow * 2, 1024);
    L.latent = off;
    off = align_up(off + rows * kDimCkv * 4, 1024);
    L.decode = off;
    // (with room for partial sums of every item: a group has one, and one more a cut)
    L.decode_lay = ws_layout(groups, kGroupRows, kPfPairs);
    const size_t items = static_cast<size_t>(groups) + kPfPairs;
    L.decode_lay.partial_o = align_up(L.decode_lay.partial_lse + sizeof(float) * items * kGroupRows, 256);
    L.decode_lay.total = align_up(L.decode_lay.partial_o + sizeof(float) * items * kGroupRows * kDimCkv, 256);
    off = align_up(off + L.decode_lay.total, 1024);
  }
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
  int clusters;      // of the decode kernel (small requests)
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
// prefill_gather.cu: tiles and row numbers, and the rows themselves
cudaError_t launch_prefill_gather(const PrefillArgs& a, cudaStream_t stream);
// prefill_expand.cu: keys and values of heads [head0, head0 + heads)
cudaError_t launch_prefill_expand(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream);
// prefill_attn.cu
cudaError_t launch_prefill_attn(const PrefillMaps& m, const PrefillArgs& a, int head0, int heads, cudaStream_t stream);
// prefill_gather.cu: split tiles' partial sums joined
cudaError_t launch_prefill_merge(const PrefillArgs& a, int head0, int heads, cudaStream_t stream);
// Whether any tile may be split (its plan decides): too few keys for two pieces otherwise.
__host__ __device__ inline bool pf_may_split(int64_t max_kv) { return max_kv > 6 * kPfKvTile; }
// prefill_absorb.cu: small requests' queries into the latent space, and their
// attention output out of it
cudaError_t launch_prefill_q_latent(const CUtensorMap& w_uk, const PrefillArgs& a, const void* q, cudaStream_t stream);
// (partial sums of the decode joined into pairs of bf16 rows)
cudaError_t launch_prefill_latent(const PrefillArgs& a, cudaStream_t stream);
cudaError_t launch_prefill_v_latent(const CUtensorMap& latent, const CUtensorMap& w_uv, const PrefillArgs& a, cudaStream_t stream);
// Streaming multiprocessors of the current device (0 on failure).
int sm_count();

}  // namespace mla
