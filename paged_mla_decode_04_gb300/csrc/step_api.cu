// Entry points of the prefill step declared in include/mla_decode.h: page
// tables, the rotary latent write and the chunk attention. Argument checks,
// tensor maps, launches; no allocation, no stream synchronisation.
#include <limits.h>
#include <string.h>

#include "host_util.h"
#include "step_internal.h"

namespace {

using mla::aligned;
using mla::make_map_2d;
using mla::valid_pool;

// Keys and values of all heads at once up to this many bytes; beyond, fewer
// heads a pass (see mla_prefill_workspace_size).
constexpr size_t kExpandedBytes = size_t(8) << 30;

int* status_of(void* workspace) { return static_cast<int*>(workspace); }

int done(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

bool make_map_3d(CUtensorMap* m, const void* base, const uint64_t (&dims)[3], const uint64_t (&strides)[2],
                 const uint32_t (&box)[3]) {
  auto fn = mla::encode_fn();
  if (!fn) return false;
  cuuint64_t d[3] = {dims[0], dims[1], dims[2]};
  cuuint64_t s[2] = {strides[0], strides[1]};
  cuuint32_t b[3] = {box[0], box[1], box[2]};
  cuuint32_t e[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), d, s, b, e,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Small requests through the decode kernel: their queries into the latent space,
// one decode over the gathered rows as its pool (pages of 64 rows, a request per
// row group), its sums joined, the result out of the latent space.
int attend_small(const mla::PrefillMaps& m, const mla::PrefillArgs& a, const void* q, cudaStream_t st) {
  const mla::PfLayout& lay = a.lay;
  const uint64_t rows = static_cast<uint64_t>(lay.kv_capacity), h = a.num_heads;
  const int groups = 2 * lay.max_pairs;
  const uint64_t q_rows = static_cast<uint64_t>(groups) * mla::kGroupRows;
  constexpr auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  uint8_t *pool = a.ws + lay.rows, *qs = a.ws + lay.q_latent, *out = a.ws + lay.latent;
  CUtensorMap maps[5], latent;
  if (!make_map_2d(&maps[0], bf16, pool, rows, mla::kDimRow, mla::kDimRow * 2, 64, 64) ||
      !make_map_2d(&maps[1], bf16, pool, rows, mla::kDimRow, mla::kDimRow * 2, 32, 64, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !make_map_2d(&maps[2], bf16, qs, q_rows, mla::kDimRow, mla::kDimRow * 2, 64, 128) ||
      !make_map_2d(&maps[3], bf16, qs, q_rows, mla::kDimRow, mla::kDimRow * 2, 32, 128, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !make_map_3d(&maps[4], pool, {64, rows, 8}, {mla::kDimRow * 2ull, 128}, {64, 64, 4}) ||
      !make_map_3d(&latent, out, {mla::kDimCkv, h, 2ull * lay.max_pairs * lay.group_tokens},
                   {mla::kDimCkv * 2ull, h * mla::kDimCkv * 2ull}, {64, 1, 128}))
    return MLA_ERR_CUDA;
  mla::DecodeArgs d = {};
  d.pool = pool;
  d.page_indptr = reinterpret_cast<const int32_t*>(a.ws + lay.group_indptr);
  d.page_ids = reinterpret_cast<const int32_t*>(a.ws + lay.group_pages);
  d.out = out;
  d.ws = a.ws + lay.decode;
  d.lay = lay.decode_lay;
  d.batch = groups;
  d.num_heads = a.num_heads;
  d.q_len = lay.group_tokens;
  d.rows = d.group_rows = mla::kGroupRows;
  d.groups = 1;
  d.page_size = mla::kBlockTokens;
  d.window = a.window;
  d.num_pages = static_cast<int>(rows / mla::kBlockTokens);
  d.num_layers = 1;
  d.dtype = MLA_DTYPE_BF16;
  d.kv_scale = 1.f;
  d.scale_log2 = a.scale_log2;
  d.out_scale = a.out_scale;
  d.infinite_scores = true;  // (as in the expanded path)
  cudaError_t e = mla::launch_prefill_q_latent(m.w_uk, a, q, st);
  if (e == cudaSuccess) e = mla::launch_decode(maps, d, a.clusters, st);
  if (e == cudaSuccess) e = mla::launch_prefill_latent(a, st);
  if (e == cudaSuccess) e = mla::launch_prefill_v_latent(latent, m.w_uv, a, st);
  return done(e);
}

// The layout with the most heads at a time that `bytes` hold, none: heads = 0.
mla::PfLayout fit(int batch, int q_rows, int64_t max_kv, int num_heads, bool absorb, size_t bytes) {
  int lo = 0, hi = num_heads;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (mla::pf_layout(batch, q_rows, max_kv, num_heads, mid, absorb).total <= bytes) lo = mid;
    else hi = mid - 1;
  }
  if (lo == 0) return mla::PfLayout{};
  const int passes = (num_heads + lo - 1) / lo;
  return mla::pf_layout(batch, q_rows, max_kv, num_heads, (num_heads + passes - 1) / passes, absorb);
}

bool prefill_sizes_ok(int batch, int q_rows, int64_t max_kv, int heads) {
  if (batch < 0 || q_rows < 0 || max_kv < 0 || heads < 1 || heads > 1024) return false;
  if (static_cast<int64_t>(q_rows) * heads >= (1ll << 31)) return false;
  return max_kv + static_cast<int64_t>(batch) * mla::kBlockTokens + 512 < (1ll << 31);
}

}  // namespace

extern "C" {

int mla_extend_tables(const int32_t* context_lens, const int32_t* new_lens, int batch, int page_size, int num_pages,
                      const int32_t* free_pages, const int32_t* free_count, int free_capacity, int32_t* block_table,
                      int max_blocks, int64_t* slot_mapping, int32_t* positions, int max_tokens, int32_t* q_indptr,
                      int32_t* page_indptr, int32_t* page_ids, int max_page_ids, int32_t* state, void* workspace,
                      void* stream) {
  if (batch < 0 || num_pages <= 0 || free_capacity < 0 || max_blocks <= 0 || max_tokens < 0 || max_page_ids < 0)
    return MLA_ERR_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return MLA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks) * page_size > INT_MAX) return MLA_ERR_ARG;  // positions are int32
  if (static_cast<int64_t>(batch) * max_blocks > INT_MAX) return MLA_ERR_ARG;  // so are the CSR lists' pointers
  if (!free_count || !q_indptr || !state || (free_capacity > 0 && !free_pages)) return MLA_ERR_ARG;
  if (batch > 0 && (!context_lens || !new_lens || !block_table)) return MLA_ERR_ARG;
  if (max_tokens > 0 && !slot_mapping) return MLA_ERR_ARG;
  if (page_indptr ? !page_ids && max_page_ids > 0 : page_ids != nullptr) return MLA_ERR_ARG;
  if (!aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  mla::TablesArgs a = {};
  a.context_lens = context_lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.block_table = block_table;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.q_indptr = q_indptr;
  a.page_indptr = page_indptr;
  a.page_ids = page_ids;
  a.state = state;
  a.status = status_of(workspace);
  a.batch = batch;
  a.page_size = page_size;
  a.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  a.num_pages = num_pages;
  a.free_capacity = free_capacity;
  a.max_blocks = max_blocks;
  a.max_tokens = max_tokens;
  a.max_page_ids = max_page_ids;
  return done(mla::launch_extend_tables(a, static_cast<cudaStream_t>(stream)));
}

int mla_rope_write(const mla_kv_pool* pool, int layer, const void* rows, const int64_t* slot_mapping, int n,
                   const int32_t* positions, int num_axes, const uint8_t* pair_axis, const float* cos_sin,
                   int max_position, int interleaved, const void* norm_weight, float norm_eps, const void* q_rope,
                   int64_t q_pitch, void* q_out, int64_t q_out_pitch, int num_heads, void* workspace, void* stream) {
  if (n < 0 || num_axes < 1 || num_axes > mla::kMaxAxes || max_position < 1) return MLA_ERR_ARG;
  mla::RopeArgs a = {};
  for (int j = 0; j < mla::kRopePairs; ++j) {
    const int axis = pair_axis ? pair_axis[j] : 0;
    if (axis >= num_axes) return MLA_ERR_ARG;
    a.pair_axis |= static_cast<uint64_t>(axis) << (2 * j);
  }
  if (!rows && !q_rope) return n == 0 ? MLA_OK : MLA_ERR_ARG;
  if (rows && (!valid_pool(pool) || layer < 0 || layer >= pool->num_layers)) return MLA_ERR_ARG;
  if (q_rope && num_heads < 1) return MLA_ERR_ARG;
  if (norm_weight && !(norm_eps >= 0.f)) return MLA_ERR_ARG;
  if (n == 0) return MLA_OK;
  if (!positions || !cos_sin || !aligned(cos_sin, 16)) return MLA_ERR_ARG;
  if (rows && (!slot_mapping || !aligned(rows, 16) || !aligned(norm_weight, 16))) return MLA_ERR_ARG;
  if (q_rope) {
    if (!q_out || !aligned(q_rope, 16) || !aligned(q_out, 16)) return MLA_ERR_ARG;
    if (q_pitch < mla::kDimRope || q_out_pitch < mla::kDimRope || q_pitch % 8 || q_out_pitch % 8) return MLA_ERR_ARG;
    const int64_t count = static_cast<int64_t>(n) * num_heads;
    if (count >= (1ll << 31)) return MLA_ERR_ARG;
    // In place, or apart: rows that overlap others' are refused (a warp would
    // read what another has turned already).
    const char *s = static_cast<const char*>(q_rope), *d = static_cast<const char*>(q_out);
    const char* s_end = s + ((count - 1) * q_pitch + mla::kDimRope) * 2;
    const char* d_end = d + ((count - 1) * q_out_pitch + mla::kDimRope) * 2;
    if (s < d_end && d < s_end && !(s == d && q_pitch == q_out_pitch)) {
      if (q_pitch != q_out_pitch) return MLA_ERR_ARG;
      const int64_t pitch = q_pitch * 2, off = (((d - s) % pitch) + pitch) % pitch;
      if (off < mla::kDimRope * 2 || off > pitch - mla::kDimRope * 2) return MLA_ERR_ARG;
    }
  }
  if (!aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  int dtype = MLA_DTYPE_BF16;
  if (rows) {
    dtype = pool->dtype;
    a.layer_rows = static_cast<int64_t>(pool->num_pages) * pool->page_size;
    a.layer_base = static_cast<uint8_t*>(pool->data) +
                   layer * a.layer_rows * mla::kDimRow * (dtype == MLA_DTYPE_BF16 ? 2 : 1);
    a.rows = static_cast<const uint4*>(rows);
    a.kv_scale = pool->kv_scale;
  }
  a.slots = slot_mapping;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.norm_weight = norm_weight;
  a.q = static_cast<const uint16_t*>(q_rope);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_pitch = q_pitch;
  a.q_out_pitch = q_out_pitch;
  a.status = status_of(workspace);
  a.norm_eps = norm_eps;
  a.n = n;
  a.num_axes = num_axes;
  a.max_position = max_position;
  a.num_heads = num_heads;
  a.interleaved = interleaved;
  return done(mla::launch_rope_write(a, dtype, static_cast<cudaStream_t>(stream)));
}

size_t mla_prefill_workspace_size(int batch, int q_rows, int64_t max_kv_tokens, int num_heads, int heads_per_pass) {
  if (!prefill_sizes_ok(batch, q_rows, max_kv_tokens, num_heads) || heads_per_pass < 0) return 0;
  // The most rows with which a call of no more requests and positions may take the latent path.
  int64_t latent_rows = q_rows;
  if (!mla::pf_may_absorb(batch, latent_rows, max_kv_tokens, num_heads) && latent_rows > 8ll * batch) latent_rows = 8ll * batch;
  const bool latent = mla::pf_may_absorb(batch, latent_rows, max_kv_tokens, num_heads);
  int h = heads_per_pass;
  if (h == 0) {
    const mla::PfLayout one = mla::pf_layout(batch, q_rows, max_kv_tokens, num_heads, 1, latent);
    const size_t per_head = static_cast<size_t>(one.kv_capacity) * ((mla::kDimNope + mla::kDimV) * 2 + 1);
    h = per_head * num_heads <= kExpandedBytes ? num_heads : static_cast<int>(kExpandedBytes / per_head);
    if (h < 1) h = 1;
  }
  if (h > num_heads) h = num_heads;
  const size_t expanded = mla::pf_layout(batch, q_rows, max_kv_tokens, num_heads, h, false).total;
  const size_t both = latent ? mla::pf_layout(batch, latent_rows, max_kv_tokens, num_heads, h, true).total : 0;
  return expanded > both ? expanded : both;
}

int mla_prefill(const mla_kv_pool* pool, int layer, const void* q, const int32_t* q_indptr, const int32_t* page_indptr,
                const int32_t* page_ids, int max_blocks, const int32_t* context_lens, int batch, int q_rows,
                int64_t max_kv_tokens, int num_heads, const void* w_uk, const void* w_uv, float softmax_scale,
                int window, void* workspace, size_t workspace_bytes, void* out, float* lse, void* stream) {
  if (!valid_pool(pool) || layer < 0 || layer >= pool->num_layers || window < 0) return MLA_ERR_ARG;
  if (!prefill_sizes_ok(batch, q_rows, max_kv_tokens, num_heads)) return MLA_ERR_ARG;
  if (!(softmax_scale > 0.f)) return MLA_ERR_ARG;
  if (batch == 0 || q_rows == 0) return MLA_OK;
  if (!q || !q_indptr || (!page_ids && !page_indptr) || !context_lens || !w_uk || !w_uv || !out) return MLA_ERR_ARG;
  if (!aligned(q, 16) || !aligned(w_uk, 16) || !aligned(w_uv, 16) || !aligned(out, 32)) return MLA_ERR_ARG;
  if (!page_indptr && (max_blocks <= 0 || static_cast<int64_t>(max_blocks) * pool->page_size > INT_MAX)) return MLA_ERR_ARG;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  // (a workspace of another call's size may lack the room for the latent path)
  const bool absorb = mla::pf_may_absorb(batch, q_rows, max_kv_tokens, num_heads);
  mla::PrefillArgs a = {};
  a.lay = fit(batch, q_rows, max_kv_tokens, num_heads, absorb, workspace_bytes);
  if (absorb && a.lay.heads == 0) a.lay = fit(batch, q_rows, max_kv_tokens, num_heads, false, workspace_bytes);
  if (a.lay.heads == 0) return MLA_ERR_WORKSPACE;
  const int per_pass = a.lay.heads;

  a.pool = pool->data;
  a.page_indptr = page_indptr;
  a.page_ids = page_ids;
  a.context_lens = context_lens;
  a.q_indptr = q_indptr;
  a.out = out;
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(workspace);
  a.max_blocks = max_blocks;
  a.max_kv = max_kv_tokens;
  a.batch = batch;
  a.q_rows = q_rows;
  a.num_heads = num_heads;
  a.page_size = pool->page_size;
  a.num_pages = pool->num_pages;
  a.layer = layer;
  a.dtype = pool->dtype;
  a.window = window;
  const bool fp8 = pool->dtype == MLA_DTYPE_FP8_E4M3;
  a.scale_log2 = softmax_scale * 1.4426950408889634f * (fp8 ? pool->kv_scale : 1.f);
  a.out_scale = fp8 ? pool->kv_scale : 1.f;

  const uint64_t cap = static_cast<uint64_t>(a.lay.kv_capacity), h = num_heads;
  mla::PrefillMaps m;
  memset(&m, 0, sizeof m);
  if (!make_map_3d(&m.q, q, {mla::kDimQk, h, static_cast<uint64_t>(q_rows)}, {mla::kDimQk * 2, h * mla::kDimQk * 2},
                   {64, 1, 128}) ||
      !make_map_2d(&m.rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.ws + a.lay.rows, cap, mla::kDimRow, mla::kDimRow * 2, 64,
                   128) ||
      !make_map_2d(&m.ropes, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.ws + a.lay.rows, cap, mla::kDimRow, mla::kDimRow * 2, 64,
                   64) ||
      !make_map_3d(&m.keys, a.ws + a.lay.keys, {mla::kDimNope, cap, static_cast<uint64_t>(per_pass)},
                   {mla::kDimNope * 2, cap * mla::kDimNope * 2}, {64, 64, 1}) ||
      !make_map_3d(&m.values, a.ws + a.lay.values, {mla::kDimV, cap, static_cast<uint64_t>(per_pass)},
                   {mla::kDimV * 2, cap * mla::kDimV * 2}, {64, 128, 1}) ||
      !make_map_2d(&m.w_uk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w_uk, h * mla::kDimNope, mla::kDimCkv, mla::kDimCkv * 2, 64,
                   64) ||
      !make_map_2d(&m.w_uv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w_uv, h * mla::kDimCkv, mla::kDimV, mla::kDimV * 2, 64, 64))
    return MLA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.lay.absorb) {
    const int c = mla::decode_max_active_clusters();
    if (c <= 0) return MLA_ERR_CUDA;
    a.clusters = c < mla::kPfPairs ? c : mla::kPfPairs;
  }
  cudaError_t e = mla::launch_prefill_gather(a, st);
  if (e == cudaSuccess && a.lay.absorb) {
    const int rc = attend_small(m, a, q, st);
    if (rc != MLA_OK) return rc;
  }
  for (int h0 = 0; h0 < num_heads && e == cudaSuccess; h0 += per_pass) {
    const int n = h0 + per_pass <= num_heads ? per_pass : num_heads - h0;
    e = mla::launch_prefill_expand(m, a, h0, n, st);
    if (e == cudaSuccess) e = mla::launch_prefill_attn(m, a, h0, n, st);
    if (e == cudaSuccess && mla::pf_may_split(max_kv_tokens)) e = mla::launch_prefill_merge(a, h0, n, st);
  }
  return done(e);
}

}  // extern "C"
