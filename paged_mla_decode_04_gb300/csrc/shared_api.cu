// Entry points of the decode over shared prefixes and of the compact latent store,
// declared in include/mla_decode.h: argument checks and launches; no allocation, no
// stream synchronisation.
#include "host_util.h"
#include "shared_internal.h"

namespace {

using mla::aligned;
using mla::valid_pool;

int done(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

bool sizes_ok(int batch, int q_len, int heads, int prefixes) {
  constexpr int kMost = 1 << 22;  // (a plan's records count in 32 bits)
  if (batch < 0 || batch > kMost || q_len < 1 || heads < 1 || heads > 1024 || prefixes < 0 || prefixes > kMost) return false;
  return static_cast<int64_t>(batch) * q_len * heads < (1ll << 31) && static_cast<int64_t>(q_len) * heads < (1ll << 30);
}

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }

bool valid_store(const mla_quant_pool* p) {
  if (!p || !p->data || p->num_layers <= 0 || p->num_pages <= 0 || !page_size_ok(p->page_size)) return false;
  return (p->format == MLA_QUANT_E4M3 || p->format == MLA_QUANT_E2M1) && aligned(p->data, 16);
}

int64_t store_row(int format) { return format == MLA_QUANT_E4M3 ? mla::kStoreE4m3Row : mla::kStoreE2m1Row; }

}  // namespace

extern "C" {

size_t mla_decode_workspace_size_shared(int batch, int q_len, int num_heads, int num_prefixes) {
  if (!sizes_ok(batch, q_len, num_heads, num_prefixes)) return 0;
  const int c = mla::shared_max_active_clusters();
  if (c <= 0) return 0;
  return mla::sh_layout(batch, q_len, num_heads, num_prefixes, c).total;
}

int mla_decode_plan_shared(const int32_t* context_lens, const int32_t* prefix_indptr, const int32_t* prefix_lens, int batch,
                           int num_prefixes, int q_len, int num_heads, int page_size, int num_clusters, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!sizes_ok(batch, q_len, num_heads, num_prefixes) || num_clusters < 0) return MLA_ERR_ARG;
  if (!page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED;
  if (!prefix_indptr || (num_prefixes > 0 && !prefix_lens) || (batch > 0 && !context_lens)) return MLA_ERR_ARG;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  const int most = mla::shared_max_active_clusters();
  if (most <= 0) return MLA_ERR_CUDA;
  mla::ShPlanArgs a = {};
  a.lay = mla::sh_layout(batch, q_len, num_heads, num_prefixes, most);
  if (workspace_bytes < a.lay.total) return MLA_ERR_WORKSPACE;
  a.context_lens = context_lens;
  a.prefix_indptr = prefix_indptr;
  a.prefix_lens = prefix_lens;
  a.ws = static_cast<uint8_t*>(workspace);
  a.batch = batch;
  a.q_len = q_len;
  a.num_heads = num_heads;
  a.num_prefixes = num_prefixes;
  a.page_size = page_size;
  a.clusters = num_clusters == 0 || num_clusters > most ? most : num_clusters;
  return done(mla::launch_shared_plan(a, static_cast<cudaStream_t>(stream)));
}

int mla_decode_shared(const mla_kv_pool* pool, int layer, const void* q, const int32_t* page_indptr, const int32_t* page_ids,
                      int max_blocks, int batch, int q_len, int num_heads, int num_prefixes, float softmax_scale,
                      void* workspace, void* out, float* lse, void* stream) {
  if (!valid_pool(pool) || layer < 0 || layer >= pool->num_layers) return MLA_ERR_ARG;
  if (!sizes_ok(batch, q_len, num_heads, num_prefixes) || !(softmax_scale > 0.f)) return MLA_ERR_ARG;
  if (batch == 0 || num_prefixes == 0) return MLA_OK;
  if (!q || (!page_ids && !page_indptr) || !out || !aligned(q, 16) || !aligned(out, 32)) return MLA_ERR_ARG;
  if (!page_indptr && max_blocks <= 0) return MLA_ERR_ARG;
  if (!workspace || !aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  const uint64_t rows = static_cast<uint64_t>(pool->num_layers) * pool->num_pages * pool->page_size;
  if (rows >= (1ull << 31)) return MLA_ERR_UNSUPPORTED;  // TMA row coordinates are int32
  const int most = mla::shared_max_active_clusters();
  if (most <= 0) return MLA_ERR_CUDA;
  const bool fp8 = pool->dtype == MLA_DTYPE_FP8_E4M3;
  mla::ShDecodeArgs a = {};
  a.lay = mla::sh_layout(batch, q_len, num_heads, num_prefixes, most);
  a.pool = pool->data;
  a.q = q;
  a.page_indptr = page_indptr;
  a.page_ids = page_ids;
  a.out = out;
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(workspace);
  a.max_blocks = max_blocks;
  a.batch = batch;
  a.q_len = q_len;
  a.num_heads = num_heads;
  a.num_prefixes = num_prefixes;
  a.page_size = pool->page_size;
  a.num_pages = pool->num_pages;
  a.num_layers = pool->num_layers;
  a.layer = layer;
  a.dtype = pool->dtype;
  a.clusters = most;
  a.scale_log2 = softmax_scale * 1.4426950408889634f * (fp8 ? pool->kv_scale : 1.f);
  a.out_scale = fp8 ? pool->kv_scale : 1.f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap maps[4] = {};
  const uint64_t q_rows = static_cast<uint64_t>(batch) * q_len * num_heads;
  if (!mla::make_map_2d(&maps[3], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, q_rows, mla::kDimRow, mla::kDimRow * 2, 64, 32))
    return MLA_ERR_CUDA;
  const uint32_t copy = mla::sh_copy_tokens(pool->page_size);
  if (fp8) {
    constexpr auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    constexpr auto plain = CU_TENSOR_MAP_SWIZZLE_NONE;
    if (!mla::make_map_2d(&maps[1], u8, pool->data, rows, mla::kDimRow, mla::kDimRow, 192, copy, plain) ||
        !mla::make_map_2d(&maps[2], u8, pool->data, rows, mla::kDimRow, mla::kDimRow, 256, copy, plain))
      return MLA_ERR_CUDA;
  } else if (!mla::make_map_2d(&maps[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pool->data, rows, mla::kDimRow, mla::kDimRow * 2, 64, copy) ||
             !mla::make_map_chunks(&maps[1], pool->data, rows, mla::kDimRow, mla::kDimRow * 2, copy, 3) ||
             !mla::make_map_chunks(&maps[2], pool->data, rows, mla::kDimRow, mla::kDimRow * 2, copy, 4)) {
    return MLA_ERR_CUDA;
  }
  cudaError_t e = mla::launch_shared_decode(maps, a, st);
  if (e == cudaSuccess) e = mla::launch_shared_merge(a, st);
  return done(e);
}

int mla_quant_write(const mla_quant_pool* pool, int layer, const void* rows, const int64_t* slot_mapping, int n,
                    void* workspace, void* stream) {
  if (n < 0 || !valid_store(pool) || layer < 0 || layer >= pool->num_layers) return MLA_ERR_ARG;
  if (n == 0) return MLA_OK;
  if (!rows || !slot_mapping || !aligned(rows, 16)) return MLA_ERR_ARG;
  if (!aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  mla::StoreWriteArgs a = {};
  a.layer_rows = static_cast<int64_t>(pool->num_pages) * pool->page_size;
  a.layer_base = static_cast<uint8_t*>(pool->data) + layer * a.layer_rows * store_row(pool->format);
  a.rows = static_cast<const uint4*>(rows);
  a.slots = slot_mapping;
  a.status = static_cast<int*>(workspace);
  a.n = n;
  return done(mla::launch_store_write(a, pool->format, static_cast<cudaStream_t>(stream)));
}

int mla_quant_read(const mla_quant_pool* pool, int layer, const int64_t* slots, int n, const mla_kv_pool* into, int into_layer,
                   const int64_t* into_slots, void* rows, void* workspace, void* stream) {
  if (n < 0 || !valid_store(pool) || layer < 0 || layer >= pool->num_layers) return MLA_ERR_ARG;
  if (into && rows) return MLA_ERR_ARG;
  if (into && (!valid_pool(into) || into_layer < 0 || into_layer >= into->num_layers)) return MLA_ERR_ARG;
  if (n == 0) return MLA_OK;
  if (!slots || (into ? !into_slots : !rows || into_slots) || !aligned(rows, 16)) return MLA_ERR_ARG;
  if (!aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
  mla::StoreReadArgs a = {};
  a.layer_rows = static_cast<int64_t>(pool->num_pages) * pool->page_size;
  a.layer_base = static_cast<const uint8_t*>(pool->data) + layer * a.layer_rows * store_row(pool->format);
  a.slots = slots;
  a.status = static_cast<int*>(workspace);
  a.n = n;
  a.out = static_cast<uint8_t*>(rows);
  a.out_rows = n;
  a.kv_scale = 1.f;
  int dtype = MLA_DTYPE_BF16;
  if (into) {
    dtype = into->dtype;
    a.out_rows = static_cast<int64_t>(into->num_pages) * into->page_size;
    a.out = static_cast<uint8_t*>(into->data) + into_layer * a.out_rows * mla::kDimRow * (dtype == MLA_DTYPE_BF16 ? 2 : 1);
    a.out_slots = into_slots;
    a.kv_scale = into->kv_scale;
  }
  return done(mla::launch_store_read(a, pool->format, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
