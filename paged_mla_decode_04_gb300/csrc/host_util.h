// Host helpers that the entry points share: the tensor-map encoder and the
// checks of pointers and pools.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mla_decode.h"

namespace mla {

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// 2-D row-major map: rows x cols elements, row pitch `pitch_bytes`, box
// {box_cols, box_rows}, zero fill out of bounds.
inline bool make_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t rows, uint64_t cols,
                 uint64_t pitch_bytes, uint32_t box_cols, uint32_t box_rows,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {pitch_bytes};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool valid_pool(const mla_kv_pool* pool) {
  if (!pool || !pool->data || pool->num_layers <= 0 || pool->num_pages <= 0) return false;
  if (pool->page_size != 16 && pool->page_size != 32 && pool->page_size != 64 && pool->page_size != 128)
    return false;
  if (pool->dtype != MLA_DTYPE_BF16 && pool->dtype != MLA_DTYPE_FP8_E4M3) return false;
  if (pool->dtype == MLA_DTYPE_FP8_E4M3 && !(pool->kv_scale > 0.f)) return false;
  return aligned(pool->data, 16);
}

}  // namespace mla
