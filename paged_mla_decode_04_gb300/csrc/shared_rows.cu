// Attention of a decode over shared prefixes: a warp a row, one position after the other.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "shared_internal.h"

namespace mla {
namespace {

constexpr int kWarps = 8;

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps) shared_rows_kernel(const ShDecodeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  ShHeader* hd = reinterpret_cast<ShHeader*>(a.ws);
  const int lane = threadIdx.x & 31, row = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (!sh_planned(hd, a)) {
    if (threadIdx.x == 0) atomicOr(&hd->status, MLA_STATUS_PLAN_MISMATCH);
    return;
  }
  if (static_cast<int>(blockIdx.x) >= hd->num_clusters) return;
  const int* start = reinterpret_cast<const int*>(a.ws + a.lay.cluster_start);
  const ShItem* items = reinterpret_cast<const ShItem*>(a.ws + a.lay.items);
  for (int k = start[blockIdx.x]; k < start[blockIdx.x + 1]; ++k) {
    const ShItem it = items[k];
    if (row >= it.rows) continue;
    const int64_t out_row = static_cast<int64_t>(it.row0) + row;
    const int i = static_cast<int>(out_row / a.num_heads) % a.q_len;
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q) + out_row * kDimRow;
    float q[18], o[16] = {};
    for (int d = 0; d < 18; ++d) q[d] = __bfloat162float(qp[lane + 32 * d]);
    float m = -1e30f, l = 0.f;
    for (int s = it.seg; s <= it.seg_last; ++s) {
      const ShSegment sg = reinterpret_cast<const ShSegment*>(a.ws + a.lay.segs)[s];
      if (row < sg.row_lo || row >= sg.row_hi) continue;
      const int lo = max(sg.tok_lo, sg.tok0 + max(it.begin - sg.block0, 0) * kShTokens);
      const int64_t till = sg.tok0 + static_cast<int64_t>(it.end - sg.block0) * kShTokens;
      const int hi = static_cast<int>(min(till, static_cast<int64_t>(min(sg.tok_hi, sg.base + i + 1))));
      const int pages = a.page_indptr ? a.page_indptr[sg.owner + 1] - a.page_indptr[sg.owner] : a.max_blocks;
      const int32_t* ids = a.page_indptr ? a.page_ids + a.page_indptr[sg.owner]
                                         : a.page_ids + static_cast<int64_t>(sg.owner) * a.max_blocks;
      for (int t = lo; t < hi; ++t) {
        const int j = t / a.page_size;
        const int id = j < pages ? ids[j] : -1;
        float x[18] = {};
        if (id < 0 || id >= a.num_pages) {
          if (lane == 0) atomicOr(&hd->status, MLA_STATUS_BAD_PAGE);
        } else {
          const int64_t at = ((static_cast<int64_t>(a.layer) * a.num_pages + id) * a.page_size + t % a.page_size) * kDimRow;
          for (int d = 0; d < 18; ++d) {
            if (kFp8) x[d] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(a.pool)[at + lane + 32 * d]);
            else x[d] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.pool)[at + lane + 32 * d]);
          }
        }
        float dot = 0.f;
        for (int d = 0; d < 18; ++d) dot = fmaf(q[d], x[d], dot);
        for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        const float sc = dot * a.scale_log2;
        const float mn = fmaxf(m, sc), f = exp2f(m - mn), p = exp2f(sc - mn);
        m = mn;
        l = fmaf(l, f, p);
        for (int d = 0; d < 16; ++d) o[d] = fmaf(p, x[d], o[d] * f);
      }
    }
    if (it.part >= 0) {
      const int64_t at = static_cast<int64_t>(it.part) * kShRows + row;
      if (lane == 0) reinterpret_cast<float2*>(a.ws + a.lay.stats)[at] = make_float2(m, l);
      float* dst = reinterpret_cast<float*>(a.ws + a.lay.partial) + at * kDimCkv;
      for (int d = 0; d < 16; ++d) dst[lane + 32 * d] = o[d];
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + out_row * kDimCkv;
      for (int d = 0; d < 16; ++d) dst[lane + 32 * d] = __float2bfloat16_rn(o[d] * (a.out_scale / l));
      if (a.lse && lane == 0) a.lse[out_row] = (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

}  // namespace

cudaError_t launch_shared_rows(const ShDecodeArgs& a, cudaStream_t stream) {
  const dim3 grid(a.clusters, kShRows / kWarps);
  if (a.dtype == MLA_DTYPE_FP8_E4M3) return launch_pdl(shared_rows_kernel<true>, grid, dim3(32 * kWarps), 0, stream, a);
  return launch_pdl(shared_rows_kernel<false>, grid, dim3(32 * kWarps), 0, stream, a);
}

}  // namespace mla
