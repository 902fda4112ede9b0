// First half of the chunk attention's preparation: which query tiles there
// are, and the cache rows that they attend, gathered from their pages.
//
// plan: one block. Request b has n = q_indptr[b + 1] - q_indptr[b] new tokens
// at positions L .. L + n - 1; its rows attend positions [lo, L + n) with
// lo = max(0, L + 1 - window), the first row's start. Those rows are packed
// request after request into a buffer, every request starting at a multiple of
// 16 rows and followed by zero rows up to the next, so that the last 16-row
// step of a P V product reads only this request's rows and zeros.
//
// gather: a warp per row copies (bf16) or widens (e4m3 codes, exact in bf16;
// kv_scale multiplies the scores and the output) the 576 values. A row whose
// c_kv holds an infinity or NaN would poison, as 0 * inf, rows that do not
// attend it once it is multiplied by their zero weights. It is stored with
// c_kv = 0 and a NaN rope part: its scores are then NaN for the rows that do
// attend it, which makes their output NaN as it should be, and masked for the
// others.
#include <cuda_bf16.h>

#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kRowVecs = kDimRow * 2 / 16;  // 72

__device__ __forceinline__ int64_t block_exclusive(int64_t x, int64_t* sh, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t x0 = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += u;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
    const int64_t u = sh[w];
    if (w < warp) before += u;
    all += u;
  }
  __syncthreads();
  *total = all;
  return x + before - x0;
}

__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const PrefillArgs a) {
  __shared__ int64_t sh[32];
  pdl_launch_dependents();
  pdl_wait();
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  PfRequest* reqs = reinterpret_cast<PfRequest*>(a.ws + a.lay.requests);
  PfTile* tiles = reinterpret_cast<PfTile*>(a.ws + a.lay.tiles);
  int64_t rows_before = 0, tiles_before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int64_t len = 0, n = 0, q0 = 0, lo = 0;
    bool ok = true;
    if (b < a.batch) {
      len = a.context_lens[b];
      q0 = a.q_indptr[b];
      n = a.q_indptr[b + 1] - q0;
      // Row pointers outside q leave nothing that could be written.
      if (q0 < 0 || n < 0 || q0 + n > a.q_rows) {
        n = 0;
        ok = false;
      }
      const int64_t nb = a.page_indptr ? a.page_indptr[b + 1] - a.page_indptr[b] : a.max_blocks;
      if (len < 0 || len + n > nb * a.page_size || len + n > INT32_MAX) ok = ok && n == 0;
      lo = a.window > 0 ? max(static_cast<int64_t>(0), len + 1 - a.window) : 0;
    }
    const int64_t want = ok && n > 0 ? len + n - lo : 0;
    const int64_t span = (want + kPfKvAlign - 1) / kPfKvAlign * kPfKvAlign;
    int64_t round_rows, round_tiles;
    const int64_t base = rows_before + block_exclusive(span, sh, &round_rows);
    bool fits = base + span <= a.lay.kv_capacity;
    const int64_t nt = (n + kPfRows - 1) / kPfRows;
    const int64_t tile0 = tiles_before + block_exclusive(nt, sh, &round_tiles);
    if (b < a.batch) {
      const bool good = ok && fits;
      if (!good) atomicOr(&hd->status, MLA_STATUS_BAD_LENGTH);
      PfRequest r;
      r.base = static_cast<int>(min(base, a.lay.kv_capacity));
      r.rows = good ? static_cast<int>(want) : 0;
      r.lo = static_cast<int>(lo);
      r.pad = 0;
      reqs[b] = r;
      for (int64_t k = 0; k < nt && tile0 + k < a.lay.max_tiles; ++k) {
        PfTile t;
        const int64_t i0 = k * kPfRows;
        t.q_row = static_cast<int>(q0 + i0);
        t.rows = static_cast<int>(min(n - i0, static_cast<int64_t>(kPfRows)));
        t.base = r.base;
        t.first_end = good ? static_cast<int>(len + i0 + 1 - lo) : 0;
        t.kv_end = good ? t.first_end + t.rows - 1 : 0;
        t.kv_begin = good && a.window > 0 ? max(0, t.first_end - a.window) / kPfKvAlign * kPfKvAlign : 0;
        t.refused = good ? 0 : 1;
        t.pad = 0;
        tiles[tile0 + k] = t;
      }
    }
    rows_before += round_rows;
    tiles_before += round_tiles;
  }
  // Tiles by falling cost (key steps, in 256 classes of the most expensive
  // one's): blocks draw them in this order, so that what is drawn last is
  // short. The order within a class varies from call to call and changes nothing
  // but who computes a tile.
  __shared__ int most, bins[256];
  const int nt = static_cast<int>(min(tiles_before, a.lay.max_tiles));
  int* order = reinterpret_cast<int*>(a.ws + a.lay.order);
  if (threadIdx.x < 256) bins[threadIdx.x] = 0;
  if (threadIdx.x == 0) most = 1;
  __syncthreads();  // (also: tiles are written)
  auto cost = [&](int i) { return pf_steps(tiles[i].kv_begin, tiles[i].kv_end); };
  for (int i = threadIdx.x; i < nt; i += kPlanThreads) atomicMax(&most, cost(i));
  __syncthreads();
  auto bin = [&](int i) { return 255 - static_cast<int>(static_cast<int64_t>(cost(i)) * 255 / most); };
  for (int i = threadIdx.x; i < nt; i += kPlanThreads) atomicAdd(&bins[bin(i)], 1);
  __syncthreads();
  int64_t first = threadIdx.x < 256 ? bins[threadIdx.x] : 0, ignored;
  first = block_exclusive(first, sh, &ignored);
  if (threadIdx.x < 256) bins[threadIdx.x] = static_cast<int>(first);
  __syncthreads();
  for (int i = threadIdx.x; i < nt; i += kPlanThreads) order[atomicAdd(&bins[bin(i)], 1)] = i;
  if (threadIdx.x == 0) {
    const int64_t used = min(rows_before, a.lay.kv_capacity);
    reqs[a.batch] = {static_cast<int>(used), 0, 0, 0};
    hd->kv_rows = static_cast<int>(used);
    hd->num_tiles = nt;
    if (tiles_before > a.lay.max_tiles) atomicOr(&hd->status, MLA_STATUS_BAD_LENGTH);
  }
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

__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool has_nonfinite(const uint4& v) {
  return has_nonfinite(v.x) || has_nonfinite(v.y) || has_nonfinite(v.z) || has_nonfinite(v.w);
}

constexpr int kGatherWarps = 8;

// A block takes runs of kPfKvAlign rows (all of one request), two a warp.
template <int kDtype>
__global__ void __launch_bounds__(32 * kGatherWarps) prefill_gather_kernel(const PrefillArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  PfHeader* hd = reinterpret_cast<PfHeader*>(a.ws);
  const PfRequest* reqs = reinterpret_cast<const PfRequest*>(a.ws + a.lay.requests);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int used = hd->kv_rows;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int64_t run = blockIdx.x; run * kPfKvAlign < used; run += gridDim.x) {
    const int row0 = static_cast<int>(run) * kPfKvAlign;
    int lo = 0, hi = a.batch;  // the last request with base <= row0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (reqs[mid].base <= row0) lo = mid;
      else hi = mid;
    }
    const PfRequest r = reqs[lo];
    const int nb = a.page_indptr ? a.page_indptr[lo + 1] - a.page_indptr[lo] : a.max_blocks;
    const int32_t* ids = a.page_indptr ? a.page_ids + a.page_indptr[lo] : a.page_ids + static_cast<int64_t>(lo) * a.max_blocks;
#pragma unroll
    for (int k = 0; k < kPfKvAlign / kGatherWarps; ++k) {
      const int row = row0 + warp + k * kGatherWarps;
      const int rel = row - r.base;
      uint4 v[3] = {zero, zero, zero};
      if (rel < r.rows) {
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
          if (__any_sync(0xffffffffu, has_nonfinite(v[0]) || has_nonfinite(v[1]))) {
            v[0] = v[1] = zero;
            v[2] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
          }
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(a.ws + a.lay.rows) + static_cast<int64_t>(row) * kRowVecs;
      dst[lane] = v[0];
      dst[lane + 32] = v[1];
      if (lane < 8) dst[lane + 64] = v[2];
    }
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

cudaError_t launch_prefill_plan(const PrefillArgs& a, cudaStream_t stream) {
  return launch_pdl(prefill_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
}

cudaError_t launch_prefill_gather(const PrefillArgs& a, cudaStream_t stream) {
  const int64_t runs = a.lay.kv_capacity / kPfKvAlign;
  const dim3 grid(static_cast<unsigned>(runs < 152 * 8 ? runs : 152 * 8)), block(32 * kGatherWarps);
  if (a.dtype == MLA_DTYPE_BF16)
    return launch_pdl(prefill_gather_kernel<MLA_DTYPE_BF16>, grid, block, 0, stream, a);
  return launch_pdl(prefill_gather_kernel<MLA_DTYPE_FP8_E4M3>, grid, block, 0, stream, a);
}

}  // namespace mla
