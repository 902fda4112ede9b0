// Page tables of one step, built on the device from request lengths.
//
// Request b holds L tokens in the first held = ceil(L / ps) blocks of its
// block table row and gets n new ones, for which it needs
// need = ceil((L + n) / ps) - held pages. With base = the needs of the
// requests before it, its k-th new page is free_pages[count - 1 - base - k]:
// the pages come off the top of the stack in the order of requests. A
// request whose base + need exceeds the stack is refused whole; since the
// sums only grow, the served needs are those of a prefix, and the stack loses
// the largest sum that fits. Token i of a request has position L + i and slot
// table[b][pos / ps] * ps + pos % ps.
//
// The sums are one block's work (a scan over the batch, 1024 requests at a
// time, in 64 bits: no sum of int32 lengths overflows); slots, positions and
// the CSR list are independent per entry once the row pointers stand. Small
// steps do both in that one block: a launch less. Larger ones spread the
// entries over the GPU in a second, dependent launch.
#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kFillThreads = 256;
constexpr int kIdsPerThread = 4;
// Entries (tokens and CSR ids) up to which one block does the whole step.
constexpr int kOneBlockEntries = 4096;

__device__ __forceinline__ int64_t ceil_div(int64_t x, int d) { return (x + d - 1) / d; }

struct Lens {
  int64_t len, add;  // cached and new tokens (new: at least 0)
  int64_t held;      // blocks of the cached tokens, 0 where the length is bad
  int64_t need;      // further pages, 0 where the lengths are bad
  bool ok;
};

__device__ __forceinline__ Lens lens_of(const TablesArgs& a, int b) {
  Lens r;
  r.len = a.context_lens[b];
  const int n = a.new_lens[b];
  r.add = max(n, 0);
  const int64_t room = static_cast<int64_t>(a.max_blocks) * a.page_size;
  const bool len_ok = r.len >= 0 && r.len <= room;
  r.ok = len_ok && n >= 0 && r.len + r.add <= room;
  r.held = len_ok ? ceil_div(r.len, a.page_size) : 0;
  r.need = r.ok ? ceil_div(r.len + r.add, a.page_size) - r.held : 0;
  return r;
}

__device__ __forceinline__ void flag(int* status, int bits) {
  if (status) atomicOr(status, bits);
}

// Exclusive prefix sums over the block of two 64-bit values; *sa and *sb
// receive the block's totals. `sh`: 64 values of shared memory.
__device__ __forceinline__ void block_scan2(int64_t& x, int64_t& y, int64_t* sh, int64_t* sa, int64_t* sb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t x0 = x, y0 = y;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    sh[warp] = x;
    sh[32 + warp] = y;
  }
  __syncthreads();
  int64_t px = 0, py = 0, tx = 0, ty = 0;
  for (int w = 0; w < warps; ++w) {
    const int64_t u = sh[w], v = sh[32 + w];
    if (w < warp) {
      px += u;
      py += v;
    }
    tx += u;
    ty += v;
  }
  __syncthreads();
  x += px - x0;
  y += py - y0;
  *sa = tx;
  *sb = ty;
}

// The last b in [lo, hi) with indptr[b] <= t (indptr[lo] <= t).
__device__ __forceinline__ int owner_of(const int32_t* indptr, int lo, int hi, int t) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (indptr[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void fill_token(const TablesArgs& a, int t, int total, int lo, int hi, int first_refused) {
  int64_t slot = -1;
  int pos = -1;
  if (t < total) {
    const int b = owner_of(a.q_indptr, lo, hi, t);
    const Lens r = lens_of(a, b);
    if (r.ok && (r.need == 0 || b < first_refused)) {
      const int p = static_cast<int>(r.len) + (t - a.q_indptr[b]);
      const int j = p / a.page_size;
      const int id = a.block_table[static_cast<int64_t>(b) * a.max_blocks + j];
      if (id >= 0 && id < a.num_pages) {
        pos = p;
        slot = static_cast<int64_t>(id) * a.page_size + p % a.page_size;
      } else {
        flag(a.status, MLA_STATUS_BAD_PAGE);
      }
    }
  }
  a.slot_mapping[t] = slot;
  if (a.positions) a.positions[t] = pos;
}

// Entries k .. k + kIdsPerThread - 1 of the CSR list.
__device__ __forceinline__ void fill_ids(const TablesArgs& a, int64_t k0, int total, int lo, int hi) {
  if (k0 >= total) return;
  int b = owner_of(a.page_indptr, lo, hi, static_cast<int>(k0));
  int begin = a.page_indptr[b], end = a.page_indptr[b + 1];
#pragma unroll
  for (int i = 0; i < kIdsPerThread; ++i) {
    const int64_t k = k0 + i;
    if (k >= total || k >= a.max_page_ids) return;
    while (k >= end) {  // empty requests in between
      ++b;
      begin = end;
      end = a.page_indptr[b + 1];
    }
    a.page_ids[k] = a.block_table[static_cast<int64_t>(b) * a.max_blocks + (k - begin)];
  }
}

// Row pointers, new pages and the stack's state; with kFill also every entry.
template <bool kFill>
__global__ void __launch_bounds__(1024) tables_scan_kernel(const TablesArgs a) {
  __shared__ int64_t sh[64];
  __shared__ unsigned long long sh_taken;
  __shared__ int sh_refused;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t count = min(max(*a.free_count, 0), a.free_capacity);
  if (tid == 0) {
    sh_taken = 0;
    sh_refused = a.batch;
    a.q_indptr[0] = 0;
    if (a.page_indptr) a.page_indptr[0] = 0;
  }
  __syncthreads();
  int64_t tokens = 0, needs = 0, blocks = 0;  // sums over the requests before this round
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + tid;
    Lens r = {0, 0, 0, 0, true};
    if (b < a.batch) {
      r = lens_of(a, b);
      if (!r.ok) flag(a.status, MLA_STATUS_BAD_LENGTH);
    }
    int64_t tok = r.add, need = r.need, round_tok, round_need;
    block_scan2(tok, need, sh, &round_tok, &round_need);
    const int64_t base = needs + need;  // pages that earlier requests ask for
    const bool served = r.ok && (r.need == 0 || base + r.need <= count);
    if (served && r.need) atomicMax(&sh_taken, static_cast<unsigned long long>(base + r.need));
    if (r.ok && !served) atomicMin(&sh_refused, b);
    if (b < a.batch) {
      const int64_t end = tokens + tok + r.add;
      a.q_indptr[b + 1] = static_cast<int>(min(end, static_cast<int64_t>(INT32_MAX)));
    }
    // New pages: a lane's own few, then the warp together for each lane with many.
    const int need_now = served ? static_cast<int>(r.need) : 0;
    auto page = [&](int64_t at) {
      int id = a.free_pages[at];
      if (id < 0 || id >= a.num_pages) {
        flag(a.status, MLA_STATUS_BAD_PAGE);
        id = -1;
      }
      return id;
    };
    if (need_now > 0 && need_now <= 4) {
      int32_t* row = a.block_table + static_cast<int64_t>(b) * a.max_blocks + r.held;
      for (int k = 0; k < need_now; ++k) row[k] = page(count - 1 - base - k);
    }
    unsigned many = __ballot_sync(0xffffffffu, need_now > 4);
    while (many) {
      const int src = __ffs(many) - 1;
      many &= many - 1;
      const int bb = __shfl_sync(0xffffffffu, b, src), nn = __shfl_sync(0xffffffffu, need_now, src);
      const int64_t base_s = __shfl_sync(0xffffffffu, base, src), held_s = __shfl_sync(0xffffffffu, r.held, src);
      int32_t* row = a.block_table + static_cast<int64_t>(bb) * a.max_blocks + held_s;
      for (int k = lane; k < nn; k += 32) row[k] = page(count - 1 - base_s - k);
    }
    if (a.page_indptr) {
      int64_t list = b < a.batch ? r.held + (served ? r.need : 0) : 0, zero = 0, round_list, ignored;
      const int64_t mine = list;
      block_scan2(list, zero, sh, &round_list, &ignored);
      if (b < a.batch)
        a.page_indptr[b + 1] = static_cast<int>(min(blocks + list + mine, static_cast<int64_t>(INT32_MAX)));
      blocks += round_list;
    }
    tokens += round_tok;
    needs += round_need;
  }
  __syncthreads();
  if (tid == 0) {
    a.state[0] = static_cast<int>(count - static_cast<int64_t>(sh_taken));
    a.state[1] = sh_refused;
    int bits = 0;
    if (sh_refused < a.batch) bits |= MLA_STATUS_NO_PAGES;
    if (tokens > a.max_tokens || (a.page_indptr && blocks > a.max_page_ids)) bits |= MLA_STATUS_BAD_LENGTH;
    if (bits) flag(a.status, bits);
  }
  if (kFill) {
    const int total = static_cast<int>(min(tokens, static_cast<int64_t>(INT32_MAX)));
    const int refused = sh_refused;
    for (int t = tid; t < a.max_tokens; t += blockDim.x) fill_token(a, t, total, 0, a.batch, refused);
    if (a.page_indptr) {
      const int ids = static_cast<int>(min(blocks, static_cast<int64_t>(a.max_page_ids)));
      for (int k = tid * kIdsPerThread; k < ids; k += blockDim.x * kIdsPerThread) fill_ids(a, k, ids, 0, a.batch);
    }
  }
}

// Entries of a large step: blocks [0, token_blocks) take kFillThreads tokens
// each, the others kFillThreads * kIdsPerThread CSR ids each. A block narrows
// the requests of its entries down first, so that a thread searches few.
__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const TablesArgs a, int token_blocks) {
  __shared__ int range[2];
  pdl_launch_dependents();
  pdl_wait();
  const bool is_token = static_cast<int>(blockIdx.x) < token_blocks;
  const int32_t* indptr = is_token ? a.q_indptr : a.page_indptr;
  const int total = is_token ? indptr[a.batch] : min(indptr[a.batch], a.max_page_ids);
  const int span = is_token ? kFillThreads : kFillThreads * kIdsPerThread;
  const int64_t first = static_cast<int64_t>(is_token ? blockIdx.x : blockIdx.x - token_blocks) * span;
  if (threadIdx.x < 2 && first < total) {
    const int64_t edge = threadIdx.x == 0 ? first : min(first + span, static_cast<int64_t>(total)) - 1;
    range[threadIdx.x] = owner_of(indptr, 0, a.batch, static_cast<int>(edge));
  }
  __syncthreads();
  const int lo = range[0], hi = range[1] + 1;
  if (is_token) {
    const int64_t t = first + threadIdx.x;
    if (t < a.max_tokens) fill_token(a, static_cast<int>(t), total, lo, hi, a.state[1]);
  } else {
    fill_ids(a, first + threadIdx.x * kIdsPerThread, total, lo, hi);
  }
}

}  // namespace

cudaError_t launch_extend_tables(const TablesArgs& a, cudaStream_t stream) {
  const int64_t ids = a.page_indptr ? a.max_page_ids : 0;
  int threads = 128;
  if (a.max_tokens + ids <= kOneBlockEntries) {
    while (threads < 1024 && (threads < a.batch || threads < a.max_tokens + ids / kIdsPerThread)) threads *= 2;
    return launch_pdl(tables_scan_kernel<true>, dim3(1), dim3(threads), 0, stream, a);
  }
  while (threads < 1024 && threads < a.batch) threads *= 2;
  const cudaError_t e = launch_pdl(tables_scan_kernel<false>, dim3(1), dim3(threads), 0, stream, a);
  if (e != cudaSuccess) return e;
  const int token_blocks = (a.max_tokens + kFillThreads - 1) / kFillThreads;
  const int id_span = kFillThreads * kIdsPerThread;
  const int64_t id_blocks = (ids + id_span - 1) / id_span;
  return launch_pdl(tables_fill_kernel, dim3(static_cast<unsigned>(token_blocks + id_blocks)), dim3(kFillThreads), 0,
                    stream, a, token_blocks);
}

}  // namespace mla
