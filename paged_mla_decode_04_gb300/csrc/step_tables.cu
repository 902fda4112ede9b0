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
// With the sums at hand every entry is independent: a page id comes from the
// table (blocks held) or straight from the stack (new blocks), whoever writes
// the new one into the table. So one launch does a step: each block makes the
// sums of the whole batch for itself, in shared memory, and fills its share of
// tokens, CSR ids and new pages. (Latency is what a small step costs; a launch
// more would be 3 us.) Where that does not work - more requests than fit in
// shared memory, or a large step whose state lies on free_count, which blocks
// still read while one would write it - a single block makes the sums and hands
// out the pages, and a second launch fills the entries from what it wrote.
// Sums are 64-bit: none of int32 lengths overflows.
//
// Bound by latency: lengths, scan, search, table entry and store wait for one another.
// 128 requests with a token each take 5.2 us a call (6.5 alone), 1,024 requests with
// 1.05 million listed pages 10.0 us, of which their 10.5 MB need 1.6.
#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "scan.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kFillThreads = 256;
constexpr int kIdsPerThread = 4;
constexpr int kStepThreads = 512;
constexpr int kStepBatch = 3840;    // requests whose sums fit in 48 KB (12 bytes each)
constexpr int kStepBlocks = 152 * 2;
constexpr int kWarpIds = 256;       // CSR ids a warp moves at a time

// Blocks of x tokens (page sizes are powers of two; a 64-bit division costs a hundred instructions).
__device__ __forceinline__ int64_t blocks_of(const TablesArgs& a, int64_t x) { return (x + a.page_size - 1) >> a.page_shift; }

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
  const int64_t room = static_cast<int64_t>(a.max_blocks) << a.page_shift;
  const bool len_ok = r.len >= 0 && r.len <= room;
  r.ok = len_ok && n >= 0 && r.len + r.add <= room;
  r.held = len_ok ? blocks_of(a, r.len) : 0;
  r.need = r.ok ? blocks_of(a, r.len + r.add) - r.held : 0;
  return r;
}

__device__ __forceinline__ void flag(int* status, int bits) {
  if (status) atomicOr(status, bits);
}

__device__ __forceinline__ int clip(int64_t x) { return static_cast<int>(min(x, static_cast<int64_t>(INT32_MAX))); }

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
      const int j = p >> a.page_shift;
      const int id = a.block_table[static_cast<int64_t>(b) * a.max_blocks + j];
      if (id >= 0 && id < a.num_pages) {
        pos = p;
        slot = (static_cast<int64_t>(id) << a.page_shift) + (p & (a.page_size - 1));
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

// A whole step (see above). Shared memory: where each request's tokens, listed
// pages and page demands start.
__global__ void __launch_bounds__(kStepThreads) tables_step_kernel(const TablesArgs a) {
  extern __shared__ int starts[];
  __shared__ int64_t sh[96];
  __shared__ unsigned long long sh_taken;
  __shared__ int sh_refused;
  int *tok0 = starts, *list0 = starts + a.batch + 1, *need0 = starts + 2 * (a.batch + 1);
  // (No early launch of what follows: its waiting blocks would share the SMs with
  // this grid's; the CSR list of a million pages took 14 us a call with it, 11 without.)
  pdl_wait();
  const int tid = threadIdx.x;
  const bool lead = blockIdx.x == 0;
  const int64_t count = min(max(*a.free_count, 0), a.free_capacity);
  if (tid == 0) {
    sh_taken = 0;
    sh_refused = a.batch;
  }
  int64_t sum[3] = {0, 0, 0};  // tokens, pages held, pages asked for by earlier requests
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + tid;
    Lens r = {0, 0, 0, 0, true};
    if (b < a.batch) {
      r = lens_of(a, b);
      if (!r.ok && lead) flag(a.status, MLA_STATUS_BAD_LENGTH);
    }
    int64_t v[3] = {r.add, r.held, r.need}, total[3];
    block_scan(v, total, sh);  // (its barriers also order the initialisation above)
    const int64_t upto = sum[2] + v[2] + r.need;
    if (r.need > 0 && upto <= count) atomicMax(&sh_taken, static_cast<unsigned long long>(upto));
    if (r.need > 0 && upto > count) atomicMin(&sh_refused, b);
    if (b < a.batch) {
      tok0[b] = clip(sum[0] + v[0]);
      list0[b] = clip(sum[1] + v[1]);  // (blocks held so far; new ones added below)
      need0[b] = clip(sum[2] + v[2]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) sum[i] += total[i];
  }
  __syncthreads();
  const int64_t taken = static_cast<int64_t>(sh_taken);
  const int refused = sh_refused;
  // Pages handed out to the requests before b: all they asked for, until the
  // stack ran out.
  for (int b = tid; b <= a.batch; b += blockDim.x) {
    if (b == a.batch) {
      tok0[b] = clip(sum[0]);
      list0[b] = clip(sum[1] + taken);
      need0[b] = clip(taken);
    } else {
      const int64_t got = need0[b] <= count ? min(static_cast<int64_t>(need0[b]), taken) : taken;
      list0[b] = clip(list0[b] + got);
      need0[b] = static_cast<int>(got);
    }
  }
  __syncthreads();
  if (lead) {
    for (int b = tid; b <= a.batch; b += blockDim.x) {
      a.q_indptr[b] = tok0[b];
      if (a.page_indptr) a.page_indptr[b] = list0[b];
    }
    if (tid == 0) {
      a.state[0] = static_cast<int>(count - taken);
      a.state[1] = refused;
      int bits = refused < a.batch ? MLA_STATUS_NO_PAGES : 0;
      if (sum[0] > a.max_tokens || (a.page_indptr && sum[1] + taken > a.max_page_ids)) bits |= MLA_STATUS_BAD_LENGTH;
      if (bits) flag(a.status, bits);
    }
  }
  // The id of block j of request b: of the listed blocks the last ones, as many
  // as the request got, come off the stack.
  auto page_of = [&](int b, int j) -> int {
    const int fresh = j - ((list0[b + 1] - list0[b]) - (need0[b + 1] - need0[b]));
    if (fresh < 0) return a.block_table[static_cast<int64_t>(b) * a.max_blocks + j];
    const int id = a.free_pages[count - 1 - need0[b] - fresh];
    return id >= 0 && id < a.num_pages ? id : -1;
  };
  const int first = blockIdx.x * blockDim.x + tid, step = gridDim.x * blockDim.x;
  const int tokens = tok0[a.batch];
  for (int64_t t = first; t < a.max_tokens; t += step) {
    int64_t slot = -1;
    int pos = -1;
    if (t < tokens) {
      const int b = owner_of(tok0, 0, a.batch, static_cast<int>(t));
      const Lens r = lens_of(a, b);
      if (r.ok && (r.need == 0 || b < refused)) {
        const int p = static_cast<int>(r.len) + (static_cast<int>(t) - tok0[b]);
        const int id = page_of(b, p >> a.page_shift);
        if (id >= 0 && id < a.num_pages) {
          pos = p;
          slot = (static_cast<int64_t>(id) << a.page_shift) + (p & (a.page_size - 1));
        } else {
          flag(a.status, MLA_STATUS_BAD_PAGE);
        }
      }
    }
    a.slot_mapping[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
  for (int64_t k = first; k < taken; k += step) {  // new pages into the table
    const int b = owner_of(need0, 0, a.batch, static_cast<int>(k));
    const int j = list0[b + 1] - list0[b] - (need0[b + 1] - need0[b]) + static_cast<int>(k - need0[b]);
    const int id = page_of(b, j);
    if (id < 0) flag(a.status, MLA_STATUS_BAD_PAGE);
    a.block_table[static_cast<int64_t>(b) * a.max_blocks + j] = id;
  }
  if (a.page_indptr) {
    // A warp takes kWarpIds consecutive ids, lane by lane next to each other: one
    // search for the first, steps to the following requests from there.
    const int ids = min(list0[a.batch], a.max_page_ids), lane = tid & 31;
    for (int64_t tile = (first >> 5) * static_cast<int64_t>(kWarpIds); tile < ids; tile += (step >> 5) * static_cast<int64_t>(kWarpIds)) {
      int b = owner_of(list0, 0, a.batch, static_cast<int>(tile));
      int id[kWarpIds / 32];
#pragma unroll
      for (int i = 0; i < kWarpIds / 32; ++i) {
        const int64_t k = tile + 32 * i + lane;
        if (k < ids) {
          while (k >= list0[b + 1]) ++b;
          id[i] = page_of(b, static_cast<int>(k) - list0[b]);
        }
      }
#pragma unroll
      for (int i = 0; i < kWarpIds / 32; ++i) {
        const int64_t k = tile + 32 * i + lane;
        if (k < ids) a.page_ids[k] = id[i];
      }
    }
  }
}

// Sums of a batch of any size by one block: row pointers, new pages, state.
__global__ void __launch_bounds__(1024) tables_scan_kernel(const TablesArgs a) {
  __shared__ int64_t sh[96];
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
  int64_t sum[3] = {0, 0, 0};  // tokens, listed pages, pages asked for by earlier requests
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + tid;
    Lens r = {0, 0, 0, 0, true};
    if (b < a.batch) {
      r = lens_of(a, b);
      if (!r.ok) flag(a.status, MLA_STATUS_BAD_LENGTH);
    }
    int64_t need[1] = {r.need}, round_need[1];
    block_scan(need, round_need, sh);  // (its barriers also order the initialisation above)
    const int64_t base = sum[2] + need[0];
    const bool served = r.ok && (r.need == 0 || base + r.need <= count);
    if (served && r.need) atomicMax(&sh_taken, static_cast<unsigned long long>(base + r.need));
    if (r.ok && !served) atomicMin(&sh_refused, b);
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
    const int64_t list = r.held + need_now;
    int64_t v[2] = {r.add, list}, total[2];
    block_scan(v, total, sh);
    if (b < a.batch) {
      a.q_indptr[b + 1] = clip(sum[0] + v[0] + r.add);
      if (a.page_indptr) a.page_indptr[b + 1] = clip(sum[1] + v[1] + list);
    }
    sum[0] += total[0];
    sum[1] += total[1];
    sum[2] += round_need[0];
  }
  __syncthreads();
  if (tid == 0) {
    a.state[0] = static_cast<int>(count - static_cast<int64_t>(sh_taken));
    a.state[1] = sh_refused;
    int bits = 0;
    if (sh_refused < a.batch) bits |= MLA_STATUS_NO_PAGES;
    if (sum[0] > a.max_tokens || (a.page_indptr && sum[1] > a.max_page_ids)) bits |= MLA_STATUS_BAD_LENGTH;
    if (bits) flag(a.status, bits);
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
  const int64_t work = a.max_tokens + ids * 32 / kWarpIds;
  const int64_t want = (work + kStepThreads - 1) / kStepThreads;
  const int blocks = static_cast<int>(want < 1 ? 1 : want < kStepBlocks ? want : kStepBlocks);
  const bool in_place = a.state == a.free_count || a.state + 1 == a.free_count;
  if (a.batch <= kStepBatch && (blocks == 1 || !in_place)) {
    int threads = kStepThreads;
    if (blocks == 1)  // a small step: no more warps than work
      while (threads > 64 && threads / 2 >= a.batch && threads / 2 >= work) threads /= 2;
    return launch_pdl(tables_step_kernel, dim3(blocks), dim3(threads), 3 * sizeof(int) * (static_cast<size_t>(a.batch) + 1),
                      stream, a);
  }
  const cudaError_t e = launch_pdl(tables_scan_kernel, dim3(1), dim3(1024), 0, stream, a);
  if (e != cudaSuccess) return e;
  const int token_blocks = static_cast<int>((static_cast<int64_t>(a.max_tokens) + kFillThreads - 1) / kFillThreads);
  const int id_span = kFillThreads * kIdsPerThread;
  const int64_t id_blocks = (ids + id_span - 1) / id_span;
  if (token_blocks + id_blocks == 0) return cudaSuccess;
  return launch_pdl(tables_fill_kernel, dim3(static_cast<unsigned>(token_blocks + id_blocks)), dim3(kFillThreads), 0,
                    stream, a, token_blocks);
}

}  // namespace mla
