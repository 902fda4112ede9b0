// Rotary positions of a step's new tokens, with the latent rows' norm and
// their write into the paged pool.
//
// A pair (x, y) of the rope part turns by the angle of its token's position:
// (x cos - y sin, x sin + y cos). The 32 pairs are dims (2j, 2j + 1) or
// (j, j + 32); pair j reads the angle of position axis pair_axis[j] (one axis
// for text, up to four for time, height and width). Latent rows: c_kv is
// scaled to unit root mean square and by the norm weight (when given), the
// rope part turns, and the row is rounded once, to bf16 or to
// e4m3(x / kv_scale); the queries' 64 rope dims of every head turn alike and
// are rounded to bf16. All arithmetic is fp32.
//
// The cost is the bytes: 256 of a (token, head)'s query read and written
// against 6 multiply-adds per pair, so bytes in flight are what counts: eight
// lanes share one row of 64 rope dims, lane i its pairs 4i .. 4i + 3 (16 bytes), and
// keep the token's eight sines and cosines in registers over all heads that the
// warp serves. (With four lanes a row the angles took 16 registers and half the
// warps fitted.) A latent row is one warp's work. Both kinds share a launch:
// blocks [0, row_blocks) write rows. 8,191 tokens of 128 heads with their rows into
// e4m3 (285 MB): 50.5 us, 5.64 TB/s, 84 % of a copy's rate; 16,384 tokens of 16 heads
// with bf16 rows and three axes (109 MB): 24.2 us, 4.5 TB/s, where the angles' table (24
// lookups of 16 bytes a token) and the short run weigh; 128 tokens of 128 heads 3.3 us
// and two of 16 heads 3.0, one round of launch, positions, angles and store.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kPairsPerLane = 4;
constexpr int kRowLanes = kRopePairs / kPairsPerLane;  // 8 lanes share a row
constexpr int kRowVecs = kDimRow * 2 / 16;             // 72
constexpr int kHeadsPerStep = 32 / kRowLanes;
constexpr int kUnroll = 4;                             // rows a lane has in flight

struct Turn {
  float c[kPairsPerLane], s[kPairsPerLane];
};

// Row of the table for each axis, or false for a pad row or a position that
// the table lacks (which sets the status word unless the row is a pad already).
__device__ __forceinline__ bool token_positions(const RopeArgs& a, int t, int (&pos)[kMaxAxes], bool real) {
  bool pad = false, bad = false;
#pragma unroll
  for (int x = 0; x < kMaxAxes; ++x) {
    pos[x] = 0;
    if (x < a.num_axes) {
      pos[x] = a.positions[static_cast<int64_t>(x) * a.n + t];
      pad |= pos[x] < 0;
      bad |= pos[x] >= a.max_position;
    }
  }
  if (bad && !pad && real && a.status) atomicOr(a.status, MLA_STATUS_BAD_POSITION);
  return !pad && !bad;
}

// Sines and cosines of pairs 4 sub .. 4 sub + 3.
__device__ __forceinline__ void load_turn(const RopeArgs& a, const int (&pos)[kMaxAxes], int sub, Turn& r) {
  const uint32_t axes = static_cast<uint32_t>(a.pair_axis >> (2 * kPairsPerLane * sub)) & 0xffu;
  auto row = [&](uint32_t axis) {
    const int p = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
    return a.cos_sin + static_cast<int64_t>(p) * kDimRope + kPairsPerLane * sub;
  };
  if (axes == (axes & 3u) * 0x55u) {  // one axis for all four
    const float4* v = reinterpret_cast<const float4*>(row(axes & 3u));
    const float4 c = __ldg(v), s = __ldg(v + kRopePairs / 4);
    r.c[0] = c.x, r.c[1] = c.y, r.c[2] = c.z, r.c[3] = c.w;
    r.s[0] = s.x, r.s[1] = s.y, r.s[2] = s.z, r.s[3] = s.w;
  } else {
#pragma unroll
    for (int i = 0; i < kPairsPerLane; ++i) {
      const float* v = row((axes >> (2 * i)) & 3u);
      r.c[i] = __ldg(v + i);
      r.s[i] = __ldg(v + kRopePairs + i);
    }
  }
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A lane's four pairs of a row, as 16 bytes: one piece, or (rotated halves) the
// four first and the four second values.
template <bool kInterleaved>
__device__ __forceinline__ uint4 load_pairs(const void* row, int sub) {
  if (kInterleaved) return static_cast<const uint4*>(row)[sub];
  const uint2 x = static_cast<const uint2*>(row)[sub], y = static_cast<const uint2*>(row)[sub + kRowLanes];
  return make_uint4(x.x, x.y, y.x, y.y);
}
template <bool kInterleaved>
__device__ __forceinline__ void store_pairs(void* row, int sub, const uint4& v) {
  if (kInterleaved) {
    static_cast<uint4*>(row)[sub] = v;
  } else {
    static_cast<uint2*>(row)[sub] = make_uint2(v.x, v.y);
    static_cast<uint2*>(row)[sub + kRowLanes] = make_uint2(v.z, v.w);
  }
}

template <bool kInterleaved>
__device__ __forceinline__ void turn_pairs(const uint4& v, const Turn& r, float (&x)[kPairsPerLane],
                                           float (&y)[kPairsPerLane]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < kPairsPerLane; ++i) {
    const float a = kInterleaved ? lo_f(w[i]) : (i & 1 ? hi_f(w[i >> 1]) : lo_f(w[i >> 1]));
    const float b = kInterleaved ? hi_f(w[i]) : (i & 1 ? hi_f(w[2 + (i >> 1)]) : lo_f(w[2 + (i >> 1)]));
    x[i] = a * r.c[i] - b * r.s[i];
    y[i] = a * r.s[i] + b * r.c[i];
  }
}

template <bool kInterleaved>
__device__ __forceinline__ uint4 pack_pairs(const float (&x)[kPairsPerLane], const float (&y)[kPairsPerLane]) {
  return kInterleaved ? make_uint4(pack_bf16x2(x[0], y[0]), pack_bf16x2(x[1], y[1]), pack_bf16x2(x[2], y[2]),
                                   pack_bf16x2(x[3], y[3]))
                      : make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]),
                                   pack_bf16x2(y[2], y[3]));
}

__device__ __forceinline__ uint32_t e4m3(float x, float scale) {
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ uint32_t e4m3x4(float p, float q, float r, float t, float scale) {
  return e4m3(p, scale) | e4m3(q, scale) << 8 | e4m3(r, scale) << 16 | e4m3(t, scale) << 24;
}

// One warp, one latent row.
template <int kDtype, bool kInterleaved>
__device__ __forceinline__ void write_row(const RopeArgs& a, int t, int lane) {
  // The row and its slot and positions are asked for together; only the angles
  // have to wait for an answer.
  const uint4* src = a.rows + static_cast<int64_t>(t) * kRowVecs;
  const int64_t slot = a.slots[t];
  const uint4 c0 = src[lane], c1 = src[lane + 32];
  uint4 rope;
  if (lane < kRowLanes) rope = load_pairs<kInterleaved>(src + 64, lane);
  int pos[kMaxAxes];
  const bool here = token_positions(a, t, pos, slot >= 0);
  if (slot < 0 || !here) return;  // pad row
  if (slot >= a.layer_rows) {
    if (lane == 0 && a.status) atomicOr(a.status, MLA_STATUS_BAD_SLOT);
    return;
  }
  Turn r;
  if (lane < kRowLanes) load_turn(a, pos, lane, r);
  float x[2][8];
  const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i >> 2][2 * (i & 3)] = lo_f(w[i]);
    x[i >> 2][2 * (i & 3) + 1] = hi_f(w[i]);
  }
  if (a.norm_weight) {
    const uint4* wt = static_cast<const uint4*>(a.norm_weight);
    const uint4 w0 = __ldg(wt + lane), w1 = __ldg(wt + lane + 32);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(x[i >> 3][i & 7], x[i >> 3][i & 7], sum);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float inv = rsqrtf(sum * (1.f / kDimCkv) + a.norm_eps);
    const uint32_t g[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i >> 2][2 * (i & 3)] *= inv * lo_f(g[i]);
      x[i >> 2][2 * (i & 3) + 1] *= inv * hi_f(g[i]);
    }
  }
  float rx[kPairsPerLane], ry[kPairsPerLane];
  if (lane < kRowLanes) turn_pairs<kInterleaved>(rope, r, rx, ry);
  if (kDtype == MLA_DTYPE_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(a.layer_base) + slot * kRowVecs;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      dst[lane + 32 * h] = make_uint4(pack_bf16x2(x[h][0], x[h][1]), pack_bf16x2(x[h][2], x[h][3]),
                                      pack_bf16x2(x[h][4], x[h][5]), pack_bf16x2(x[h][6], x[h][7]));
    if (lane < kRowLanes) store_pairs<kInterleaved>(dst + 64, lane, pack_pairs<kInterleaved>(rx, ry));
  } else {
    uint2* dst = reinterpret_cast<uint2*>(a.layer_base + slot * kDimRow);
    const float s = a.kv_scale;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      dst[lane + 32 * h] = make_uint2(e4m3x4(x[h][0], x[h][1], x[h][2], x[h][3], s), e4m3x4(x[h][4], x[h][5], x[h][6], x[h][7], s));
    if (lane < kRowLanes) {
      if (kInterleaved) {
        dst[64 + lane] = make_uint2(e4m3x4(rx[0], ry[0], rx[1], ry[1], s), e4m3x4(rx[2], ry[2], rx[3], ry[3], s));
      } else {
        uint32_t* half = reinterpret_cast<uint32_t*>(dst + 64);
        half[lane] = e4m3x4(rx[0], rx[1], rx[2], rx[3], s);
        half[lane + kRowLanes] = e4m3x4(ry[0], ry[1], ry[2], ry[3], s);
      }
    }
  }
}

// One warp: heads [h0, h1) of one token's query. The first rows are asked for
// together with the token's slot and positions, the next ones before the current
// ones are turned.
template <bool kInterleaved>
__device__ __forceinline__ void turn_query(const RopeArgs& a, int t, int h0, int h1, int lane) {
  const int sub = lane % kRowLanes;
  const int64_t row0 = static_cast<int64_t>(t) * a.num_heads;
  uint4 u[kUnroll];
  auto load = [&](int h, int k) {
    const int hh = h + k * kHeadsPerStep;
    if (hh < h1) u[k] = load_pairs<kInterleaved>(a.q + (row0 + hh) * a.q_pitch, sub);
  };
  int h = h0 + lane / kRowLanes;
  const int64_t slot = a.slots ? a.slots[t] : 0;
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) load(h, k);
  int pos[kMaxAxes];
  const bool here = token_positions(a, t, pos, slot >= 0);
  if (slot < 0 || !here) return;  // pad row
  Turn r;
  load_turn(a, pos, sub, r);
  for (; h < h1; h += kHeadsPerStep * kUnroll) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int hh = h + k * kHeadsPerStep;
      const uint4 v = u[k];
      load(h + kHeadsPerStep * kUnroll, k);
      if (hh < h1) {
        float x[kPairsPerLane], y[kPairsPerLane];
        turn_pairs<kInterleaved>(v, r, x, y);
        store_pairs<kInterleaved>(a.q_out + (row0 + hh) * a.q_out_pitch, sub, pack_pairs<kInterleaved>(x, y));
      }
    }
  }
}

template <int kDtype, bool kInterleaved>
__global__ void __launch_bounds__(32 * kWarps, 4) rope_write_kernel(const RopeArgs a, int row_blocks, int heads_per_warp,
                                                                 int warps_per_token) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    const int t = blockIdx.x * kWarps + warp;
    if (t < a.n) write_row<kDtype, kInterleaved>(a, t, lane);
    return;
  }
  const int64_t w = static_cast<int64_t>(blockIdx.x - row_blocks) * kWarps + warp;
  const int t = static_cast<int>(w / warps_per_token);
  if (t >= a.n) return;
  const int h0 = static_cast<int>(w % warps_per_token) * heads_per_warp;
  turn_query<kInterleaved>(a, t, h0, min(h0 + heads_per_warp, a.num_heads), lane);
}

}  // namespace

cudaError_t launch_rope_write(const RopeArgs& a, int dtype, cudaStream_t stream) {
  const int row_blocks = a.layer_base ? (a.n + kWarps - 1) / kWarps : 0;
  // A warp serves as many heads of a token as leave enough warps to fill the
  // GPU (a token's angles are then loaded once for all of them).
  int heads_per_warp = 0, warps_per_token = 0;
  int64_t q_blocks = 0;
  if (a.q) {
    heads_per_warp = a.num_heads;
    auto per_token = [&] { return (a.num_heads + heads_per_warp - 1) / heads_per_warp; };
    while (heads_per_warp > kHeadsPerStep && static_cast<int64_t>(a.n) * per_token() < 152 * 16)
      heads_per_warp = (heads_per_warp / 2 + kHeadsPerStep - 1) / kHeadsPerStep * kHeadsPerStep;
    warps_per_token = per_token();
    q_blocks = (static_cast<int64_t>(a.n) * warps_per_token + kWarps - 1) / kWarps;
  }
  const dim3 grid(static_cast<unsigned>(row_blocks + q_blocks)), block(32 * kWarps);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, stream, a, row_blocks, heads_per_warp, warps_per_token);
  };
  if (dtype == MLA_DTYPE_BF16)
    return a.interleaved ? go(rope_write_kernel<MLA_DTYPE_BF16, true>) : go(rope_write_kernel<MLA_DTYPE_BF16, false>);
  return a.interleaved ? go(rope_write_kernel<MLA_DTYPE_FP8_E4M3, true>)
                       : go(rope_write_kernel<MLA_DTYPE_FP8_E4M3, false>);
}

}  // namespace mla
