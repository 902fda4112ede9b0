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
// against 12 multiply-adds per pair. So everything moves in 16-byte pieces:
// four lanes share one row of 64 rope dims, lane i its pairs 8i .. 8i + 7
// (two 16-byte pieces in either layout), and keep the token's 16 sines and
// cosines in registers over all heads that the warp serves. A latent row is one
// warp's work. Both kinds share a launch: blocks [0, row_blocks) write rows.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "step_internal.h"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kPairsPerLane = 8;
constexpr int kRowVecs = kDimRow * 2 / 16;  // 72
constexpr int kHeadsPerStep = 8;            // 32 lanes / 4 lanes a row
constexpr int kUnroll = 4;                  // rows a lane has in flight

struct Turn {
  float c[kPairsPerLane], s[kPairsPerLane];
};

// Row of the table for each axis, or false for a pad row or a position that
// the table lacks (which sets the status word).
__device__ __forceinline__ bool token_positions(const RopeArgs& a, int t, int (&pos)[kMaxAxes]) {
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
  if (bad && !pad && a.status) atomicOr(a.status, MLA_STATUS_BAD_POSITION);
  return !pad && !bad;
}

// Sines and cosines of pairs 8 sub .. 8 sub + 7.
__device__ __forceinline__ void load_turn(const RopeArgs& a, const int (&pos)[kMaxAxes], int sub, Turn& r) {
  const uint32_t axes = static_cast<uint32_t>(a.pair_axis >> (16 * sub)) & 0xffffu;
  auto row = [&](uint32_t axis) {
    const int p = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
    return a.cos_sin + static_cast<int64_t>(p) * kDimRope + 8 * sub;
  };
  if (axes == (axes & 3u) * 0x5555u) {  // one axis for all eight
    const float4* v = reinterpret_cast<const float4*>(row(axes & 3u));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = __ldg(v + i), s = __ldg(v + 8 + i);
      r.c[4 * i] = c.x, r.c[4 * i + 1] = c.y, r.c[4 * i + 2] = c.z, r.c[4 * i + 3] = c.w;
      r.s[4 * i] = s.x, r.s[4 * i + 1] = s.y, r.s[4 * i + 2] = s.z, r.s[4 * i + 3] = s.w;
    }
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

// Turns the lane's eight pairs: u, v are its two 16-byte pieces. x[], y[]
// receive the pairs' two values; the caller packs them.
__device__ __forceinline__ void turn_pairs(const uint4& u, const uint4& v, const Turn& r, bool interleaved,
                                           float (&x)[kPairsPerLane], float (&y)[kPairsPerLane]) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < kPairsPerLane; ++i) {
    const float a = interleaved ? lo_f(w[i]) : (i & 1 ? hi_f(w[i >> 1]) : lo_f(w[i >> 1]));
    const float b = interleaved ? hi_f(w[i]) : (i & 1 ? hi_f(w[4 + (i >> 1)]) : lo_f(w[4 + (i >> 1)]));
    x[i] = a * r.c[i] - b * r.s[i];
    y[i] = a * r.s[i] + b * r.c[i];
  }
}

// The two 16-byte bf16 pieces of turned pairs.
__device__ __forceinline__ void pack_pairs(const float (&x)[kPairsPerLane], const float (&y)[kPairsPerLane],
                                           bool interleaved, uint4& u, uint4& v) {
  if (interleaved) {
    u = make_uint4(pack_bf16x2(x[0], y[0]), pack_bf16x2(x[1], y[1]), pack_bf16x2(x[2], y[2]), pack_bf16x2(x[3], y[3]));
    v = make_uint4(pack_bf16x2(x[4], y[4]), pack_bf16x2(x[5], y[5]), pack_bf16x2(x[6], y[6]), pack_bf16x2(x[7], y[7]));
  } else {
    u = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    v = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
  }
}

__device__ __forceinline__ uint32_t e4m3(float x, float scale) {
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float scale) {
  uint2 r;
  r.x = e4m3(x[0], scale) | e4m3(x[1], scale) << 8 | e4m3(x[2], scale) << 16 | e4m3(x[3], scale) << 24;
  r.y = e4m3(x[4], scale) | e4m3(x[5], scale) << 8 | e4m3(x[6], scale) << 16 | e4m3(x[7], scale) << 24;
  return r;
}

// One warp, one latent row.
template <int kDtype>
__device__ __forceinline__ void write_row(const RopeArgs& a, int t, int lane) {
  const int64_t slot = a.slots[t];
  if (slot < 0) return;  // pad row
  if (slot >= a.layer_rows) {
    if (lane == 0 && a.status) atomicOr(a.status, MLA_STATUS_BAD_SLOT);
    return;
  }
  int pos[kMaxAxes];
  if (!token_positions(a, t, pos)) return;
  const uint4* src = a.rows + static_cast<int64_t>(t) * kRowVecs;
  const uint4 c0 = src[lane], c1 = src[lane + 32];
  const bool il = a.interleaved != 0;
  uint4 ru, rv;
  Turn r;
  if (lane < 4) {
    ru = src[64 + (il ? 2 * lane : lane)];
    rv = src[64 + (il ? 2 * lane + 1 : lane + 4)];
    load_turn(a, pos, lane, r);
  }
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
  if (lane < 4) turn_pairs(ru, rv, r, il, rx, ry);
  if (kDtype == MLA_DTYPE_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(a.layer_base) + slot * kRowVecs;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      dst[lane + 32 * h] = make_uint4(pack_bf16x2(x[h][0], x[h][1]), pack_bf16x2(x[h][2], x[h][3]),
                                      pack_bf16x2(x[h][4], x[h][5]), pack_bf16x2(x[h][6], x[h][7]));
    if (lane < 4) {
      uint4 u, v;
      pack_pairs(rx, ry, il, u, v);
      dst[64 + (il ? 2 * lane : lane)] = u;
      dst[64 + (il ? 2 * lane + 1 : lane + 4)] = v;
    }
  } else {
    uint2* dst = reinterpret_cast<uint2*>(a.layer_base + slot * kDimRow);
    dst[lane] = e4m3x8(x[0], a.kv_scale);
    dst[lane + 32] = e4m3x8(x[1], a.kv_scale);
    if (lane < 4) {
      float p[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = il ? (i & 1 ? ry[i >> 1] : rx[i >> 1]) : rx[i];
        q[i] = il ? (i & 1 ? ry[4 + (i >> 1)] : rx[4 + (i >> 1)]) : ry[i];
      }
      dst[64 + (il ? 2 * lane : lane)] = e4m3x8(p, a.kv_scale);
      dst[64 + (il ? 2 * lane + 1 : lane + 4)] = e4m3x8(q, a.kv_scale);
    }
  }
}

// One warp: heads [h0, h1) of one token's query.
template <bool kInterleaved>
__device__ __forceinline__ void turn_query(const RopeArgs& a, int t, int h0, int h1, int lane) {
  if (a.slots && a.slots[t] < 0) return;  // pad row
  int pos[kMaxAxes];
  if (!token_positions(a, t, pos)) return;
  const int sub = lane & 3;
  Turn r;
  load_turn(a, pos, sub, r);
  const int off0 = kInterleaved ? 16 * sub : 8 * sub;
  const int off1 = kInterleaved ? 16 * sub + 8 : 8 * sub + 32;
  const int64_t row0 = static_cast<int64_t>(t) * a.num_heads;
  for (int h = h0 + (lane >> 2); h < h1; h += kHeadsPerStep * kUnroll) {
    uint4 u[kUnroll], v[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int hh = h + k * kHeadsPerStep;
      if (hh < h1) {
        const uint16_t* src = a.q + (row0 + hh) * a.q_pitch;
        u[k] = *reinterpret_cast<const uint4*>(src + off0);
        v[k] = *reinterpret_cast<const uint4*>(src + off1);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int hh = h + k * kHeadsPerStep;
      if (hh < h1) {
        float x[kPairsPerLane], y[kPairsPerLane];
        turn_pairs(u[k], v[k], r, kInterleaved, x, y);
        pack_pairs(x, y, kInterleaved, u[k], v[k]);
        uint16_t* dst = a.q_out + (row0 + hh) * a.q_out_pitch;
        *reinterpret_cast<uint4*>(dst + off0) = u[k];
        *reinterpret_cast<uint4*>(dst + off1) = v[k];
      }
    }
  }
}

template <int kDtype, bool kInterleaved>
__global__ void __launch_bounds__(32 * kWarps) rope_write_kernel(const RopeArgs a, int row_blocks, int heads_per_warp,
                                                                 int warps_per_token) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    const int t = blockIdx.x * kWarps + warp;
    if (t < a.n) write_row<kDtype>(a, t, lane);
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
