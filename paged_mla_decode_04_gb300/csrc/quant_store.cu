// Compact latent store: rows of codes with scales of their own groups, written from
// bf16 rows and read back.
//
// Per group of dims (128 for e4m3, 32 for e2m1) a = max |x|:
//   e4m3: scale = a / 448 in fp32,              code = e4m3(x / scale)
//   e2m1: scale = a / 6 rounded to bf16 (once), code = e2m1(x / scale)
// with IEEE fp32 divisions, rounded to the nearest code (ties to even) and saturating.
// Groups of zeros, or so small that the scale is zero, have codes of zero; a group with an
// infinity or NaN has scale NaN and reads as NaN throughout.
//
// A warp a row: reading and writing is all there is to it, 1,816 bytes a token (e4m3). 131,072
// rows: written in 40.7 us (e4m3; 5.9 TB/s, 87 % of a copy's rate) and 37.0 (e2m1; 5.6), read
// from e2m1 into a bf16 pool in 40.2 (5.2 TB/s; three quarters of the bytes are writes), from e4m3
// in 41.8 (5.7). A few rows: 2.3 us. Into an e4m3 pool it is the divisions by its kv_scale, one a
// value: 58 us from e4m3 and 113 from e2m1, whose bytes take 24 and 20. (As products with the
// reciprocal, which round otherwise, 37 from either.)
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "../../include/mla_decode.h"
#include "ptx.cuh"
#include "shared_internal.h"

namespace mla {
namespace {

constexpr int kWarps = 4;  // (a percent or two more than eight of the bandwidth, of large calls)
constexpr int kRowVecs = kDimRow * 2 / 16;  // 16-byte pieces of a bf16 row: 64 of c_kv, 8 of rope

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Largest magnitude among a piece's eight values, as bf16 bits (NaN above infinity).
__device__ __forceinline__ uint32_t largest(const uint4& v) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
  return max(a & 0xffffu, a >> 16);
}

__device__ __forceinline__ float scale_of(uint32_t top, float most) {
  return top >= 0x7f80u ? CUDART_NAN_F : __fdiv_rn(__uint_as_float(top << 16), most);
}

// Division of many numbers by one, as IEEE division rounds it: by Markstein's theorem the
// quotient q = x y is put right by its exact remainder, q + (x - q s) y, where y is 1 / s
// rounded (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990). Held to IEEE division for every pair of significands that a value and
// its group's scale can have, and for scales down to 2^-60, whose remainders keep their
// bits; smaller ones, zero and NaN go the long way. (Divisions for every value took the
// store's write 48 us for 131,072 rows; so it takes 41.)
struct Divisor {
  float s, y;
  bool quick;
  __device__ __forceinline__ explicit Divisor(float scale) : s(scale), quick(scale >= 0x1p-60f) {
    y = quick ? __frcp_rn(scale) : 0.f;
  }
};

template <bool kQuick>
__device__ __forceinline__ float over(float x, const Divisor& d) {
  if (!kQuick) return d.s > 0.f ? __fdiv_rn(x, d.s) : 0.f;
  const float q = __fmul_rn(x, d.y);
  return __fmaf_rn(__fmaf_rn(-q, d.s, x), d.y, q);
}

template <bool kQuick>
__device__ __forceinline__ uint32_t e4m3x4(uint32_t a, uint32_t b, const Divisor& s) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(over<kQuick>(lo_f(a), s), over<kQuick>(hi_f(a), s)), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(over<kQuick>(lo_f(b), s), over<kQuick>(hi_f(b), s)), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

template <bool kQuick>
__device__ __forceinline__ uint32_t e2m1x2(uint32_t a, const Divisor& s) {
  return __nv_cvt_float2_to_fp4x2(make_float2(over<kQuick>(lo_f(a), s), over<kQuick>(hi_f(a), s)), __NV_E2M1, cudaRoundNearest);
}

template <bool kQuick>
__device__ __forceinline__ uint2 e4m3x8(const uint4& v, const Divisor& s) {
  return make_uint2(e4m3x4<kQuick>(v.x, v.y, s), e4m3x4<kQuick>(v.z, v.w, s));
}
template <bool kQuick>
__device__ __forceinline__ uint32_t e2m1x8(const uint4& v, const Divisor& s) {
  return e2m1x2<kQuick>(v.x, s) | e2m1x2<kQuick>(v.y, s) << 8 | e2m1x2<kQuick>(v.z, s) << 16 | e2m1x2<kQuick>(v.w, s) << 24;
}

template <int kFormat>
__global__ void __launch_bounds__(32 * kWarps) store_write_kernel(const StoreWriteArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= a.n) return;
  const uint4* src = a.rows + t * kRowVecs;
  const int64_t slot = a.slots[t];
  const uint4 v[2] = {src[lane], src[lane + 32]};
  uint4 rope;
  if (lane < 8) rope = src[64 + lane];
  if (slot < 0) return;  // pad row
  if (slot >= a.layer_rows) {
    if (lane == 0 && a.status) atomicOr(a.status, MLA_STATUS_BAD_SLOT);
    return;
  }
  if (kFormat == MLA_QUANT_E4M3) {
    uint8_t* dst = a.layer_base + slot * kStoreE4m3Row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // piece 32 h + lane: group 2 h + lane / 16
      uint32_t top = largest(v[h]);
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float s = scale_of(top, 448.f);
      const Divisor d(s);
      reinterpret_cast<uint2*>(dst)[lane + 32 * h] = d.quick ? e4m3x8<true>(v[h], d) : e4m3x8<false>(v[h], d);
      if ((lane & 15) == 0) reinterpret_cast<float*>(dst + kDimCkv)[2 * h + (lane >> 4)] = s;
    }
    if (lane < 8) reinterpret_cast<uint4*>(dst + kDimCkv + 16)[lane] = rope;
  } else {
    uint8_t* dst = a.layer_base + slot * kStoreE2m1Row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // piece 32 h + lane: group 8 h + lane / 4
      uint32_t top = largest(v[h]);
#pragma unroll
      for (int d = 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      const __nv_bfloat16 sb = __float2bfloat16_rn(scale_of(top, 6.f));
      const float s = __bfloat162float(sb);
      const Divisor d(s);
      reinterpret_cast<uint32_t*>(dst)[lane + 32 * h] = d.quick ? e2m1x8<true>(v[h], d) : e2m1x8<false>(v[h], d);
      if ((lane & 3) == 0) reinterpret_cast<__nv_bfloat16*>(dst + 256)[8 * h + (lane >> 2)] = sb;
    }
    if (lane < 8) reinterpret_cast<uint4*>(dst + 288)[lane] = rope;
  }
}

// Two e4m3 codes, as floats.
__device__ __forceinline__ float2 of_e4m3x2(uint32_t v) {
  const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(v));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 of_e2m1x2(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(v), __NV_E2M1);
  return __half22float2(__half2(h));
}

__device__ __forceinline__ uint32_t to_e4m3x4(float p, float q, float r, float t, float s) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(p, s), __fdiv_rn(q, s)), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(r, s), __fdiv_rn(t, s)), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// A lane has pieces of eight dims as in the write, so that each load and store of a warp is
// of bytes next to each other. (With 16 dims next to each other a lane 33 rows took 2.6 us
// instead of 2.3 and 8,192 rows 3.8 instead of 3.5; the largest reads as long.)
template <int kFormat, int kOut>
__global__ void __launch_bounds__(32 * kWarps) store_read_kernel(const StoreReadArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= a.n) return;
  const int64_t slot = a.slots[t], to = a.out_slots ? a.out_slots[t] : t;
  if (slot < 0 || to < 0) return;
  if (slot >= a.layer_rows || to >= a.out_rows) {
    if (lane == 0 && a.status) atomicOr(a.status, MLA_STATUS_BAD_SLOT);
    return;
  }
  float x[2][8];
  const uint8_t* src = a.layer_base + slot * (kFormat == MLA_QUANT_E4M3 ? kStoreE4m3Row : kStoreE2m1Row);
  uint4 rope;
  if (lane < 8) rope = reinterpret_cast<const uint4*>(src + (kFormat == MLA_QUANT_E4M3 ? 528 : 288))[lane];
  if (kFormat == MLA_QUANT_E4M3) {
    const uint2 c[2] = {reinterpret_cast<const uint2*>(src)[lane], reinterpret_cast<const uint2*>(src)[lane + 32]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // group 2 h + lane / 16
      const float s = reinterpret_cast<const float*>(src + kDimCkv)[2 * h + (lane >> 4)];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = of_e4m3x2((i < 2 ? c[h].x : c[h].y) >> (16 * (i & 1)) & 0xffffu);
        x[h][2 * i] = f.x * s;
        x[h][2 * i + 1] = f.y * s;
      }
    }
  } else {
    const uint32_t c[2] = {reinterpret_cast<const uint32_t*>(src)[lane], reinterpret_cast<const uint32_t*>(src)[lane + 32]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // group 8 h + lane / 4
      const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src + 256)[8 * h + (lane >> 2)]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = of_e2m1x2(c[h] >> (8 * i) & 0xffu);
        x[h][2 * i] = f.x * s;
        x[h][2 * i + 1] = f.y * s;
      }
    }
  }
  if (kOut == MLA_DTYPE_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(a.out) + to * kRowVecs;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      dst[lane + 32 * h] = make_uint4(pack_bf16x2(x[h][0], x[h][1]), pack_bf16x2(x[h][2], x[h][3]),
                                      pack_bf16x2(x[h][4], x[h][5]), pack_bf16x2(x[h][6], x[h][7]));
    if (lane < 8) dst[64 + lane] = rope;
  } else {
    uint2* dst = reinterpret_cast<uint2*>(a.out + to * kDimRow);
    const float k = a.kv_scale;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      dst[lane + 32 * h] = make_uint2(to_e4m3x4(x[h][0], x[h][1], x[h][2], x[h][3], k), to_e4m3x4(x[h][4], x[h][5], x[h][6], x[h][7], k));
    if (lane < 8)
      dst[64 + lane] = make_uint2(to_e4m3x4(lo_f(rope.x), hi_f(rope.x), lo_f(rope.y), hi_f(rope.y), k),
                                  to_e4m3x4(lo_f(rope.z), hi_f(rope.z), lo_f(rope.w), hi_f(rope.w), k));
  }
}

}  // namespace

cudaError_t launch_store_write(const StoreWriteArgs& a, int format, cudaStream_t stream) {
  const dim3 grid((a.n - 1) / kWarps + 1), block(32 * kWarps);
  if (format == MLA_QUANT_E4M3) return launch_pdl(store_write_kernel<MLA_QUANT_E4M3>, grid, block, 0, stream, a);
  return launch_pdl(store_write_kernel<MLA_QUANT_E2M1>, grid, block, 0, stream, a);
}

cudaError_t launch_store_read(const StoreReadArgs& a, int format, int out_dtype, cudaStream_t stream) {
  const dim3 grid((a.n - 1) / kWarps + 1), block(32 * kWarps);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, stream, a); };
  if (format == MLA_QUANT_E4M3)
    return out_dtype == MLA_DTYPE_BF16 ? go(store_read_kernel<MLA_QUANT_E4M3, MLA_DTYPE_BF16>)
                                       : go(store_read_kernel<MLA_QUANT_E4M3, MLA_DTYPE_FP8_E4M3>);
  return out_dtype == MLA_DTYPE_BF16 ? go(store_read_kernel<MLA_QUANT_E2M1, MLA_DTYPE_BF16>)
                                     : go(store_read_kernel<MLA_QUANT_E2M1, MLA_DTYPE_FP8_E4M3>);
}

}  // namespace mla
