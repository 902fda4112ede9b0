// PTX wrappers that only the decode over shared prefixes uses: products of a pair of
// blocks within a cluster of four, and stores into another block's shared memory.
#pragma once

#include "ptx_prefill.cuh"

namespace mla {

// Low word of a descriptor of an MN-major operand whose blocks of 64 columns lie
// `lbo` bytes apart (128-byte swizzle).
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

// mma2_bf16_ss that leaves the rows (lanes of the pair's accumulators) whose bit is set in
// `off` as they are.
__device__ __forceinline__ void mma2_bf16_ss_rows(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                                  const uint32_t (&off)[8], uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, {%6, %7, %8, %9, %10, %11, %12, %13}, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]),
      "r"(off[4]), "r"(off[5]), "r"(off[6]), "r"(off[7])
      : "memory");
}

// Arrive once on the barrier at this offset in the blocks of `mask` when the products that
// this thread issued so far are complete.
__device__ __forceinline__ void mma2_commit_to(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// Arrival on any block's barrier that expects `bytes` more; publishes nothing (what is
// expected completes on the barrier by itself).
__device__ __forceinline__ void mbar_arrive_expect_tx_relaxed(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes)
               : "memory");
}

// Copies `bytes` (a multiple of 16, as the addresses are) of this block's shared memory into
// another block's and completes them on a barrier of that block.
__device__ __forceinline__ void bulk_copy_to(uint32_t cluster_dst, uint32_t src, uint32_t bytes, uint32_t cluster_bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   cluster_dst),
               "r"(src), "r"(bytes), "r"(cluster_bar)
               : "memory");
}

__device__ __forceinline__ void st_async_v2(uint32_t addr, uint32_t a, uint32_t b, uint32_t remote_bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr), "r"(a),
               "r"(b), "r"(remote_bar)
               : "memory");
}

// Asks for `bytes` (a multiple of 16, as the address is) to be brought into L2.
__device__ __forceinline__ void prefetch_l2(const void* ptr, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ptr), "r"(bytes) : "memory");
}

// A pair of bf16 as f16, saturating.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v) {
  return pack_f16x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// 32-byte vector load from global memory.
__device__ __forceinline__ void ld_global_v8(const float* ptr, float* v) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(ptr));
}

}  // namespace mla
