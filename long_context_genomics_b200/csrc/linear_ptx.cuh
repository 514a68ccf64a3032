// linear_ptx.cuh -- the forms of TMA and of the matrix instruction that the
// linear layers use beyond the attention's (sm100.cuh, whose text identifies the
// attention kernel that a profile was taken of).
#pragma once

#include "sm100.cuh"

namespace ag {

// tma_load_2d with the default L2 policy.
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// The same by either CTA of a pair into its own shared memory, the bytes
// counted on a barrier of the pair's even CTA (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map,
                                                 uint32_t cluster_bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int c0,
                                             int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Instruction descriptor of kind::f16 with a float32 accumulator for 16-bit
// operands of either type and major-ness: bf16 or f16 (both operands), A and B
// K-major (0) or MN-major (1).
__host__ __device__ constexpr uint32_t idesc_half_f32(uint32_t M, uint32_t N, bool bf16,
                                                      uint32_t a_mn_major, uint32_t b_mn_major) {
  return (1u << 4)                         // D format: f32
         | ((bf16 ? 1u : 0u) << 7)         // A format
         | ((bf16 ? 1u : 0u) << 10)        // B format
         | (a_mn_major << 15) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

}  // namespace ag
