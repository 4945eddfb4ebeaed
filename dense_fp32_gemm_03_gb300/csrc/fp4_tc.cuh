// fp4_tc.cuh -- the tcgen05 operations that the 4-bit products share: descriptors,
// block-scaled MMAs, copies of scales to tensor memory and commits.
#pragma once

#include "fp4_device.cuh"
#include "sgemm_device.cuh"

namespace gb300 {
namespace fp4 {

// Instruction descriptor: E2M1 operands, K-major, 32-bit accumulator; `id` is
// the first of the block scales within a 4-byte group of each operand.
template <int kFormat>
__host__ __device__ constexpr uint32_t instr_desc(uint32_t m, uint32_t n, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | (n >> 3 << 17) | (uint32_t(kFormat == FP4_MXFP4 ? 1 : 0) << 23) |
         (m >> 4 << 24) | (id << 29);
}

// Rows of 128 bytes with the 128-byte swizzle: groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
         uint64_t(2) << 61;
}
// A 512-byte atom of scales: 32 rows of 16 bytes, groups of eight 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | uint64_t(1) << 16 | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
}

template <int kFormat, int kCtas>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                    uint32_t accumulate) {
#define GB300_FP4_MMA(GROUP, KIND, VEC)                                                                    \
  asm volatile(                                                                                            \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                    \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC                        \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                                   \
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)                                        \
      : "memory")
  if constexpr (kFormat == FP4_MXFP4) {
    if constexpr (kCtas == 2)
      GB300_FP4_MMA("2", "mxf4", "2X");
    else
      GB300_FP4_MMA("1", "mxf4", "2X");
  } else {
    if constexpr (kCtas == 2)
      GB300_FP4_MMA("2", "mxf4nvf4", "4X");
    else
      GB300_FP4_MMA("1", "mxf4nvf4", "4X");
  }
#undef GB300_FP4_MMA
}

// One atom of scales into four columns of tensor memory (of both CTAs of a pair).
template <int kCtas>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (kCtas == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Arrives on `bar` (of both CTAs of a pair) once this thread's tcgen05 operations so far completed.
template <int kCtas>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (kCtas == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            dev::smem_addr(bar)),
        "h"(uint16_t(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     dev::smem_addr(bar))
                 : "memory");
}

}  // namespace fp4
}  // namespace gb300
