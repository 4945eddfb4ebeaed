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

// The single-thread instructions below are executed by a whole warp in uniform
// control flow, predicated on `e` (one elected lane): operands then stay in uniform
// registers.  Behind a branch on the elected lane, with the warp's number taken from
// threadIdx alone, 8 copies of scales, 4 MMAs and a commit took 544 cycles to issue;
// like this, with the warp's number through a shuffle (uniform_warp()), 292.
// A predicate that depends on more than the election undoes it (8192^3: 250 us instead
// of 167), so MMAs are issued also after a wait gave up: they read shared memory that
// may be stale, and the output is invalid anyway.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0); }
__device__ __forceinline__ uint32_t elected() { return dev::elect_one() ? 1u : 0u; }

// A kernel that allocates all 512 columns of tensor memory gets the base address 0.
constexpr uint32_t kTmemColumns = 512, kTmemBase = 0;

template <int kFormat, int kCtas>
__device__ __forceinline__ void mma(uint32_t e, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                    uint32_t sb, uint32_t accumulate) {
#define GB300_FP4_MMA(GROUP, KIND, VEC)                                                                    \
  asm volatile(                                                                                            \
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"                        \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC                     \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                                   \
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(e)                                \
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
__device__ __forceinline__ void copy_scales(uint32_t e, uint32_t taddr, uint64_t desc) {
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(
            taddr),
        "l"(desc), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(
            taddr),
        "l"(desc), "r"(e)
        : "memory");
}

// Arrives on `bar` (of both CTAs of a pair) once the tcgen05 operations issued so far completed.
template <int kCtas>
__device__ __forceinline__ void commit(uint32_t e, uint64_t* bar) {
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            dev::smem_addr(bar)),
        "h"(uint16_t(3)), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(dev::smem_addr(bar)),
        "r"(e)
        : "memory");
}

__device__ __forceinline__ void expect_bytes(uint32_t e, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(dev::smem_addr(bar)),
      "r"(bytes), "r"(e)
      : "memory");
}

// `bytes` contiguous bytes (a multiple of 16, both addresses too) to shared memory.
__device__ __forceinline__ void load_bytes(uint32_t e, void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(
          dev::smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(dev::smem_addr(bar)), "r"(e)
      : "memory");
}

// The box at (x, y) of a tensor map; `bar` is the address of a barrier of the pair's first CTA (kCtas = 2) or of this one.
template <int kCtas>
__device__ __forceinline__ void load_box(uint32_t e, void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (kCtas == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dev::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dev::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(e)
        : "memory");
}

}  // namespace fp4
}  // namespace gb300
