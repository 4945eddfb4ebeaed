// fp4_stream.cuh -- what the kernels that stream 4-bit weights past a few columns
// share: the form of a stage in shared memory, the ring, and values passed
// between CTAs.
#pragma once

#include "fp4_device.cuh"
#include "fp4_tc.cuh"
#include "sgemm_device.cuh"

namespace gb300 {
namespace fp4 {

constexpr int kMaxStages = 8;
constexpr int kSmemBytes = 232448;  // of a CTA

// 128 rows x 256 columns of weights: the codes as the 128-byte swizzle lays them
// out in shared memory, then the scale atoms.  One stage of the ring; the
// columns' blocks (`cols` rows x 256) have the same form.
template <int kFormat>
struct Block {
  static constexpr int kAtoms = Format<kFormat>::kAtomsPerStage;
  static constexpr uint32_t kScales = kAtoms * 512;
  static constexpr uint32_t kBytes = 16384 + kScales;
};

// Byte of 16-byte piece `piece` of row r in a block's codes.
__host__ __device__ __forceinline__ uint32_t piece_at(uint32_t r, uint32_t piece) {
  return r * 128 + ((piece ^ (r & 7)) << 4);
}
// Byte of the scale of row r, block b (of 256 / kBlock) among a block's scales.
__host__ __device__ __forceinline__ uint32_t scale_at(uint32_t r, uint32_t b) {
  return (b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
}

// Ring position: slot, and how often the ring went round.
struct At {
  uint32_t slot = 0, lap = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++slot == stages) slot = 0, ++lap;
  }
};

// Orders global writes of ordinary stores before later bulk copies, and the other way round.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// A value passed between CTAs and the mark that it is there, in one 64-bit word: no flag, no fence.
__device__ __forceinline__ void put_share(uint64_t* p, float v, uint32_t mark) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(uint64_t(mark) << 32 | __float_as_uint(v)) : "memory");
}
__device__ __forceinline__ uint64_t peek_share(const uint64_t* p) {
  uint64_t w;
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(w) : "l"(p) : "memory");
  return w;
}

}  // namespace fp4
}  // namespace gb300
