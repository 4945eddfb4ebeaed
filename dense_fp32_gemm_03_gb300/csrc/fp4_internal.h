// fp4_internal.h -- declarations shared by the 4-bit operators' translation
// units.  Not installed; the public interface is include/fp4.h.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "fp4.h"

namespace gb300 {

cudaError_t launch_fp4_quantize(int dtype, const void* x, int64_t ldx, const fp4_matrix_t& q,
                                cudaStream_t stream);
cudaError_t launch_fp4_dequantize(const fp4_matrix_t& q, int dtype, void* y, int64_t ldy,
                                  cudaStream_t stream);
cudaError_t launch_fp4_pack(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                            const fp4_matrix_t& q, cudaStream_t stream);

// C (type dtype) = A B^T with bounds-checked loads (fp4_simple.cu).
cudaError_t launch_fp4_simple(const fp4_matrix_t& A, const fp4_matrix_t& B, int dtype, void* C, int64_t ldc,
                              cudaStream_t stream);

// The expert weights' order (fp4_moe.cu): tiles of 16 rows; a tile's rows are
// cut into chunks of 128 columns, stored one after another.
int64_t fp4_expert_chunk_bytes(int format);
cudaError_t launch_fp4_experts_pack(const fp4_matrix_t& gate_up, const fp4_matrix_t& down,
                                    const fp4_experts_t& w, cudaStream_t stream);

constexpr int kMoeTokens = 16;  // tokens of one launch
struct MoeArgs {
  const void* x;
  int64_t ldx;
  const float* router;
  int64_t ldr;
  const uint8_t* gate_up;
  const uint8_t* down;
  const float* gate_up_factor;
  const float* down_factor;
  void* y;
  int64_t ldy;
  int32_t* ids;
  float* p;
  int32_t tokens, experts, d, f, top, renormalize;
  // Scratch.
  float* logits;      // tokens x experts
  int32_t* pick;      // tokens x top
  float* weight;      // tokens x top
  float* x_scale;     // tokens: the power of two that x was multiplied by
  uint32_t* h_max;    // tokens: the largest |h| of the token's pairs, as bits
  void* x_frag;       // x as 16-bit floats in fragment order
  float* h;           // (tokens x top) x f rounded up to 128
  int32_t* counters;  // three, zero on entry and on exit
  uint32_t* status;
  uint64_t wait_limit_ns;
};
struct MoeScratch {
  size_t logits, pick, weight, x_scale, h_max, x_frag, h, bytes;  // offsets, and the size of all
};
MoeScratch fp4_moe_scratch(int dtype, int64_t tokens, int64_t experts, int64_t d, int64_t f, int64_t top);
cudaError_t launch_fp4_moe(int dtype, int format, const MoeArgs& args, int sms, cudaStream_t stream);

}  // namespace gb300
