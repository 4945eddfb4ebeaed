// fp4_internal.h -- declarations shared by the 4-bit operators' translation
// units.  Not installed; the public interface is include/fp4.h.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "fp4.h"
#include "sgemm_plan.h"

namespace gb300 {

cudaError_t launch_fp4_quantize(int dtype, const void* x, int64_t ldx, const fp4_matrix_t& q,
                                cudaStream_t stream);
cudaError_t launch_fp4_dequantize(const fp4_matrix_t& q, int dtype, void* y, int64_t ldy,
                                  cudaStream_t stream);
cudaError_t launch_fp4_pack(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                            const fp4_matrix_t& q, cudaStream_t stream);

// Products on the tensor cores (fp4_tc.cu): tiles of a row operand by a column
// operand.  Swapped shapes take B as the row operand.
enum Fp4TcShape { kFp4Pair, kFp4Single128, kFp4Swap16, kFp4Swap32, kFp4Swap64, kFp4TcShapes };
struct Fp4TcTile {
  int rows, cols, ctas;
  bool swap;
};
Fp4TcTile fp4_tc_tile(Fp4TcShape shape);
// Sets the kernels' attributes on the current device; the CTA pairs that run at once, or < 0.
int fp4_tc_prepare();
struct Fp4TcArgs {
  int32_t rows, cols;  // of the row and the column operand
  void* out;
  int64_t ld;
  const float* factor_r;
  const float* factor_c;
  float* partials;    // shares of split tiles: (tiles split + units - 1) slots of a tile
  int32_t* counters;  // one per CTA of a split tile, zero on entry and on exit
  uint32_t* status;
  uint64_t wait_limit_ns;
  int32_t tma_out;    // the output's rows can be addressed by TMA (map_out)
  int32_t tma_edge;   // and its row bytes are a multiple of 16
};
// maps: codes of the row and the column operand (boxes of 128 rows and of the
// columns that one CTA stages), their scales (boxes of the atoms of 256
// columns), the output (boxes of 32 rows x 128 bytes).
cudaError_t launch_fp4_tc(int dtype, int format, Fp4TcShape shape, const CUtensorMap (&maps)[5],
                          const Fp4TcArgs& args, const Sched& sc, int grid, cudaStream_t stream);

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
  float* x_scale;     // tokens: the power of two that x was multiplied by
  uint32_t* h_max;    // tokens: the largest |h| of the token's pairs, as bits
  void* x_frag;       // x as 16-bit floats in fragment order
  float* h;           // (tokens x top) x f rounded up to 128
  float* partial;     // shares of the tiles of y: tile x part x token x row
  int32_t* counters;  // three, zero on entry and on exit
  int32_t* tile_counters;  // one per tile of y (16 rows), zero on entry and on exit
  int32_t tile_counter_count;
  uint32_t* status;
  uint64_t wait_limit_ns;
};
struct MoeScratch {
  size_t logits, x_scale, h_max, x_frag, h, partial, bytes;  // offsets, and the size of all
};
MoeScratch fp4_moe_scratch(int dtype, int64_t tokens, int64_t experts, int64_t d, int64_t f, int64_t top);
cudaError_t launch_fp4_moe(int dtype, int format, const MoeArgs& args, int sms, cudaStream_t stream);

}  // namespace gb300
