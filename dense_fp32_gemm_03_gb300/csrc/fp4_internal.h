// fp4_internal.h -- declarations shared by the 4-bit operators' translation
// units.  Not installed; the public interface is include/fp4.h.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "fp4.h"
#include "sgemm_plan.h"

namespace gb300 {

cudaError_t launch_fp4_quantize(int dtype, const void* x, int64_t ldx, const fp4_matrix_t& q, int sms,
                                cudaStream_t stream);
cudaError_t launch_fp4_dequantize(const fp4_matrix_t& q, int dtype, void* y, int64_t ldy, int sms,
                                  cudaStream_t stream);
cudaError_t launch_fp4_pack(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                            const fp4_matrix_t& q, int sms, cudaStream_t stream);

// Products on the tensor cores (fp4_tc.cu): tiles of a row operand by a column
// operand.  Swapped shapes take B as the row operand.
enum Fp4TcShape { kFp4Pair256, kFp4Pair128, kFp4Single128, kFp4Swap16, kFp4Swap32, kFp4Swap64, kFp4TcShapes };
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
// The kernel may start beside the end of the one before on the stream, and waits for it by itself.
cudaError_t launch_fp4_tc(int dtype, int format, Fp4TcShape shape, const CUtensorMap (&maps)[5],
                          const Fp4TcArgs& args, const Sched& sc, int grid, cudaStream_t stream);

// The linear layer for few tokens (fp4_linear.cu).
int fp4_linear_tokens();  // the most
int fp4_linear_steps();   // stages (256 columns) of K that one CTA of a cluster takes at most
struct Fp4LinearArgs {
  const void* x;
  int64_t ldx;
  const float* x_factor;
  const uint8_t* scales;  // W's
  const float* w_factor;
  void* y;
  int64_t ldy;
  int32_t tokens, n, k;
  int32_t steps, ctas, per;  // stages of K, CTAs of a cluster, stages of each
  uint32_t* status;
  uint64_t wait_limit_ns;
};
// Sets the kernels' attributes on the current device; the clusters of 1, 2, 4 and 8 CTAs that run at once.
bool fp4_linear_prepare(int (&clusters)[4]);
// map: W's codes in boxes of 128 rows x 128 bytes, 128-byte swizzle.
cudaError_t launch_fp4_linear(int dtype, int format, const CUtensorMap& map, const Fp4LinearArgs& args, int clusters,
                              cudaStream_t stream);

// The expert weights' order (fp4_moe.cu): blocks of 128 rows x 256 columns as
// one stage of the layer's kernel takes them; after the gate-and-up blocks one 32-bit bound an expert.
int64_t fp4_gate_up_bytes(int format, int64_t experts, int64_t d, int64_t f);
int64_t fp4_down_bytes(int format, int64_t experts, int64_t d, int64_t f);
const uint32_t* fp4_expert_bounds(const fp4_experts_t& w);
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
  const uint32_t* bound;  // per expert (fp4_expert_bounds)
  int32_t cols;           // columns of a product: tokens x terms, rounded up to 16
  // Scratch.
  float* logits;      // tokens x experts
  int32_t* x_exp;     // tokens: x was multiplied by 2^x_exp
  float* x_norm;      // tokens: log2 of x's 2-norm
  uint32_t* h_max;    // tokens: largest |h|, as bits
  float* h;           // h in 32 bits: token, place of the expert among its own, f rounded up to 64
  uint8_t* x_image;   // x as terms: a block of columns for each 256 of d
  uint8_t* h_image;   // h as terms: the same for each expert in use and 256 of f
  uint64_t* share;    // shares of units cut between CTAs: CTA x phase (2, 3) x token x row
  int32_t* counters;  // the workspace's counters, zero on entry and on exit
  uint32_t* status;
  uint64_t wait_limit_ns;
};
struct MoeScratch {
  size_t logits, x_exp, x_norm, h_max, h, x_image, h_image, share, bytes;  // offsets, and the size of all
  int cols;
};
MoeScratch fp4_moe_scratch(int dtype, int format, int64_t tokens, int64_t experts, int64_t d, int64_t f, int64_t top,
                           int sms);
bool fp4_moe_prepare();  // the kernels' attributes on the current device
cudaError_t launch_fp4_moe(int dtype, int format, const MoeArgs& args, int sms, cudaStream_t stream);

}  // namespace gb300
