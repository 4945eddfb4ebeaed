// int8_internal.h -- declarations shared by the 8-bit integer operators'
// translation units.  Not installed; the public interface is include/int8.h.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>

#include "int8.h"

namespace gb300 {

// ---- conversions (int8_convert.cu)
cudaError_t launch_int8_quantize(int dtype, const void* x, int64_t ldx, const int8_matrix_t& q, cudaStream_t stream);
cudaError_t launch_int8_dequantize(const int8_matrix_t& q, int dtype, void* y, int64_t ldy, int sms,
                                   cudaStream_t stream);
// Rows of integers as 16-bit floats, cols rounded up to 8 with zeros (the pitch, in elements, too): quantised on the way ...
cudaError_t launch_int8_rows16(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, uint16_t* out,
                               int64_t ld, float* scales, cudaStream_t stream);
// ... or from integers.
cudaError_t launch_int8_widen(const int8_matrix_t& q, uint16_t* out, int64_t ld, int sms, cudaStream_t stream);
// x (rows x cols, 16-bit or 32-bit) as `terms` matrices of 16 bits one after the other, `ld` elements (a multiple of 8,
// zeros behind cols) a row: 16-bit types as they are, 32 bits as three bfloat16 whose sum they are.
cudaError_t launch_int8_split(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, uint16_t* out,
                              int64_t ld, int sms, cudaStream_t stream);
cudaError_t launch_int8_keep(const void* x, int64_t ldx, const int8_checkpoint_t& c, cudaStream_t stream);
cudaError_t launch_int8_restore(const int8_checkpoint_t& c, int dtype, void* y, int64_t ldy, int sms,
                                cudaStream_t stream);
cudaError_t launch_int8_swiglu(int dtype, int64_t M, int64_t F, const void* gate, int64_t ldg, const void* up,
                               int64_t ldu, void* h, int64_t ldh, const int8_checkpoint_t& kg,
                               const int8_checkpoint_t& ku, int sms, cudaStream_t stream);
cudaError_t launch_int8_swiglu_backward(const void* dh, int64_t lddh, const int8_checkpoint_t& kg,
                                        const int8_checkpoint_t& ku, void* dgate, int64_t ldg, void* dup, int64_t ldu,
                                        int sms, cudaStream_t stream);

// ---- products on the tensor cores (int8_tc.cu)
// D[r, c] = sum over k of a[r, k] b[c, k], stored at out[c * ld + r]; `a` 8-bit integers, times units if it is a
// checkpoint; b 16-bit floats.
// The kind of `a`, whether sums leave the accumulator after some stages, and the columns of a tile.
enum Int8TcShape {
  kInt8Whole32, kInt8Whole64, kInt8Whole128,
  kInt8Bf16N128, kInt8Bf16N256, kInt8Bf16Runs, kInt8Bf16Runs256,
  kInt8F16N128, kInt8F16N256, kInt8F16Runs, kInt8F16Runs256,
  kInt8TcShapes
};
constexpr int64_t kInt8TcStep = 128;  // elements of k a stage
// How many clusters of one, two and four pairs of CTAs run at once.
struct Int8TcClusters {
  int pairs, twos, fours;
};
bool int8_tc_prepare(Int8TcClusters* n);  // sets the kernels' attributes on the current device, too
struct Int8TcArgs {
  int32_t rows, cols, depth;
  int32_t steps, terms;      // stages of k; matrices b, one after the other with depth rows each, whose products are added
  int32_t run;               // stages of k whose sums an accumulator takes, where it does not take all
  int32_t tiles_r, tiles_c, splits, units;  // units = tiles x splits
  const float* scale_r;      // of integers
  const float* scale_c;
  int32_t dtype;             // of out
  int32_t accumulate;        // out += D
  void* out;
  int64_t ld;
  int32_t early;             // the launch before prepared b (one of those above): `a` is read before it ends
  int32_t join;              // a tile's shares are the pairs of a cluster, which add them; otherwise a kernel of its own does
  uint32_t* partials;        // splits x cols x rows 32-bit sums for that
  uint32_t* status;
  uint64_t wait_limit_ns;
};
// maps: `a` (boxes of 128 rows x 128 bytes), its units (4 rows x 128 bytes), b (rows of k in boxes of half the tile's
// columns x 128 bytes, or for checkpoints rows of columns in boxes of 128 rows x 128 bytes).  May start beside the end of the kernel
// before on the stream, and waits for it by itself.
cudaError_t launch_int8_tc(Int8TcShape shape, const CUtensorMap (&maps)[3], const Int8TcArgs& args, int pairs,
                           cudaStream_t stream);

// ---- the same for few tokens and for small products (int8_few.cu): y = X W^T
constexpr int kInt8FewTokens = 8;  // up to which it is always taken
struct Int8FewArgs {
  const int8_t* w;
  int64_t ldw;
  const float* scale_w;
  const void* x;         // tokens of integers, pitch ldx, and their scales; or one unquantised
  int64_t ldx;
  const float* scale_x;
  int32_t early;         // the launch before prepared x: w is read before it ends
  int32_t vec;           // the unquantised one starts at a multiple of 16 bytes
  void* y;
  int64_t ldy;
  int32_t n, k, tokens;
  int32_t dtype;         // of y
};
bool int8_few_quantises(int64_t tokens, int64_t n, int64_t k, int sms);  // whether it takes unquantised tokens (one)
// type_x: the unquantised token's type, or < 0.
cudaError_t launch_int8_few(int type_x, const Int8FewArgs& args, int sms, cudaStream_t stream);

// ---- a small weight gradient (int8_grad.cu): dw (n x cols, + dw if asked) = dy^T X, dy of the type that was kept
struct Int8GradArgs {
  const int8_t* codes;  // channels x tokens
  int64_t ld;
  const uint16_t* units;  // blocks of 32 channels x tokens
  int64_t ldu;
  const void* dy;  // tokens x n
  int64_t lddy;
  int32_t tokens, cols, n;
  int32_t dtype, accumulate;  // of dw
  void* dw;
  int64_t ldw;
};
constexpr int kInt8GradTile = 32, kInt8GradWarps = 4, kInt8GradStep = 64;  // channels and columns of dy a block, its warps, tokens of a warp's step
bool int8_grad_vec(const Int8GradArgs& args);  // whether it reads dy 16 bytes at a time
cudaError_t launch_int8_grad(int dtype, const Int8GradArgs& args, cudaStream_t stream);

}  // namespace gb300
