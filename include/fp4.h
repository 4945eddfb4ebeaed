/*
 * fp4.h -- C ABI of the microscaled 4-bit operators: quantisation, products
 * of quantised matrices, a linear layer on unquantised activations and a
 * mixture-of-experts layer for a few tokens.  Part of the same library as
 * sgemm.h, with its status codes, streams, workspaces and error rules.
 *
 * Number formats.  A code has 4 bits: sign (bit 3), two exponent bits and one
 * fraction bit, and stands for 0, 0.5, 1, 1.5, 2, 3, 4 or 6 (codes 0 to 7) or
 * the negative (8 to 15).  A row's consecutive values are divided into
 * blocks, and each block has a unit u by which its codes are multiplied:
 *
 *   FP4_MXFP4  blocks of 32, a scale byte b, u = 2^(b - 127); 255 means NaN.
 *   FP4_NVFP4  blocks of 16, a scale byte that is an unsigned 8-bit float s (4
 *              exponent bits, bias 7, 3 fraction bits; 127 means NaN, from 128 on
 *              a byte is no scale), and one 32-bit factor g >= 0 of the whole
 *              matrix; u = s * g.
 *
 * Quantising a block whose largest magnitude is a gives
 *
 *   FP4_MXFP4  b = clamp(floor(log2 a) - 2, -127, 127) + 127 (0 if a = 0)
 *   FP4_NVFP4  s = a / (6 g) rounded to nearest even, at most 448 (0 if a = 0)
 *
 * and each code is the value divided by u, rounded to nearest with ties to
 * the even code, at most 6 in magnitude.  Everything is computed in 32 bits
 * (s * g and the quotients are correctly rounded).  A block with u = 0 has
 * zero codes.  A block that holds a NaN or an infinity gets the NaN scale and
 * reads back as NaN.
 *
 * Memory and ownership are those of sgemm.h: device pointers owned by the
 * caller, calls asynchronous on `stream`, scratch from the per-(device,
 * stream) cache (so calls on one stream must not be made from several host
 * threads at the same time, and the first call that needs more scratch is
 * made outside stream capture).  Outputs are write-only and must not overlap
 * inputs (factors included) or one another.
 */
#ifndef GB300_FP4_H
#define GB300_FP4_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FP4_MXFP4 = 0, FP4_NVFP4 = 1 } fp4_format_t;

/* Types of unquantised matrices. */
typedef enum { FP4_F32 = 0, FP4_BF16 = 1, FP4_F16 = 2 } fp4_dtype_t;

/*
 * A quantised matrix of rows x cols values.  Value (r, c) is the code in byte
 * codes[r * ld + c / 2], low four bits for an even c.  Codes beyond cols in a
 * row are zero.  The scale byte of block k of row r is at
 *
 *   scales[(((r / 128) * atoms + k / 4) * 32 + r % 32) * 16 + (r % 128) / 32 * 4 + k % 4]
 *
 * with atoms = ceil(cols / 256) * 64 / block: the order in which the tensor
 * core takes the scales of 128 rows.  Bytes of blocks beyond cols are zero.
 * fp4_layout() gives ld and both sizes.  codes and scales are 16-byte
 * aligned.  factor points to g on the device (NULL: 1; unused for FP4_MXFP4).
 */
typedef struct {
  int32_t format;
  int64_t rows, cols;
  uint8_t *codes;
  int64_t ld; /* bytes from one row to the next, a multiple of 16 */
  uint8_t *scales;
  const float *factor;
} fp4_matrix_t;

/* Row pitch (bytes) and sizes (bytes) of the two arrays of a quantised matrix. */
sgemm_status_t fp4_layout(int format, int64_t rows, int64_t cols, int64_t *ld, int64_t *code_bytes,
                          int64_t *scale_bytes);

/*
 * Quantises x (q->rows x q->cols, type `dtype`, row stride ldx elements, any
 * alignment that the type allows) into q, whose pointers, sizes and factor
 * the caller has set.
 */
sgemm_status_t fp4_quantize(int dtype, const void *x, int64_t ldx, const fp4_matrix_t *q,
                            cudaStream_t stream);

/*
 * Fills q from row-major arrays as checkpoints hold them: `codes` with two
 * codes a byte (low four bits first) and row stride ld_codes bytes, `scales`
 * with one byte a block and row stride ld_scales bytes.
 */
sgemm_status_t fp4_pack(const uint8_t *codes, int64_t ld_codes, const uint8_t *scales,
                        int64_t ld_scales, const fp4_matrix_t *q, cudaStream_t stream);

/* y (type `dtype`, row stride ldy) = the values of q: code * u in 32 bits, rounded once. */
sgemm_status_t fp4_dequantize(const fp4_matrix_t *q, int dtype, void *y, int64_t ldy,
                              cudaStream_t stream);

/*
 * C = A * B^T: A is M x K, B is N x K, both quantised in the same format; C
 * (type `dtype`, row stride ldc) is M x N.  Sums are kept in 32 bits and
 * rounded once.  K = 0 writes zeros.
 */
sgemm_status_t fp4_gemm(const fp4_matrix_t *A, const fp4_matrix_t *B, int dtype, void *C,
                        int64_t ldc, cudaStream_t stream);

/*
 * y = Q(x) * W^T: x (M x W->cols, type `dtype`, row stride ldx) is quantised
 * in W's format, with factor x_factor (device pointer, NULL: 1) for
 * FP4_NVFP4, and multiplied by W (N x K); y (M x N, row stride ldy) has x's
 * type.  The result is that of fp4_quantize() and fp4_gemm(), up to M = 16 with the 32-bit
 * sums in another order.
 */
sgemm_status_t fp4_linear(int dtype, const void *x, int64_t ldx, int64_t M, const float *x_factor,
                          const fp4_matrix_t *W, void *y, int64_t ldy, cudaStream_t stream);

/*
 * The weights of a mixture-of-experts layer, in the order in which the layer's
 * kernel reads them (made once by fp4_experts_pack()): per expert a gate and
 * an up matrix (f x d each) and a down matrix (d x f), d the layer's width.
 * Both arrays are 16-byte aligned; the factors are those of the matrices that
 * they were packed from.
 */
typedef struct {
  int32_t format;
  int64_t experts, d, f;
  uint8_t *gate_up;
  uint8_t *down;
  const float *gate_up_factor;
  const float *down_factor;
} fp4_experts_t;

/* Sizes (bytes) of the two arrays. */
sgemm_status_t fp4_experts_layout(int format, int64_t experts, int64_t d, int64_t f,
                                  int64_t *gate_up_bytes, int64_t *down_bytes);

/*
 * Fills w's arrays.  gate_up is (experts * 2 f) x d, each expert's f gate
 * rows followed by its f up rows; down is (experts * d) x f.  Both have w's
 * format.
 */
sgemm_status_t fp4_experts_pack(const fp4_matrix_t *gate_up, const fp4_matrix_t *down,
                                const fp4_experts_t *w, cudaStream_t stream);

/*
 * The layer for M tokens x (M x d, type `dtype`, row stride ldx):
 *
 *   logits = x R^T                       R: router, experts x d, 32-bit, row stride ldr
 *   ids    = the `top` experts of the largest logits, in that order; equal
 *            logits in the order of their index, NaN after every number
 *   p      = softmax(logits)[ids], divided by its sum if `renormalize`
 *   h_j    = silu(G x) * (U x)           G, U, D: gate, up and down of expert ids[j]
 *   y      = sum_j p_j D h_j
 *
 * y is M x d (row stride ldy) of x's type.  ids (int32) and p (32-bit), M x top
 * each and contiguous, are written if not NULL.  1 <= top <= 32, top <=
 * experts <= 1024.  Activations are not quantised to one 4-bit number: x and h
 * enter the products as sums of 4-bit terms with the format's block scales, each
 * the quantisation of what the terms before it left: 5 terms for bfloat16, 6 for
 * 16-bit float, 8 for 32 bits.  What is left is about 2^-16, 2^-19 and 2^-25 of a
 * block's largest value in the mean and 2^-13, 2^-16 and 2^-22 at most; or, where that
 * is more (FP4_NVFP4, blocks far below the token's largest value of x or h), 2^-21, 2^-24
 * and 2^-30 of that value.  Logits, softmax and sums are in 32 bits.  Values of x
 * that are not finite give results that are not finite, in their token alone; blocks of
 * the weights that are NaN do so for the tokens that go to their expert alone.  Meant for few tokens: more than 16 are done 16 at a time.
 * One kernel on all SMs, launched cooperatively: it waits for the whole GPU.
 */
sgemm_status_t fp4_moe(int dtype, const void *x, int64_t ldx, int64_t M, const float *router,
                       int64_t ldr, const fp4_experts_t *w, int32_t top, int32_t renormalize,
                       void *y, int64_t ldy, int32_t *ids, float *p, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GB300_FP4_H */
