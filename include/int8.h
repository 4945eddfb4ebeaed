/*
 * int8.h -- C ABI of the 8-bit integer operators: products with a scale for
 * each token and each channel, linear layers on such weights, and activations
 * kept in 8 bits between a forward pass and the gradients that need them.
 * Part of the same library as sgemm.h, with its status codes, streams,
 * workspaces and error rules.
 *
 * Rows.  A row of weights or activations is held as integers q from -127 to
 * 127 and one 32-bit scale s; the values are q * s.  Quantising a row gives
 *
 *   s = max(c * largest |x|, 2^-126), with c = 1/127 and the product rounded to 32 bits
 *   q = the integer nearest to x / s (the exact quotient), ties to even
 *
 * A row that holds a NaN or an infinity gets s = NaN and q = 0.
 *
 * Checkpoints.  A token's channels are divided into blocks of 32 consecutive
 * ones, and each block has a unit u, a power of two; the values are q * u.
 * With a the block's largest magnitude,
 *
 *   u = 2^max(floor(log2 a) - 6, e0), e0 = -126 (INT8_F32, INT8_BF16) or -24 (INT8_F16)
 *   q = x / u rounded to the nearest integer, ties to even, at most 127 in magnitude
 *
 * so that every value is exact in bfloat16, or, kept from 16-bit floats
 * (INT8_F16), in those.  A block that holds a NaN or an infinity gets u = NaN
 * and q = 0.  x is kept with an error of at most u / 2 (u where |x| > 127 u): 2^-7 of a
 * block's largest value, where e0 does not bound the exponent (a block below 2^-127 is
 * kept as zeros; 16-bit floats of INT8_F16 lose nothing there).
 *
 * Memory and ownership are those of sgemm.h: device pointers owned by the
 * caller, calls asynchronous on `stream`, scratch from the per-(device,
 * stream) cache (so calls on one stream must not be made from several host
 * threads at the same time, the first call that needs more scratch is made
 * outside stream capture, and two graphs captured on one stream, which share
 * its scratch, must not run at the same time).  The stream keeps the most that a call on it took: int8_linear()
 * up to 2 bytes for each element of x (its columns rounded up to 64), int8_gemm() as much for A;
 * int8_weight_grad() of INT8_F32 6 bytes for each element of dY, of 16-bit
 * types 2 if dY's rows are not at multiples of 16 bytes; and where sums are cut into shares, up to 20 MB for them.
 * sgemm_release_workspaces() frees it.  Outputs are write-only unless
 * said otherwise and must not overlap inputs or one another.
 */
#ifndef GB300_INT8_H
#define GB300_INT8_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of unquantised matrices. */
typedef enum { INT8_F32 = 0, INT8_BF16 = 1, INT8_F16 = 2 } int8_dtype_t;

/*
 * rows x cols integers, row r at codes + r * ld, and a scale for each row.
 * codes is 16-byte aligned and ld a multiple of 16.  Codes may hold any
 * integer from -128 on.  A row takes cols bytes rounded up to 16: what follows
 * its codes there may be read and is not used, and int8_quantize() writes
 * zeros to it.
 */
typedef struct {
  int64_t rows, cols;
  int8_t *codes;
  int64_t ld; /* bytes from one row to the next */
  float *scales;
} int8_matrix_t;

/* q = x (q->rows x q->cols, type `dtype`, row stride ldx, any alignment that the type allows). */
sgemm_status_t int8_quantize(int dtype, const void *x, int64_t ldx, const int8_matrix_t *q, cudaStream_t stream);

/* y (type `dtype`, row stride ldy) = the values of q: q * s in 32 bits, rounded once. */
sgemm_status_t int8_dequantize(const int8_matrix_t *q, int dtype, void *y, int64_t ldy, cudaStream_t stream);

/*
 * C = A * B^T: A is M x K, B is N x K; C (type `dtype`, row stride ldc) is M x N.
 * The integer sums are exact; a sum is rounded to 32 bits, multiplied there
 * by the smaller and then the larger of its row's and its column's scale
 * (so that scales far apart do not overflow on the way), and rounded to the
 * type.  K = 0 writes zeros; K is at most 131071.
 */
sgemm_status_t int8_gemm(const int8_matrix_t *A, const int8_matrix_t *B, int dtype, void *C, int64_t ldc,
                         cudaStream_t stream);

/*
 * y = Q(x) * W^T: x (M x W->cols, type `dtype`, row stride ldx) is quantised
 * row by row and multiplied by W (N x K); y (M x N, row stride ldy) has x's
 * type.  The result is bit for bit that of int8_quantize() and int8_gemm().
 */
sgemm_status_t int8_linear(int dtype, const void *x, int64_t ldx, int64_t M, const int8_matrix_t *W, void *y,
                           int64_t ldy, cudaStream_t stream);

/*
 * Orders of a checkpoint of `rows` tokens with `cols` channels:
 *
 *   INT8_CHANNELS  codes[c * ld + t], units[(c / 32) * ld_units + t]: the order in which a
 *                  weight gradient's product takes them
 *   INT8_TOKENS    codes[t * ld + c], units[t * ld_units + c / 32]
 *
 * codes and units are 16-byte aligned, ld a multiple of 16 and ld_units of 8.
 * Codes and units that pad a row to the next such multiple are zero.  A unit
 * is the bits of a bfloat16, or of a 16-bit float where dtype is INT8_F16.
 */
typedef enum { INT8_CHANNELS = 0, INT8_TOKENS = 1 } int8_order_t;
typedef struct {
  int32_t dtype; /* type of what was kept */
  int32_t order;
  int64_t rows, cols;
  int8_t *codes;
  int64_t ld; /* bytes */
  uint16_t *units;
  int64_t ld_units; /* elements */
} int8_checkpoint_t;

/* Pitches of the two arrays (bytes and elements) and their sizes in bytes. */
sgemm_status_t int8_checkpoint_layout(int order, int64_t rows, int64_t cols, int64_t *ld, int64_t *ld_units,
                                      int64_t *code_bytes, int64_t *unit_bytes);

/* Keeps x (c->rows x c->cols, type c->dtype, row stride ldx) in c, of order INT8_CHANNELS. */
sgemm_status_t int8_checkpoint(const void *x, int64_t ldx, const int8_checkpoint_t *c, cudaStream_t stream);

/* y (type `dtype`, row stride ldy) = the values of c, of either order. */
sgemm_status_t int8_restore(const int8_checkpoint_t *c, int dtype, void *y, int64_t ldy, cudaStream_t stream);

/*
 * A linear layer's weight gradient from its kept input: dW = dY^T * X, with dY
 * (c->rows x N, type c->dtype, row stride lddy) and X the values of c, of order
 * INT8_CHANNELS.  dW is N x c->cols (row stride ldw) of type `dtype`, which is
 * c->dtype or INT8_F32; if `accumulate`, dW is added to (read, and rounded once).
 * Every product is exact and sums are kept in 32 bits: INT8_F32 gradients are
 * taken as three bfloat16 terms, which hold all of their 24 bits from 2^-110
 * on, 16-bit ones as they are.  The tensor core cuts off what is below an
 * accumulator's last place, at most 6.5e-9 of a sum for each token (measured on sums of one sign); the sums
 * leave it, and are added, correctly rounded, elsewhere, after at most 512 tokens for dW of INT8_F32,
 * 2048 for INT8_F16 and 16384 for INT8_BF16, which is 1/30 of half a step of the 16-bit types.
 * No tokens: zeros, or dW as it was.  At most 2^27 tokens and an N of 2^29.
 */
sgemm_status_t int8_weight_grad(const void *dy, int64_t lddy, int64_t N, const int8_checkpoint_t *c, int dtype,
                                int32_t accumulate, void *dw, int64_t ldw, cudaStream_t stream);

/*
 * The gated activation h = gate * sigmoid(gate) * up, elementwise on M x F
 * matrices of type `dtype`, each with a row stride of its own; the two
 * checkpoints (M x F, that type, order INT8_TOKENS) receive gate and up for
 * the backward pass.  h is computed in 32 bits from gate and up themselves, the
 * sigmoid within 2^-22 of itself, or for 16-bit types within (|gate| + 4) 2^-22 (approximate
 * exponential and reciprocal).  Where the sigmoid leaves the range of 32 bits, for gates below -80,
 * its products are computed in 64 (not for INT8_F16, which cannot hold what comes out).
 */
sgemm_status_t int8_swiglu(int dtype, int64_t M, int64_t F, const void *gate, int64_t ld_gate, const void *up,
                           int64_t ld_up, void *h, int64_t ld_h, const int8_checkpoint_t *kept_gate,
                           const int8_checkpoint_t *kept_up, cudaStream_t stream);

/*
 * Its backward pass from the kept values g and u, with s = sigmoid(g):
 * dgate = dh * u * s * (1 + g * (1 - s)) and dup = dh * g * s, in 32 bits
 * (from left to right; gates below -80 as above), rounded once to the checkpoints' type, which all matrices have.
 */
sgemm_status_t int8_swiglu_backward(const void *dh, int64_t ld_dh, const int8_checkpoint_t *kept_gate,
                                    const int8_checkpoint_t *kept_up, void *dgate, int64_t ld_dgate, void *dup,
                                    int64_t ld_dup, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GB300_INT8_H */
