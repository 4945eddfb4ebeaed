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
// zeros behind cols) a row: 16-bit types as they are (1 term), 32 bits as three bfloat16 whose sum they are.
int int8_terms(int dtype);
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

// ---- products (int8_product.cu)
// D[r, c] = sum over k of a[r, k] b[c, k], stored at out[c * ld + r]: `a` integers (rows x depth, depth contiguous),
// times units[(r / 32) * ld_units + k] if there are units.
struct Int8Product {
  int32_t rows, cols, depth;
  const int8_t* a;
  int64_t lda;
  const uint16_t* units;  // NULL: b holds integers as 16-bit floats, sums are integers
  int64_t ldu;
  const uint16_t* b;      // without units cols x depth, depth contiguous; with them depth x cols, cols contiguous
  int64_t ldb;            // elements, a multiple of 8
  int32_t half;           // units and b are 16-bit floats, not bfloat16
  int32_t terms;          // matrices b one after the other (depth * ldb elements each) whose products are added
  const float* scale_r;   // without units
  const float* scale_c;
  int32_t dtype;          // of out
  int32_t accumulate;     // with units: out += D
  void* out;
  int64_t ld;
};
cudaError_t launch_int8_product(const Int8Product& p, cudaStream_t stream);

}  // namespace gb300
