// fp4_simple.cu -- the bounds-checked product of two 4-bit matrices: 64 x 64
// tiles, both operands turned into 32-bit values in shared memory, FFMA.
#include <cuda_runtime.h>

#include "fp4_device.cuh"
#include "fp4_internal.h"

namespace gb300 {
namespace {

using namespace fp4;

template <int kFormat>
__device__ __forceinline__ float value_at(const fp4_matrix_t& q, int64_t r, int64_t c, int64_t atoms) {
  if (r >= q.rows || c >= q.cols) return 0.f;
  const uint32_t byte = q.codes[r * q.ld + c / 2];
  const float2 v = __half22float2(decode2<0>(byte));
  return ((c & 1) ? v.y : v.x) *
         decode_scale<kFormat>(q.scales[scale_offset(r, c / Format<kFormat>::kBlock, atoms)]);
}

template <typename T, int kFormat>
__global__ void __launch_bounds__(256)
    simple_kernel(const fp4_matrix_t A, const fp4_matrix_t B, T* __restrict__ C, int64_t ldc) {
  __shared__ float sa[16][65], sb[16][65];
  const int64_t m0 = int64_t(blockIdx.y) * 64, n0 = int64_t(blockIdx.x) * 64;
  const int64_t atoms = (A.cols + 255) / 256 * Format<kFormat>::kAtomsPerStage;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < A.cols; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i >> 4, k = i & 15;
      sa[k][r] = value_at<kFormat>(A, m0 + r, k0 + k, atoms);
      sb[k][r] = value_at<kFormat>(B, n0 + r, k0 + k, atoms);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  float alpha = 1.f;
  if (kFormat == FP4_NVFP4) {
    if (A.factor) alpha = *A.factor;
    if (B.factor) alpha *= *B.factor;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < A.rows && n < B.rows) C[m * ldc + n] = from_f32<T>(acc[i][j] * alpha);
    }
}

template <typename T>
cudaError_t launch_t(const fp4_matrix_t& A, const fp4_matrix_t& B, void* C, int64_t ldc, cudaStream_t stream) {
  const dim3 grid(unsigned((B.rows + 63) / 64), unsigned((A.rows + 63) / 64));
  if (A.format == FP4_MXFP4)
    simple_kernel<T, FP4_MXFP4><<<grid, 256, 0, stream>>>(A, B, static_cast<T*>(C), ldc);
  else
    simple_kernel<T, FP4_NVFP4><<<grid, 256, 0, stream>>>(A, B, static_cast<T*>(C), ldc);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_simple(const fp4_matrix_t& A, const fp4_matrix_t& B, int dtype, void* C, int64_t ldc,
                              cudaStream_t stream) {
  return dtype == FP4_F32    ? launch_t<float>(A, B, C, ldc, stream)
         : dtype == FP4_BF16 ? launch_t<__nv_bfloat16>(A, B, C, ldc, stream)
                             : launch_t<__half>(A, B, C, ldc, stream);
}

}  // namespace gb300
