// int8_product.cu -- products of the 8-bit integer operators.
//
// D[r, c] = sum over k of a[r, k] b[c, k] with `a` 8-bit integers and `b` 16-bit
// floats, which hold integers exactly (sums of integers, then scales), or a
// gradient's values (a's integers times the units of a checkpoint).
//
// 64 x 64 tiles, 16 elements of k at a time through shared memory, 16 sums a thread.
#include <cuda_runtime.h>

#include "int8_device.cuh"
#include "int8_internal.h"

namespace gb300 {
namespace {

using namespace int8;

constexpr int kTile = 64, kStep = 16, kThreads = 256;

template <typename T>
__device__ __forceinline__ void put(const Int8Product& p, int64_t at, float v) {
  T* out = static_cast<T*>(p.out) + at;
  if (p.accumulate) v += to_f32(*out);
  *out = from_f32<T>(v);
}

template <bool kUnits>
__global__ void __launch_bounds__(kThreads) product_kernel(const Int8Product p) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int tiles_r = (p.rows + kTile - 1) / kTile;
  const int r0 = int(blockIdx.x % tiles_r) * kTile, c0 = int(blockIdx.x / tiles_r) * kTile;
  const int tr = threadIdx.x % 16, tc = threadIdx.x / 16;
  float acc[4][4] = {}, total[4][4] = {};
  int whole[4][4] = {};
  for (int t = 0; t < p.terms; ++t) {
    const uint16_t* b = p.b + t * p.depth * p.ldb;
    for (int64_t k0 = 0; k0 < p.depth; k0 += kStep) {
      for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
        const int k = i % kStep, r = i / kStep;
        float v = 0.f;
        if (k0 + k < p.depth && r0 + r < p.rows) {
          v = float(p.a[int64_t(r0 + r) * p.lda + k0 + k]);
          if (kUnits) v *= unit_value(p.units[int64_t((r0 + r) / kBlock) * p.ldu + k0 + k], p.half);
        }
        sa[k][r] = v;
      }
      for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
        const int k = kUnits ? i / kTile : i % kStep, c = kUnits ? i % kTile : i / kStep;
        float v = 0.f;
        if (k0 + k < p.depth && c0 + c < p.cols) {
          const uint16_t w = kUnits ? b[(k0 + k) * p.ldb + c0 + c] : b[int64_t(c0 + c) * p.ldb + k0 + k];
          v = kUnits && !p.half ? __uint_as_float(uint32_t(w) << 16) : __half2float(__ushort_as_half(w));
        }
        sb[k][c] = v;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][tr + 16 * i] * sb[k][tc + 16 * j];
      __syncthreads();
      if ((k0 / kStep) % 64 == 63 || k0 + kStep >= p.depth) {  // 1024 products at a time
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (kUnits)
              total[i][j] += acc[i][j];
            else
              whole[i][j] += __float2int_rn(acc[i][j]);
            acc[i][j] = 0.f;
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + tr + 16 * i, c = c0 + tc + 16 * j;
      if (r >= p.rows || c >= p.cols) continue;
      float v = total[i][j];
      if (!kUnits) {
        const float s = p.scale_r[r], t = p.scale_c[c];
        const bool first = fabsf(s) <= fabsf(t);
        v = float(whole[i][j]) * (first ? s : t) * (first ? t : s);
      }
      const int64_t at = int64_t(c) * p.ld + r;
      if (p.dtype == INT8_F32)
        put<float>(p, at, v);
      else if (p.dtype == INT8_BF16)
        put<__nv_bfloat16>(p, at, v);
      else
        put<__half>(p, at, v);
    }
}

}  // namespace

cudaError_t launch_int8_product(const Int8Product& p, cudaStream_t stream) {
  const int64_t grid = int64_t((p.rows + kTile - 1) / kTile) * ((p.cols + kTile - 1) / kTile);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (p.units)
    product_kernel<true><<<unsigned(grid), kThreads, 0, stream>>>(p);
  else
    product_kernel<false><<<unsigned(grid), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gb300
