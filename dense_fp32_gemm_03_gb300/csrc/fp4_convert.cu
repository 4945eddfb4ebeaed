// fp4_convert.cu -- quantisation to the microscaled 4-bit formats, its
// inverse, and the re-ordering of row-major codes and scales (fp4.h).
//
// All three kernels walk the matrix in pieces of 256 columns of one row, a
// piece to a warp and eight columns to a lane: one or two 16-byte loads and
// one 4-byte store of codes, both contiguous over the warp.  A block of 16
// (32) columns is two (four) lanes, so its largest magnitude takes one (two)
// shuffles; the four scale bytes that lie together in the scale layout are
// joined by two more.  The kernels are bound by the bytes that they move.
#include <cuda_runtime.h>

#include "fp4_device.cuh"
#include "fp4_internal.h"

namespace gb300 {
namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xffffffffu;

// Joins the scale bytes of the four blocks of one atom: every lane passes its
// block's byte, and the first lane of each 4 * kLanes lanes gets the word.
template <int kLanes>
__device__ __forceinline__ uint32_t join_scales(uint32_t byte, int lane) {
  uint32_t w = byte << (8 * ((lane / kLanes) & 3));
  w |= __shfl_xor_sync(kFull, w, kLanes);
  w |= __shfl_xor_sync(kFull, w, 2 * kLanes);
  return w;
}

template <typename T, int kFormat, bool kVector>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T* __restrict__ x, int64_t ldx, const float* __restrict__ factor, int rows,
                    int cols, int pieces, uint8_t* __restrict__ codes, int64_t ld,
                    uint8_t* __restrict__ scales) {
  using F = Format<kFormat>;
  constexpr int kLanes = F::kBlock / 8;  // lanes of a block
  const int lane = threadIdx.x & 31;
  const float g = kFormat == FP4_NVFP4 && factor != nullptr ? __ldg(factor) : 1.f;
  const int64_t atoms = int64_t(pieces) * F::kAtomsPerStage;
  const int64_t items = int64_t(rows) * pieces;
  for (int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items;
       item += int64_t(gridDim.x) * kWarps) {
    const int r = int(item / pieces), piece = int(item - int64_t(r) * pieces);
    const int c = piece * 256 + lane * 8;
    const T* p = x + int64_t(r) * ldx + c;
    float v[8];
    if (kVector && c + 8 <= cols) {
      load8(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_f32(p[i]) : 0.f;
    }
    // The largest magnitude as an integer: NaN > infinity > every finite value.
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int s = 1; s < kLanes; s *= 2) top = max(top, __shfl_xor_sync(kFull, top, s));

    uint32_t byte, word = 0;
    if constexpr (kFormat == FP4_MXFP4) {
      // floor(log2 a) is the exponent field; a subnormal a clamps to -127 as field 0 does.
      const int e = max(int(top >> 23) - 127 - 2, -127);
      byte = top >= 0x7f800000u ? 255u : top == 0 ? 0u : uint32_t(e + 127);
      const float inv = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e, at most 2^127
#pragma unroll
      for (int i = 0; i < 4; ++i) word |= encode2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
    } else {
      const float a = __uint_as_float(top);
      byte = top >= 0x7f800000u ? 127u : top == 0 ? 0u : encode_e4m3(__fdiv_rn(a, 6.f * g));
      const float unit = decode_e4m3(byte) * g;
      if (unit > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          word |= encode2(__fdiv_rn(v[2 * i], unit), __fdiv_rn(v[2 * i + 1], unit)) << (8 * i);
      }
    }
    if (c < (cols + 31) / 32 * 32) *reinterpret_cast<uint32_t*>(codes + int64_t(r) * ld + c / 2) = word;
    const uint32_t four = join_scales<kLanes>(byte, lane);
    if (lane % (4 * kLanes) == 0)
      *reinterpret_cast<uint32_t*>(scales + scale_offset(r, c / F::kBlock, atoms)) = four;
  }
}

template <typename T, int kFormat, bool kVector>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ld, const uint8_t* __restrict__ scales,
                      const float* __restrict__ factor, int rows, int cols, int pieces,
                      T* __restrict__ y, int64_t ldy) {
  using F = Format<kFormat>;
  const int lane = threadIdx.x & 31;
  const float g = kFormat == FP4_NVFP4 && factor != nullptr ? __ldg(factor) : 1.f;
  const int64_t atoms = int64_t(pieces) * F::kAtomsPerStage;
  const int64_t items = int64_t(rows) * pieces;
  for (int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items;
       item += int64_t(gridDim.x) * kWarps) {
    const int r = int(item / pieces), piece = int(item - int64_t(r) * pieces);
    const int c = piece * 256 + lane * 8;
    if (c >= cols) continue;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + int64_t(r) * ld + c / 2));
    const float s = decode_scale<kFormat>(__ldg(scales + scale_offset(r, c / F::kBlock, atoms)));
    const float unit = kFormat == FP4_NVFP4 ? s * g : s;
    const float2 a = __half22float2(decode2<0>(w)), b = __half22float2(decode2<1>(w)),
                 d = __half22float2(decode2<2>(w)), e = __half22float2(decode2<3>(w));
    const float v[8] = {a.x * unit, a.y * unit, b.x * unit, b.y * unit,
                        d.x * unit, d.y * unit, e.x * unit, e.y * unit};
    T* p = y + int64_t(r) * ldy + c;
    if (kVector && c + 8 <= cols) {
      store8(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) p[i] = from_f32<T>(v[i]);
    }
  }
}

// Row-major codes (any pitch and alignment) and scales into the library's layout.
template <int kFormat>
__global__ void __launch_bounds__(kThreads)
    pack_codes_kernel(const uint8_t* __restrict__ src, int64_t ld_src, const uint8_t* __restrict__ src_scales,
                      int64_t ld_scales, int rows, int cols, int pieces, uint8_t* __restrict__ codes,
                      int64_t ld, uint8_t* __restrict__ scales) {
  using F = Format<kFormat>;
  constexpr int kLanes = F::kBlock / 8;
  const int lane = threadIdx.x & 31;
  const int64_t atoms = int64_t(pieces) * F::kAtomsPerStage;
  const int64_t items = int64_t(rows) * pieces;
  for (int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items;
       item += int64_t(gridDim.x) * kWarps) {
    const int r = int(item / pieces), piece = int(item - int64_t(r) * pieces);
    const int c = piece * 256 + lane * 8;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = c + 2 * i;
      if (k < cols) {
        uint32_t b = src[int64_t(r) * ld_src + k / 2];
        if (k + 1 >= cols) b &= 0xfu;
        w |= b << (8 * i);
      }
    }
    if (c < (cols + 31) / 32 * 32) *reinterpret_cast<uint32_t*>(codes + int64_t(r) * ld + c / 2) = w;
    const uint32_t byte = c < cols ? src_scales[int64_t(r) * ld_scales + c / F::kBlock] : 0u;
    const uint32_t four = join_scales<kLanes>(byte, lane);
    if (lane % (4 * kLanes) == 0)
      *reinterpret_cast<uint32_t*>(scales + scale_offset(r, c / F::kBlock, atoms)) = four;
  }
}

unsigned grid_of(int64_t rows, int pieces) {
  const int64_t blocks = (rows * pieces + kWarps - 1) / kWarps;
  return unsigned(blocks < (int64_t(1) << 30) ? blocks : (int64_t(1) << 30));
}

template <typename T>
bool vector_ok(const void* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % int64_t(16 / sizeof(T)) == 0;
}

template <typename T, int kFormat>
cudaError_t quantize_t(const void* x, int64_t ldx, const fp4_matrix_t& q, int pieces, cudaStream_t stream) {
  auto* kernel = vector_ok<T>(x, ldx) ? quantize_kernel<T, kFormat, true> : quantize_kernel<T, kFormat, false>;
  kernel<<<grid_of(q.rows, pieces), kThreads, 0, stream>>>(static_cast<const T*>(x), ldx, q.factor, int(q.rows),
                                                           int(q.cols), pieces, q.codes, q.ld, q.scales);
  return cudaGetLastError();
}

template <typename T, int kFormat>
cudaError_t dequantize_t(const fp4_matrix_t& q, void* y, int64_t ldy, int pieces, cudaStream_t stream) {
  auto* kernel = vector_ok<T>(y, ldy) ? dequantize_kernel<T, kFormat, true> : dequantize_kernel<T, kFormat, false>;
  kernel<<<grid_of(q.rows, pieces), kThreads, 0, stream>>>(q.codes, q.ld, q.scales, q.factor, int(q.rows),
                                                           int(q.cols), pieces, static_cast<T*>(y), ldy);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_quantize(int dtype, const void* x, int64_t ldx, const fp4_matrix_t& q,
                                cudaStream_t stream) {
  const int pieces = int((q.cols + 255) / 256);
  const bool mx = q.format == FP4_MXFP4;
  switch (dtype) {
    case FP4_F32:
      return mx ? quantize_t<float, FP4_MXFP4>(x, ldx, q, pieces, stream)
                : quantize_t<float, FP4_NVFP4>(x, ldx, q, pieces, stream);
    case FP4_BF16:
      return mx ? quantize_t<__nv_bfloat16, FP4_MXFP4>(x, ldx, q, pieces, stream)
                : quantize_t<__nv_bfloat16, FP4_NVFP4>(x, ldx, q, pieces, stream);
    default:
      return mx ? quantize_t<__half, FP4_MXFP4>(x, ldx, q, pieces, stream)
                : quantize_t<__half, FP4_NVFP4>(x, ldx, q, pieces, stream);
  }
}

cudaError_t launch_fp4_dequantize(const fp4_matrix_t& q, int dtype, void* y, int64_t ldy,
                                  cudaStream_t stream) {
  const int pieces = int((q.cols + 255) / 256);
  const bool mx = q.format == FP4_MXFP4;
  switch (dtype) {
    case FP4_F32:
      return mx ? dequantize_t<float, FP4_MXFP4>(q, y, ldy, pieces, stream)
                : dequantize_t<float, FP4_NVFP4>(q, y, ldy, pieces, stream);
    case FP4_BF16:
      return mx ? dequantize_t<__nv_bfloat16, FP4_MXFP4>(q, y, ldy, pieces, stream)
                : dequantize_t<__nv_bfloat16, FP4_NVFP4>(q, y, ldy, pieces, stream);
    default:
      return mx ? dequantize_t<__half, FP4_MXFP4>(q, y, ldy, pieces, stream)
                : dequantize_t<__half, FP4_NVFP4>(q, y, ldy, pieces, stream);
  }
}

cudaError_t launch_fp4_pack(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                            const fp4_matrix_t& q, cudaStream_t stream) {
  const int pieces = int((q.cols + 255) / 256);
  auto* kernel = q.format == FP4_MXFP4 ? pack_codes_kernel<FP4_MXFP4> : pack_codes_kernel<FP4_NVFP4>;
  kernel<<<grid_of(q.rows, pieces), kThreads, 0, stream>>>(codes, ld_codes, scales, ld_scales, int(q.rows),
                                                           int(q.cols), pieces, q.codes, q.ld, q.scales);
  return cudaGetLastError();
}

}  // namespace gb300
