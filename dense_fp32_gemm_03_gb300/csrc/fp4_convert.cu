// fp4_convert.cu -- quantisation to the microscaled 4-bit formats, its
// inverse, and the re-ordering of row-major codes and scales (fp4.h).
//
// The kernels walk the matrix in pieces of one row, a piece to a warp.
// Quantising takes 512 columns, 16 to a lane: a lane then holds a whole block
// (mxfp4: half a one), so that a block's scale is found once by one lane, and the
// work beside the 16 quotients is spread over twice as many values as with eight
// columns to a lane (177 instructions a lane for 8, which bound it).  The four
// scale bytes that lie together in the scale layout are joined by two shuffles.
// Reading back takes 256 columns, 16 bytes of output to a lane at a time.
#include <cuda_runtime.h>

#include <type_traits>

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

// The pieces of one warp: every `warps`-th one, row by row.
struct PieceIter {
  int r, piece, rows, pieces, dr, dp;
  __device__ __forceinline__ PieceIter(int rows_, int pieces_, int64_t warp, int64_t warps)
      : rows(rows_), pieces(pieces_) {
    const int64_t first = warp / pieces;
    r = first < rows ? int(first) : rows;
    piece = int(warp - first * pieces);
    const int64_t step = warps / pieces;
    dr = step < rows ? int(step) : rows;
    dp = int(warps - step * pieces);
  }
  __device__ __forceinline__ bool valid() const { return r < rows; }
  __device__ __forceinline__ void next() {
    r = r + dr < rows ? r + dr : rows;
    piece += dp;
    if (piece >= pieces) piece -= pieces, ++r;
  }
};

constexpr int kPieceCols = 512;  // of quantising
constexpr int kLaneCols = 16;

// Sixteen consecutive values a lane, 32 lanes, of a row that starts at any address
// the type allows.  16-byte loads at aligned addresses bring the lanes' bytes
// (kWords words each) from the piece's first address rounded down; lane 31 brings
// 16 bytes more.  values() moves them into place with the next lane's first words.
// Nothing outside the row is read: 16 bytes that reach over an end of it are
// gathered value by value, which only the first and the last piece meet.
template <typename T, bool kAligned>
struct Piece {
  static constexpr int kWords = kLaneCols * int(sizeof(T)) / 4;
  uint32_t w[kWords], extra[4];
  uint32_t shift;  // bytes from the aligned address to the piece's first value

  // 16 bytes at `at`; those from `from` up to `to` (bytes of the 16) are the row's.
  __device__ __forceinline__ static uint4 load16(const uint8_t* at, int from, int to) {
    if (from <= 0 && to >= 16) return __ldg(reinterpret_cast<const uint4*>(at));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (to > 0) {
      T* t = reinterpret_cast<T*>(&v);
#pragma unroll
      for (int i = 0; i < int(16 / sizeof(T)); ++i) {
        const int byte = i * int(sizeof(T));
        if (byte >= from && byte < to) t[i] = *reinterpret_cast<const T*>(at + byte);
      }
    }
    return v;
  }

  __device__ __forceinline__ void load(const T* row, int cols, int piece, int lane) {
    const uint8_t* first = reinterpret_cast<const uint8_t*>(row) + int64_t(piece) * (kPieceCols * sizeof(T));
    shift = kAligned ? 0u : uint32_t(reinterpret_cast<uintptr_t>(first) & 15u);
    const int off = lane * (kWords * 4) - int(shift);  // of this lane's bytes from the piece's first
    const uint8_t* at = first + off;
    const int before = piece == 0 ? 0 : -16;                                             // the row reaches back to here
    const int left = min(cols - piece * kPieceCols, 2 * kPieceCols) * int(sizeof(T));  // and to here
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = load16(at + 16 * i, before - (off + 16 * i), left - (off + 16 * i));
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
    if (!kAligned) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (lane == 31 && shift != 0) v = load16(at + kWords * 4, 0, left - (off + kWords * 4));
      extra[0] = v.x, extra[1] = v.y, extra[2] = v.z, extra[3] = v.w;
    }
  }

  template <int kBy>
  __device__ __forceinline__ void place(const uint32_t (&next)[4], uint32_t (&out)[kWords]) const {
    const uint32_t bits = (shift & 3u) * 8;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t lo = i + kBy < kWords ? w[(i + kBy) % kWords] : next[(i + kBy - kWords) & 3];
      const uint32_t hi = i + kBy + 1 < kWords ? w[(i + kBy + 1) % kWords] : next[(i + kBy + 1 - kWords) & 3];
      out[i] = __funnelshift_r(lo, hi, bits);
    }
  }

  __device__ __forceinline__ void values(float (&v)[kLaneCols], int lane) const {
    uint32_t out[kWords];
    if (kAligned) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) out[i] = w[i];
    } else {
      uint32_t next[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        next[i] = __shfl_down_sync(kFull, w[i], 1);
        if (lane == 31) next[i] = extra[i];
      }
      switch (shift >> 2) {
        case 0: place<0>(next, out); break;
        case 1: place<1>(next, out); break;
        case 2: place<2>(next, out); break;
        default: place<3>(next, out);
      }
    }
    const T* t = reinterpret_cast<const T*>(out);
#pragma unroll
    for (int i = 0; i < kLaneCols; ++i) v[i] = to_f32(t[i]);
  }
};

// Four blocks an SM, that is 64 registers: with 72 three run, and 8192^2 nvfp4 fp32 takes 50.6 us, not 47.8.
template <typename T, int kFormat, bool kAligned>
__global__ void __launch_bounds__(kThreads, 4)
    quantize_kernel(const T* __restrict__ x, int64_t ldx, const float* __restrict__ factor, int rows,
                    int cols, uint8_t* __restrict__ codes, int64_t ld, uint8_t* __restrict__ scales) {
  using F = Format<kFormat>;
  constexpr int kLanes = F::kBlock / kLaneCols;  // lanes of a block
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Quantizer<kFormat> quantizer(factor);
  const int code_cols = (cols + 31) / 32 * 32, scale_cols = (cols + 255) / 256 * 256;
  const int64_t atoms = int64_t(scale_cols / F::kAtom);
  PieceIter it(rows, (cols + kPieceCols - 1) / kPieceCols, int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5),
               int64_t(gridDim.x) * kWarps);
  Piece<T, kAligned> in;
  if (it.valid()) in.load(x + int64_t(it.r) * ldx, cols, it.piece, lane);
  // A product of what this kernel writes may set itself up meanwhile; it waits for the
  // end (linear 17 x 4096 x 4096 bf16 9.2 -> 8.6 us, 1000 x 4096 x 4096 17.4 -> 16.6).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  while (it.valid()) {
    const int r = it.r, c = it.piece * kPieceCols + lane * kLaneCols;
    float v[kLaneCols];
    in.values(v, lane);
    it.next();
    if (it.valid()) in.load(x + int64_t(it.r) * ldx, cols, it.piece, lane);  // on its way during the arithmetic
    float a = largest(v), unit;
    if (kLanes == 2) a = max_abs(a, __shfl_xor_sync(kFull, a, 1));
    const uint32_t byte = quantizer.scale(a, unit);
    uint32_t word[2];
    quantizer.encode(v, a, unit, word);
    if (c < code_cols) *reinterpret_cast<uint2*>(codes + int64_t(r) * ld + c / 2) = make_uint2(word[0], word[1]);
    const uint32_t four = join_scales<kLanes>(byte, lane);
    if (lane % (4 * kLanes) == 0 && c < scale_cols)
      *reinterpret_cast<uint32_t*>(scales + scale_offset(r, c / F::kBlock, atoms)) = four;
  }
}

// Stores 16 bytes of values a lane to a row that starts at any address the type
// allows, `first` being where lane 0's belong: 16-byte stores at aligned addresses,
// their words taken from this lane and the one before; the warp's first and last 16
// bytes, and those past `left` bytes, value by value.
template <typename T>
__device__ __forceinline__ void store_shifted(uint8_t* first, int left, int lane, const uint4& mine) {
  uint32_t w[8] = {0u, 0u, 0u, 0u, mine.x, mine.y, mine.z, mine.w};  // the previous lane's words, then this lane's
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(kFull, w[4 + i], 1);
  const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(first) & 15u), bits = (shift & 3u) * 8;
  // Aligned word j of this lane holds the bytes from 4 j - shift on of its own 16;
  // words 4 to 7 are lane 31's, behind its own.
  uint32_t out[8];
  auto place = [&](auto by) {
    constexpr int kBy = decltype(by)::value;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = j + 4 - kBy;  // w[s] starts at or after aligned word j
      const uint32_t hi = s < 8 ? w[s & 7] : 0u, lo = s - 1 < 8 ? w[(s - 1) & 7] : 0u;
      out[j] = bits == 0 ? hi : __funnelshift_r(lo, hi, 32 - bits);
    }
  };
  switch (shift >> 2) {
    case 0: place(std::integral_constant<int, 0>()); break;
    case 1: place(std::integral_constant<int, 1>()); break;
    case 2: place(std::integral_constant<int, 2>()); break;
    default: place(std::integral_constant<int, 3>());
  }
  const int off = lane * 16 - int(shift);
  uint8_t* at = first + off;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int from = -(off + 16 * i), to = left + from;  // the row's bytes among these 16
    if (i == 1 && (lane != 31 || shift == 0)) break;
    if (i == 0 && from <= 0 && to >= 16) {
      *reinterpret_cast<uint4*>(at) = make_uint4(out[0], out[1], out[2], out[3]);
    } else if (to > 0) {
      const T* t = reinterpret_cast<const T*>(out + 4 * i);
#pragma unroll
      for (int k = 0; k < int(16 / sizeof(T)); ++k) {
        const int byte = k * int(sizeof(T));
        // The extra 16 bytes of lane 31 end where its own values do.
        if (byte >= from && byte < to && (i == 0 || byte < int(shift))) *reinterpret_cast<T*>(at + 16 * i + byte) = t[k];
      }
    }
  }
}

template <typename T, int kFormat, bool kAligned>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ld, const uint8_t* __restrict__ scales,
                      const float* __restrict__ factor, int rows, int cols, int pieces,
                      T* __restrict__ y, int64_t ldy) {
  using F = Format<kFormat>;
  constexpr int kV = 16 / int(sizeof(T)), kParts = 256 / (32 * kV);  // values of a lane and part
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float g = kFormat == FP4_NVFP4 && factor != nullptr ? __ldg(factor) : 1.f;
  const int64_t atoms = int64_t(pieces) * F::kAtomsPerStage;
  PieceIter it(rows, pieces, int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5), int64_t(gridDim.x) * kWarps);
  uint32_t w[kParts] = {}, byte[kParts] = {};
  auto load = [&]() {
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const int c = it.piece * 256 + (p * 32 + lane) * kV;
      if (c < cols) {
        const uint8_t* at = codes + int64_t(it.r) * ld + c / 2;
        w[p] = kV == 8 ? __ldg(reinterpret_cast<const uint32_t*>(at)) : uint32_t(__ldg(reinterpret_cast<const uint16_t*>(at)));
        byte[p] = __ldg(scales + scale_offset(it.r, c / F::kBlock, atoms));
      }
    }
  };
  if (it.valid()) load();
  while (it.valid()) {
    const int r = it.r, piece = it.piece;
    uint4 out[kParts];
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const float s = decode_scale<kFormat>(byte[p]);
      const float unit = kFormat == FP4_NVFP4 ? s * g : s;
      T* t = reinterpret_cast<T*>(&out[p]);
      const float2 a = __half22float2(decode2<0>(w[p])), b = __half22float2(decode2<1>(w[p]));
      t[0] = from_f32<T>(a.x * unit), t[1] = from_f32<T>(a.y * unit);
      t[2] = from_f32<T>(b.x * unit), t[3] = from_f32<T>(b.y * unit);
      if constexpr (kV == 8) {
        const float2 d = __half22float2(decode2<2>(w[p])), e = __half22float2(decode2<3>(w[p]));
        t[4] = from_f32<T>(d.x * unit), t[5] = from_f32<T>(d.y * unit);
        t[6] = from_f32<T>(e.x * unit), t[7] = from_f32<T>(e.y * unit);
      }
    }
    it.next();
    if (it.valid()) load();
    uint8_t* row = reinterpret_cast<uint8_t*>(y + int64_t(r) * ldy + piece * 256);
    const int left = min(cols - piece * 256, 256) * int(sizeof(T));
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (!kAligned) {
        store_shifted<T>(row + p * 512, left - p * 512, lane, out[p]);
      } else {
        const int at = p * 512 + lane * 16;
        if (at + 16 <= left) {
          *reinterpret_cast<uint4*>(row + at) = out[p];
        } else {
          const T* t = reinterpret_cast<const T*>(&out[p]);
#pragma unroll
          for (int i = 0; i < kV; ++i)
            if (at + (i + 1) * int(sizeof(T)) <= left) reinterpret_cast<T*>(row + at)[i] = t[i];
        }
      }
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

// Blocks that cover the pieces once, or eight an SM, whose warps walk on: four to six run at once
// (40 to 64 registers), the others follow and even out the end.  8192^2 nvfp4 fp32 there and
// back with 4, 8 and 16 an SM: 137, 112 and 108 us; 1000 x 5003: 12.5, 11.4 and 12.3.
unsigned grid_of(int64_t rows, int pieces, int sms) {
  const int64_t blocks = (rows * pieces + kWarps - 1) / kWarps, most = int64_t(sms) * 8;
  return unsigned(blocks < most ? blocks : most);
}

template <typename T>
bool vector_ok(const void* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % int64_t(16 / sizeof(T)) == 0;
}

// A kernel that may start beside the end of the one before on the stream and waits for it by itself
// (16 x 4096 quantised and read back in a graph: 3.6 us in order, 2.8 so).
template <typename... P>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, cudaStream_t stream, P... params) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, params...);
}

template <typename T, int kFormat>
cudaError_t quantize_t(const void* x, int64_t ldx, const fp4_matrix_t& q, int pieces, int sms,
                       cudaStream_t stream) {
  auto* kernel = vector_ok<T>(x, ldx) ? quantize_kernel<T, kFormat, true> : quantize_kernel<T, kFormat, false>;
  return launch_early(kernel, grid_of(q.rows, pieces, sms), stream, static_cast<const T*>(x), ldx,
                      static_cast<const float*>(q.factor), int(q.rows), int(q.cols), q.codes, q.ld, q.scales);
}

template <typename T, int kFormat>
cudaError_t dequantize_t(const fp4_matrix_t& q, void* y, int64_t ldy, int pieces, int sms, cudaStream_t stream) {
  auto* kernel = vector_ok<T>(y, ldy) ? dequantize_kernel<T, kFormat, true> : dequantize_kernel<T, kFormat, false>;
  return launch_early(kernel, grid_of(q.rows, pieces, sms), stream, static_cast<const uint8_t*>(q.codes), q.ld,
                      static_cast<const uint8_t*>(q.scales), static_cast<const float*>(q.factor), int(q.rows),
                      int(q.cols), pieces, static_cast<T*>(y), ldy);
}

}  // namespace

cudaError_t launch_fp4_quantize(int dtype, const void* x, int64_t ldx, const fp4_matrix_t& q, int sms,
                                cudaStream_t stream) {
  const int pieces = int((q.cols + kPieceCols - 1) / kPieceCols);
  const bool mx = q.format == FP4_MXFP4;
  switch (dtype) {
    case FP4_F32:
      return mx ? quantize_t<float, FP4_MXFP4>(x, ldx, q, pieces, sms, stream)
                : quantize_t<float, FP4_NVFP4>(x, ldx, q, pieces, sms, stream);
    case FP4_BF16:
      return mx ? quantize_t<__nv_bfloat16, FP4_MXFP4>(x, ldx, q, pieces, sms, stream)
                : quantize_t<__nv_bfloat16, FP4_NVFP4>(x, ldx, q, pieces, sms, stream);
    default:
      return mx ? quantize_t<__half, FP4_MXFP4>(x, ldx, q, pieces, sms, stream)
                : quantize_t<__half, FP4_NVFP4>(x, ldx, q, pieces, sms, stream);
  }
}

cudaError_t launch_fp4_dequantize(const fp4_matrix_t& q, int dtype, void* y, int64_t ldy, int sms,
                                  cudaStream_t stream) {
  const int pieces = int((q.cols + 255) / 256);
  const bool mx = q.format == FP4_MXFP4;
  switch (dtype) {
    case FP4_F32:
      return mx ? dequantize_t<float, FP4_MXFP4>(q, y, ldy, pieces, sms, stream)
                : dequantize_t<float, FP4_NVFP4>(q, y, ldy, pieces, sms, stream);
    case FP4_BF16:
      return mx ? dequantize_t<__nv_bfloat16, FP4_MXFP4>(q, y, ldy, pieces, sms, stream)
                : dequantize_t<__nv_bfloat16, FP4_NVFP4>(q, y, ldy, pieces, sms, stream);
    default:
      return mx ? dequantize_t<__half, FP4_MXFP4>(q, y, ldy, pieces, sms, stream)
                : dequantize_t<__half, FP4_NVFP4>(q, y, ldy, pieces, sms, stream);
  }
}

cudaError_t launch_fp4_pack(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                            const fp4_matrix_t& q, int sms, cudaStream_t stream) {
  const int pieces = int((q.cols + 255) / 256);
  auto* kernel = q.format == FP4_MXFP4 ? pack_codes_kernel<FP4_MXFP4> : pack_codes_kernel<FP4_NVFP4>;
  kernel<<<grid_of(q.rows, pieces, sms), kThreads, 0, stream>>>(codes, ld_codes, scales, ld_scales, int(q.rows),
                                                           int(q.cols), pieces, q.codes, q.ld, q.scales);
  return cudaGetLastError();
}

}  // namespace gb300
