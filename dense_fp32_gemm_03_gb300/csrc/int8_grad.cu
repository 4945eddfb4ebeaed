// int8_grad.cu -- weight gradients of few tokens and small layers from 8-bit checkpoints.
//
// Mathematics.  dw[n, c] = sum over tokens of dy[t, n] q[t, c] u[t, c / 32].  q u is exact in 16 bits (bfloat16, or 16-bit
// floats if those were kept); dy is in that type, or in 32 bits the sum of three bfloat16, of which the two small ones have
// sums of their own.  Everything is added up in 32 bits.
//
// Structure.  A block has 32 channels and 32 columns of dy, and its four warps take 64 tokens in turn, each by itself: a lane
// loads 16 tokens' integers of four channels and the tokens' units (its share of four steps of mma.m16n8k16, whose k can be any if
// both operands take the same ones), and turns them to 16 bits in registers; dy goes through the warp's part of shared
// memory as it is, whatever its pitch, and is turned by ldmatrix.  The warps' sums are added up at the end.
//
// What bounds it: latencies (one launch; the tiled kernel needs dy on aligned rows, in terms if it has 32 bits, which is
// a kernel before it).  64 tokens of 256 x 256 bf16 2.7 us, in tiles 6.3; 333 x 520 x 1001 fp16 with odd rows 7.1 and 7.7.
#include <cuda_runtime.h>

#include <type_traits>

#include "int8_device.cuh"
#include "int8_internal.h"

namespace gb300 {
namespace {

using namespace int8;

constexpr int kTile = kInt8GradTile, kWarps = kInt8GradWarps, kThreads = 32 * kWarps, kStep = kInt8GradStep;

template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where 16 bytes (columns 8 q ..) of a token's 64 are: the eight rows of a matrix that ldmatrix reads, tokens 16 apart and
// pairs of neighbours, lie in different banks.
__device__ __forceinline__ int place(int token, int q) { return token * 64 + ((q ^ (token >> 4)) & 3) * 16; }

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) grad_kernel(const Int8GradArgs a) {
  constexpr int kTerms = sizeof(T) == 4 ? 3 : 1, kSets = kTerms == 1 ? 1 : 2;  // sums: of the first terms, of the others
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int kBytes = kStep * kTile * 2;  // of a term of a warp's step
  __shared__ __align__(128) unsigned char staged[kWarps][kTerms][kBytes];
  static_assert(sizeof(staged) >= kWarps * kTile * kTile * 4, "the sums take the same memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int tiles = (a.n + kTile - 1) / kTile;
  const int c0 = blockIdx.x / tiles * kTile, n0 = blockIdx.x % tiles * kTile;
  const int8_t* codes[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) codes[r] = a.codes + min(c0 + 8 * r + g, a.cols - 1) * a.ld + 16 * t;
  const uint16_t* units = a.units + c0 / kBlock * a.ldu + 16 * t;
  const int left_n = a.n - n0;
  unsigned char* mine = staged[warp][0];
  const uint32_t mine_at = uint32_t(__cvta_generic_to_shared(mine));
  float acc[kSets][2][4][4] = {};
#pragma unroll 1
  for (int t0 = kStep * warp; t0 < a.tokens; t0 += kStep * kWarps) {
    const int left = a.tokens - t0;  // of which 16 t .. are this lane's
    uint4 q[4] = {}, u[2] = {};
    if (16 * t < left) {
#pragma unroll
      for (int r = 0; r < 4; ++r) q[r] = *reinterpret_cast<const uint4*>(codes[r] + t0);
      u[0] = *reinterpret_cast<const uint4*>(units + t0);
      if (16 * t + 8 < left) u[1] = *reinterpret_cast<const uint4*>(units + t0 + 8);
    }
    const T* dy = static_cast<const T*>(a.dy) + t0 * a.lddy + n0;
    __syncwarp();  // the step before has been read
    if constexpr (kVec) {
      uint4 v[kStep * kTile / 256];
#pragma unroll
      for (int i = 0; i < kStep * kTile / 256; ++i) {
        const int token = 8 * i + lane / 4, c = 8 * (lane % 4);
        v[i] = token < left && c < left_n ? *reinterpret_cast<const uint4*>(dy + token * a.lddy + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kStep * kTile / 256; ++i) *reinterpret_cast<uint4*>(mine + place(8 * i + lane / 4, lane % 4)) = v[i];
    } else {
      // 32 values a lane at a time, of one column; in 32 bits of two, whose terms are written together (64 tokens of 256 x 256
      // 7.0 -> 4.5 us; 16 bits are better off with one, 333 x 520 x 1001 8.3 and 7.1).
      constexpr int kCols = kTerms == 1 ? 1 : 2, kLanes = 32 / kCols, kBatch = 32 / kCols;
      const int c = lane % kLanes * kCols;
      const T* from = dy + lane / kLanes * a.lddy + c;
#pragma unroll 1
      for (int i0 = 0; i0 < kStep; i0 += 32) {
        T v[kBatch][kCols];
#pragma unroll
        for (int i = 0; i < kBatch; ++i, from += kCols * a.lddy) {
          const bool here = i0 + kCols * i + lane / kLanes < left;
#pragma unroll
          for (int e = 0; e < kCols; ++e) v[i][e] = here && c + e < left_n ? from[e] : from_f32<T>(0.f);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          unsigned char* to = mine + place(i0 + kCols * i + lane / kLanes, c / 8) + c % 8 * 2;
          if constexpr (kTerms == 1) {
            *reinterpret_cast<T*>(to) = v[i][0];
          } else {
            float x = v[i][0], y = v[i][kCols - 1];
#pragma unroll
            for (int s = 0; s < kTerms; ++s) {
              const uint32_t low = take16(x);
              *reinterpret_cast<uint32_t*>(to + s * kBytes) = low | take16(y) << 16;
            }
          }
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // Four tokens of four channels, as two steps' rows.
      const uint32_t word[4] = {(&q[0].x)[i], (&q[1].x)[i], (&q[2].x)[i], (&q[3].x)[i]};
      const uint32_t u0 = (&u[i / 2].x)[i % 2 * 2], u1 = (&u[i / 2].x)[i % 2 * 2 + 1];
      uint32_t x[2][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (kHalf) {
          const uint32_t v = word[r] ^ 0x80808080u;
          x[r / 2][r % 2] = hmul2(to_f16<0>(v), u0);
          x[r / 2][r % 2 + 2] = hmul2(to_f16<1>(v), u1);
        } else {
          x[r / 2][r % 2] = bmul2(to_bf16<0>(word[r]), u0);
          x[r / 2][r % 2 + 2] = bmul2(to_bf16<1>(word[r]), u1);
        }
      }
      const int token = 16 * (lane % 8 / 2) + 4 * i + lane % 2 + 2 * (lane / 8 % 2);
#pragma unroll
      for (int s = 0; s < kTerms; ++s)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          uint32_t b[4];
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                       : "r"(mine_at + s * kBytes + place(token, j + lane / 16))
                       : "memory");
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma<kHalf>(acc[s ? kSets - 1 : 0][m][j], x[m], b[0], b[1]);
            mma<kHalf>(acc[s ? kSets - 1 : 0][m][j + 1], x[m], b[2], b[3]);
          }
        }
    }
  }
  __syncthreads();
  // sums[warp][column of dy][channel], lanes of a column two banks apart.
  float* sums = reinterpret_cast<float*>(staged);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 16 * m + g + e / 2 * 8, n = 8 * j + 2 * t + e % 2;
        sums[(warp * kTile + n) * kTile + (c ^ (8 * t))] = acc[0][m][j][e] + (kSets > 1 ? acc[kSets - 1][m][j][e] : 0.f);
      }
  __syncthreads();
  for (int i = threadIdx.x; i < kTile * kTile; i += kThreads) {
    const int n = i / kTile, c = i % kTile;
    if (n >= left_n || c0 + c >= a.cols) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[(w * kTile + n) * kTile + (c ^ (8 * (n / 2 % 4)))];
    const int64_t at = (n0 + n) * a.ldw + c0 + c;
    if (a.dtype == INT8_F32) {
      float* to = static_cast<float*>(a.dw) + at;
      *to = a.accumulate ? v + *to : v;
    } else {  // (the type that was kept)
      using O = std::conditional_t<sizeof(T) == 4, __half, T>;  // 32-bit ones have no other
      O* to = static_cast<O*>(a.dw) + at;
      *to = from_f32<O>(a.accumulate ? v + to_f32(*to) : v);
    }
  }
}

}  // namespace

bool int8_grad_vec(const Int8GradArgs& a) {
  // (32-bit values are split on the way)
  return reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.lddy % 8 == 0 && a.n % 8 == 0;
}
static int64_t blocks_of(const Int8GradArgs& a) {
  return (int64_t(a.cols) + kTile - 1) / kTile * ((int64_t(a.n) + kTile - 1) / kTile);
}

cudaError_t launch_int8_grad(int dtype, const Int8GradArgs& args, cudaStream_t stream) {
  const int64_t blocks = blocks_of(args);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const bool vec = int8_grad_vec(args);
  void (*const kernel)(Int8GradArgs) = dtype == INT8_F32    ? grad_kernel<float, false>
                                       : dtype == INT8_BF16 ? vec ? grad_kernel<__nv_bfloat16, true> : grad_kernel<__nv_bfloat16, false>
                                       : vec                ? grad_kernel<__half, true>
                                                            : grad_kernel<__half, false>;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace gb300
