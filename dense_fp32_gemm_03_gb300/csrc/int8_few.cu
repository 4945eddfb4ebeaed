// int8_few.cu -- products of 8-bit integer weights with a few tokens.
//
// Mathematics.  y[m, n] = sx[m] sw[n] sum over k of qx[m, k] qw[n, k].  Up to 16 tokens the
// weights' bytes are what counts, so they go from memory to registers without a stop in shared
// memory: a lane loads 16 bytes of a row, which are its share of four m16n8k16 products (the k that a
// lane supplies can be any, if both operands take the same ones), turned to 16-bit
// floats in registers.  The sums are exact: 1024 products at a time in the 32-bit
// accumulator, then integers.  (The legacy mma serves here: a tile has 8 columns, and tensor
// memory would be two more stops on the way.)
//
// Structure.  A block has 16 or 32 rows of W, its eight warps take 64 columns of K in
// turn and add up their sums at the end.  Each warp has 64 registers of W on the
// way, the first of them before the kernel that quantises x is done.
#include <cuda_runtime.h>

#include "int8_device.cuh"
#include "int8_internal.h"

namespace gb300 {
namespace {

using namespace int8;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStep = 64;             // columns of K of a warp's step
constexpr int kRun = 1024 / kStep;    // steps whose sums stay exact
constexpr int kMost = 16;             // tokens

__device__ __forceinline__ uint4 load_once(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ void put(const Int8FewArgs& a, int token, int row, float v) {
  static_cast<T*>(a.y)[token * a.ldy + row] = from_f32<T>(v);
}

// kR x 16 rows, kT x 8 tokens.
template <int kR, int kT>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const Int8FewArgs a) {
  constexpr int kAhead = 8 / kR;  // steps on the way
  __shared__ int sums[kWarps][kR * kT * 4][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int row0 = blockIdx.x * 16 * kR, steps = (a.k + kStep - 1) / kStep, bytes = (a.k + 15) / 16 * 16;
  const int8_t* rows[kR][2];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) rows[r][h] = a.w + min(row0 + 16 * r + 8 * h + g, a.n - 1) * a.ldw + 16 * t;
  uint4 w[kAhead][kR][2];
  auto fetch = [&](int slot, int step) {
    const bool there = kStep * step + 16 * t < bytes;
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[slot][r][h] = there ? load_once(rows[r][h] + int64_t(kStep) * step) : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) fetch(j, warp + j * kWarps);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  float acc[kR][kT][4] = {};
  int total[kR][kT][4] = {};
  int run = 0;
  const uint4* x = reinterpret_cast<const uint4*>(a.x) + lane;
#pragma unroll 1
  for (int step0 = warp; step0 < steps; step0 += kAhead * kWarps) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int step = step0 + j * kWarps;
      if (step >= steps) break;
      uint32_t b[kT][8];
#pragma unroll
      for (int c = 0; c < kT; ++c) {
        const uint4 v = x[(int64_t(c) * steps + step) * 32];
        const uint32_t word[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
        for (int i = 0; i < 4; ++i) b[c][2 * i] = to_f16<0>(word[i]), b[c][2 * i + 1] = to_f16<1>(word[i]);
      }
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const uint32_t lo[4] = {w[j][r][0].x, w[j][r][0].y, w[j][r][0].z, w[j][r][0].w};
        const uint32_t hi[4] = {w[j][r][1].x, w[j][r][1].y, w[j][r][1].z, w[j][r][1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t p = lo[i] ^ 0x80808080u, q = hi[i] ^ 0x80808080u;
          const uint32_t a0 = to_f16<0>(p), a1 = to_f16<0>(q), a2 = to_f16<1>(p), a3 = to_f16<1>(q);
#pragma unroll
          for (int c = 0; c < kT; ++c) mma(acc[r][c], a0, a1, a2, a3, b[c][2 * i], b[c][2 * i + 1]);
        }
      }
      fetch(j, step + kAhead * kWarps);
      if (++run == kRun) {
        run = 0;
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
          for (int c = 0; c < kT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[r][c][i] += __float2int_rn(acc[r][c][i]), acc[r][c][i] = 0.f;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int c = 0; c < kT; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[warp][(r * kT + c) * 4 + i][lane] = total[r][c][i] + __float2int_rn(acc[r][c][i]);
  __syncthreads();
  for (int i = threadIdx.x; i < kR * kT * 128; i += kThreads) {
    const int row = i % (16 * kR), token = i / (16 * kR);
    const int at = ((row / 16) * kT + token / 8) * 4 + (row / 8 % 2) * 2 + token % 2, from = row % 8 * 4 + token % 8 / 2;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += sums[v][at][from];
    if (token < a.tokens && row0 + row < a.n) {
      const float v = scaled(sum, a.scale_w[row0 + row], a.scale_x[token]);
      if (a.dtype == INT8_F32)
        put<float>(a, token, row0 + row, v);
      else if (a.dtype == INT8_BF16)
        put<__nv_bfloat16>(a, token, row0 + row, v);
      else
        put<__half>(a, token, row0 + row, v);
    }
  }
}

}  // namespace

int int8_few_tokens() { return kMost; }

cudaError_t launch_int8_few(const Int8FewArgs& args, cudaStream_t stream) {
  const bool wide = args.tokens > 8;
  const int rows = wide ? 32 : 16;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(args.n) + rows - 1) / rows), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, wide ? few_kernel<2, 2> : few_kernel<1, 1>, args);
}

}  // namespace gb300
