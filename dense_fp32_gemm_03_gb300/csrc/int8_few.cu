// int8_few.cu -- products of 8-bit integer weights with a few tokens.
//
// Mathematics.  y[m, n] = sx[m] sw[n] sum over k of qx[m, k] qw[n, k].  Up to eight tokens the
// weights' bytes are what counts, so they go from memory to registers without a stop in shared
// memory: a lane loads 16 bytes of a row, which are its share of four m16n8k16 products (the k that a
// lane supplies can be any, if both operands take the same ones), turned to 16-bit
// floats in registers.  The sums are exact: 1024 products at a time in the 32-bit
// accumulator, then integers.  (Integer instructions are no way here: the chip's dp4a takes 5.5 cycles of
// an SM, its integer mma 27 for 16 x 8 x 32: 80 and 17 us for 8 tokens of 8192 x 8192.)
//
// Structure.  A block has 16 or 32 rows of W, and its warps take 128 columns of K in turn; each has
// 8 KB of W on the way.  Products take the tokens as 16-bit floats in the lanes' order.  A single token of
// moderate length is quantised by every block for itself, into shared memory while its first loads of W
// are on the way; others by a kernel of their own, and the first of W is requested before that is done.
#include <cuda_runtime.h>

#include <type_traits>

#include "int8_device.cuh"
#include "int8_internal.h"

namespace gb300 {
namespace {

using namespace int8;

constexpr int kStep = 64;           // columns of K of a warp's step
constexpr int kRun = 1024 / kStep;  // steps whose sums stay exact
constexpr int kMost = 8;            // tokens

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

// kR x 16 rows.  T: the tokens' type, void if they come quantised.
template <typename T, int kR, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps) few_kernel(const Int8FewArgs a) {
  constexpr int kThreads = 32 * kWarps, kAhead = 8 / kR, kXAhead = kR == 1 ? 4 : 2;
  constexpr bool kQuantise = !std::is_same<T, void>::value;
  extern __shared__ __align__(16) unsigned char s_x[];  // 16 bytes for each step, half and t
  __shared__ int sums[kWarps][kR * 4][32];
  __shared__ uint32_t s_top;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int row0 = blockIdx.x * 16 * kR, steps = (a.k + kStep - 1) / kStep;
  const int8_t* rows[kR][2];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) rows[r][h] = a.w + min(row0 + 16 * r + 8 * h + g, a.n - 1) * a.ldw + 16 * t;
  // A warp's i-th step: pairs next to one another, so that it is a whole line of a row (16384 x 16384 51.1 -> 49.8 us).
  auto step_of = [&](int i) { return (i >> 1) * (2 * kWarps) + 2 * warp + (i & 1); };
  uint4 w[kAhead][kR][2];
  auto fetch = [&](int slot, int step) {
    const bool there = kStep * step + 16 * t < a.k;  // (what follows a row's end in its 16 bytes meets zeros of x)
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[slot][r][h] = there ? load_once(rows[r][h] + int64_t(kStep) * step) : make_uint4(0, 0, 0, 0);
  };
  if constexpr (kQuantise) {
    // W may be what the kernel before wrote.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) s_top = 0;
    __syncthreads();
    const int chunks = (a.k + 7) / 8;
    auto read = [&](int c, float (&v)[8]) {
      const T* p = static_cast<const T*>(a.x) + 8 * c;
      if (a.vec && 8 * c + 8 <= a.k)
        load8<true>(p, 8, v);
      else
        load8<false>(p, a.k - 8 * c, v);
    };
    // Magnitudes compare as their bits do, NaN above infinity.
    uint32_t top = 0;
#pragma unroll 2
    for (int c = threadIdx.x; c < chunks; c += kThreads) {
      float v[8];
      read(c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) fetch(j, step_of(j));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicMax(&s_top, top);
    __syncthreads();
    const float s = row_scale(__uint_as_float(s_top)), inv = __frcp_rn(s);
#pragma unroll 2
    for (int c = threadIdx.x; c < 8 * steps; c += kThreads) {
      float v[8], n[8];
      read(c, v);
      nearest8(v, s, inv, n);
      uint4 h;
      __half2* p = reinterpret_cast<__half2*>(&h);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = __floats2half2_rn(n[2 * e] - kRound, n[2 * e + 1] - kRound);
      reinterpret_cast<uint4*>(s_x)[((c >> 3) * 2 + (c & 1)) * 4 + (c & 7) / 2] = h;
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) fetch(j, step_of(j));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }

  // Lanes of tokens that are not there keep zeros.
  const uint4* x = (kQuantise ? reinterpret_cast<const uint4*>(s_x) : static_cast<const uint4*>(a.x)) + lane;
  constexpr int kPitch = kQuantise ? 4 : 32;  // of a half
  uint4 b[kXAhead][2] = {};
  auto fetch_x = [&](int slot, int step) {
    if (g < a.tokens && step < steps) {
#pragma unroll
      for (int h = 0; h < 2; ++h) b[slot][h] = x[(2 * step + h) * kPitch];
    }
  };
#pragma unroll
  for (int j = 0; j < kXAhead; ++j) fetch_x(j, step_of(j));
  float acc[kR][4] = {};
  int total[kR][4] = {}, run = 0;
  auto flush = [&]() {
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[r][i] += __float2int_rn(acc[r][i]), acc[r][i] = 0.f;
  };
#pragma unroll 1
  for (int base = 0; step_of(base) < steps; base += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (step_of(base + j) >= steps) break;
      const uint4 b0 = b[j % kXAhead][0], b1 = b[j % kXAhead][1];
      const uint32_t xs[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const uint32_t lo[4] = {w[j][r][0].x, w[j][r][0].y, w[j][r][0].z, w[j][r][0].w};
        const uint32_t hi[4] = {w[j][r][1].x, w[j][r][1].y, w[j][r][1].z, w[j][r][1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t p = lo[i] ^ 0x80808080u, q = hi[i] ^ 0x80808080u;
          mma(acc[r], to_f16<0>(p), to_f16<0>(q), to_f16<1>(p), to_f16<1>(q), xs[2 * i], xs[2 * i + 1]);
        }
      }
      fetch(j, step_of(base + j + kAhead));
      fetch_x(j % kXAhead, step_of(base + j + kXAhead));
    }
    if ((run += kAhead) == kRun) run = 0, flush();
  }
  flush();
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][4 * r + i][lane] = total[r][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * kR * a.tokens; i += kThreads) {
    const int row = i % (16 * kR), m = i / (16 * kR);
    if (row0 + row >= a.n) continue;
    const float sw = a.scale_w[row0 + row], sx = kQuantise ? row_scale(__uint_as_float(s_top)) : a.scale_x[m];
    int sum = 0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += sums[v][row / 16 * 4 + (row / 8 % 2) * 2 + m % 2][row % 8 * 4 + m / 2];
    const float v = scaled(sum, sw, sx);
    const int64_t to = m * a.ldy + row0 + row;
    if (a.dtype == INT8_F32)
      static_cast<float*>(a.y)[to] = v;
    else if (a.dtype == INT8_BF16)
      static_cast<__nv_bfloat16*>(a.y)[to] = __float2bfloat16_rn(v);
    else
      static_cast<__half*>(a.y)[to] = __float2half_rn(v);
  }
}

typedef void (*Kernel)(Int8FewArgs);
template <typename T, int kR>
Kernel by_warps(int warps) {
  return warps == 4 ? few_kernel<T, kR, 4> : warps == 8 ? few_kernel<T, kR, 8> : few_kernel<T, kR, 16>;
}

}  // namespace

int int8_few_tokens() { return kMost; }

// As many warps a block as leave all blocks at work at once, 16 warps on an SM (5000 x 4096 in 313 blocks of eight warps
// takes 9.6 us, 4096 x 4096 in 256 7.1): 4096 rows are 256 blocks of eight warps, 8192 rows 512 of four.  Beyond four tokens a
// block has 32 rows, so that its tokens are half as many bytes as its weights, where that leaves 200 blocks (8 tokens of
// 8192 x 8192 18.2 -> 16.5 us; of 1024 x 8192, 32 blocks, 7 -> 10).
static int64_t block_rows(int64_t tokens, int64_t n) { return tokens > 4 && n >= 32 * 200 ? 32 : 16; }
static int block_warps(int64_t tokens, int64_t n, int sms) {
  const int64_t blocks = (n + block_rows(tokens, n) - 1) / block_rows(tokens, n);
  return blocks <= sms ? 16 : blocks <= 2 * sms ? 8 : 4;
}

// Up to 16 values a thread (1024 x 1024: 2.9 us in a graph, 4.0 with a kernel before; 4096 x 4096: 7.5 and 7.3, but 1.5 us
// less of host time; 8192 x 8192, 64 a thread: 17.7 and 16.3).
bool int8_few_quantises(int64_t tokens, int64_t n, int64_t k, int sms) {
  return tokens == 1 && k <= 16 * 32 * block_warps(1, n, sms);
}

cudaError_t launch_int8_few(int type_x, const Int8FewArgs& args, int sms, cudaStream_t stream) {
  const int warps = block_warps(args.tokens, args.n, sms);
  const int64_t rows = block_rows(args.tokens, args.n), blocks = (args.n + rows - 1) / rows;
  const Kernel kernel = rows == 32 ? by_warps<void, 2>(warps)
                        : type_x < 0 ? by_warps<void, 1>(warps)
                        : type_x == INT8_F32 ? by_warps<float, 1>(warps)
                        : type_x == INT8_BF16 ? by_warps<__nv_bfloat16, 1>(warps) : by_warps<__half, 1>(warps);
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks), 1, 1);
  cfg.blockDim = dim3(32 * warps, 1, 1);
  cfg.dynamicSmemBytes = type_x < 0 ? 0 : size_t((args.k + kStep - 1) / kStep) * kStep * 2;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace gb300
