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
// 8 KB of W on the way.  Tokens are integers, too, and turned to 16-bit floats in the same way (8192 x 8192 takes 15.2 us with the
// kernel that quantises, 16.2 if that one writes 16-bit floats in the lanes' order); the first of W is requested before
// that kernel is done.  A single token of moderate length is quantised by every block for itself, into shared memory
// while its first loads of W are on the way.  More tokens are taken eight by eight where the product is so small that the
// launches of the tiled kernel and of the one before it would be most of its time (300 x 520 x 200 6.1 -> 3.4 us, 128 tokens
// of 512 x 512 6.8 -> 2.7).
#include <cuda_runtime.h>

#include <type_traits>

#include "int8_device.cuh"
#include "int8_internal.h"

namespace gb300 {
namespace {

using namespace int8;

constexpr int kStep = 64;           // columns of K of a warp's step
constexpr int kRun = 1024 / kStep;  // steps whose sums stay exact
constexpr int kMost = kInt8FewTokens;

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

// kR x 16 rows, eight tokens.  T: int8_t for tokens of integers, or an unquantised one's type.
template <typename T, int kR, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps) few_kernel(const Int8FewArgs a) {
  constexpr bool kQuantise = !std::is_same<T, int8_t>::value;
  constexpr int kThreads = 32 * kWarps, kAhead = 8 / kR, kXAhead = 2 / kR;
  extern __shared__ __align__(16) unsigned char s_x[];  // 16 bytes for each step, half and t
  __shared__ int sums[kWarps][kR * 4][32];
  __shared__ uint32_t s_top;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int steps = (a.k + kStep - 1) / kStep, blocks = (a.n + 16 * kR - 1) / (16 * kR);  // of one group of tokens
  const int group = kQuantise ? 0 : blockIdx.x / blocks, row0 = (blockIdx.x - group * blocks) * 16 * kR;
  const int token0 = group * kMost, tokens = min(a.tokens - token0, kMost);
  const int8_t* rows[kR][2];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) rows[r][h] = a.w + min(row0 + 16 * r + 8 * h + g, a.n - 1) * a.ldw + 16 * t;
  // A warp's i-th step: pairs next to one another, so that it is a whole line of a row (16384 x 16384 51.1 -> 49.8 us).
  // `from`: that of an even one.
  auto step_of = [&](int from, int i) { return from + (i >> 1) * (2 * kWarps) + (i & 1); };
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
    for (int j = 0; j < kAhead; ++j) fetch(j, step_of(2 * warp, j));
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
    if (a.early) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(j, step_of(2 * warp, j));
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (!a.early) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(j, step_of(2 * warp, j));
    }
  }

  // The tokens of eight lanes each: 16 bytes of integers a step, or from shared memory twice 16 of 16-bit floats.  (A
  // token that is not there is another one, whose sums are not stored; lanes 4.. of a single one keep zeros.)
  const int8_t* x_row = kQuantise ? nullptr : static_cast<const int8_t*>(a.x) + (token0 + min(g, tokens - 1)) * a.ldx + 16 * t;
  uint4 b[kXAhead][kQuantise ? 2 : 1] = {};
  auto fetch_x = [&](int slot, int step) {
    if constexpr (kQuantise) {
      if (g == 0 && step < steps) {
#pragma unroll
        for (int h = 0; h < 2; ++h) b[slot][h] = reinterpret_cast<const uint4*>(s_x)[(2 * step + h) * 4 + t];
      }
    } else {
      const int left = a.k - kStep * step - 16 * t;  // what follows the row's end is made 0
      uint4 v = make_uint4(0, 0, 0, 0);
      if (left > 0) v = *reinterpret_cast<const uint4*>(x_row + int64_t(kStep) * step);
      if (left > 0 && left < 16) {
        auto some = [&](uint32_t word, int n) { return n <= 0 ? 0u : n >= 4 ? word : word & ((1u << 8 * n) - 1u); };
        v = make_uint4(some(v.x, left), some(v.y, left - 4), some(v.z, left - 8), some(v.w, left - 12));
      }
      b[slot][0] = v;
    }
  };
#pragma unroll
  for (int j = 0; j < kXAhead; ++j) fetch_x(j, step_of(2 * warp, j));
  float acc[kR][4] = {};
  int total[kR][4] = {}, run = 0;
  auto flush = [&]() {
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[r][i] += __float2int_rn(acc[r][i]), acc[r][i] = 0.f;
  };
#pragma unroll 1
  for (int from = 2 * warp; from < steps; from += kAhead * kWarps) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (step_of(from, j) >= steps) break;
      uint32_t xs[8];
      const uint4 v = b[j % kXAhead][0];
      if constexpr (kQuantise) {
        const uint4 u = b[j % kXAhead][1];
        xs[0] = v.x, xs[1] = v.y, xs[2] = v.z, xs[3] = v.w, xs[4] = u.x, xs[5] = u.y, xs[6] = u.z, xs[7] = u.w;
      } else {
        const uint32_t word[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
        for (int i = 0; i < 4; ++i) xs[2 * i] = to_f16<0>(word[i]), xs[2 * i + 1] = to_f16<1>(word[i]);
      }
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
      fetch(j, step_of(from, j + kAhead));
      fetch_x(j % kXAhead, step_of(from, j + kXAhead));
    }
    if ((run += kAhead) == kRun) run = 0, flush();
  }
  flush();
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][4 * r + i][lane] = total[r][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * kR * tokens; i += kThreads) {
    const int row = i % (16 * kR), m = i / (16 * kR);
    if (row0 + row >= a.n) continue;
    const float sw = a.scale_w[row0 + row], sx = kQuantise ? row_scale(__uint_as_float(s_top)) : a.scale_x[token0 + m];
    int sum = 0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += sums[v][row / 16 * 4 + (row / 8 % 2) * 2 + m % 2][row % 8 * 4 + m / 2];
    const float v = scaled(sum, sw, sx);
    const int64_t to = (token0 + m) * a.ldy + row0 + row;
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
  if constexpr (std::is_same<T, int8_t>::value) {
    if (warps == 2) return few_kernel<T, kR, 2>;
  }
  return warps == 4 ? few_kernel<T, kR, 4> : warps == 8 ? few_kernel<T, kR, 8> : few_kernel<T, kR, 16>;
}
template <typename T>
Kernel kernel_of(int64_t rows, int warps) {
  return rows == 32 ? by_warps<T, 2>(warps) : by_warps<T, 1>(warps);
}

// How W is shared out.  Up to eight tokens, as many warps a block as leave all blocks at work at once, 16 warps on an SM (5000 x
// 4096 in 313 blocks of eight warps takes 9.6 us, 4096 x 4096 in 256 6.9): 4096 rows are 256 blocks of eight warps, 8192 rows
// 256 of eight or 512 of four.  A block has 32 rows, which halves what it spends on its tokens, where that leaves 200 blocks
// (products with one token of integers, 16384 x 16384 55 -> 46.4 us, 14336 x 4096 16.2 -> 12.9; 8 tokens of 1024 x 8192, 32
// blocks, 7 -> 10).  More tokens come eight by eight, in blocks of two to eight warps (300 x 520 x 200, 646 blocks: four warps
// each 4.3 us, two 3.4).
struct Shares {
  int64_t rows, blocks;
  int warps;
};
Shares shares(int64_t tokens, int64_t n, int64_t k, int sms) {
  const int64_t groups = (tokens + kMost - 1) / kMost;
  const int64_t rows = groups == 1 ? (n >= 32 * 200 ? 32 : 16) : (n + 31) / 32 * groups >= 4 * sms ? 32 : 16;
  const int64_t blocks = (n + rows - 1) / rows * groups;
  if (groups > 1) return {rows, blocks, blocks > 4 * sms ? 2 : blocks <= 2 * sms && k > 512 ? 8 : 4};
  return {rows, blocks, blocks <= sms ? 16 : blocks <= 2 * sms ? 8 : 4};
}

}  // namespace

// Up to 16 values a thread (1024 x 1024: 2.8 us in a graph, 3.9 with a kernel before; 4096 x 4096, 6.9 us, 0.3 less, and 1.5 us
// less of host time; 8192 x 8192, 32 a thread: 15.4 and 14.6).
bool int8_few_quantises(int64_t tokens, int64_t n, int64_t k, int sms) {
  return tokens == 1 && k <= 16 * 32 * shares(1, n, k, sms).warps;
}

cudaError_t launch_int8_few(int type_x, const Int8FewArgs& args, int sms, cudaStream_t stream) {
  const Shares s = shares(args.tokens, args.n, args.k, sms);
  if (s.blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const Kernel kernel = type_x == INT8_F32    ? kernel_of<float>(s.rows, s.warps)
                        : type_x == INT8_BF16 ? kernel_of<__nv_bfloat16>(s.rows, s.warps)
                        : type_x == INT8_F16  ? kernel_of<__half>(s.rows, s.warps)
                                              : kernel_of<int8_t>(s.rows, s.warps);
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(s.blocks), 1, 1);
  cfg.blockDim = dim3(32 * s.warps, 1, 1);
  cfg.dynamicSmemBytes = type_x < 0 ? 0 : size_t((args.k + kStep - 1) / kStep) * kStep * 2;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace gb300
