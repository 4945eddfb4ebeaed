// int8_convert.cu -- conversions of the 8-bit integer operators: rows to
// integers and back, operands of the products, checkpoints, and the gated
// activation that keeps its inputs in 8 bits.
//
// All of them are bound by memory: each element is read once and written once.  A
// thread takes eight consecutive values (16 bytes of 16-bit types, 8 of integers) at a time.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "int8_device.cuh"
#include "int8_internal.h"

namespace gb300 {
namespace {

using namespace int8;

constexpr int kThreads = 256;
constexpr int kPer = 2;  // chunks that a thread has on the way where it does little else

bool aligned16(const void* p, int64_t ld_bytes) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld_bytes % 16 == 0; }

// Waits for the kernel before on the stream; the next one may then set itself up beside this one.
__device__ __forceinline__ void begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int threads, cudaStream_t stream, const A&... args) {
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid), 1, 1);
  cfg.blockDim = dim3(unsigned(threads), 1, 1);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

#define GB300_INT8_BY_TYPE(dtype, call)      \
  switch (dtype) {                           \
    case INT8_F32: {                         \
      using T = float;                       \
      return call;                           \
    }                                        \
    case INT8_BF16: {                        \
      using T = __nv_bfloat16;               \
      return call;                           \
    }                                        \
    default: {                               \
      using T = __half;                      \
      return call;                           \
    }                                        \
  }

// ------------------------------------------------------------------------- rows
enum RowForm { kBytes, kWide };  // integers as bytes, or as 16-bit floats

struct RowArgs {
  const void* x;
  int64_t ldx;
  int64_t rows, cols;
  void* out;
  int64_t ld;  // of out, in its elements
  float* scales;
};

// kGroup threads to a row: the row's first 32 kGroup values stay in registers, as they are in memory, between
// the search for the largest and the rounding; the rest is read again (from L2).
template <typename T, int kGroup, RowForm kForm, bool kVec>
__global__ void __launch_bounds__(kGroup <= 32 ? kThreads : kGroup) rows_kernel(const RowArgs a) {
  begin();
  constexpr int kRows = kGroup <= 32 ? kThreads / kGroup : 1, kKept = 4;
  const int t = threadIdx.x % kGroup;
  const int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kGroup;
  if (kGroup <= 32 && row >= a.rows) return;  // whole warps
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const int cols = int(a.cols), chunks = (cols + 7) / 8;
  Eight<T> kept[kKept];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int c = t + i * kGroup;
    if constexpr (kVec) {
      if (c < chunks)
        kept[i] = reinterpret_cast<const Eight<T>*>(x)[c];
      else
        kept[i] = Eight<T>{};
    } else {
      T* to = reinterpret_cast<T*>(&kept[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) to[e] = 8 * c + e < cols ? x[8 * c + e] : from_f32<T>(0.f);
    }
  }
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    float v[8];
    values(kept[i], v);
    top = max_abs(top, largest8(v));
  }
#pragma unroll 1
  for (int c = t + kKept * kGroup; c < chunks; c += kGroup) {
    float v[8];
    load8<kVec>(x + 8 * c, cols - 8 * c, v);
    top = max_abs(top, largest8(v));
  }
#pragma unroll
  for (int d = 16; d; d /= 2) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, d));
  if constexpr (kGroup > 32) {
    __shared__ float warps[kGroup / 32];
    if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = top;
    __syncthreads();
    top = warps[threadIdx.x % 32 % (kGroup / 32)];  // (each of them in some lane)
#pragma unroll
    for (int d = 16; d; d /= 2) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, d));
  }
  const float s = row_scale(top), inv = __frcp_rn(s);
  if (t == 0) a.scales[row] = s;
  const int out_chunks = kForm == kBytes ? (cols + 15) / 16 * 2 : chunks;
  auto write = [&](int c, const float (&w)[8]) {
    float n[8];
    nearest8(w, s, inv, n);
    if constexpr (kForm == kBytes) {
      *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.out) + row * a.ld + 8 * c) = pack8(n);
    } else {
      uint4 h;
      __half2* p = reinterpret_cast<__half2*>(&h);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = __floats2half2_rn(n[2 * e] - kRound, n[2 * e + 1] - kRound);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * a.ld + 8 * c) = h;
    }
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int c = t + i * kGroup;
    if (c < out_chunks) {
      float v[8];
      values(kept[i], v);
      write(c, v);
    }
  }
#pragma unroll 1
  for (int c = t + kKept * kGroup; c < out_chunks; c += kGroup) {
    float v[8];
    if (kVec && c >= chunks) {  // zeros that fill up
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    } else {
      load8<kVec>(x + 8 * c, cols - 8 * c, v);
    }
    write(c, v);
  }
}

// Whether the kernels read and write 16 bytes at a time: rows start at multiples of 16 bytes and hold whole chunks.
bool whole(int64_t cols, bool aligned) { return aligned && cols % 8 == 0; }

// As few threads to a row as keep all of it.
template <typename T, RowForm kForm, bool kVec>
cudaError_t launch_rows_of(const RowArgs& a, cudaStream_t stream) {
  if (a.cols <= 1024) return launch(rows_kernel<T, 32, kForm, kVec>, (a.rows + kThreads / 32 - 1) / (kThreads / 32), kThreads, stream, a);
  if (a.cols <= 2048) return launch(rows_kernel<T, 64, kForm, kVec>, a.rows, 64, stream, a);
  if (a.cols <= 4096) return launch(rows_kernel<T, 128, kForm, kVec>, a.rows, 128, stream, a);
  if (a.cols <= 6144) return launch(rows_kernel<T, 192, kForm, kVec>, a.rows, 192, stream, a);
  if (a.cols <= 8192) return launch(rows_kernel<T, 256, kForm, kVec>, a.rows, 256, stream, a);
  return launch(rows_kernel<T, 1024, kForm, kVec>, a.rows, 1024, stream, a);
}
template <RowForm kForm>
cudaError_t launch_rows(int dtype, const RowArgs& a, bool vec, cudaStream_t stream) {
  GB300_INT8_BY_TYPE(dtype, (vec ? launch_rows_of<T, kForm, true>(a, stream) : launch_rows_of<T, kForm, false>(a, stream)))
}

// A matrix's chunks of eight columns, divided into one run of consecutive chunks for each block.
struct Chunks {
  int64_t all, per_block;
  int64_t row_chunks;
  Divider div;
};
// This thread's kPer chunks in each step of its block's run.
template <int kPer>
struct Walk {
  int64_t row0, left;
  uint32_t c0;

  __device__ __forceinline__ explicit Walk(const Chunks& n) {
    const int64_t first = int64_t(blockIdx.x) * n.per_block;
    row0 = first / n.row_chunks;
    c0 = uint32_t(first - row0 * n.row_chunks);
    left = min(n.per_block, n.all - first);
  }
  // Whether this thread has a j-th one; its row and its place in the row.
  __device__ __forceinline__ bool at(const Chunks& n, int j, int64_t& row, int64_t& c) const {
    const uint32_t i = c0 + threadIdx.x + j * kThreads, r = divide(i, n.div);
    row = row0 + r;
    c = i - r * n.div.d;
    return threadIdx.x + j * kThreads < left;
  }
  __device__ __forceinline__ void next(const Chunks& n) {
    const uint32_t i = c0 + kPer * kThreads, r = divide(i, n.div);
    row0 += r;
    c0 = i - r * n.div.d;
    left -= kPer * kThreads;
  }
};

struct BackArgs {
  const int8_t* codes;
  int64_t ld;
  const float* scales;
  int64_t rows, cols;
  void* out;
  int64_t ld_out;
  Chunks n;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const BackArgs a) {
  begin();
  __shared__ __align__(16) float scratch_[kVec ? 4 : 8 * kThreads];
  float* const scratch = scratch_ + (kVec ? 0 : threadIdx.x / 32 * 256);
  for (Walk<1> w(a.n); w.left > 0; w.next(a.n)) {
    int64_t row, c;
    const bool here = w.at(a.n, 0, row, c);
    float v[8] = {};
    if (here) {
      const uint2 q = *reinterpret_cast<const uint2*>(a.codes + row * a.ld + 8 * c);
      const float s = a.scales[row];
      widen4(q.x, v);
      widen4(q.y, v + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= s;
    }
    write8<kVec>(static_cast<T*>(a.out) + row * a.ld_out + 8 * c, here ? a.cols - 8 * c : 0, scratch, v);
  }
}

__global__ void __launch_bounds__(kThreads) widen_kernel(const BackArgs a) {
  begin();
  for (Walk<kPer> w(a.n); w.left > 0; w.next(a.n)) {
    int64_t row[kPer], c[kPer];
    bool here[kPer];
    uint2 q[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      here[j] = w.at(a.n, j, row[j], c[j]);
      if (here[j]) q[j] = *reinterpret_cast<const uint2*>(a.codes + row[j] * a.ld + 8 * c[j]);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (!here[j]) break;
      float v[8];
      widen4(q[j].x, v);
      widen4(q[j].y, v + 4);
      if (8 * c[j] + 8 > a.cols) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 8 * c[j] + e < a.cols ? v[e] : 0.f;
      }
      uint4 h;
      __half2* p = reinterpret_cast<__half2*>(&h);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row[j] * a.ld_out + 8 * c[j]) = h;
    }
  }
}

// ---------------------------------------------------------------- gradients' terms
struct SplitArgs {
  const void* x;
  int64_t ldx;
  int64_t rows, cols;
  uint16_t* out;
  int64_t ld;
  Chunks n;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) split_kernel(const SplitArgs a) {
  begin();
  for (Walk<kPer> w(a.n); w.left > 0; w.next(a.n)) {
    int64_t row[kPer], c[kPer];
    bool here[kPer];
    float v[kPer][8];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      here[j] = w.at(a.n, j, row[j], c[j]);
      if (here[j]) load8<kVec>(static_cast<const T*>(a.x) + row[j] * a.ldx + 8 * c[j], a.cols - 8 * c[j], v[j]);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (!here[j]) break;
      uint16_t* out = a.out + row[j] * a.ld + 8 * c[j];
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          uint4 term;
          uint16_t* p = reinterpret_cast<uint16_t*>(&term);
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = uint16_t(take16(v[j][e]));
          *reinterpret_cast<uint4*>(out + t * a.rows * a.ld) = term;
        }
      } else {
        store8(reinterpret_cast<T*>(out), v[j]);
      }
    }
  }
}

// ------------------------------------------------------------------ checkpoints
struct KeepArgs {
  const void* x;
  int64_t ldx;
  int64_t rows, cols;
  int8_t* codes;
  int64_t ld;
  uint16_t* units;
  int64_t ldu;
  int32_t vec;  // rows start at multiples of 16 bytes
  int32_t tiles_t;
};

// A tile of 128 tokens x 128 channels, turned in shared memory.  A thread takes eight
// channels of four tokens (a quarter of a block of 32), and writes for each channel
// a word of four tokens; the word of tokens 4 m.. of channel k is at k * 32 + (m ^ 2 (k / 8 % 16)):
// no two lanes of a warp (16 groups of channels, two m) meet in a bank, and 16-byte reads along a
// channel find their four words within one group of four.
template <typename T>
__global__ void __launch_bounds__(kThreads) keep_kernel(const KeepArgs a) {
  begin();
  constexpr bool kHalf = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
  __shared__ __align__(16) uint32_t codes[128 * 32];
  __shared__ __align__(16) uint16_t units[4][128];
  const int64_t t0 = int64_t(blockIdx.x % a.tiles_t) * 128, k0 = int64_t(blockIdx.x / a.tiles_t) * 128;
  const int g = threadIdx.x % 16;  // group of eight channels
  const T* x = static_cast<const T*>(a.x) + t0 * a.ldx + k0 + 8 * g;
  const int left_t = int(min(a.rows - t0, int64_t(128))), left_k = int(min(a.cols - k0, int64_t(128))) - 8 * g;
  auto turn = [&](auto full) {
#pragma unroll 1
    for (int m = threadIdx.x / 16; m < 32; m += kThreads / 16) {
      float v[4][8], q[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * m + i;
        if constexpr (decltype(full)::value) {
          load8<true>(x + t * a.ldx, 8, v[i]);
        } else {
          load8<false>(x + t * a.ldx, t < left_t ? left_k : 0, v[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = largest8(v[i]);
        top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const Unit u = unit_of<kHalf>(top);
        keep8(v[i], top, u.inverse, q[i]);
        if (g % 4 == 0) units[g / 4][4 * m + i] = decltype(full)::value || 4 * m + i < left_t ? uint16_t(u.bits) : 0;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        codes[(8 * g + e) * 32 + (m ^ (2 * g))] =
            pack4(__float_as_int(q[0][e]), __float_as_int(q[1][e]), __float_as_int(q[2][e]), __float_as_int(q[3][e]));
    }
  };
  if (a.vec && left_t == 128 && k0 + 128 <= a.cols)
    turn(std::true_type());
  else
    turn(std::false_type());
  __syncthreads();
  // 16 tokens of a channel a thread; `ld` covers the tokens rounded up to 16.
  const int64_t end = (a.rows + 15) / 16 * 16;
#pragma unroll
  for (int i = 0; i < 128 * 8 / kThreads; ++i) {
    const int k = (threadIdx.x + i * kThreads) / 8, p = threadIdx.x % 8, s = 2 * (k / 8);
    if (k0 + k < a.cols && t0 + 16 * p < end) {
      uint4 w = *reinterpret_cast<const uint4*>(&codes[k * 32 + ((4 * p) ^ (s & ~3))]);
      if (s & 2) w = make_uint4(w.z, w.w, w.x, w.y);
      *reinterpret_cast<uint4*>(a.codes + (k0 + k) * a.ld + t0 + 16 * p) = w;
    }
  }
  if (threadIdx.x < 64) {
    const int b = threadIdx.x / 16, p = threadIdx.x % 16;
    if (k0 + 32 * b < a.cols && t0 + 8 * p < (a.rows + 7) / 8 * 8)
      *reinterpret_cast<uint4*>(a.units + (k0 / 32 + b) * a.ldu + t0 + 8 * p) = *reinterpret_cast<const uint4*>(&units[b][8 * p]);
  }
}

struct RestoreArgs {
  const int8_t* codes;
  int64_t ld;
  const uint16_t* units;
  int64_t ldu;
  int64_t rows, cols;
  int32_t half;
  void* out;
  int64_t ld_out;
  Chunks n;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) restore_tokens_kernel(const RestoreArgs a) {
  begin();
  __shared__ __align__(16) float scratch_[kVec ? 4 : 8 * kThreads];
  float* const scratch = scratch_ + (kVec ? 0 : threadIdx.x / 32 * 256);
  for (Walk<1> w(a.n); w.left > 0; w.next(a.n)) {
    int64_t row, c;
    const bool here = w.at(a.n, 0, row, c);
    float v[8] = {};
    if (here) {
      const uint2 q = *reinterpret_cast<const uint2*>(a.codes + row * a.ld + 8 * c);
      const float u = unit_value(a.units[row * a.ldu + c / 4], a.half);
      widen4(q.x, v);
      widen4(q.y, v + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= u;
    }
    write8<kVec>(static_cast<T*>(a.out) + row * a.ld_out + 8 * c, here ? a.cols - 8 * c : 0, scratch, v);
  }
}

// Tiles of 32 channels (a block) x 64 tokens: reads 16 tokens of a channel, writes 8 channels of a token.
template <typename T, bool kVec>
__global__ void __launch_bounds__(128) restore_channels_kernel(const RestoreArgs a) {
  begin();
  __shared__ __align__(16) int8_t tile[32][68];
  __shared__ __align__(16) float scratch_[kVec ? 4 : 8 * 128];
  float* const scratch = scratch_ + (kVec ? 0 : threadIdx.x / 32 * 256);
  const int64_t blocks = (a.cols + 31) / 32, tiles = (a.rows + 63) / 64 * blocks;
  for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int64_t t0 = i / blocks * 64, b = i % blocks;
    const int k = threadIdx.x / 4, p = threadIdx.x % 4;
    int4 w = make_int4(0, 0, 0, 0);
    if (32 * b + k < a.cols && t0 + 16 * p < a.rows)
      w = *reinterpret_cast<const int4*>(a.codes + (32 * b + k) * a.ld + t0 + 16 * p);
    int32_t* to = reinterpret_cast<int32_t*>(&tile[k][16 * p]);
    to[0] = w.x, to[1] = w.y, to[2] = w.z, to[3] = w.w;
    __syncthreads();
    for (int j = threadIdx.x; j < 256; j += 128) {
      const int t = j / 4, c = j % 4;
      const bool here = t0 + t < a.rows;
      const float u = here ? unit_value(a.units[b * a.ldu + t0 + t], a.half) : 0.f;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = float(tile[8 * c + e][t]) * u;
      write8<kVec>(static_cast<T*>(a.out) + (t0 + t) * a.ld_out + 32 * b + 8 * c, here ? a.cols - 32 * b - 8 * c : 0, scratch, v);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- gated activation
struct SwigluArgs {
  const void *gate, *up;
  int64_t ldg, ldu;
  int64_t rows, cols;
  void* h;
  int64_t ldh;
  int8_t *kg, *ku;
  int64_t ldkg, ldku;
  uint16_t *ug, *uu;
  int64_t ldug, lduu;
  Chunks n;
};

// For x >= kFar.  16-bit types: the exponential of the rounded product x log2(e), within (|x| + 2) 2^-23 of itself, and a reciprocal
// within 2^-23: far below the types' own steps.  32 bits: within 2^-22.
constexpr float kFar = -80.f;
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (sizeof(T) == 4) {
    return __frcp_rn(1.f + expf(-x));
  } else {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * -1.44269504f));  // (flushed only where 1 + r is 1 anyway)
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + r));
    return r;
  }
}

// Below kFar the sigmoid is e^x, which leaves the range of 32 bits where a product with it need not (e^x times 1e38 counts
// down to x = -176): what depends on such a gate is computed again, in 64 bits, and written over, by a second pass of the
// threads that saw one.  (Each goes over its own values; what other lanes wrote for it, write8() has ordered.  fp16 cannot hold
// what comes out.)  Hardly any thread does; within the first pass it would cost that registers (8192 x 8192 bf16, back: 84 us,
// with a branch in the loop 100).
__device__ __forceinline__ double far_sigmoid(float x) {
  const double t = expf(0.5f * x);
  return t * t;
}
template <typename T>
__device__ __forceinline__ void far_swiglu(const T* gate, const T* up, T* h, int n) {
#pragma unroll 1
  for (int e = 0; e < n; ++e) {
    const float g = to_f32(gate[e]);
    if (g < kFar) h[e] = from_f32<T>(float(double(g) * far_sigmoid(g) * double(to_f32(up[e]))));
  }
}
template <typename T>
__device__ __forceinline__ void far_gradients(const T* dh, const int8_t* kg, float ug, const int8_t* ku, float uu, T* dgate, T* dup, int n) {
#pragma unroll 1
  for (int e = 0; e < n; ++e) {
    const float g = float(kg[e]) * ug, u = float(ku[e]) * uu;
    if (!(g < kFar)) continue;
    const double s = far_sigmoid(g), d = double(to_f32(dh[e])) * s;
    dgate[e] = from_f32<T>(float(d * double(u) * (1.0 + double(g) * (1.0 - s))));
    dup[e] = from_f32<T>(float(d * double(g)));
  }
}

// Keeps kN of a block's values (the block's 32 / kN lanes together); the largest magnitude of them all.
template <bool kHalf, int kN>
__device__ __forceinline__ float keep_block(const float (&v)[kN / 8][8], int8_t* codes, uint16_t* unit, bool first, bool write) {
  float top = largest8(v[0]), t[8];
  if constexpr (kN > 8) top = max_abs(top, largest8(v[1]));
  top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 1));
  if constexpr (kN == 8) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const Unit of = unit_of<kHalf>(top);
  uint2 w[kN / 8];
#pragma unroll
  for (int p = 0; p < kN / 8; ++p) {
    keep8(v[p], top, of.inverse, t);
    w[p] = pack8(t);
  }
  if constexpr (kN == 8) {
    if (write) *reinterpret_cast<uint2*>(codes) = w[0];
  } else {
    if (write) *reinterpret_cast<uint4*>(codes) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
  }
  if (write && first) *unit = uint16_t(of.bits);
  return top;
}

// 32 / kN lanes to a block; a row's columns are rounded up to whole blocks so that a block's lanes stay together.
template <typename T, bool kVec, int kN>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluArgs a) {
  begin();
  __shared__ __align__(16) float scratch_[kVec ? 4 : 8 * kThreads];
  float* const scratch = scratch_ + (kVec ? 0 : threadIdx.x / 32 * 256);
  constexpr bool kHalf = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
  constexpr int kLanes = 32 / kN;
  const int64_t blocks = (a.cols + 31) / 32;
  bool far = false;
  for (Walk<1> w(a.n); w.left > 0; w.next(a.n)) {
    int64_t row, c;
    const bool here = w.at(a.n, 0, row, c);
    const int64_t left = here ? a.cols - kN * c : 0;
    float g[kN / 8][8] = {}, u[kN / 8][8] = {}, h[8];
    if (left > 0) {
#pragma unroll
      for (int p = 0; p < kN / 8; ++p) {
        load8<kVec>(static_cast<const T*>(a.gate) + row * a.ldg + kN * c + 8 * p, left, g[p]);
        load8<kVec>(static_cast<const T*>(a.up) + row * a.ldu + kN * c + 8 * p, left, u[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < kN / 8; ++p) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = g[p][e] * sigmoid<T>(g[p][e]) * u[p][e];
      write8<kVec>(static_cast<T*>(a.h) + row * a.ldh + kN * c + 8 * p, left, scratch, h);
    }
    const bool write = here && kN * c < (a.cols + 15) / 16 * 16;
    const float top = keep_block<kHalf, kN>(g, a.kg + row * a.ldkg + kN * c, a.ug + row * a.ldug + c / kLanes, c % kLanes == 0, write);
    far = far || !(top <= -kFar);
    keep_block<kHalf, kN>(u, a.ku + row * a.ldku + kN * c, a.uu + row * a.lduu + c / kLanes, c % kLanes == 0, write);
    // Units that pad the row.
    if (here && c % kLanes == 0 && c / kLanes == blocks - 1)
      for (int64_t b = blocks; b < (blocks + 7) / 8 * 8; ++b) a.ug[row * a.ldug + b] = a.uu[row * a.lduu + b] = 0;
  }
  if constexpr (!kHalf) {
    if (!far) return;
    for (Walk<1> w(a.n); w.left > 0; w.next(a.n)) {
      int64_t row, c;
      if (w.at(a.n, 0, row, c))
        far_swiglu(static_cast<const T*>(a.gate) + row * a.ldg + kN * c, static_cast<const T*>(a.up) + row * a.ldu + kN * c,
                   static_cast<T*>(a.h) + row * a.ldh + kN * c, int(min(a.cols - kN * c, int64_t(kN))));
    }
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && kVec ? 8 : 5) swiglu_backward_kernel(const SwigluArgs a, const T* dh, int64_t lddh, T* dgate,
                                                                   int64_t lddg, T* dup, int64_t lddu) {
  begin();
  constexpr bool kHalf = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
  __shared__ __align__(16) float scratch_[kVec ? 4 : 8 * kThreads];
  float* const scratch = scratch_ + (kVec ? 0 : threadIdx.x / 32 * 256);
  bool far = false;
  for (Walk<1> w(a.n); w.left > 0; w.next(a.n)) {
    int64_t row, c;
    const bool here = w.at(a.n, 0, row, c);
    const int64_t left = here ? a.cols - 8 * c : 0;
    float d[8] = {}, g[8], u[8];
    uint2 wg = make_uint2(0, 0), wu = wg;
    float ug = 0.f, uu = 0.f;
    if (here) {
      wg = *reinterpret_cast<const uint2*>(a.kg + row * a.ldkg + 8 * c);
      wu = *reinterpret_cast<const uint2*>(a.ku + row * a.ldku + 8 * c);
      ug = unit_value(a.ug[row * a.ldug + c / 4], kHalf), uu = unit_value(a.uu[row * a.lduu + c / 4], kHalf);
      load8<kVec>(dh + row * lddh + 8 * c, left, d);
    }
    widen4(wg.x, g), widen4(wg.y, g + 4);
    widen4(wu.x, u), widen4(wu.y, u + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = g[e] * ug, s = sigmoid<T>(x);
      g[e] = d[e] * (u[e] * uu) * s * (1.f + x * (1.f - s));
      u[e] = d[e] * (x * s);
    }
    write8<kVec>(dgate + row * lddg + 8 * c, left, scratch, g);
    write8<kVec>(dup + row * lddu + 8 * c, left, scratch, u);
    far = far || !(ug <= 0.5f);  // (a block whose values are below 64 has a unit of 1/2 or less)
  }
  if constexpr (!kHalf) {
    if (!far) return;
    for (Walk<1> w(a.n); w.left > 0; w.next(a.n)) {
      int64_t row, c;
      if (!w.at(a.n, 0, row, c)) continue;
      const float ug = unit_value(a.ug[row * a.ldug + c / 4], false), uu = unit_value(a.uu[row * a.lduu + c / 4], false);
      if (!(ug <= 0.5f))
        far_gradients(dh + row * lddh + 8 * c, a.kg + row * a.ldkg + 8 * c, ug, a.ku + row * a.ldku + 8 * c, uu,
                      dgate + row * lddg + 8 * c, dup + row * lddu + 8 * c, int(min(a.cols - 8 * c, int64_t(8))));
    }
  }
}

// Rows of `row_chunks` chunks over blocks, 96 to an SM at most: with 8, which start and end together, the gated
// activation of 8192 x 8192 fp32 takes 163 us instead of 139, and 158 instead of 141 back.
Chunks chunks_of(int64_t rows, int64_t row_chunks, int sms, int per = 1) {
  Chunks n{};
  n.all = rows * row_chunks;
  n.row_chunks = row_chunks;
  n.div = divider(uint32_t(row_chunks));
  const int64_t step = int64_t(per) * kThreads, steps = (n.all + step - 1) / step, blocks = std::min(steps, int64_t(sms) * 96);
  n.per_block = (steps + blocks - 1) / blocks * step;
  return n;
}
int64_t blocks_of(const Chunks& n) { return (n.all + n.per_block - 1) / n.per_block; }
int64_t bytes_of(int dtype) { return dtype == INT8_F32 ? 4 : 2; }

}  // namespace

cudaError_t launch_int8_quantize(int dtype, const void* x, int64_t ldx, const int8_matrix_t& q, cudaStream_t stream) {
  const RowArgs a{x, ldx, q.rows, q.cols, q.codes, q.ld, q.scales};
  return launch_rows<kBytes>(dtype, a, whole(q.cols, aligned16(x, ldx * bytes_of(dtype))), stream);
}

cudaError_t launch_int8_rows16(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, uint16_t* out,
                               int64_t ld, float* scales, cudaStream_t stream) {
  const RowArgs a{x, ldx, rows, cols, out, ld, scales};
  return launch_rows<kWide>(dtype, a, whole(cols, aligned16(x, ldx * bytes_of(dtype))), stream);
}

cudaError_t launch_int8_dequantize(const int8_matrix_t& q, int dtype, void* y, int64_t ldy, int sms,
                                   cudaStream_t stream) {
  const BackArgs a{q.codes, q.ld, q.scales, q.rows, q.cols, y, ldy, chunks_of(q.rows, (q.cols + 7) / 8, sms)};
  const bool vec = whole(q.cols, aligned16(y, ldy * bytes_of(dtype)));
  GB300_INT8_BY_TYPE(dtype, launch(vec ? dequantize_kernel<T, true> : dequantize_kernel<T, false>, blocks_of(a.n), kThreads, stream, a))
}

cudaError_t launch_int8_widen(const int8_matrix_t& q, uint16_t* out, int64_t ld, int sms, cudaStream_t stream) {
  const BackArgs a{q.codes, q.ld, q.scales, q.rows, q.cols, out, ld, chunks_of(q.rows, (q.cols + 7) / 8, sms, kPer)};
  return launch(widen_kernel, blocks_of(a.n), kThreads, stream, a);
}

cudaError_t launch_int8_split(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols, uint16_t* out,
                              int64_t ld, int sms, cudaStream_t stream) {
  const SplitArgs a{x, ldx, rows, cols, out, ld, chunks_of(rows, (cols + 7) / 8, sms, kPer)};
  const bool vec = whole(cols, aligned16(x, ldx * bytes_of(dtype)));
  GB300_INT8_BY_TYPE(dtype, launch(vec ? split_kernel<T, true> : split_kernel<T, false>, blocks_of(a.n), kThreads, stream, a))
}

cudaError_t launch_int8_keep(const void* x, int64_t ldx, const int8_checkpoint_t& c, cudaStream_t stream) {
  const int64_t tiles_t = (c.rows + 127) / 128, tiles = tiles_t * ((c.cols + 127) / 128);
  const KeepArgs a{x, ldx, c.rows, c.cols, c.codes, c.ld, c.units, c.ld_units, aligned16(x, ldx * bytes_of(c.dtype)),
                   int32_t(tiles_t)};
  GB300_INT8_BY_TYPE(c.dtype, launch(keep_kernel<T>, tiles, kThreads, stream, a))
}

cudaError_t launch_int8_restore(const int8_checkpoint_t& c, int dtype, void* y, int64_t ldy, int sms,
                                cudaStream_t stream) {
  const RestoreArgs a{c.codes, c.ld, c.units, c.ld_units, c.rows, c.cols, c.dtype == INT8_F16, y, ldy,
                      chunks_of(c.rows, (c.cols + 7) / 8, sms)};
  const bool vec = whole(c.cols, aligned16(y, ldy * bytes_of(dtype)));
  if (c.order == INT8_TOKENS) {
    GB300_INT8_BY_TYPE(dtype, launch(vec ? restore_tokens_kernel<T, true> : restore_tokens_kernel<T, false>, blocks_of(a.n), kThreads, stream, a))
  }
  const int64_t tiles = std::min((c.rows + 63) / 64 * ((c.cols + 31) / 32), int64_t(sms) * 16);
  GB300_INT8_BY_TYPE(dtype, launch(vec ? restore_channels_kernel<T, true> : restore_channels_kernel<T, false>, tiles, 128, stream, a))
}

cudaError_t launch_int8_swiglu(int dtype, int64_t M, int64_t F, const void* gate, int64_t ldg, const void* up,
                               int64_t ldu, void* h, int64_t ldh, const int8_checkpoint_t& kg,
                               const int8_checkpoint_t& ku, int sms, cudaStream_t stream) {
  const int64_t es = bytes_of(dtype);
  const bool vec = whole(F, aligned16(gate, ldg * es) && aligned16(up, ldu * es) && aligned16(h, ldh * es));
  // 16 of a row's values a thread halve what it spends on addresses and on the block's largest (8192 x 8192 bf16 92 -> 82 us;
  // back, where there is less of that, 83 -> 86), where that leaves a block to each SM (33 x 1024: 1.9 -> 2.3 us).
  const int n = vec && es == 2 && F % 16 == 0 && M * F >= int64_t(sms) * kThreads * 16 ? 16 : 8;
  const SwigluArgs a{gate, up, ldg, ldu, M, F, h, ldh, kg.codes, ku.codes, kg.ld, ku.ld, kg.units, ku.units,
                     kg.ld_units, ku.ld_units, chunks_of(M, (F + 31) / 32 * (32 / n), sms)};
  GB300_INT8_BY_TYPE(dtype, launch(n == 16 ? swiglu_kernel<T, true, sizeof(T) == 2 ? 16 : 8>
                                           : vec ? swiglu_kernel<T, true, 8> : swiglu_kernel<T, false, 8>,
                                   blocks_of(a.n), kThreads, stream, a))
}

cudaError_t launch_int8_swiglu_backward(const void* dh, int64_t lddh, const int8_checkpoint_t& kg,
                                        const int8_checkpoint_t& ku, void* dgate, int64_t ldg, void* dup, int64_t ldu,
                                        int sms, cudaStream_t stream) {
  const int64_t es = bytes_of(kg.dtype);
  SwigluArgs a{};
  a.rows = kg.rows;
  a.cols = kg.cols;
  a.kg = kg.codes, a.ku = ku.codes, a.ldkg = kg.ld, a.ldku = ku.ld;
  a.ug = kg.units, a.uu = ku.units, a.ldug = kg.ld_units, a.lduu = ku.ld_units;
  const bool vec = whole(kg.cols, aligned16(dh, lddh * es) && aligned16(dgate, ldg * es) && aligned16(dup, ldu * es));
  a.n = chunks_of(kg.rows, (kg.cols + 7) / 8, sms);
  GB300_INT8_BY_TYPE(kg.dtype,
                     launch(vec ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>, blocks_of(a.n), kThreads, stream, a, static_cast<const T*>(dh), lddh,
                            static_cast<T*>(dgate), ldg, static_cast<T*>(dup), ldu))
}

}  // namespace gb300
