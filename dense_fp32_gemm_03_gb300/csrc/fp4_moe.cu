// fp4_moe.cu -- the mixture-of-experts layer on 4-bit weights for a few
// tokens (fp4_moe in fp4.h), and the order of its weights.
//
// Mathematics.  A token takes part in `top` of the experts, so a few tokens
// touch each expert's weights for one or two columns only: the layer is bound
// by reading the weights once.  Turning each weight into a wider number in
// registers takes more instructions than the memory allows time for (an
// mma.m16n8k16 form of this kernel ran at a quarter of the bandwidth), so the
// weights go to the tensor core as they are stored, block-scaled 4-bit, and the
// activations are brought to the same form without loss that matters: a value is
// the sum of kTerms terms 8^-j u_j q_j, each the 4-bit quantisation of what the
// terms before it left, times 8: a term takes off a factor of about 8 in the mean, so
// that the units stay where they began (at least 5.6 for nvfp4 and 5 for mxfp4, so a
// block grows by 1.42 or 1.6 a term at most).  With 5 terms (bfloat16) the rest is
// about 2^-16 of the block's largest value in the mean and 2^-13 at most, with 6 (16-bit
// float) 2^-19 and 2^-16, with 8 (32 bits) 2^-25 and 2^-22.  (bfloat16 with 4 terms, 2^-13 in
// the mean, rounded a few per cent of the outputs the other way: 1 token 15.5 us, 16 tokens
// 142.2; with 5 15.9 and 142.8, with 6 16.3 and 145.0.)  A token and term is one column of
// the product, and the columns' 32-bit sums are added with their powers of 8 at the end.
//
// nvfp4's units reach from 2^-6 to 448 at full precision (2^-9 at less), so each token's
// x and h are brought near the top of that by a power of two first: blocks of 2^-10 of
// the token's largest value and more keep the precision above, smaller ones lose bits
// that lie 8^-kTerms 2^-14 below that value (h: 2^-6).  For h the largest
// value is known only after phase 2, so its power of two is a guess from the norms of the
// weights and of x, which is checked: phase 2 also keeps h in 32 bits and finds each
// token's largest value, the barrier behind it carries one bit a token that says whether
// some value was high enough and one for too high, and tokens whose guess was off are
// written again with the measured power of two (a pass over h between two more barriers: 5 us
// with 1 token of 64 experts of 2048 x 768, 10 with 16 of 4096 x 2048).
//
// What bounds it, measured.  16 tokens (nvfp4, 64 experts of 4096 x 2048, top 8: 800 MB of
// weights) take 142.5 us, 5.6 TB/s; about 10 us of that are the start, the two grid barriers
// and the last sums, between which nothing streams.  One token (64 of 2048 x 768: 22 MB) takes
// 15.9 us, a chain of latencies: the router (3 us), a barrier (1), the selection (1), the first
// weights' round to memory, sums and h (5), a barrier (1), the second products and sums (4).
#include <cuda_runtime.h>

#include "fp4_device.cuh"
#include "fp4_internal.h"
#include "fp4_stream.cuh"
#include "sgemm_device.cuh"

namespace gb300 {
namespace {

using namespace fp4;

constexpr int kPackThreads = 256;
constexpr int kThreads = 512;  // of the layer's kernel, one CTA to an SM
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 3;  // of four warps that join, activate and store
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;
constexpr int kMaxPairs = kMoeTokens * kMaxTop;
constexpr uint32_t kStatusTimeout = 3;

template <typename T>
struct Terms {
  static constexpr int kCount = 8;  // 32 bits
};
template <>
struct Terms<__nv_bfloat16> {
  static constexpr int kCount = 5;
};
template <>
struct Terms<__half> {
  static constexpr int kCount = 6;
};
static_assert(kMoeTokens * 8 <= 128, "columns of one product");
constexpr float kStep = 8.f;  // from one term to the next

// Exponents of a token's largest value once it is scaled: x's is kHigh - 1; h's is aimed at
// kAim and taken from kLow on below kHigh.  nvfp4: the block may grow 1.42 times a term and
// stays below 6 * 448 (2^7 1.42^7 = 1490, 2^8 1.42^5 = 1478); from 2^kLow down there are three
// octaves to the smallest unit of full precision.  mxfp4's units have all exponents.
template <int kFormat, int kTerms>
struct Window {
  static constexpr int kHigh = kTerms == 8 ? 7 : 8, kAim = 5, kLow = 0;
};
template <int kTerms>
struct Window<FP4_MXFP4, kTerms> {
  static constexpr int kHigh = 90, kAim = 5, kLow = -60;
};

// ------------------------------------------------------------------ packing
// One thread moves one 16-byte piece of codes, and the first threads of a row
// its scales.  A gate-and-up tile has 64 gate rows and the 64 up rows beside them.
//
// The layer multiplies an expert's down weights also by the zeros of tokens that do not go
// to it, so NaN may not enter that product: a down block whose scale is NaN is kept as
// scale 0 with every code -0 (which no other block is left with), the expert's bound is
// marked in its last bit, and the layer looks for such blocks in the rows of marked
// experts, for the tokens that go to them.
constexpr uint32_t kHidden = 0x88888888u;  // eight codes of -0

template <int kFormat>
__device__ __forceinline__ bool nan_scale(uint32_t byte) {
  return kFormat == FP4_MXFP4 ? byte == 255u : (byte & 127u) == 127u;
}

template <int kFormat, bool kGateUp>
__global__ void __launch_bounds__(kPackThreads)
    pack_experts_kernel(const fp4_matrix_t q, int64_t experts, int64_t rows_per, uint8_t* __restrict__ out,
                        uint32_t* __restrict__ bound) {
  using B = Block<kFormat>;
  const int64_t tiles = kGateUp ? (rows_per + 63) / 64 : (rows_per + 127) / 128;
  const int64_t stages = (q.cols + 255) / 256, atoms = stages * B::kAtoms;
  const int64_t pitch = (q.cols + 31) / 32 * 16;
  const int64_t items = experts * tiles * stages * 1024;
  for (int64_t i = int64_t(blockIdx.x) * kPackThreads + threadIdx.x; i < items;
       i += int64_t(gridDim.x) * kPackThreads) {
    const int piece = int(i & 7), r = int(i >> 3) & 127;
    const int64_t block = i >> 10, s = block % stages, tile = block / stages % tiles, e = block / stages / tiles;
    int64_t row;
    bool in;
    if (kGateUp) {
      const int64_t f = tile * 64 + (r & 63);
      in = f < rows_per;
      row = (2 * e + (r >> 6)) * rows_per + f;
    } else {
      const int64_t d = tile * 128 + r;
      in = d < rows_per;
      row = e * rows_per + d;
    }
    uint8_t* dst = out + block * B::kBytes;
    const int64_t at = s * 128 + piece * 16;
    uint4 codes = in && at < pitch ? *reinterpret_cast<const uint4*>(q.codes + row * q.ld + at) : make_uint4(0u, 0u, 0u, 0u);
    if (!kGateUp && in) {
      constexpr int kBlocks = 32 / Format<kFormat>::kBlock;  // of a piece
      uint32_t* w = reinterpret_cast<uint32_t*>(&codes);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const uint32_t byte = q.scales[scale_offset(row, (s * 8 + piece) * kBlocks + b, atoms)];
        bool hidden = byte == 0;
#pragma unroll
        for (int j = 0; j < 4 / kBlocks; ++j) hidden = hidden && w[b * (4 / kBlocks) + j] == kHidden;
#pragma unroll
        for (int j = 0; j < 4 / kBlocks; ++j)
          if (nan_scale<kFormat>(byte) || hidden) w[b * (4 / kBlocks) + j] = hidden ? 0u : kHidden;
      }
    }
    *reinterpret_cast<uint4*>(dst + piece_at(r, piece)) = codes;
    if (piece < B::kAtoms) {
      uint32_t four = in ? *reinterpret_cast<const uint32_t*>(q.scales + scale_offset(row, (s * B::kAtoms + piece) * 4, atoms)) : 0u;
      if (!kGateUp) {
        bool any = false;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (nan_scale<kFormat>(four >> (8 * b) & 255u)) any = true, four &= ~(255u << (8 * b));
        if (any) atomicOr(bound + e, 1u);
      }
      *reinterpret_cast<uint32_t*>(dst + 16384 + scale_at(r, piece * 4)) = four;
    }
  }
}

// Whether a row of an expert's down weights (one tile's blocks, `steps` of them) holds a hidden NaN.
template <int kFormat>
__device__ __noinline__ bool row_is_nan(const uint8_t* blocks, int row, int steps) {
  using B = Block<kFormat>;
  constexpr int kBlocks = 32 / Format<kFormat>::kBlock;
  bool found = false;
  for (int i = 0; i < steps * 8; ++i) {
    const uint8_t* block = blocks + int64_t(i >> 3) * B::kBytes;
    const uint4 codes = __ldg(reinterpret_cast<const uint4*>(block + piece_at(uint32_t(row), uint32_t(i & 7))));
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      bool hidden = true;
#pragma unroll
      for (int j = 0; j < 4 / kBlocks; ++j) hidden = hidden && w[b * (4 / kBlocks) + j] == kHidden;
      found = found || (hidden && __ldg(block + 16384 + scale_at(uint32_t(row), uint32_t((i & 7) * kBlocks + b))) == 0);
    }
  }
  return found;
}

// bound[e] = the largest |gate row| |up row| (2-norms, with the factor) of expert e, as
// bits: with the token's norm it bounds h.  The last bit is left for NaN among the down
// weights.  One warp to a pair of rows.
template <int kFormat>
__global__ void __launch_bounds__(kPackThreads)
    bound_kernel(const fp4_matrix_t q, int64_t experts, int64_t f, uint32_t* __restrict__ bound) {
  using F = Format<kFormat>;
  const int lane = threadIdx.x & 31;
  const int64_t atoms = (q.cols + 255) / 256 * F::kAtomsPerStage;
  const float g = kFormat == FP4_NVFP4 && q.factor != nullptr ? __ldg(q.factor) : 1.f;
  const int64_t warps = int64_t(gridDim.x) * (kPackThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kPackThreads / 32) + (threadIdx.x >> 5); i < experts * f; i += warps) {
    const int64_t e = i / f, row = 2 * e * f + (i - e * f);
    float sum[2] = {0.f, 0.f};
    for (int s = 0; s < 2; ++s)
      for (int64_t c = lane * 8; c < q.cols; c += 256) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q.codes + (row + s * f) * q.ld + c / 2));
        const float u = decode_scale<kFormat>(__ldg(q.scales + scale_offset(row + s * f, c / F::kBlock, atoms))) * g;
        const float2 v[4] = {__half22float2(decode2<0>(w)), __half22float2(decode2<1>(w)),
                             __half22float2(decode2<2>(w)), __half22float2(decode2<3>(w))};
        float part = 0.f;
        for (int j = 0; j < 4; ++j) part += v[j].x * v[j].x + v[j].y * v[j].y;
        sum[s] += part * u * u;
      }
    for (int s = 16; s; s >>= 1) {
      sum[0] += __shfl_xor_sync(kFull, sum[0], s);
      sum[1] += __shfl_xor_sync(kFull, sum[1], s);
    }
    if (lane == 0) atomicMax(bound + e, __float_as_uint(sqrtf(sum[0]) * sqrtf(sum[1])) & ~1u);
  }
}

// ------------------------------------------------------------------ helpers
__device__ __forceinline__ float pow2f(int e) {  // 2^e for -126 <= e <= 127
  return __uint_as_float(uint32_t(127 + e) << 23);
}

// Scale byte of a term whose block's largest magnitude has the bits `top`, and its
// unit: nearest 8-bit float to a / 6, or the smallest power of two from a / 6 up.
template <int kFormat>
__device__ __forceinline__ uint32_t term_scale(uint32_t top, float& unit) {
  if (top >= 0x7f800000u) {
    unit = 0.f;
    return kFormat == FP4_MXFP4 ? 255u : 127u;
  }
  const float s = __uint_as_float(top) * (1.f / 6.f);
  if constexpr (kFormat == FP4_MXFP4) {
    const uint32_t bits = __float_as_uint(s);
    const uint32_t byte = min((bits >> 23) + ((bits & 0x7fffffu) != 0 ? 1u : 0u), 254u);
    unit = byte == 0 ? 0.f : __uint_as_float(byte << 23);
    return byte;
  } else {
    const uint32_t byte = encode_e4m3(s);
    unit = decode_e4m3(byte);
    return byte;
  }
}

// The code of r / unit; r becomes what the term leaves, times kStep.
__device__ __forceinline__ uint32_t term_code(float& r, float unit, float inv) {
  const uint32_t code = encode2(r * inv, 0.f) & 15u;
  r = fmaf(-__low2float(decode2<0>(code)), unit, r) * kStep;
  return code;
}

// Four values of a row of activations, columns col .. col + 3, as kTerms rows of `image` (a
// block of columns) from `row` on.  A block is kBlock / 4 neighbouring lanes.
template <int kFormat, int kTerms>
__device__ __forceinline__ void write_terms(float4 x, uint8_t* image, uint32_t cols, uint32_t row, uint32_t col) {
  constexpr int kBlock = Format<kFormat>::kBlock;
  float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < kTerms; ++j, ++row) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int s = 1; s < kBlock / 4; s *= 2) top = max(top, __shfl_xor_sync(kFull, top, s));
    float unit;
    const uint32_t byte = term_scale<kFormat>(top, unit);
    const float inv = unit > 0.f ? __fdividef(1.f, unit) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= term_code(v[i], unit, inv) << (4 * i);
    *reinterpret_cast<uint16_t*>(image + piece_at(row, col >> 5) + (col & 31) / 2) = uint16_t(w);
    if (col % kBlock == 0) image[cols * 128 + scale_at(row, col / kBlock)] = uint8_t(byte);
  }
}

// The same for 32 columns from `col`, a value to a lane.
template <int kFormat, int kTerms>
__device__ __forceinline__ void write_terms_warp(float r, uint8_t* image, uint32_t cols, uint32_t row, uint32_t col,
                                                 int lane) {
  constexpr int kBlock = Format<kFormat>::kBlock;
#pragma unroll
  for (int j = 0; j < kTerms; ++j, ++row) {
    uint32_t top = __float_as_uint(r) & 0x7fffffffu;
    if constexpr (kBlock == 32) {
      top = __reduce_max_sync(kFull, top);
    } else {
#pragma unroll
      for (int s = 8; s; s >>= 1) top = max(top, __shfl_xor_sync(kFull, top, s));
    }
    float unit;
    const uint32_t byte = term_scale<kFormat>(top, unit);
    uint32_t w = term_code(r, unit, unit > 0.f ? __fdividef(1.f, unit) : 0.f);
    w |= __shfl_xor_sync(kFull, w, 1) << 4;
    w |= __shfl_xor_sync(kFull, w, 2) << 8;
    w |= __shfl_xor_sync(kFull, w, 4) << 16;
    if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(image + piece_at(row, col >> 5) + lane / 2) = w;
    if (lane % kBlock == 0) image[cols * 128 + scale_at(row, (col + lane) / kBlock)] = uint8_t(byte);
  }
}

// ------------------------------------------------------------------ routing
// Order of logits as integers: larger first; NaN last, below every number.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x7fffffffu) > 0x7f800000u ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key == 1u ? 0x7fffffffu : key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// One warp: the `top` largest of one token's logits (equal ones by index) and
// their softmax weights.  A lane keeps the logits of its experts in registers, and
// its largest at hand: a choice is two reductions over the warp.  chosen() is called with
// the experts' numbers stored, before the weights, which nobody waits for as long.
template <int kPerLane, typename Chosen>
__device__ __forceinline__ void select_top(const float* logits, int experts, int top, int renorm, int lane,
                                           uint16_t* ids, float* weight, Chosen chosen) {
  uint32_t key[kPerLane];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < experts ? order_key(__ldcg(logits + e)) : 0u;
    nan = nan || key[i] == 1u;
  }
  float exps[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) exps[i] = key[i] != 0 ? logit_of(key[i]) : -INFINITY;
  uint32_t mine_key = 0, peak_key = 0;
  int mine_id = 0;
  for (int j = 0; j < top; ++j) {
    uint32_t most = 0, at = 0;  // the lane's largest, the first of equal ones
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (key[i] > most) most = key[i], at = uint32_t(lane + 32 * i);
    const uint32_t best = __reduce_max_sync(kFull, most);
    const uint32_t id = __reduce_min_sync(kFull, most == best ? at : ~0u);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (uint32_t(lane + 32 * i) == id) key[i] = 0;
    if (j == 0) peak_key = best;
    if (lane == j) mine_key = best, mine_id = int(id);
  }
  if (lane < top) ids[lane] = uint16_t(mine_id);
  chosen(mine_id);
  const float peak = logit_of(peak_key);
  float sum = __any_sync(kFull, nan) ? __uint_as_float(0x7fffffffu) : 1.f;
  if (!renorm) {  // the sum over all experts cancels otherwise, unless it is NaN
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (lane + 32 * i < experts) sum += expf(exps[i] - peak);
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
  }
  float mine = lane < top ? expf(logit_of(mine_key) - peak) / sum : 0.f;
  if (renorm) {
    float total = mine;
    for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(kFull, total, s);
    mine /= total;
  }
  if (lane < top) weight[lane] = mine;
}

// The same for any number of experts, reading the logits again for each choice.
template <typename Chosen>
__device__ __forceinline__ void select_top_any(const float* logits, int experts, int top, int renorm, int lane,
                                               uint16_t* ids, float* weight, Chosen chosen) {
  float peak = -INFINITY, sum = 0.f;
  for (int e = lane; e < experts; e += 32) peak = fmaxf(peak, __ldcg(logits + e));
  for (int s = 16; s; s >>= 1) peak = fmaxf(peak, __shfl_xor_sync(kFull, peak, s));
  for (int e = lane; e < experts; e += 32) sum += expf(__ldcg(logits + e) - peak);
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
  uint64_t last = ~0ull;  // larger key and smaller index first
  float mine = 0.f;
  int mine_id = 0;
  for (int j = 0; j < top; ++j) {
    uint64_t best = 0;
    for (int e = lane; e < experts; e += 32) {
      const uint64_t k = uint64_t(order_key(__ldcg(logits + e))) << 32 | (0xffffffffu - uint32_t(e));
      if (k < last && k > best) best = k;
    }
    for (int s = 16; s; s >>= 1) {
      const uint64_t o = __shfl_xor_sync(kFull, best, s);
      best = o > best ? o : best;
    }
    last = best;
    const int id = int(0xffffffffu - uint32_t(best));
    if (lane == j) mine = expf(__ldcg(logits + id) - peak) / sum, mine_id = id;
  }
  if (renorm) {
    float total = mine;
    for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(kFull, total, s);
    mine /= total;
  }
  if (lane < top) {
    ids[lane] = uint16_t(mine_id);
    weight[lane] = mine;
  }
  chosen(mine_id);
}

// Four consecutive values of a row, zeros beyond `n`.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, int k, int n, bool vector) {
  if (vector && k + 4 <= n) {
    if constexpr (sizeof(T) == 4) {
      return __ldg(reinterpret_cast<const float4*>(p + k));
    } else {
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(p + k));
      const T* t = reinterpret_cast<const T*>(&r);
      return make_float4(to_f32(t[0]), to_f32(t[1]), to_f32(t[2]), to_f32(t[3]));
    }
  }
  float4 v;
  v.x = k < n ? to_f32(p[k]) : 0.f;
  v.y = k + 1 < n ? to_f32(p[k + 1]) : 0.f;
  v.z = k + 2 < n ? to_f32(p[k + 2]) : 0.f;
  v.w = k + 3 < n ? to_f32(p[k + 3]) : 0.f;
  return v;
}

// Four consecutive values as they are stored.
template <typename T>
struct Four {
  uint2 raw;
  __device__ __forceinline__ void load(const T* p) { raw = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ float4 value() const {
    const T* t = reinterpret_cast<const T*>(&raw);
    return make_float4(to_f32(t[0]), to_f32(t[1]), to_f32(t[2]), to_f32(t[3]));
  }
};
template <>
struct Four<float> {
  float4 raw;
  __device__ __forceinline__ void load(const float* p) { raw = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ float4 value() const { return raw; }
};

// ------------------------------------------------------------- grid barrier
// All CTAs are resident (cooperative launch).  `word` counts the CTAs in its low half and
// takes up the flags that they bring in its high half: flags() is called by the whole first
// warp once the CTA's threads have met, and answer[1] becomes all CTAs' flags together.
// Every thread returns the same answer: false once the bounded wait ran out.
template <typename Flags>
__device__ __forceinline__ bool grid_barrier(uint64_t* word, const MoeArgs& args, uint32_t* answer, Flags flags) {
  __syncthreads();
  if (threadIdx.x < 32) {
    const uint32_t mine = flags();
    __syncwarp();
    if (threadIdx.x == 0) {
      // The fence covers the CTA's writes, which the barrier above ordered before it.  The two
      // updates of one word stay in their order without another wait for the first to arrive.
      asm volatile("fence.acq_rel.gpu;" ::: "memory");
      if (mine != 0) asm volatile("red.relaxed.gpu.global.or.b64 [%0], %1;" ::"l"(word), "l"(uint64_t(mine) << 32) : "memory");
      asm volatile("red.relaxed.gpu.global.add.u64 [%0], %1;" ::"l"(word), "l"(uint64_t(1)) : "memory");
      uint32_t ok = 1;
      uint64_t seen;
      const uint64_t t0 = dev::global_timer_ns();
      for (;;) {
        asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(seen) : "l"(word) : "memory");
        if (uint32_t(seen) >= gridDim.x) break;
        if (dev::global_timer_ns() - t0 > args.wait_limit_ns) {
          dev::record_status(args.status, kStatusTimeout, kWaitTileStage);
          ok = 0;
          break;
        }
      }
      answer[0] = ok;
      answer[1] = uint32_t(seen >> 32);
    }
  }
  __syncthreads();
  return answer[0] != 0;
}

// -------------------------------------------------------------------- layer
// A phase's work: `units` sums of `steps` stages each, cut into runs of nearly
// equal length, one to a CTA, of kLeast stages at least where there are few.  A
// unit that is cut between CTAs is finished by the first of them.
constexpr int kLeast = 4;
struct Runs {
  int steps, count, base, extra;
  __device__ __forceinline__ Runs(int units, int steps_, int ctas) : steps(steps_) {
    const int total = units * steps, runs = min(ctas, max(total / kLeast, 1));
    base = total / runs;
    extra = total - base * runs;
    count = runs;
  }
  __device__ __forceinline__ int start(int cta) const { return min(cta, count) * base + min(min(cta, count), extra); }
  __device__ __forceinline__ int owner(int at) const {
    const int big = extra * (base + 1);
    return at < big ? at / (base + 1) : extra + (at - big) / base;
  }
};

struct Smem {
  float weight[kMoeTokens][kMaxTop];
  float gate_up[kMoeTokens][128];       // finished sums of a tile, by the expert's tokens
  float red[kWarps];
  float norm[kWarps];
  int x_exp[kMoeTokens], h_exp[kMoeTokens];  // x and h are multiplied by these powers of two
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint16_t ids[kMoeTokens][kMaxTop];
  alignas(16) uint8_t slot[kMaxPairs][kMoeTokens];  // place of an expert in use among a token's, or 255
  uint8_t nth[kMaxPairs][kMoeTokens];               // the tokens of an expert in use
  uint32_t mask[kMaxExperts];           // tokens that go to an expert
  float bound[kMaxExperts];             // log2 of MoeArgs::bound; last bit: some down weights are NaN
  uint32_t nan_down[kMoeTokens];        // which of a token's experts have such weights
  uint16_t index[kMaxExperts];          // place of an expert among those in use
  uint16_t active[kMaxPairs];           // experts in use, in order
  uint32_t h_max[kMoeTokens];           // largest |h| of this CTA's, as bits; infinity where h is known to be 0
  uint32_t tmem, top, flag[2];
  int count;
  volatile int abort;
};
constexpr int kStageArea = kSmemBytes - 1024 - int((sizeof(Smem) + 127) / 128 * 128);

// This lane's row of kTerms columns of tensor memory, as one value.
template <int kTerms>
__device__ __forceinline__ float read_terms(uint32_t taddr) {
  static_assert(kTerms <= 8 && (kMoeTokens - 1) * kTerms + 8 <= 128, "columns of an accumulator");
  float v[8];
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  float sum = v[kTerms - 1];
#pragma unroll
  for (int j = kTerms - 2; j >= 0; --j) sum = fmaf(sum, 1.f / kStep, v[j]);
  return sum;
}

// Three phases with a grid barrier between them.
//  1. Router: a CTA to an expert computes the logits of all tokens; a CTA to a
//     token turns x into terms.
//  2. Every CTA selects the experts (the same way).  Units are (expert in use,
//     64 values of h); a stage is 256 columns of x.  Where h's powers of two were guessed
//     wrong, its terms are written again, between two more barriers.
//  3. Units are 128 rows of y; the stages run over all experts in use, h of a token
//     that does not go to one being zero there.
// In phases 2 and 3 one thread streams stages (weights and columns, one bulk copy
// each), one issues the MMAs, and four warps join, activate and store.  The
// weights of phase 3's first stages are asked for before its barrier.
template <typename T, int kFormat>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const MoeArgs args) {
  using B = Block<kFormat>;
  constexpr int kTerms = Terms<T>::kCount, kBlock = Format<kFormat>::kBlock;
  using W = Window<kFormat, kTerms>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* area = smem_raw + ((1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u);
  Smem& sm = *reinterpret_cast<Smem*>(area + kStageArea);
  const int warp = uniform_warp(), lane = threadIdx.x & 31, cta = blockIdx.x, ctas = gridDim.x;
  const int tokens = args.tokens, experts = args.experts, top = args.top, d = args.d, f = args.f;
  const int d_steps = (d + 255) / 256, f_steps = (f + 255) / 256;
  const int f_tiles = (f + 63) / 64, d_tiles = (d + 127) / 128;
  uint64_t* words = reinterpret_cast<uint64_t*>(args.counters);  // of the grid barriers
  const uint32_t cols = uint32_t(args.cols), col_bytes = cols * 128 + B::kScales;
  const uint32_t stage_bytes = B::kBytes + col_bytes;
  const uint32_t stages = min(uint32_t(kStageArea) / stage_bytes, uint32_t(kMaxStages));
  const uint64_t limit = args.wait_limit_ns;

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_addr(&sm.tmem)),
                 "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      dev::mbar_init(&sm.full[s], 1);
      dev::mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      dev::mbar_init(&sm.acc_full[b], 1);
      dev::mbar_init(&sm.acc_empty[b], 4 * kGroups);
    }
    dev::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    dev::mbar_init_fence();
  }

  // ---- phase 1
  {
    for (int e = threadIdx.x; e < experts; e += kThreads) {
      sm.mask[e] = 0;
      const uint32_t b = __ldg(args.bound + e);
      sm.bound[e] = __uint_as_float((__float_as_uint(log2f(__uint_as_float(b & ~1u))) & ~1u) | (b & 1u));
    }
    if (threadIdx.x < kMoeTokens) {
      sm.h_max[threadIdx.x] = 0;
      if (cta == 0) args.h_max[threadIdx.x] = 0;
    }
    for (int i = threadIdx.x; i < kMaxPairs; i += kThreads)
      *reinterpret_cast<uint4*>(sm.slot[i]) = make_uint4(~0u, ~0u, ~0u, ~0u);
    // This CTA's shares, in both phases, are not there yet.
    for (int i = threadIdx.x; i < 2 * tokens * 64; i += kThreads)
      *reinterpret_cast<uint4*>(args.share + (int64_t(cta) * 2 + i / (tokens * 64)) * (kMoeTokens * 128) +
                                i % (tokens * 64) * 2) = make_uint4(0u, 0u, 0u, 0u);
    const T* x = static_cast<const T*>(args.x);
    const bool vec_x = (reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T))) == 0 && args.ldx % 4 == 0;
    const bool vec_r = (reinterpret_cast<uintptr_t>(args.router) & 15u) == 0 && args.ldr % 4 == 0;
    const int share = kWarps / tokens;  // warps to a token
    // CTAs to a token's terms, of those that the experts leave: each finds the token's
    // largest value and writes its part of the columns.  One more item: the spare columns.
    const int slices = max(min((ctas - experts - 1) / tokens, 4), 1);
    const int items = experts + tokens * slices + 1;
    for (int item = cta; item < items; item += ctas) {
      if (item < experts) {
        const float* r = args.router + item * args.ldr;
        float sum = 0.f;
        const int t = warp / share, part = warp % share;
        if (t < tokens) {
          const T* xt = x + t * args.ldx;
          const int step = share * 128;
          int k = (part * 32 + lane) * 4;
          if (vec_x && vec_r && d % 4 == 0) {
            // Eight pieces of both rows under way at a time.
            for (; k < d; k += 8 * step) {
              Four<T> a[8];
              float4 b[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const bool in = k + j * step < d;
                a[j].load(xt + (in ? k + j * step : 0));
                b[j] = in ? __ldg(reinterpret_cast<const float4*>(r + k + j * step)) : make_float4(0.f, 0.f, 0.f, 0.f);
              }
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 v = k + j * step < d ? a[j].value() : make_float4(0.f, 0.f, 0.f, 0.f);
                sum = fmaf(v.x, b[j].x, fmaf(v.y, b[j].y, fmaf(v.z, b[j].z, fmaf(v.w, b[j].w, sum))));
              }
            }
          } else {
            for (; k < d; k += step) {
              const float4 a = load4(xt, k, d, vec_x), b = load4(r, k, d, vec_r);
              sum = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, sum))));
            }
          }
          for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
          if (lane == 0) sm.red[warp] = sum;
        }
        __syncthreads();
        if (threadIdx.x < tokens) {
          float total = 0.f;
          for (int w = 0; w < share; ++w) total += sm.red[threadIdx.x * share + w];
          args.logits[threadIdx.x * experts + item] = total;
        }
        __syncthreads();
      } else if (item == items - 1) {
        const uint32_t spare = cols - uint32_t(tokens * kTerms);  // columns beyond the tokens' are zero
        for (int s = warp; spare != 0 && s < d_steps; s += kWarps) {
          uint8_t* image = args.x_image + int64_t(s) * col_bytes;
          for (uint32_t i = uint32_t(lane); i < spare * 8; i += 32) {
            const uint32_t row = uint32_t(tokens * kTerms) + (i >> 3), piece = i & 7;
            *reinterpret_cast<uint4*>(image + piece_at(row, piece)) = make_uint4(0u, 0u, 0u, 0u);
            if (piece < B::kAtoms) *reinterpret_cast<uint32_t*>(image + cols * 128 + scale_at(row, piece * 4)) = 0u;
          }
        }
        fence_proxy_async_all();
      } else {
        const int t = (item - experts) / slices, slice = (item - experts) - t * slices;
        const T* xt = x + t * args.ldx;
        if (threadIdx.x == 0) sm.top = 0;
        __syncthreads();
        uint32_t most = 0;
        float square = 0.f;
        for (int k = threadIdx.x * 4; k < d; k += kThreads * 4) {
          const float4 v = load4(xt, k, d, vec_x);
          most = max(max(max(most, __float_as_uint(v.x) & 0x7fffffffu), __float_as_uint(v.y) & 0x7fffffffu),
                     max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
          square += v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
        }
        most = __reduce_max_sync(kFull, most);
        for (int s = 16; s; s >>= 1) square += __shfl_xor_sync(kFull, square, s);
        if (lane == 0) {
          atomicMax(&sm.top, most);
          sm.norm[warp] = square;
        }
        __syncthreads();
        // x 2^e has its largest magnitude in [2^(kHigh - 1), 2^kHigh).
        constexpr int kTop = kFormat == FP4_NVFP4 ? W::kHigh - 1 : W::kAim;
        int e = 0;
        if (sm.top != 0 && sm.top < 0x7f800000u) e = max(min(kTop - (int(sm.top >> 23) - 127), 126), -126);
        const float scale = pow2f(e);
        const int width = (d_steps + slices - 1) / slices * 256, stop = min((slice + 1) * width, d_steps * 256);
        for (int k = slice * width + threadIdx.x * 4; k < stop; k += kThreads * 4) {
          float4 v = load4(xt, k, d, vec_x);
          v.x *= scale, v.y *= scale, v.z *= scale, v.w *= scale;
          write_terms<kFormat, kTerms>(v, args.x_image + int64_t(k >> 8) * col_bytes, cols, uint32_t(t * kTerms),
                                       uint32_t(k) & 255u);
        }
        if (warp == kWarps - 1 && slice == 0) {
          float total = lane < kWarps ? sm.norm[lane] : 0.f;
          for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(kFull, total, s);
          if (lane == 0) {
            // log2 of x's 2-norm, or of a bound where its square leaves the range of 32 bits.
            args.x_norm[t] = total > 1e-30f && total < 1e30f ? 0.5f * log2f(total)
                                                             : log2f(__uint_as_float(sm.top)) + 0.5f * log2f(float(d));
            args.x_exp[t] = e;
          }
        }
        fence_proxy_async_all();
        __syncthreads();
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  bool ok = grid_barrier(words, args, sm.flag, [] { return 0u; });
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  constexpr uint32_t tmem = kTmemBase;

  // ---- selection, the same in every CTA: the experts' numbers first, which the weights'
  // copies wait for; the softmax weights and the places of tokens beside the first copies.
  // A token to a warp from the last one down: with up to 14 tokens the producer and the MMA
  // warp take none.
  const int token = kWarps - 1 - warp;
  if (!ok) {
    for (int e = threadIdx.x; e < experts; e += kThreads) sm.mask[e] = 0;
    __syncthreads();
  } else {
    if (token < tokens) {
      const float* l = args.logits + token * experts;
      const float norm = __ldcg(args.x_norm + token);
      const int exponent = __ldcg(args.x_exp + token);
      auto chosen = [&](int e) {
        if (lane < top) atomicOr(&sm.mask[e], 1u << token);
        __syncthreads();
      };
      uint16_t* ids = sm.ids[token];
      float* weight = sm.weight[token];
      if (experts <= 64)
        select_top<2>(l, experts, top, args.renormalize, lane, ids, weight, chosen);
      else if (experts <= 128)
        select_top<4>(l, experts, top, args.renormalize, lane, ids, weight, chosen);
      else if (experts <= 256)
        select_top<8>(l, experts, top, args.renormalize, lane, ids, weight, chosen);
      else
        select_top_any(l, experts, top, args.renormalize, lane, ids, weight, chosen);
      __syncwarp();
      // |h| <= p |gate row| |up row| |x|^2.  Where the rows and x have nothing to do with one another
      // each product is about that over sqrt(d), and the largest of them eight times the usual h.
      float bound = lane < top ? sm.bound[ids[lane]] : 0.f;
      const uint32_t marked = __ballot_sync(kFull, lane < top && (__float_as_uint(bound) & 1u) != 0);
      bound = lane < top ? log2f(weight[lane]) + bound : -INFINITY;
      for (int s = 16; s; s >>= 1) bound = fmaxf(bound, __shfl_xor_sync(kFull, bound, s));
      if (lane == 0) {
        sm.nan_down[token] = marked;
        bound += 2.f * norm;
        const float e = floorf(float(W::kAim) - 3.f - bound + log2f(float(d)));
        sm.h_exp[token] = e >= -126.f && e <= 126.f ? int(e) : e > 126.f ? 126 : e < -126.f ? -126 : 0;
        if (bound == -INFINITY) sm.h_max[token] = 0x7f800000u;
        sm.x_exp[token] = exponent;
      }
      if (cta == 0 && lane < top) {
        if (args.ids) args.ids[token * top + lane] = ids[lane];
        if (args.p) args.p[token * top + lane] = weight[lane];
      }
    } else {
      __syncthreads();
    }
  }
  // The experts in use, in order: the producer's warp writes them down, the MMA warp counts.
  int used = 0;
  if (warp < 2) {
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int e = e0 + lane;
      const bool in = e < experts && sm.mask[e] != 0;
      const uint32_t vote = __ballot_sync(kFull, in);
      const int at = used + __popc(vote & ((1u << lane) - 1u));
      if (in && warp == 0) {
        sm.active[at] = uint16_t(e);
        sm.index[e] = uint16_t(at);
      }
      used += __popc(vote);
    }
    if (threadIdx.x == 0) sm.count = used;
    __syncwarp();
    asm volatile("bar.arrive 2, %0;" ::"n"(kThreads) : "memory");
  } else {
    dev::named_barrier(2, kThreads);
    used = sm.count;
    for (int i = threadIdx.x - 64; ok && i < tokens * top; i += kThreads - 64) {
      const int t = i / top, j = i - t * top, e = sm.ids[t][j], a = sm.index[e];
      sm.slot[a][t] = uint8_t(j);
      sm.nth[a][__popc(sm.mask[e] & ((1u << t) - 1u))] = uint8_t(t);
    }
    dev::named_barrier(3, kThreads - 64);
  }

  // ---- phases 2 and 3
  const Runs up(used * f_tiles, d_steps, ctas);
  const int up_begin = up.start(cta), up_end = up.start(cta + 1);
  At put, got;             // of the producer and of the MMA thread
  uint32_t runs_done = 0;  // accumulators handed over so far (MMA thread and epilogue)

  auto fail = [&]() {
    if (!sm.abort) {
      sm.abort = 1;
      dev::record_status(args.status, kStatusTimeout, kWaitTileStage);
    }
  };
  auto produce_weights = [&](const uint8_t* weights) {
    if (put.lap > 0 && !dev::mbar_wait_abortable(&sm.empty[put.slot], (put.lap - 1) & 1u, limit, &sm.abort)) fail();
    if (__shfl_sync(kFull, sm.abort, 0)) return false;
    const uint32_t e = elected();
    expect_bytes(e, &sm.full[put.slot], stage_bytes);
    load_bytes(e, area + put.slot * stage_bytes, weights, B::kBytes, &sm.full[put.slot]);
    return true;
  };
  auto produce_columns = [&](const uint8_t* columns, uint32_t slot) {
    load_bytes(elected(), area + slot * stage_bytes + B::kBytes, columns, col_bytes, &sm.full[slot]);
  };
  // Streams the stages [begin, end) of a phase.  weights(at) and columns(at) are called for
  // consecutive stages.  Phase 3's first weights, which nothing in this kernel writes, go
  // ahead of the barrier that the columns wait for.  Elsewhere each stage's columns follow its
  // weights: after a ring of weights they would arrive last (1 token 17.2 us, not 16.5; a
  // second warp for them, whose copies queue behind the same weights, 17.2 too).
  int ahead = 0;
  auto produce_ahead = [&](int begin, int end, auto& weights) {
    for (ahead = 0; ahead < int(stages) && begin + ahead < end; ++ahead) {
      if (!produce_weights(weights.next())) break;
      put.next(stages);
    }
  };
  auto produce = [&](int begin, int end, auto& weights, auto& columns) {
    fence_proxy_async_all();
    uint32_t slot = (put.slot + stages - uint32_t(ahead)) % stages;
    for (int i = 0; i < ahead; ++i) {
      produce_columns(columns.next(), slot);
      if (++slot == stages) slot = 0;
    }
    for (int at = begin + ahead; at < end; ++at) {
      if (!produce_weights(weights.next())) break;
      produce_columns(columns.next(), put.slot);
      put.next(stages);
    }
  };
  auto multiply = [&](const Runs& runs, int begin, int end) {
    for (int at = begin; at < end;) {
      const int stop = min(end, at - at % runs.steps + runs.steps);
      const uint32_t b = runs_done & 1u, nb = runs_done >> 1;
      if (nb > 0 && !dev::mbar_wait_abortable(&sm.acc_empty[b], (nb - 1) & 1u, limit, &sm.abort)) fail();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int i = at; i < stop; ++i) {
        if (!dev::mbar_wait_abortable(&sm.full[got.slot], got.lap & 1u, limit, &sm.abort)) fail();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t e = elected();
        const uint32_t base = dev::smem_addr(area + got.slot * stage_bytes);
        const uint32_t sr = tmem + 256 + got.slot * (8 * B::kAtoms), sc = sr + 4 * B::kAtoms;
        const uint64_t drs = scale_desc(base + 16384), dcs = scale_desc(base + B::kBytes + cols * 128);
#pragma unroll
        for (int a = 0; a < B::kAtoms; ++a) {
          copy_scales<1>(e, sr + 4 * a, drs + 32 * a);
          copy_scales<1>(e, sc + 4 * a, dcs + 32 * a);
        }
        const uint64_t dr = operand_desc(base), dc = operand_desc(base + B::kBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          constexpr int kPer = 4 / B::kAtoms;  // MMAs that share an atom
          const int a = j / kPer;
          mma<kFormat, 1>(e, tmem + b * 128, dr + 2 * j, dc + 2 * j,
                          instr_desc<kFormat>(128, cols, kPer == 2 ? (j & 1) * 2 : 0), sr + 4 * a, sc + 4 * a,
                          (i != at || j != 0) ? 1u : 0u);
        }
        commit<1>(e, &sm.empty[got.slot]);
        got.next(stages);
      }
      commit<1>(elected(), &sm.acc_full[b]);
      ++runs_done;
      at = stop;
    }
  };
  // The epilogue of one phase: value(unit, k, v) takes this lane's row of the finished sum of a
  // unit's k-th token, of count(unit), whose columns are token(unit, k)'s; then done(unit, n).
  // The groups of four warps take a token each in turn: one group alone waits for one token's
  // shares after another's (5 tokens 20.8 us, 17.3 with three groups; 16 tokens 148 and 141).
  const int q = warp & 3, group = (warp - 2) >> 2, row_local = 32 * q + lane, etid = threadIdx.x - 64;
  auto join = [&](const Runs& runs, int begin, int end, uint64_t* shares, auto count, auto token, auto value, auto done) {
    int unit = begin < end ? begin / runs.steps : 0;
    for (int at = begin; at < end; ++unit) {
      const int unit_at = unit * runs.steps, unit_end = unit_at + runs.steps, stop = min(end, unit_end);
      const uint32_t b = runs_done & 1u, nb = runs_done >> 1;
      if (!dev::mbar_wait_abortable(&sm.acc_full[b], nb & 1u, limit, &sm.abort)) fail();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      __syncwarp();
      const uint32_t taddr = tmem + b * 128 + (uint32_t(32 * q) << 16);
      const int n = count(unit);
      if (at != unit_at) {  // begun by another CTA: this is a share (each CTA has one such run at most)
        uint64_t* mine = shares + int64_t(cta) * 2 * (kMoeTokens * 128) + row_local;
        for (int k = group; k < n; k += kGroups)
          put_share(mine + k * 128, read_terms<kTerms>(taddr + token(unit, k) * kTerms), 1u);
      } else {
        const int c_last = stop == unit_end ? cta : runs.owner(unit_end - 1);
        // The other shares in the CTAs' order, kC under way at a time.  (With four tokens' at once,
        // which is more code, 1 token took 16.5 us, not 15.2.)
        constexpr int kC = 8;
        for (int k = group; k < n; k += kGroups) {
          float v = read_terms<kTerms>(taddr + token(unit, k) * kTerms);
          for (int c0 = cta + 1; c0 <= c_last; c0 += kC) {
            uint64_t w[kC];
            const uint64_t* from = shares + int64_t(c0) * 2 * (kMoeTokens * 128) + k * 128 + row_local;
            uint64_t t0 = 0;
            for (uint32_t tries = 0;; ++tries) {
              uint32_t missing = 0;
#pragma unroll
              for (int c = 0; c < kC; ++c)
                if (tries == 0 || uint32_t(w[c] >> 32) == 0)
                  w[c] = c0 + c <= c_last ? peek_share(from + int64_t(c) * 2 * (kMoeTokens * 128)) : uint64_t(1) << 32;
#pragma unroll
              for (int c = 0; c < kC; ++c) missing += uint32_t(w[c] >> 32) == 0 ? 1u : 0u;
              if (missing == 0) break;
              if (tries == 0) t0 = dev::global_timer_ns();
              if (sm.abort || (tries % 32 == 31 && dev::global_timer_ns() - t0 > limit)) {
                fail();
                break;
              }
            }
#pragma unroll
            for (int c = 0; c < kC; ++c)
              if (c0 + c <= c_last) v += __uint_as_float(uint32_t(w[c]));
          }
          value(unit, k, v);
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&sm.acc_empty[b]);
      ++runs_done;
      if (at == unit_at) done(unit, n);
      at = stop;
    }
  };

  // Where the stages' bytes are.  Blocks of an expert follow one another tile by tile.
  struct UpWeights {
    const uint8_t* base;
    const Smem& sm;
    int per_expert, a, left;  // blocks of an expert; expert in use; blocks of it still to come
    const uint8_t* at;
    __device__ const uint8_t* next() {
      if (left == 0) {
        ++a;
        left = per_expert;
        at = base + int64_t(sm.active[a]) * per_expert * B::kBytes;
      }
      const uint8_t* p = at;
      at += B::kBytes;
      --left;
      return p;
    }
  };
  struct DownWeights {
    const uint8_t* base;
    const Smem& sm;
    int used, tiles, steps, tile, a, left;
    const uint8_t* at;
    __device__ const uint8_t* next() {
      if (left == 0) {
        if (++a == used) a = 0, ++tile;
        left = steps;
        at = base + (int64_t(sm.active[a]) * tiles + tile) * steps * B::kBytes;
      }
      const uint8_t* p = at;
      at += B::kBytes;
      --left;
      return p;
    }
  };
  struct Columns {
    const uint8_t* base;
    uint32_t bytes;
    int steps, step;
    __device__ const uint8_t* next() {
      const uint8_t* p = base + int64_t(step) * bytes;
      if (++step == steps) step = 0;
      return p;
    }
  };

  // Phase 2, and phase 3's first weights.
  DownWeights down_weights{args.down, sm, used, d_tiles, f_steps, 0, 0, 0, nullptr};
  if (warp == 0) {
    if (up_begin < up_end) {
      const int per = f_tiles * d_steps, a = up_begin / per;
      UpWeights weights{args.gate_up, sm, per, a, per - (up_begin - a * per),
                        args.gate_up + (int64_t(sm.active[a]) * per + (up_begin - a * per)) * B::kBytes};
      Columns columns{args.x_image, col_bytes, d_steps, up_begin % d_steps};
      produce(up_begin, up_end, weights, columns);
    }
    ahead = 0;
    const Runs down(used > 0 ? d_tiles : 0, max(used * f_steps, 1), ctas);
    const int down_begin = down.start(cta), down_end = down.start(cta + 1);
    if (down_begin < down_end) {
      const int tile = down_begin / down.steps, i = down_begin - tile * down.steps, a = i / f_steps;
      down_weights.tile = tile;
      down_weights.a = a;
      down_weights.left = f_steps - (i - a * f_steps);
      down_weights.at = args.down + ((int64_t(sm.active[a]) * d_tiles + tile) * f_steps + (i - a * f_steps)) * B::kBytes;
      produce_ahead(down_begin, down_end, down_weights);
    }
  } else if (warp == 1) {
    multiply(up, up_begin, up_end);
  } else if (warp < 2 + 4 * kGroups) {
    const float factor = args.gate_up_factor ? __ldg(args.gate_up_factor) : 1.f;
    join(
        up, up_begin, up_end, args.share, [&](int unit) { return __popc(uint32_t(sm.mask[sm.active[unit / f_tiles]])); },
        [&](int unit, int k) { return int(sm.nth[unit / f_tiles][k]); },
        [&](int, int k, float v) { sm.gate_up[k][row_local] = v; },
        [&](int unit, int n) {
          dev::named_barrier(1, 128 * kGroups);
          const int a = unit / f_tiles, tile = unit - a * f_tiles;
          uint8_t* image = args.h_image + (int64_t(a) * f_steps + tile / 4) * col_bytes;
          const uint32_t col = uint32_t(tile % 4) * 64, half = uint32_t(q & 1);
          for (int k = 2 * group + (q >> 1); k < n; k += 2 * kGroups) {
            const int t = sm.nth[a][k];
            const float u = factor * pow2f(-sm.x_exp[t]);
            const float g = sm.gate_up[k][32 * half + lane] * u, up_value = sm.gate_up[k][64 + 32 * half + lane] * u;
            const int place = sm.slot[a][t];
            const float h = g / (1.f + expf(-g)) * up_value * sm.weight[t][place];
            const uint32_t most = __reduce_max_sync(kFull, __float_as_uint(h) & 0x7fffffffu);
            if (lane == 0) atomicMax(&sm.h_max[t], most);
            args.h[int64_t(t * top + place) * (f_tiles * 64) + tile * 64 + 32 * half + lane] = h;
            write_terms_warp<kFormat, kTerms>(h * pow2f(sm.h_exp[t]), image, cols, uint32_t(t * kTerms), col + 32 * half, lane);
          }
          // Zeros in the other columns, and beyond f up to the stage's end.
          const uint32_t end = tile == f_tiles - 1 ? 256 : col + 64;
          for (uint32_t row = uint32_t(etid); row < cols; row += 128 * kGroups) {
            const int t = int(row) / kTerms;
            const bool taken = t < tokens && sm.slot[a][t] != 255;
            for (uint32_t c = taken ? col + 64 : col; c < end; c += 32) {
              *reinterpret_cast<uint4*>(image + piece_at(row, c >> 5)) = make_uint4(0u, 0u, 0u, 0u);
              for (uint32_t i = 0; i < 32 / kBlock; ++i) image[cols * 128 + scale_at(row, c / kBlock + i)] = 0;
            }
          }
          dev::named_barrier(1, 128 * kGroups);  // sm.gate_up may be written again
        });
    fence_proxy_async_all();
  }
  __syncwarp();
  const Runs down(used > 0 ? d_tiles : 0, max(used * f_steps, 1), ctas);
  const int down_begin = down.start(cta), down_end = down.start(cta + 1);
  // One bit a token: some |h| reached the window (or there is nothing to check); 16 bits up: it passed it.
  auto h_flags = [&]() {
    bool seen = false, over = false;
    if (lane < tokens) {
      const uint32_t most = sm.h_max[lane];
      const int exponent = int(most >> 23) - 127 + sm.h_exp[lane];
      seen = most >= 0x7f800000u || (most != 0 && exponent >= W::kLow);
      over = most < 0x7f800000u && exponent >= W::kHigh;
    }
    return __ballot_sync(kFull, seen) | __ballot_sync(kFull, over) << 16;
  };
  if (ok && !grid_barrier(words + 1, args, sm.flag, h_flags)) ok = false;
  const uint32_t off = ok ? (~sm.flag[1] | sm.flag[1] >> 16) & ((1u << tokens) - 1u) : 0u;
  if (off != 0) {
    // The same in every CTA: h's terms again, with the tokens' largest values in [2^(kHigh - 1), 2^kHigh).
    if (threadIdx.x < tokens)
      asm volatile("red.relaxed.gpu.global.max.u32 [%0], %1;" ::"l"(args.h_max + threadIdx.x), "r"(sm.h_max[threadIdx.x])
                   : "memory");
    ok = grid_barrier(words + 2, args, sm.flag, [] { return 0u; });
  }
  if (off != 0 && ok) {
    if (threadIdx.x < tokens && (off >> threadIdx.x & 1u) != 0) {
      const uint32_t most = __ldcg(args.h_max + threadIdx.x);
      constexpr int kTop = kFormat == FP4_NVFP4 ? W::kHigh - 1 : W::kAim;
      sm.h_exp[threadIdx.x] =
          most != 0 && most < 0x7f800000u ? max(min(kTop - (int(most >> 23) - 127), 126), -126) : 0;
    }
    __syncthreads();
    const int chunks = f_tiles * 2;  // of 32 values
    const int64_t items = int64_t(tokens * top) * chunks;
    const int64_t stride = int64_t(ctas) * kWarps;
    int64_t i = int64_t(cta) * kWarps + warp;
    float ahead_h = i < items ? __ldcg(args.h + i * 32 + lane) : 0.f;  // on its way during the arithmetic
    for (; i < items; i += stride) {
      const int pair = int(i / chunks), chunk = int(i - int64_t(pair) * chunks), t = pair / top;
      const float h = ahead_h;
      if (i + stride < items) ahead_h = __ldcg(args.h + (i + stride) * 32 + lane);
      if ((off >> t & 1u) == 0) continue;
      const int a = sm.index[sm.ids[t][pair - t * top]];
      write_terms_warp<kFormat, kTerms>(h * pow2f(sm.h_exp[t]), args.h_image + (int64_t(a) * f_steps + chunk / 8) * col_bytes,
                                        cols, uint32_t(t * kTerms), uint32_t(chunk % 8) * 32, lane);
    }
    fence_proxy_async_all();
    ok = grid_barrier(words + 3, args, sm.flag, [] { return 0u; });
  }
  if (!ok) sm.abort = 1;

  // Phase 3.
  if (warp == 0) {
    if (down_begin < down_end) {
      Columns columns{args.h_image, col_bytes, down.steps, down_begin % down.steps};
      produce(down_begin, down_end, down_weights, columns);
    }
  } else if (warp == 1) {
    multiply(down, down_begin, down_end);
    commit<1>(elected(), &sm.drain);
    dev::mbar_wait(&sm.drain, 0u, limit);
  } else if (warp < 2 + 4 * kGroups) {
    const float factor = args.down_factor ? __ldg(args.down_factor) : 1.f;
    join(
        down, down_begin, down_end, args.share + kMoeTokens * 128, [&](int) { return tokens; }, [&](int, int k) { return k; },
        [&](int unit, int k, float v) {
          const int row = unit * 128 + row_local;
          for (uint32_t m = sm.nan_down[k]; m != 0 && row < d; m &= m - 1) {
            const int64_t e = sm.ids[k][__ffs(int(m)) - 1];
            if (row_is_nan<kFormat>(args.down + (e * d_tiles + unit) * f_steps * B::kBytes, row_local, f_steps))
              v = __uint_as_float(0x7fffffffu);
          }
          if (row < d) static_cast<T*>(args.y)[k * args.ldy + row] = from_f32<T>(v * factor * pow2f(-sm.h_exp[k]));
        },
        [&](int, int) {});
  }
  __syncwarp();
  if (sm.abort && threadIdx.x == 0) {
    // Copies still under way get a bounded time to land before the CTA's memory goes.
    const uint64_t t0 = dev::global_timer_ns();
    while (dev::global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
  // The last CTA to leave clears the barriers' counters for the next call.
  if (threadIdx.x == 0 && atomicAdd(args.counters + 8, 1) == ctas - 1) {
    words[0] = words[1] = words[2] = words[3] = 0;
    args.counters[8] = 0;
  }
}

const void* moe_instance(int dtype, int format) {
  const bool mx = format == FP4_MXFP4;
  auto pointer = [](auto* k) { return reinterpret_cast<const void*>(k); };
  switch (dtype) {
    case FP4_F32: return mx ? pointer(&moe_kernel<float, FP4_MXFP4>) : pointer(&moe_kernel<float, FP4_NVFP4>);
    case FP4_BF16:
      return mx ? pointer(&moe_kernel<__nv_bfloat16, FP4_MXFP4>) : pointer(&moe_kernel<__nv_bfloat16, FP4_NVFP4>);
    default: return mx ? pointer(&moe_kernel<__half, FP4_MXFP4>) : pointer(&moe_kernel<__half, FP4_NVFP4>);
  }
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

int64_t block_bytes(int format) { return format == FP4_MXFP4 ? Block<FP4_MXFP4>::kBytes : Block<FP4_NVFP4>::kBytes; }

int64_t gate_up_blocks(int64_t experts, int64_t d, int64_t f) { return experts * ((f + 63) / 64) * ((d + 255) / 256); }
int64_t down_blocks(int64_t experts, int64_t d, int64_t f) { return experts * ((d + 127) / 128) * ((f + 255) / 256); }

int terms_of(int dtype) {
  return dtype == FP4_F32 ? Terms<float>::kCount : dtype == FP4_BF16 ? Terms<__nv_bfloat16>::kCount : Terms<__half>::kCount;
}

}  // namespace

int64_t fp4_gate_up_bytes(int format, int64_t experts, int64_t d, int64_t f) {
  return gate_up_blocks(experts, d, f) * block_bytes(format) + (experts + 3) / 4 * 16;
}
int64_t fp4_down_bytes(int format, int64_t experts, int64_t d, int64_t f) {
  return down_blocks(experts, d, f) * block_bytes(format);
}
const uint32_t* fp4_expert_bounds(const fp4_experts_t& w) {
  return reinterpret_cast<const uint32_t*>(w.gate_up + gate_up_blocks(w.experts, w.d, w.f) * block_bytes(w.format));
}

MoeScratch fp4_moe_scratch(int dtype, int format, int64_t tokens, int64_t experts, int64_t d, int64_t f, int64_t top,
                           int sms) {
  MoeScratch s{};
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += round_up(size_t(bytes));
    return here;
  };
  const int64_t used = experts < tokens * top ? experts : tokens * top;
  s.cols = int((tokens * terms_of(dtype) + 15) / 16 * 16);
  const int64_t col_bytes = s.cols * 128 + block_bytes(format) - 16384;
  s.logits = take(tokens * experts * 4);
  s.x_exp = take(tokens * 4);
  s.x_norm = take(tokens * 4);
  s.h_max = take(kMoeTokens * 4);
  s.h = take(tokens * top * ((f + 63) / 64) * 64 * 4);
  s.x_image = take((d + 255) / 256 * col_bytes);
  s.h_image = take(used * ((f + 255) / 256) * col_bytes);
  s.share = take(int64_t(sms) * 2 * kMoeTokens * 128 * 8);
  s.bytes = at;
  return s;
}

cudaError_t launch_fp4_experts_pack(const fp4_matrix_t& gate_up, const fp4_matrix_t& down,
                                    const fp4_experts_t& w, cudaStream_t stream) {
  auto grid = [](int64_t items) {
    const int64_t b = (items + kPackThreads - 1) / kPackThreads;
    return unsigned(b < (1 << 20) ? b : (1 << 20));
  };
  uint32_t* bound = const_cast<uint32_t*>(fp4_expert_bounds(w));
  const cudaError_t e = cudaMemsetAsync(bound, 0, size_t(w.experts) * 4, stream);
  if (e != cudaSuccess) return e;
  const unsigned up = grid(gate_up_blocks(w.experts, w.d, w.f) * 1024), dn = grid(down_blocks(w.experts, w.d, w.f) * 1024);
  const unsigned bd = grid(w.experts * w.f * 32);
  if (w.format == FP4_MXFP4) {
    pack_experts_kernel<FP4_MXFP4, true><<<up, kPackThreads, 0, stream>>>(gate_up, w.experts, w.f, w.gate_up, nullptr);
    bound_kernel<FP4_MXFP4><<<bd, kPackThreads, 0, stream>>>(gate_up, w.experts, w.f, bound);
    pack_experts_kernel<FP4_MXFP4, false><<<dn, kPackThreads, 0, stream>>>(down, w.experts, w.d, w.down, bound);
  } else {
    pack_experts_kernel<FP4_NVFP4, true><<<up, kPackThreads, 0, stream>>>(gate_up, w.experts, w.f, w.gate_up, nullptr);
    bound_kernel<FP4_NVFP4><<<bd, kPackThreads, 0, stream>>>(gate_up, w.experts, w.f, bound);
    pack_experts_kernel<FP4_NVFP4, false><<<dn, kPackThreads, 0, stream>>>(down, w.experts, w.d, w.down, bound);
  }
  return cudaGetLastError();
}

bool fp4_moe_prepare() {
  for (int dtype = FP4_F32; dtype <= FP4_F16; ++dtype)
    for (int format = FP4_MXFP4; format <= FP4_NVFP4; ++format)
      if (cudaFuncSetAttribute(moe_instance(dtype, format), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
          cudaSuccess)
        return false;
  return true;
}

cudaError_t launch_fp4_moe(int dtype, int format, const MoeArgs& args, int sms, cudaStream_t stream) {
  MoeArgs copy = args;
  void* params[] = {&copy};
  return cudaLaunchCooperativeKernel(moe_instance(dtype, format), dim3(unsigned(sms)), dim3(kThreads), params, kSmemBytes,
                                     stream);
}

}  // namespace gb300
