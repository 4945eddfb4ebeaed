// int8_device.cuh -- device helpers of the 8-bit integer operators: loads of
// eight values, quantisation of a row's and of a block's values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fp4_device.cuh"
#include "int8.h"

namespace gb300 {
namespace int8 {

using fp4::from_f32;
using fp4::max_abs;
using fp4::to_f32;

constexpr int kBlock = 32;  // channels that share a checkpoint's unit

// Eight consecutive values as they are in memory.
template <typename T>
struct alignas(16) Eight {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void values(const Eight<T>& x, float (&v)[8]) {
  const T* t = reinterpret_cast<const T*>(&x);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
}

// Eight consecutive values from p on in 32 bits, of which `left` exist (the others are 0).  kVec: p is 16-byte aligned and all exist.
template <bool kVec, typename T>
__device__ __forceinline__ void load8(const T* p, int64_t left, float (&v)[8]) {
  if constexpr (kVec) {
    Eight<T> x;  // (read as vectors: values() of the memory itself would read one element at a time)
#pragma unroll
    for (uint32_t i = 0; i < sizeof(T) / 2; ++i) x.w[i] = reinterpret_cast<const uint4*>(p)[i];
    values(x, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  Eight<T> x;
  T* t = reinterpret_cast<T*>(&x);
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = from_f32<T>(v[i]);
#pragma unroll
  for (uint32_t i = 0; i < sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = x.w[i];
}

// The same for rows that start anywhere, by whole warps: each lane's eight values pass through `scratch`, 256 numbers of the
// warp's, so that 32 elements after one another are written at a time and not every eighth (dequantising 16384 x 4097
// bfloat16 177 -> 61 us).  Reads are better off with every eighth, which the L1 cache serves (quantising it 55 to 65 us, with
// reads like this 123).  `left` may be anything; lanes of none do not touch memory.
template <typename T>
__device__ __forceinline__ void scatter8(T* p, int64_t left, float* scratch, const float (&v)[8]) {
  const int lane = threadIdx.x % 32, mine = int(max(int64_t(0), min(left, int64_t(8))));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(scratch + 8 * lane)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int owner = 4 * i + lane / 8, n = __shfl_sync(0xffffffffu, mine, owner);
    T* to = reinterpret_cast<T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), owner));
    if (lane % 8 < n) to[lane % 8] = from_f32<T>(scratch[32 * i + lane]);
  }
  __syncwarp();
}
// Whichever of the two a kernel takes.
template <bool kVec, typename T>
__device__ __forceinline__ void write8(T* p, int64_t left, float* scratch, const float (&v)[8]) {
  if constexpr (!kVec)
    scatter8(p, left, scratch, v);
  else if (left > 0)
    store8(p, v);
}

__device__ __forceinline__ float largest8(const float (&v)[8]) {
  return max_abs(max_abs(max_abs(v[0], v[1]), max_abs(v[2], v[3])), max_abs(max_abs(v[4], v[5]), max_abs(v[6], v[7])));
}

__device__ __forceinline__ bool finite(float a) { return __float_as_uint(a) < 0x7f800000u; }  // of a >= 0

// The integer nearest to x / s, ties to even, for |x| <= 127 s (1 + 2^-22) and s >= 2^-126,
// with inv the rounded reciprocal of s.  x inv is within 2^-15 of x / s, so its nearest
// integer n is the answer or next to it, and the remainder x - n s says which: it is a
// multiple of the last place of s and at most s, so that the fma gives it exactly.  Twice the remainder is exact too; half of
// s would not be below 2^-125.
__device__ __forceinline__ int nearest(float x, float s, float inv) {
  const float n = rintf(x * inv), r = fmaf(-n, s, x), d = fabsf(r) + fabsf(r);
  int q = int(n);
  if (d > s || (d == s && (q & 1))) q += r > 0.f ? 1 : -1;
  return q;
}

// A row's scale (NaN unless every value is finite) from its largest magnitude.
__device__ __forceinline__ float row_scale(float a) {
  return finite(a) ? fmaxf(a * (1.f / 127.f), 0x1p-126f) : __uint_as_float(0x7fffffffu);
}

// Four integers in bytes, the first lowest.
__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return __byte_perm(__byte_perm(uint32_t(a), uint32_t(b), 0x0040), __byte_perm(uint32_t(c), uint32_t(d), 0x0040), 0x5410);
}

// A block's unit from its largest magnitude.
struct Unit {
  uint32_t bits;  // bfloat16, or a 16-bit float (exponents -24 to 9: subnormal below -14)
  float inverse;  // what values are multiplied by before they are rounded (exact): 0 where the block is not finite
};
template <bool kHalf>
__device__ __forceinline__ Unit unit_of(float a) {
  const int e = max(int(__float_as_uint(a) >> 23) - 127 - 6, kHalf ? -24 : -126);  // the field of a subnormal clamps too
  Unit u;
  u.bits = kHalf ? (e >= -14 ? uint32_t(e + 15) << 10 : 1u << (e + 24)) : uint32_t(e + 127) << 7;
  u.inverse = __uint_as_float(uint32_t(127 - e) << 23);
  if (!finite(a)) u.bits = kHalf ? 0x7e00u : 0x7fc0u, u.inverse = 0.f;
  return u;
}
__device__ __forceinline__ float unit_value(uint32_t bits, bool half) {
  return half ? __half2float(__ushort_as_half(uint16_t(bits))) : __uint_as_float(bits << 16);
}

// 3 * 2^22: a number up to 2^22 in magnitude that is added to it is rounded to the nearest integer, ties to
// even, which the low bits of the sum then hold.  (A conversion instruction has an eighth of the rate of an addition.)
constexpr float kRound = 12582912.f;

__device__ __forceinline__ uint2 pack8(const float (&t)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = pack4(__float_as_int(t[4 * i]), __float_as_int(t[4 * i + 1]), __float_as_int(t[4 * i + 2]), __float_as_int(t[4 * i + 3]));
  return make_uint2(w[0], w[1]);
}

// Eight values of a block whose largest magnitude is `top`, as integers on kRound.
__device__ __forceinline__ void keep8(const float (&v)[8], float top, float inverse, float (&t)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = fmaf(v[e], inverse, kRound);
  if (!(top * inverse < 127.5f)) {  // one may round to 128, or the block is not finite
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = finite(top) ? fminf(fmaxf(t[e], kRound - 127.f), kRound + 127.f) : kRound;
  }
}

// Eight values of a row of scale s, as integers on kRound.  x inv is within 2^-16 of x / s, so its nearest integer
// is the answer unless it lies within 2^-13 of a tie.
__device__ __forceinline__ void nearest8(const float (&v)[8], float s, float inv, float (&t)[8]) {
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t[e] = fmaf(v[e], inv, kRound);
    far = fmaxf(far, fabsf(fmaf(v[e], inv, kRound - t[e])));
  }
  if (far > 0.5f - 0x1p-13f || !(s < 0x1p127f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = kRound + float(nearest(v[e], s, inv));
  }
}

// A word's four integers as numbers: the low bits of 2^23 + 128 + q, of which 2^23 + 128 is taken off.
__device__ __forceinline__ void widen4(uint32_t word, float* v) {
  const uint32_t biased = word ^ 0x80808080u;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7540 + e)) - 8388736.f;
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two of a word's four integers as 16-bit floats: in the low bits of 1024 + 128 + q, of which
// 1024 + 128 is taken off.  `biased`: the word with each byte's top bit flipped (q + 128).
template <int kPair>
__device__ __forceinline__ uint32_t to_f16(uint32_t biased) {
  return hsub2(__byte_perm(biased, 0x64646464u, kPair ? 0x4342 : 0x4140), 0x64806480u);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two of a word's four integers in bfloat16: of 128 + (the low seven bits) 128 is taken off where q >= 0 and 256 where
// q < 0, the number whose bits are 0x4300 and q's top bit.
template <int kPair>
__device__ __forceinline__ uint32_t to_bf16(uint32_t word) {
  const uint32_t p = __byte_perm(word, 0x43434343u, kPair ? 0x4342 : 0x4140);
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(p & 0xff7fff7fu), "r"(p & 0xff80ff80u));
  return d;
}
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The upper 16 bits of v's 32 (v's first eight significant bits), and v less that; a value that is
// not finite is its own first term.
__device__ __forceinline__ uint32_t take16(float& v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7fffffffu) >= 0x7f800000u) {
    v = 0.f;
    return (b & 0x7fffffffu) > 0x7f800000u ? 0x7fc0u : b >> 16;
  }
  v -= __uint_as_float(b & 0xffff0000u);
  return b >> 16;
}

// A sum of integers times its scales, the smaller first (NaN stays).
__device__ __forceinline__ float scaled(int sum, float s, float t) {
  const bool first = fabsf(s) <= fabsf(t);
  return float(sum) * (first ? s : t) * (first ? t : s);
}

// n / d for 0 <= n < 2^31, with m = floor(2^(31 + s) / d) + 1 and 2^s >= d: n m / 2^(31 + s) is above n / d by
// less than 1 / d.
struct Divider {
  uint64_t m;
  uint32_t s, d;
};
inline Divider divider(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return {(uint64_t(1) << (31 + s)) / d + 1, s, d};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider& v) { return uint32_t(uint64_t(n) * v.m >> (31 + v.s)); }

}  // namespace int8
}  // namespace gb300
