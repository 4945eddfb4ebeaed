// fp4_device.cuh -- device helpers of the microscaled 4-bit operators: the
// formats' block sizes, code and scale conversions, and 32-bit reads and
// writes of the unquantised types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fp4.h"

namespace gb300 {
namespace fp4 {

template <int kFormat>
struct Format {
  static constexpr int kBlock = kFormat == FP4_MXFP4 ? 32 : 16;
  static constexpr int kAtom = 4 * kBlock;                // columns whose scales make one 512-byte atom
  static constexpr int kAtomsPerStage = 256 / kAtom;      // atoms of 256 columns
};

// Offset of the scale byte of block `k` of row `r` (fp4.h).
__host__ __device__ __forceinline__ int64_t scale_offset(int64_t r, int64_t k, int64_t atoms) {
  return (((r >> 7) * atoms + (k >> 2)) * 32 + (r & 31)) * 16 + ((r & 127) >> 5) * 4 + (k & 3);
}

// Two codes from two values (each rounded to nearest even, at most 6 in magnitude): lo in bits 0-3.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "mov.b32 %0, {b, b, b, b};\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r & 0xffu;
}

// Eight codes from eight values.
__device__ __forceinline__ uint32_t encode8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The larger magnitude; NaN if there is one.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// The two values of byte kByte of w, exact in 16-bit floats (low code in .x).
template <int kByte>
__device__ __forceinline__ __half2 decode2(uint32_t w) {
  uint32_t h;
  if constexpr (kByte == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
  else if constexpr (kByte == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(w));
  else if constexpr (kByte == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(h) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(h) : "r"(w));
  return *reinterpret_cast<__half2*>(&h);
}

// 8-bit float scale (4 exponent bits, 3 fraction bits) of v >= 0: nearest even, at most 448.
__device__ __forceinline__ uint32_t encode_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xffu;
}

__device__ __forceinline__ float decode_e4m3(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(byte)));
  return __low2float(*reinterpret_cast<__half2*>(&h));
}

// Two scale bytes, low one first.
__device__ __forceinline__ float2 decode_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// 2^(byte - 127); 255: NaN.
__device__ __forceinline__ float decode_e8m0(uint32_t byte) {
  const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23;
  return __uint_as_float(bits);
}

// The unit of a block without the matrix's factor.
template <int kFormat>
__device__ __forceinline__ float decode_scale(uint32_t byte) {
  return kFormat == FP4_MXFP4 ? decode_e8m0(byte) : decode_e4m3(byte);
}

// The two matrices' factors, by which a finished sum is multiplied one after the other:
// their product and 1, as long as that is a normal number, else the smaller one first.  (One
// factor may be far above and the other far below 1: sum * 1e35 * 1e-30 would overflow on
// the way.)
__device__ __forceinline__ float2 join_factors(float a, float b) {
  const float p = a * b, m = fabsf(p);
  return m >= 0x1p-126f && m <= 0x1.fffffep127f ? make_float2(p, 1.f) : fabsf(a) <= fabsf(b) ? make_float2(a, b) : make_float2(b, a);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// x / unit, correctly rounded.  With r the correctly rounded reciprocal, the
// quotient x r corrected once by its residual is correctly rounded (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990) as long as the residual is not subnormal, which holds for units between
// 2^-100 and 2^100 wherever the quotient is not far below the smallest level, and as
// long as x r does not overflow (infinity less infinity): the callers keep x below.
// The residual is taken as q unit - x: it is +0 where it vanishes, so that a q of -0 stays -0.
__device__ __forceinline__ float quotient(float x, float unit, float r) {
  const float q = x * r;
  return fmaf(-fmaf(q, unit, -x), r, q);
}

// Quantisation of a block, 16 of its values at a time (fp4.h has the definition).
template <int kFormat>
struct Quantizer {
  float g, g6, g6_inv;
  bool plain;

  __device__ __forceinline__ explicit Quantizer(const float* factor) {
    g = kFormat == FP4_NVFP4 && factor != nullptr ? __ldg(factor) : 1.f;
    g6 = 6.f * g;
    g6_inv = __frcp_rn(g6);
    plain = g6 >= 0x1p-100f && g6 <= 0x1p100f;
  }

  // The scale byte of a block whose largest magnitude is `a` (NaN if one value is),
  // and what encode() needs: the unit, or for powers of two its inverse.
  __device__ __forceinline__ uint32_t scale(float a, float& unit) const {
    const uint32_t top = __float_as_uint(a);  // NaN and infinity: from 0x7f800000 on
    if constexpr (kFormat == FP4_MXFP4) {
      // floor(log2 a) is the exponent field; a subnormal a clamps to -127 as field 0 does.
      const int e = max(int(top >> 23) - 127 - 2, -127);
      unit = __uint_as_float(uint32_t(127 - e) << 23);  // 2^-e, at most 2^127
      return top >= 0x7f800000u ? 255u : top == 0 ? 0u : uint32_t(e + 127);
    } else {
      // From 448 * 6 g on the scale is 448 (a / (6 g) may pass the largest number of 32 bits).
      const float s = !plain ? __fdiv_rn(a, g6) : a < 448.f * g6 ? quotient(a, g6, g6_inv) : 448.f;
      const uint32_t byte = top >= 0x7f800000u ? 127u : top == 0 ? 0u : encode_e4m3(s);
      unit = decode_e4m3(byte) * g;
      return byte;
    }
  }

  // `a` and `unit`: as scale() got and gave them.
  __device__ __forceinline__ void encode(float (&v)[16], float a, float unit, uint32_t (&word)[2]) const {
    if constexpr (kFormat == FP4_MXFP4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= unit;
      word[0] = encode8(v);
      word[1] = encode8(v + 8);
    } else {
      word[0] = word[1] = 0u;
      if (unit >= 0x1p-100f && unit <= 0x1p100f) {
        const float inv = __frcp_rn(unit);
        if (a > 16.f * unit) {  // the scale is at its largest; from 6 units on every value has the last code
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = fminf(fmaxf(v[i], -16.f * unit), 16.f * unit);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = quotient(v[i], unit, inv);
        word[0] = encode8(v);
        word[1] = encode8(v + 8);
      } else if (unit > 0.f) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          float q[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) q[k] = __fdiv_rn(i ? v[8 + k] : v[k], unit);
          const uint32_t w = encode8(q);
          if (i) word[1] = w; else word[0] = w;
        }
      }
    }
  }
};

// The largest magnitude of 16 values; NaN if there is one.
__device__ __forceinline__ float largest(const float (&v)[16]) {
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max_abs(v[i], v[i + 8]);
#pragma unroll
  for (int n = 4; n; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) a[i] = max_abs(a[i], a[i + n]);
  return a[0];
}

}  // namespace fp4
}  // namespace gb300
