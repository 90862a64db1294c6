// The row format of the 4-bit cache: d e2m1 numbers, the even elements in the low nibbles, then d / 16
// scale bytes, one for each 16 numbers.
//
// A scale byte is the upper half of an f16 number without its sign: five exponent bits (bias 15), three
// fraction bits; it becomes a half by a shift.  Scales reach from 2^-17 to 10240, so e2m1 (two significant
// bits, at most 6) times scale (four) is exact in f16, below 2^16 and a multiple of 2^-18, and in bf16.
#pragma once

#include "kv_common.cuh"

namespace cpattn {
namespace kv4 {

template <int D>
constexpr int kRow = D / 2 + D / 16;  // bytes of a row: 72 or 36

constexpr uint32_t kNaN = 255;         // scale byte of a group with a number that is not finite
constexpr uint32_t kMostScale = 0xe2;  // 10240: 6 times the next one is beyond f16

// x times a constant c given in two parts, hi near c and lo = c - hi: off by 2^-42 before its one rounding (Brisebarre and
// Muller's multiplication by a constant of twice the precision).  So x / 6 and x / scale, taken by the reciprocals, are
// never rounded onto a tie of the next step but where they are one: numbers that are a divisor times a tie are exact in fp32,
// and the next number of fp32 is at least 0.53 of a step of the quotient away.
__device__ __forceinline__ float times(float x, float hi, float lo) { return __fmaf_rn(x, hi, __fmul_rn(x, lo)); }

// The byte of the scale nearest to amax / 6 (ties to even).
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const float x = times(amax, 0x1.555556p-3f, -0x1.555556p-28f);
  const uint32_t small = static_cast<uint32_t>(__float2int_rn(x * 0x1p17f));
  uint32_t u = __float_as_uint(x);
  u += 0x7ffffu + ((u >> 20) & 1u);
  const uint32_t code = x < 0x1p-14f ? small : (u >> 20) - ((127u - 15u) << 3);
  return code < kMostScale ? code : kMostScale;
}
__device__ __forceinline__ float scale_of(uint32_t code) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<uint16_t>(code << 7)));
  return f;
}

// The reciprocal of a scale in two parts.  hi is the approximation less two steps of fp32, which is below the reciprocal, as
// the approximation is off by one at most: with lo above 0 the sum of a minus zero's two products is a minus zero.
__device__ __forceinline__ void reciprocal(float scale, float& hi, float& lo) {
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(hi) : "f"(scale));
  hi = __uint_as_float(__float_as_uint(hi) - 2u);
  lo = __fmul_rn(__fmaf_rn(-scale, hi, 1.0f), hi);
}

// Eight fp32 to a word of e2m1 numbers, the first in the lowest nibble: round to nearest even, at most 6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
// The eight e2m1 numbers of a word as f16 pairs, exact: byte i's low nibble is the low half of h[i].
__device__ __forceinline__ void to_f16x2(uint32_t word, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(word));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Scale bytes as halves: byte `at` (0 or 1) of `bytes` in both, and of two words below 256 one in each.
__device__ __forceinline__ uint32_t scale_twice(uint32_t bytes, int at) {
  return __byte_perm(bytes, 0u, at == 0 ? 0x0404 : 0x1414) >> 1;
}
__device__ __forceinline__ uint32_t scale_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x4101) >> 1; }

}  // namespace kv4
}  // namespace cpattn
