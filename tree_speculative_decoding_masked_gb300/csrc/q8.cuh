// Paged caches held in 8 bits: e4m3 codes, and for each KV head a block of 2^block_shift rows of a
// page shares one scale 2^(s - 127), held as the byte s.  A cached number is code * 2^(s - 127).
//
// Powers of two, because then a block that takes a larger scale can code its rows anew by moving
// their exponents, without a rounding but where a code falls below e4m3's normal numbers, and a
// cached number is a bf16 number exactly, which is what the attention's products take.  e4m3 is a
// floating format: a scale off by up to 2 costs no precision, as it would with integer codes.
#pragma once

#include "tv_common.cuh"

namespace tv {

// Smallest scale exponent that is written: the codes' smallest step, 2^-9, then stands for a normal
// number in 32 bits and in bf16.
constexpr int kQ8Least = -117;
constexpr int kQ8MaxBlock = 64;  // rows that share a scale

// 2^e for e in -149..127 (0 below, infinite above)
__device__ __forceinline__ float q8_two(int e) {
  if (e < -126) return e < -149 ? 0.f : __uint_as_float(1u << (e + 149));
  return e > 127 ? INFINITY : __uint_as_float((uint32_t)(e + 127) << 23);
}
// the number that a scale byte stands for; 255 is no number
__device__ __forceinline__ float q8_scale(unsigned s) { return s == 255u ? __uint_as_float(0x7fffffffu) : q8_two((int)s - 127); }

// The smallest e >= kQ8Least with amax <= 448 * 2^e, amax >= 0 and finite: 448 = 1.75 * 2^8.
__device__ __forceinline__ int q8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
  return max(e, kQ8Least);
}

// two finite numbers or NaNs to e4m3 (nearest, ties to even), `lo` in the low byte
__device__ __forceinline__ uint32_t q8_cvt2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// a number, or NaN for what is not finite
__device__ __forceinline__ float q8_finite(float x) { return fabsf(x) <= 3.4028234e38f ? x : __uint_as_float(0x7fffffffu); }
__device__ __forceinline__ uint32_t q8_code2(float lo, float hi) { return q8_cvt2(q8_finite(lo), q8_finite(hi)); }
// two codes to f16x2, exact
__device__ __forceinline__ uint32_t q8_half2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
__device__ __forceinline__ float q8_half_lo(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float q8_half_hi(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, hi;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
// four codes
__device__ __forceinline__ float4 q8_quad(uint32_t w) {
  const uint32_t a = q8_half2((uint16_t)w), b = q8_half2((uint16_t)(w >> 16));
  return make_float4(q8_half_lo(a), q8_half_hi(a), q8_half_lo(b), q8_half_hi(b));
}
// four codes times a scale
__device__ __forceinline__ float4 q8_numbers(uint32_t w, float scale) {
  const float4 f = q8_quad(w);
  return make_float4(f.x * scale, f.y * scale, f.z * scale, f.w * scale);
}
__device__ __forceinline__ uint32_t q8_code4(float a, float b, float c, float d) {
  return q8_code2(a, b) | q8_code2(c, d) << 16;
}
// four codes to two f16x2
__device__ __forceinline__ void q8_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Attention with P = 2^(z + e - m + 7), e the value's exponent and m at most 8 below the row's largest z + e, takes the
// row's sum of weights from 2^-e P while every e is at most 40 either way.  With z' the largest z, m <= z' + 40, so a P
// below fp32's 2^-126 has z < z' - 53; a term 2^(z - m + 7) is at most 2^(8 - e + 7), 2^55, and that of the key
// that m comes from at least 2^-33.  Of tiles with an e beyond that (2^-117, say, of a block of zeros) it is taken from z
// alone, and of all tiles once an e is that large, which lifts m over z.
constexpr float kQ8Near = 40.f;
__device__ __forceinline__ bool q8_far(float e) { return !(fabsf(e) <= kQ8Near); }
// l > 0 to 2^-12..2^-11 times a power of two, whose exponent it returns; 0 and NaN stay.  O against the same
// reference is then the values' mean times that: the sum of a row's parts, whose weights add up to less than 1, stays
// below the largest value, and the least, 2^-126, keeps more bits than bf16's 2^-133.
__device__ __forceinline__ int q8_norm(float& l) {
  if (!(l > 0.f)) return 0;
  const int k = (int)(__float_as_uint(l) >> 23) - 127 + 12;
  l *= q8_two(-k);
  return k;
}

// four codes under the scale 2^from, coded for 2^to >= 2^from
__device__ __forceinline__ uint32_t q8_recode(uint32_t w, float ratio) {
  const float4 f = q8_numbers(w, ratio);
  return q8_cvt2(f.x, f.y) | q8_cvt2(f.z, f.w) << 16;
}

}  // namespace tv
