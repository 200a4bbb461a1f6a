// cache8.cuh -- the numbers of the 8-bit paged cache.
//
// A code is an e4m3 byte (1 sign, 4 exponent, 3 mantissa bits; up to 448, steps
// of 2^-9 below 2^-6, 0x7f and 0xff NaN).  scale_rows consecutive positions of a
// page and one kv head share a scale 2^e, kept as the byte 127 + e, with e from
// -14 to 7.  A value is code * 2^e: at most four significant bits between 2^-23
// and 448 * 2^7 = 57344, so every value is exactly a bf16 number and an fp16
// number, and a block's codes move to a larger scale without a new rounding
// except where they become subnormal.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace attn {
namespace c8 {

constexpr int kMinExp = -14, kMaxExp = 7;

// Exponent of a scale byte; bytes outside the range read as its nearest end.
__device__ __forceinline__ int exp_of(uint32_t byte) { return min(max((int)byte - 127, kMinExp), kMaxExp); }

// The smallest exponent in range with amax <= 448 * 2^e (448 = 1.75 * 2^8).  An
// infinite amax gives the largest.
__device__ __forceinline__ int exp_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

// Two codes (low byte first) as two fp16 numbers.
__device__ __forceinline__ uint32_t to_half2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(two));
  return h;
}
// The four codes of a word as two pairs of fp16 numbers.
__device__ __forceinline__ void to_half4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
__device__ __forceinline__ void to_float4(uint32_t four, float (&v)[4]) {
  uint32_t lo, hi;
  to_half4(four, lo, hi);
  const float2 a = half2_to_float2(lo), b = half2_to_float2(hi);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
// Two numbers as codes, rounded to nearest even, magnitudes above 448 to 448;
// lo in the low byte.
__device__ __forceinline__ uint32_t from_float2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}
__device__ __forceinline__ uint32_t from_float4(float a, float b, float c, float d) {
  return from_float2(a, b) | (from_float2(c, d) << 16);
}
// 2^e as an fp16 number in both halves, -14 <= e <= 15.
__device__ __forceinline__ uint32_t pow2_half2(int e) { return (uint32_t)(e + 15) * 0x04000400u; }
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace c8

// Q of bf16 as an fp16 operand: a row is multiplied by the power of two that
// brings its largest magnitude to [2^14, 2^15) (pow2_scale_exp), which every
// score of the row is divided by again.  Entries down to 2^-28 of the largest
// keep all their bits, smaller ones are off by at most 2^-39 of it.
namespace q16 {

// Largest magnitude of two bf16 numbers, and the two as fp16, times mul.
__device__ __forceinline__ float largest2(uint32_t w) {
  return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u)));
}
__device__ __forceinline__ uint32_t to_half2(uint32_t w, float mul) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;"
      : "=r"(r)
      : "f"(__uint_as_float(w & 0xffff0000u) * mul), "f"(__uint_as_float(w << 16) * mul));
  return r;
}
// Largest magnitude of eight, in shared memory (16 bytes).
__device__ __forceinline__ float largest(const unsigned char* p) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, largest2(w[i]));
  return m;
}
// Eight bf16 numbers in shared memory become fp16, times mul.
__device__ __forceinline__ void to_half(unsigned char* p, float mul) {
  uint4 x = *reinterpret_cast<uint4*>(p);
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_half2(w[i], mul);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace q16
}  // namespace attn
