// The 4-bit cache format: e2m1 codes (sign, two exponent bits of bias 1, one
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) packed two a byte, the even feature
// in the low nibble; one e4m3fn scale code for 16 consecutive features of a
// cached row; one fp32 scale a tensor.  A feature's value is
// e2m1 * e4m3 * scale.  The product e2m1 * e4m3 has at most six significant
// bits and lies between 2^-10 and 2688 (or is 0): exact in f16.
#pragma once

#include <stdint.h>

namespace pa {

constexpr int kQ4Group = 16;   // features that share a scale code

// Eight floats -> eight e2m1 codes (nibble i = x[i]), round to nearest even,
// magnitudes above 6 saturate.
__device__ __forceinline__ uint32_t e2m1x8_from_f32(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Eight e2m1 codes -> four f16 pairs (nibble 2i in the low half of h[i]).  Exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Products of two f16 pairs, rounded to nearest (exact for an e2m1 value by an e4m3 value).
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One half of a pair in both halves.
__device__ __forceinline__ uint32_t half_lo2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t half_hi2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float f16_lo(uint32_t x) {
  float r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float f16_hi(uint32_t x) {
  float r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(r) : "r"(x));
  return r;
}

// Transpose of an 8x8 matrix of 16-bit elements held one row pair a lane (row
// lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

}  // namespace pa
