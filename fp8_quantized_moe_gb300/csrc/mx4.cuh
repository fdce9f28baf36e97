// MXFP4 device helpers (OCP Microscaling Formats v1.0, e2m1 elements): 32
// consecutive values of a row along the contracted dimension share one E8M0
// scale 2^X, X = floor(log2(amax)) - 2 (2 is the exponent of e2m1's largest
// power of two, 4), at least -127; the element codes are e2m1(x / 2^X).
#pragma once

#include "common.cuh"

namespace moe {

constexpr uint32_t kE8M0NaN = 255u;

// E8M0 code X + 127 of a block from the largest |x| of its bf16 bit patterns
// (sign cleared).  The bf16 exponent field is floor(log2) + 127 for a normal
// amax, so the code is field - 2; zero and subnormal amax clamp to code 0.  A
// block that holds an infinity or a NaN has no e2m1 form and takes the NaN
// code, so that everything computed from it is NaN.
__device__ __forceinline__ uint32_t mx4_scale_code(uint32_t amax_bits) {
  const uint32_t field = amax_bits >> 7;
  return field == 255u ? kE8M0NaN : (field > 2u ? field - 2u : 0u);
}

// 2^(code - 127) in fp32: code 0 is the subnormal 2^-127, code 255 NaN.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return __uint_as_float(code == 0u ? 0x00400000u : (code == kE8M0NaN ? 0x7FC00000u : code << 23));
}

// 2^(127 - code) for a code that mx4_scale_code gives to finite values (code
// <= 252, so the result is normal); 0 for the NaN code.
__device__ __forceinline__ float mx4_inv_scale(uint32_t code) {
  return code == kE8M0NaN ? 0.0f : __uint_as_float((254u - code) << 23);
}

// Eight fp32 values -> eight e2m1 codes, round to nearest even, saturating to
// +-6; value 2i lands in the low half of byte i.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// e2m1 code (low 4 bits of n) -> its value.  Sign at bit 15 and the three
// magnitude bits at bits 9..11 make an f16 of 2^-14 times the value (the f16
// subnormals hold 0 and 0.5), so one exact product gives it.
__device__ __forceinline__ float e2m1_value(uint32_t n) {
  const uint16_t h = static_cast<uint16_t>(((n & 8u) << 12) | ((n & 7u) << 9));
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
  return __fmul_rn(f, 16384.0f);
}

}  // namespace moe
