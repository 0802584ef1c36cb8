// fp8.cuh -- E4M3 values with a power of two per group of channels: the checkpoints of training.
//
// The scale is the smallest power of two 2^e with max|v| / 2^e <= 448, E4M3's largest value; being
// a power of two it costs no bit of the codes' four, and code times scale is exact in bf16 and f32.
// e lies in [-118, 120], so that 2^e and 2^-e are normal f32: every 16-bit or f32 maximum is
// within (smaller groups than 448 * 2^-118 lose their last bits).  Infinities and NaN are NaN.
#pragma once

#include "common.cuh"

namespace gb300moe {

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= 3.402823466e38f ? a : 0.0f;
}

// e of a group whose largest finite value is `top`; 0 (a scale of 1) for zeros.
__device__ __forceinline__ int fp8_exponent(float top) {
  const uint32_t bits = __float_as_uint(top);
  // top = m 2^x with m in [1, 2), and 448 = 1.75 * 2^8
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return top == 0.0f ? 0 : max(-118, min(120, e));
}
__device__ __forceinline__ float fp8_scale(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Codes of four values, finite or NaN, times `inv`, the first in the lowest byte.
__device__ __forceinline__ uint32_t fp8_pack4_finite(float a, float b, float c, float d, float inv) {
  a *= inv, b *= inv, c *= inv, d *= inv;
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// The same of any values: the conversion would take infinities to 448, and v - v is NaN for them.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d, float inv) {
  return fp8_pack4_finite(a + (a - a), b + (b - b), c + (c - c), d + (d - d), inv);
}

// Four codes (lowest byte first) -> their values in f32, not scaled.
__device__ __forceinline__ void fp8_unpack4(uint32_t q, float (&v)[4]) {
  uint32_t h01, h23;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}\n"
      : "=r"(h01), "=r"(h23)
      : "r"(q));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h23));
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

}  // namespace gb300moe
