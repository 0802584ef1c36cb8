// vec16.cuh -- eight 16-bit values as one 16-byte vector, and their f32 values.
#pragma once

#include "common.cuh"

namespace gb300moe {

constexpr int kVec = 8;

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[kVec]);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& v, float (&f)[kVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <>
__device__ __forceinline__ void unpack<__half>(const uint4& v, float (&f)[kVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[kVec]);
template <>
__device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float (&f)[kVec]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack<__half>(const float (&f)[kVec]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two f32 values in a 64-bit register: sm_103a multiplies and adds them in one instruction, each
// rounded as alone.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float f2_sum(F2 a) {
  const float2 x = f2_get(a);
  return x.x + x.y;
}
template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, F2 (&f)[kVec / 2]) {
  float x[kVec];
  unpack<T>(v, x);
#pragma unroll
  for (int i = 0; i < kVec / 2; ++i) f[i] = f2(x[2 * i], x[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const F2 (&f)[kVec / 2]) {
  float x[kVec];
#pragma unroll
  for (int i = 0; i < kVec / 2; ++i) {
    const float2 p = f2_get(f[i]);
    x[2 * i] = p.x;
    x[2 * i + 1] = p.y;
  }
  return pack<T>(x);
}

}  // namespace gb300moe
