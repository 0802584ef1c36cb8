// rows.cuh -- what the products that decode or stream weight rows share (dense_rows.cu, dense_w4.cu):
// copies into shared memory, E4M3 scales, and the end of an output.
#pragma once

#include "activation.cuh"
#include "dense_ops.cuh"
#include "nvfp4.cuh"
#include "pipe.cuh"
#include "vec16.cuh"

namespace gb300moe {

// Into L2 alone: also before the wait for the kernel before this one, which may write what is there.
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
// `bytes` of the 16; zeros behind them.
__device__ __forceinline__ void copy16_part(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds2(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
// Two E4M3 scales (the low bytes of `v`), each in both halves of an f16x2 word.
__device__ __forceinline__ void two_scales(uint32_t v, uint32_t (&s)[2]) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}\n"
      : "=r"(h)
      : "r"(v));
  s[0] = __byte_perm(h, h, 0x1010);
  s[1] = __byte_perm(h, h, 0x3232);
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int c) {
  return c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
}

// One output from its f32 sum (or sums, gated).
template <typename T, bool kGated>
__device__ __forceinline__ void finish(const RowsCall& p, int64_t row, int64_t n, float z, float up) {
  const int64_t o = row * p.N + n;
  if constexpr (kGated) {
    z = (p.act == MOE_ACT_SILU ? gate_value<MOE_ACT_SILU>(z) : gate_value<MOE_ACT_GELU_TANH>(z)) * up;
  } else {
    if (p.bias) z += DT<T>::to_f(static_cast<const T*>(p.bias)[n]);
    z = activate(z, p.act);
    if (p.res) z += DT<T>::to_f(static_cast<const T*>(p.res)[o]);
  }
  static_cast<T*>(p.out)[o] = DT<T>::from_f(z);
}

}  // namespace gb300moe
