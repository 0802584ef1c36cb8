// rows.cuh -- what the products of few rows of x share (dense_rows.cu, dense_w4.cu, dense_few.cu):
// copies into shared memory, E4M3 scales, the end of a tile, and in how many parts K is split.
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
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
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

// bf16 x in f16.  A row whose largest magnitude lies in [0.5, 65504] is taken as it is: exact down to
// 2^-14, at most 2^-25 off below, which is 2^-24 of its largest at most, as f32 sums are.  Another is
// taken times a power of two that brings the largest to [2^14, 2^15), and its sums times the inverse:
// 2^-39 of its largest at most, over all of bf16's range.
struct RowScale {
  float down, up;  // of x, of the sums
};
// The largest magnitude of eight values as its bits; NaN does not count (its row is NaN).
__device__ __forceinline__ uint32_t top_bits(const uint4& v) {
  const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
  uint32_t zero = 0u;
  __nv_bfloat162 top = *reinterpret_cast<const __nv_bfloat162*>(&zero);
#pragma unroll
  for (int i = 0; i < 4; ++i) top = __hmax2(top, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
  const uint32_t t = *reinterpret_cast<const uint32_t*>(&top);
  return max(t & 0xffffu, t >> 16);
}
__device__ __forceinline__ bool past_f16(uint32_t top) { return top >= 0x4780u; }  // 65536
__device__ __forceinline__ bool needs_scale(uint32_t top) {
  return top != 0u && (top < 0x3f00u || past_f16(top));  // 0.5
}
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  if (!needs_scale(top)) return RowScale{1.0f, 1.0f};
  const int k = max((int)min(top >> 7, 254u) - 127 - 14, -126);  // both powers are normal f32
  return RowScale{__uint_as_float((uint32_t)(127 - k) << 23), __uint_as_float((uint32_t)(127 + k) << 23)};
}
__device__ __forceinline__ uint4 bf16x8_times(const uint4& v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    const __half2 h = __floats2half2_rn(f.x * scale, f.y * scale);
    r[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Blocks of K that one of kAccs accumulators takes, of `all` in a part: `most` (kChainK), or more where
// the accumulators are not enough for that.
template <int kAccs>
__device__ __forceinline__ int chain_of(int all, int most) {
  const int least = (all - 1) / kAccs + 1;
  return least > most ? least : most;
}
// Adds `more` further accumulators, `cols` columns apart, to 16 columns of the first.
__device__ __forceinline__ void add_accumulators(uint32_t t, int cols, int more, float (&v)[16]) {
  for (int a = 1; a <= more; ++a) {
    float u[16];
    tmem_ld_x16(t + (uint32_t)(a * cols), u);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += u[i];
  }
}

constexpr int kMaxParts = 8;  // of K: a portable cluster

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

// A tile's share of its outputs, once the CTAs of its cluster (`parts` of K, this one the part-th) have
// written their sums [columns][pitch]: kOuts of them, a gated product's up rows kOuts further.
// Consecutive threads have consecutive columns of out; the parts are added in their order.
// x_scale: of the sums of each row of x, or null.
template <typename T, bool kGated, int kOuts, int kThreads>
__device__ __forceinline__ void finish_tile(const RowsCall& p, uint32_t base, const float* sums,
                                            int pitch, int64_t group, int part, int parts,
                                            int64_t t0, int cols, float alpha,
                                            const float* x_scale) {
  const int64_t n0 = group * kOuts;
  const int end = (part + 1) * kOuts * cols / parts;
  for (int i = part * kOuts * cols / parts + (int)threadIdx.x; i < end; i += kThreads) {
    const int c = i / kOuts, r = i % kOuts;
    if (n0 + r >= p.N) continue;  // (every read of a peer is waited for by its output)
    float z = 0.0f, up = 0.0f;
    if (parts > 1) {
      const uint32_t at = base + (uint32_t)((c * pitch + r) * 4);
      float a[kMaxParts], b[kMaxParts];  // all asked for before the first is added
#pragma unroll
      for (int q = 0; q < kMaxParts; ++q) {
        const uint32_t peer = cluster_map(at, (uint32_t)(q < parts ? q : 0));
        a[q] = q < parts ? ld_cluster(peer) : 0.0f;
        b[q] = kGated && q < parts ? ld_cluster(peer + kOuts * 4u) : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < kMaxParts; ++q) z += a[q], up += b[q];
    } else {
      z = sums[c * pitch + r];
      if (kGated) up = sums[c * pitch + kOuts + r];
    }
    z *= alpha, up *= alpha;
    if (x_scale) {  // behind alpha, so that what is not past f32 at the end is not before
      const float s = x_scale[t0 + c];
      z *= s, up *= s;
    }
    finish<T, kGated>(p, t0 + c, n0 + r, z, up);
  }
}

// ---- host side ---------------------------------------------------------------------------------
// Clusters of `parts` CTAs that the GPU holds at a time, asked for once per device.
template <auto Kernel>
inline int max_clusters(int parts, int threads, int smem) {
  static std::once_flag once[64];
  static int most[64][kMaxParts + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::call_once(once[dev], [dev, threads, smem] {
    for (int q = 1; q <= kMaxParts; ++q) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)q);
      cfg.blockDim = dim3((unsigned)threads);
      cfg.dynamicSmemBytes = (size_t)smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)q;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      most[dev][q] = cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) == cudaSuccess ? n : 0;
    }
  });
  return most[dev][parts];
}

// Parts of K in which `tiles` tiles of `all` blocks take the least time, in blocks, of which a CTA is
// taken to cost `start` beside its own (its start, the first block and the join): the fastest of one
// to eight, or within 3% of it, at 30 of 31 sizes of both kernels, 8% behind at the other (4 x 4096 x
// 1536).  0: no launch is possible.
template <auto Kernel>
inline int parts_of(int64_t tiles, int all, int start, int threads, int smem) {
  int64_t best = 0;
  int parts = 0;
  for (int q = 1; q <= kMaxParts && q <= all; ++q) {
    const int64_t most = max_clusters<Kernel>(q, threads, smem);
    if (most <= 0) continue;
    const int64_t t = ((tiles + most - 1) / most) * ((all + q - 1) / q + start);
    if (parts == 0 || t < best) best = t, parts = q;
  }
  return parts;
}

}  // namespace gb300moe
