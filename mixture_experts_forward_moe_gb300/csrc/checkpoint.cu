// checkpoint.cu -- 8-bit checkpoints of activations (include/moe.h: moe_checkpoint,
// moe_checkpoint_restore; the format is in fp8.cuh) and the element-wise parts of the dense
// block's gradients: the gated product's from its checkpoint, and the sum of a bias.
//
// All of these stream their tensors once.  A thread takes sixteen channels (two 16-byte vectors of
// 16-bit values, one of codes), eight threads a group of 128 channels, and asks for several such
// units before it uses the first; a CTA takes a block of whole rows, so that rows and channels come
// from a 32-bit division.
// They may start before the kernel that wrote their inputs has ended, and wait for it: what they read
// is not read-only while they run, so no pointer is __restrict__ and no load goes past pdl_wait().
#include "activation.cuh"
#include "dense_ops.cuh"
#include "fp8.cuh"
#include "pipe.cuh"
#include "vec16.cuh"

namespace gb300moe {

namespace {

constexpr int kThreads = 256;

// Rows of a CTA: about `each` units per thread, one row at least, and fewer where the SMs would not
// all have a block.
int rows_per_cta(int64_t T, int64_t units, int each) {
  int64_t r = each * kThreads / units;
  while (r > 1 && (T + r - 1) / r < 2 * num_sms()) r /= 2;
  return r < 1 ? 1 : (int)r;
}

// Units of sixteen channels; `per_row` of them.
struct Rows {
  int64_t row0;
  int per_row, end;
  __device__ __forceinline__ Rows(int rows, int T, int units) {
    row0 = (int64_t)blockIdx.x * rows;
    per_row = units;
    end = (T - row0 < rows ? (int)(T - row0) : rows) * units;
  }
  __device__ __forceinline__ void at(int i, int64_t& row, int& u) const {
    const int r = (unsigned)i / (unsigned)per_row;
    row = row0 + r;
    u = i - r * per_row;
  }
};

constexpr int kAhead = 4;  // units that a thread asks for together

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
};
template <>
struct Pair<__half> {
  using type = __half2;
};
// The largest magnitude of sixteen values; NaN does not count.
template <typename T>
__device__ __forceinline__ float top16(const uint4& a, const uint4& b) {
  using P = typename Pair<T>::type;
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t t = 0u;
  P top = *reinterpret_cast<const P*>(&t);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t m = w[j] & 0x7fff7fffu;
    top = __hmax2(top, *reinterpret_cast<const P*>(&m));
  }
  return fmaxf(DT<T>::to_f(top.x), DT<T>::to_f(top.y));
}

// x [T, vecs] vectors of eight values.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    save_kernel(int rows, int T_, int vecs, int groups, const uint4* x,
                uint4* codes, float* scales) {
  pdl_wait();
  pdl_trigger();
  const Rows b(rows, T_, groups * 8);
  // All lanes of a warp stay for the reductions: `first` is its first lane's unit.
  for (int first = threadIdx.x & ~31; first < b.end; first += kAhead * kThreads) {
    uint4 v[kAhead][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = first + k * kThreads + (threadIdx.x & 31);
      int64_t row;
      int u;
      b.at(i, row, u);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[k][h] = i < b.end && 2 * u + h < vecs ? __ldcs(x + row * vecs + 2 * u + h)
                                                : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (first + k * kThreads >= b.end) break;
      const int i = first + k * kThreads + (threadIdx.x & 31);
      // The largest magnitude of 16 bits two by two, NaN left out; where it is an infinity, again
      // without those.
      float top = top16<T>(v[k][0], v[k][1]);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      float f[2][8];
      unpack<T>(v[k][0], f[0]);
      unpack<T>(v[k][1], f[1]);
      const bool far = !(top <= 3.402823466e38f);
      if (__any_sync(0xffffffffu, far)) {
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t = fmaxf(t, fmaxf(finite_abs(f[0][j]), finite_abs(f[1][j])));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        top = t;
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // infinities become NaN, as the conversion does not make them
          f[0][j] += f[0][j] - f[0][j];
          f[1][j] += f[1][j] - f[1][j];
        }
      }
      if (i >= b.end) continue;
      int64_t row;
      int u;
      b.at(i, row, u);
      const int e = fp8_exponent(top);
      const float inv = fp8_scale(-e);
      codes[row * b.per_row + u] =
          make_uint4(fp8_pack4_finite(f[0][0], f[0][1], f[0][2], f[0][3], inv),
                     fp8_pack4_finite(f[0][4], f[0][5], f[0][6], f[0][7], inv),
                     fp8_pack4_finite(f[1][0], f[1][1], f[1][2], f[1][3], inv),
                     fp8_pack4_finite(f[1][4], f[1][5], f[1][6], f[1][7], inv));
      if ((u & 7) == 0) scales[row * groups + (u >> 3)] = fp8_scale(e);
    }
  }
}

// Eight channels from two words of codes.
__device__ __forceinline__ void restore8(uint32_t q0, uint32_t q1, float scale, float (&f)[8]) {
  float a[4], b[4];
  fp8_unpack4(q0, a);
  fp8_unpack4(q1, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = a[j] * scale;
    f[4 + j] = b[j] * scale;
  }
}

template <typename T>
struct Largest;
template <>
struct Largest<__half> {
  static constexpr float value = 65504.0f;
};
template <>
struct Largest<__nv_bfloat16> {
  static constexpr float value = 3.3895313892515355e38f;
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
    restore_kernel(int rows, int T_, int vecs, int groups, const uint4* codes,
                   const float* scales, uint4* out) {
  pdl_wait();
  pdl_trigger();
  const Rows b(rows, T_, (vecs + 1) / 2);
  for (int first = threadIdx.x; first < b.end; first += kAhead * kThreads) {
    uint4 q[kAhead];
    float scale[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = first + k * kThreads;
      int64_t row;
      int u;
      b.at(i < b.end ? i : first, row, u);
      q[k] = __ldcs(codes + row * groups * 8 + u);
      scale[k] = scales[row * groups + (u >> 3)];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = first + k * kThreads;
      if (i >= b.end) break;
      int64_t row;
      int u;
      b.at(i, row, u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
        restore8(h == 0 ? q[k].x : q[k].z, h == 0 ? q[k].y : q[k].w, scale[k], f);
        // a value next to the type's largest may have been rounded past it; NaN stays
        constexpr float top = Largest<T>::value;
        if (scale[k] > top / 512.0f) {  // else 448 scales are within
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = f[j] > top ? top : (f[j] < -top ? -top : f[j]);
        }
        if (2 * u + h < vecs) out[row * vecs + 2 * u + h] = pack<T>(f);
      }
    }
  }
}

// d_pre [T, 2F]: dg = dh u act'(g), du = dh act(g), and h = act(g) u (out, if wanted); F = 8 vecs.
template <typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
    gated_grad_kernel(int rows, int T_, int vecs, int groups, const uint4* d_out,
                      const uint4* gate, const float* gate_scales,
                      const uint4* up, const float* up_scales,
                      uint4* d_pre, uint4* out) {  // out may be d_out
  pdl_wait();
  pdl_trigger();
  const Rows b(rows, T_, (vecs + 1) / 2);
  for (int i = threadIdx.x; i < b.end; i += kThreads) {
    int64_t row;
    int u;
    b.at(i, row, u);
    const bool second = 2 * u + 1 < vecs;
    const uint4 d0 = d_out[row * vecs + 2 * u];
    const uint4 d1 = second ? d_out[row * vecs + 2 * u + 1] : make_uint4(0u, 0u, 0u, 0u);
    const uint4 gq = __ldcs(gate + row * groups * 8 + u), uq = __ldcs(up + row * groups * 8 + u);
    const float gs = gate_scales[row * groups + (u >> 3)];
    const float us = up_scales[row * groups + (u >> 3)];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float dh[8], g[8], v[8], dg[8], du[8], h[8];
      unpack<T>(k == 0 ? d0 : d1, dh);
      restore8(k == 0 ? gq.x : gq.z, k == 0 ? gq.y : gq.w, gs, g);
      restore8(k == 0 ? uq.x : uq.z, k == 0 ? uq.y : uq.w, us, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float a, s;
        gate_slope<kAct>(g[j], a, s);
        h[j] = a * v[j];
        dg[j] = dh[j] * v[j] * s;
        du[j] = dh[j] * a;
      }
      if (k == 1 && !second) break;
      d_pre[2 * row * vecs + 2 * u + k] = pack<T>(dg);
      d_pre[(2 * row + 1) * vecs + 2 * u + k] = pack<T>(du);
      if (out) out[row * vecs + 2 * u + k] = pack<T>(h);
    }
  }
}

// Sixteen bytes from `at` on (a multiple of 16) of a tensor of `bytes`: zeros behind its end.
__device__ __forceinline__ uint4 load_end(const char* base, int64_t at, int64_t bytes) {
  if (at + 16 <= bytes) return *reinterpret_cast<const uint4*>(base + at);
  uint32_t w[4] = {};
  for (int j = 0; j < 8; ++j)
    if (at + 2 * j < bytes)
      w[j >> 1] |= (uint32_t) * reinterpret_cast<const uint16_t*>(base + at + 2 * j) << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight 16-bit values from the i-th on, anywhere in a tensor of `bytes` on a 16-byte boundary: the two
// vectors that hold them, moved together.
__device__ __forceinline__ uint4 load8(const void* tensor, int64_t i, int64_t bytes) {
  const char* base = static_cast<const char*>(tensor);
  const int64_t at = 2 * i & ~int64_t(15);
  const int off = (int)(2 * i & 15);
  const uint4 a = load_end(base, at, bytes);
  if (off == 0) return a;
  const uint4 b = load_end(base, at + 16, bytes);
  uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  uint32_t last = b.w;
  if (off & 8) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 2];
    w[5] = last;
  }
  if (off & 4) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
  }
  const int shift = (off & 2) * 8;
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], shift);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA adds 64 columns, eight threads side by side and 32 rows at a time; a cluster of `parts` CTAs
// shares the rows of the same columns, and its first CTA adds their sums.  The order depends on T
// alone.  (One CTA for all of 4096 rows: 39 us for 4096 columns.)
// kPad: the rows start anywhere, `pitch` = N; they are copied to `out`, whose rows lie out_pitch apart,
// with anything behind N.
template <typename T, bool kPad>
__global__ void __launch_bounds__(kThreads)
    column_sum_kernel(int T_, int N, int parts, int64_t pitch, int64_t out_pitch,
                      const T* v, T* out, T* sum) {
  __shared__ float part[32][65];
  __shared__ float total[64];
  pdl_wait();
  pdl_trigger();
  const int group = blockIdx.x / (unsigned)parts, mine = blockIdx.x % (unsigned)parts;
  const int n = group * 64 + (threadIdx.x & 7) * 8, r = threadIdx.x >> 3;
  constexpr int kRows = kPad ? 4 : 8;  // that a thread asks for together
  float s[8] = {};
  if (n < N) {
    const int step = 32 * parts;
    for (int64_t t = mine * 32 + r; t < T_; t += kRows * step) {
      uint4 q[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t row = t + k * step;
        if (row >= T_)
          q[k] = make_uint4(0u, 0u, 0u, 0u);
        else if constexpr (kPad)
          q[k] = load8(v, row * pitch + n, T_ * pitch * 2);
        else
          q[k] = *reinterpret_cast<const uint4*>(v + row * pitch + n);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t row = t + k * step;
        float f[8];
        unpack<T>(q[k], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += f[j];
        if (kPad && row < T_) *reinterpret_cast<uint4*>(out + row * out_pitch + n) = q[k];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[r][(threadIdx.x & 7) * 8 + j] = s[j];
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 64) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += part[i][c];
    total[c] = a;
  }
  if (parts > 1)
    cluster_sync();
  else
    __syncthreads();
  if (mine == 0 && c < 64 && group * 64 + c < N) {
    float a = total[c];
    for (int q = 1; q < parts; ++q) {
      float b;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(b)
                   : "r"(cluster_map(smem_u32(&total[c]), (uint32_t)q))
                   : "memory");
      a += b;
    }
    sum[group * 64 + c] = DT<T>::from_f(a);
  }
  if (parts > 1) cluster_leave();  // the first CTA may still read the others' sums
}

__global__ void __launch_bounds__(kThreads)
    pad_kernel(int rows, int T_, int N, int per_row, const void* v, uint4* out) {
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int left = T_ - row0 < rows ? (int)(T_ - row0) : rows;
  const int end = left * per_row;
  for (int i = threadIdx.x; i < end; i += kThreads) {
    const int r = (unsigned)i / (unsigned)per_row, c = i - r * per_row;
    out[(row0 + r) * per_row + c] = load8(v, (row0 + r) * N + c * 8, (int64_t)T_ * N * 2);
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_blocks(void (*kern)(int, int, KArgs...), int T, int64_t units, int each,
                          cudaStream_t s, Args... args) {
  if (T == 0) return cudaSuccess;
  const int rows = rows_per_cta(T, units, each);
  return launch_k(kern, dim3((unsigned)((T - 1) / rows + 1)), dim3(kThreads), 0, s, true, rows, T,
                  args...);
}
const uint4* vectors(const void* p) { return static_cast<const uint4*>(p); }

template <typename T>
cudaError_t launch_grad(int act, int T_, int F, const void* d_out, CkptIn gate, CkptIn up,
                        void* d_pre, void* out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(F);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T_, (F / 8 + 1) / 2, 1, s, F / 8, groups, vectors(d_out),
                         vectors(gate.codes), gate.scales, vectors(up.codes), up.scales,
                         static_cast<uint4*>(d_pre), static_cast<uint4*>(out));
  };
  return act == MOE_ACT_SILU ? go(gated_grad_kernel<T, MOE_ACT_SILU>)
                             : go(gated_grad_kernel<T, MOE_ACT_GELU_TANH>);
}

}  // namespace

cudaError_t launch_checkpoint(int dtype, int T, int C, const void* x, Ckpt out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(C);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T, (int64_t)groups * 8, kAhead, s, C / 8, groups, vectors(x),
                         reinterpret_cast<uint4*>(out.codes), out.scales);
  };
  return dtype == MOE_BF16 ? go(save_kernel<__nv_bfloat16>) : go(save_kernel<__half>);
}

cudaError_t launch_restore(int dtype, int T, int C, CkptIn in, void* out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(C);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T, (C / 8 + 1) / 2, kAhead, s, C / 8, groups, vectors(in.codes), in.scales,
                         static_cast<uint4*>(out));
  };
  return dtype == MOE_BF16 ? go(restore_kernel<__nv_bfloat16>) : go(restore_kernel<__half>);
}

cudaError_t launch_gated_grad_saved(int dtype, int act, int T, int F, const void* d_out, CkptIn gate,
                                    CkptIn up, void* d_pre, void* out, cudaStream_t s) {
  return dtype == MOE_BF16 ? launch_grad<__nv_bfloat16>(act, T, F, d_out, gate, up, d_pre, out, s)
                           : launch_grad<__half>(act, T, F, d_out, gate, up, d_pre, out, s);
}

namespace {
template <typename T>
cudaError_t sum_columns(int T_, int N, int64_t pitch, const void* v, void* padded, void* sum,
                        cudaStream_t s) {
  int parts = 1;
  while (parts < 8 && T_ > 128 * parts) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((N - 1) / 64 + 1) * parts);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)parts;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  const T* from = static_cast<const T*>(v);
  T *out = static_cast<T*>(padded), *to = static_cast<T*>(sum);
  return padded ? cudaLaunchKernelEx(&cfg, column_sum_kernel<T, true>, T_, N, parts, (int64_t)N, pitch,
                                     from, out, to)
                : cudaLaunchKernelEx(&cfg, column_sum_kernel<T, false>, T_, N, parts, pitch, pitch,
                                     from, out, to);
}
}  // namespace

cudaError_t launch_column_sum(int dtype, int T, int N, int64_t pitch, const void* v, void* padded,
                              void* sum, cudaStream_t s) {
  return dtype == MOE_BF16 ? sum_columns<__nv_bfloat16>(T, N, pitch, v, padded, sum, s)
                           : sum_columns<__half>(T, N, pitch, v, padded, sum, s);
}

cudaError_t launch_pad_rows(int T, int N, int64_t pitch, const void* v, void* out, cudaStream_t s) {
  return launch_blocks(pad_kernel, T, pitch / 8, kAhead, s, N, (int)(pitch / 8),
                       v, static_cast<uint4*>(out));
}

}  // namespace gb300moe
