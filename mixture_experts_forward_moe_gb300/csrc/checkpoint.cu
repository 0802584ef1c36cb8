// checkpoint.cu -- 8-bit checkpoints of activations (include/moe.h: moe_checkpoint,
// moe_checkpoint_restore; the format is in fp8.cuh) and the element-wise parts of the dense
// block's gradients: the gated product's from its checkpoint, and the sum of a bias.
//
// All of these stream their tensors once.  A thread takes sixteen channels (two 16-byte vectors of
// 16-bit values, one of codes), eight threads a group of 128 channels, and asks for several such
// units before it uses the first; a CTA takes a block of whole rows, so that rows and channels come
// from a 32-bit division.
#include "activation.cuh"
#include "dense_ops.cuh"
#include "fp8.cuh"
#include "ptx.cuh"
#include "vec16.cuh"

namespace gb300moe {

namespace {

constexpr int kThreads = 256;

// Rows of a CTA: about four units per thread, one row at least, and fewer where the SMs would not
// all have a block.
int rows_per_cta(int64_t T, int64_t units) {
  int64_t r = 4 * kThreads / units;
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

// x [T, vecs] vectors of eight values.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    save_kernel(int rows, int T_, int vecs, int groups, const uint4* __restrict__ x,
                uint4* __restrict__ codes, float* __restrict__ scales) {
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
      float f[2][8], top = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unpack<T>(v[k][h], f[h]);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(f[h][j]));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (i >= b.end) continue;
      int64_t row;
      int u;
      b.at(i, row, u);
      const int e = fp8_exponent(top);
      const float inv = fp8_scale(-e);
      codes[row * b.per_row + u] =
          make_uint4(fp8_pack4(f[0][0], f[0][1], f[0][2], f[0][3], inv),
                     fp8_pack4(f[0][4], f[0][5], f[0][6], f[0][7], inv),
                     fp8_pack4(f[1][0], f[1][1], f[1][2], f[1][3], inv),
                     fp8_pack4(f[1][4], f[1][5], f[1][6], f[1][7], inv));
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
    restore_kernel(int rows, int T_, int vecs, int groups, const uint4* __restrict__ codes,
                   const float* __restrict__ scales, uint4* __restrict__ out) {
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
      scale[k] = __ldg(scales + row * groups + (u >> 3));
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
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] > top ? top : (f[j] < -top ? -top : f[j]);
        if (2 * u + h < vecs) out[row * vecs + 2 * u + h] = pack<T>(f);
      }
    }
  }
}

// d_pre [T, 2F]: dg = dh u act'(g), du = dh act(g), and h = act(g) u (out, if wanted); F = 8 vecs.
template <typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
    gated_grad_kernel(int rows, int T_, int vecs, int groups, const uint4* d_out,
                      const uint4* __restrict__ gate, const float* __restrict__ gate_scales,
                      const uint4* __restrict__ up, const float* __restrict__ up_scales,
                      uint4* __restrict__ d_pre, uint4* out) {  // out may be d_out
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
    const float gs = __ldg(gate_scales + row * groups + (u >> 3));
    const float us = __ldg(up_scales + row * groups + (u >> 3));
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

// A CTA adds 64 columns: eight threads side by side, 32 rows at a time, in an order that depends on
// T alone.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    column_sum_kernel(int T_, int N, int64_t pitch, const T* __restrict__ v, T* __restrict__ sum) {
  __shared__ float part[32][65];
  pdl_wait();
  pdl_trigger();
  const int n = blockIdx.x * 64 + (threadIdx.x & 7) * 8, r = threadIdx.x >> 3;
  float s[8] = {};
  if (n < N) {
#pragma unroll 8
    for (int64_t t = r; t < T_; t += 32) {
      float f[8];
      unpack<T>(__ldg(reinterpret_cast<const uint4*>(v + t * pitch + n)), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += f[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[r][(threadIdx.x & 7) * 8 + j] = s[j];
  __syncthreads();
  if (threadIdx.x < 64 && blockIdx.x * 64 + (int)threadIdx.x < N) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += part[i][threadIdx.x];
    sum[blockIdx.x * 64 + threadIdx.x] = DT<T>::from_f(a);
  }
}

__global__ void __launch_bounds__(kThreads)
    pad_kernel(int rows, int T_, int N, int per_row, const uint16_t* __restrict__ v,
               uint4* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int left = T_ - row0 < rows ? (int)(T_ - row0) : rows;
  const int end = left * per_row;
  for (int i = threadIdx.x; i < end; i += kThreads) {
    const int r = (unsigned)i / (unsigned)per_row, c = i - r * per_row;
    const uint16_t* from = v + (row0 + r) * N;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = c * 8 + 2 * j;
      const uint32_t lo = n < N ? from[n] : 0u, hi = n + 1 < N ? from[n + 1] : 0u;
      w[j] = lo | (hi << 16);
    }
    out[(row0 + r) * per_row + c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_blocks(void (*kern)(int, int, KArgs...), int T, int64_t units, cudaStream_t s,
                          Args... args) {
  if (T == 0) return cudaSuccess;
  const int rows = rows_per_cta(T, units);
  return launch_k(kern, dim3((unsigned)((T - 1) / rows + 1)), dim3(kThreads), 0, s, true, rows, T,
                  args...);
}
const uint4* vectors(const void* p) { return static_cast<const uint4*>(p); }

template <typename T>
cudaError_t launch_grad(int act, int T_, int F, const void* d_out, CkptIn gate, CkptIn up,
                        void* d_pre, void* out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(F);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T_, (F / 8 + 1) / 2, s, F / 8, groups, vectors(d_out),
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
    return launch_blocks(kern, T, (int64_t)groups * 8, s, C / 8, groups, vectors(x),
                         reinterpret_cast<uint4*>(out.codes), out.scales);
  };
  return dtype == MOE_BF16 ? go(save_kernel<__nv_bfloat16>) : go(save_kernel<__half>);
}

cudaError_t launch_restore(int dtype, int T, int C, CkptIn in, void* out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(C);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T, (C / 8 + 1) / 2, s, C / 8, groups, vectors(in.codes), in.scales,
                         static_cast<uint4*>(out));
  };
  return dtype == MOE_BF16 ? go(restore_kernel<__nv_bfloat16>) : go(restore_kernel<__half>);
}

cudaError_t launch_gated_grad_saved(int dtype, int act, int T, int F, const void* d_out, CkptIn gate,
                                    CkptIn up, void* d_pre, void* out, cudaStream_t s) {
  return dtype == MOE_BF16 ? launch_grad<__nv_bfloat16>(act, T, F, d_out, gate, up, d_pre, out, s)
                           : launch_grad<__half>(act, T, F, d_out, gate, up, d_pre, out, s);
}

cudaError_t launch_column_sum(int dtype, int T, int N, int64_t pitch, const void* v, void* sum,
                              cudaStream_t s) {
  const dim3 grid((unsigned)((N - 1) / 64 + 1));
  if (dtype == MOE_BF16)
    return launch_k(column_sum_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, true, T, N, pitch,
                    static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(sum));
  return launch_k(column_sum_kernel<__half>, grid, dim3(kThreads), 0, s, true, T, N, pitch,
                  static_cast<const __half*>(v), static_cast<__half*>(sum));
}

cudaError_t launch_pad_rows(int dtype, int T, int N, int64_t pitch, const void* v, void* out,
                            cudaStream_t s) {
  (void)dtype;  // 16 bits either way
  return launch_blocks(pad_kernel, T, pitch / 8, s, N, (int)(pitch / 8),
                       static_cast<const uint16_t*>(v), static_cast<uint4*>(out));
}

}  // namespace gb300moe
