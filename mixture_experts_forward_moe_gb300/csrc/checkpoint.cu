// checkpoint.cu -- 8-bit checkpoints of activations (include/moe.h: moe_checkpoint,
// moe_checkpoint_restore; the format is in fp8.cuh) and the element-wise parts of the dense
// block's gradients: the gated product's from its checkpoint, and the sum of a bias.
//
// All of these stream their tensors once.  A thread takes eight channels (16 bytes of 16-bit
// values, 8 bytes of codes), sixteen threads a group of 128 channels; a CTA takes a block of whole
// rows, so that rows and channels come from a 32-bit division.
#include "activation.cuh"
#include "dense_ops.cuh"
#include "fp8.cuh"
#include "vec16.cuh"

namespace gb300moe {

namespace {

constexpr int kThreads = 256;

// Rows of a CTA: about four vectors per thread, one row at least, and fewer where the SMs would not
// all have a block.
int rows_per_cta(int64_t T, int64_t vectors) {
  int64_t r = 4 * kThreads / vectors;
  while (r > 1 && (T + r - 1) / r < 2 * num_sms()) r /= 2;
  return r < 1 ? 1 : (int)r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    save_kernel(int rows, int T_, int C, int groups, const uint4* __restrict__ x,
                uint2* __restrict__ codes, float* __restrict__ scales) {
  const int per_row = groups * 16, live = C / 8;
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int left = T_ - row0 < rows ? (int)(T_ - row0) : rows;
  const int end = left * per_row;
  // All lanes of a warp stay for the reduction: `first` is its first lane's vector.
  for (int first = threadIdx.x & ~31; first < end; first += kThreads) {
    const int i = first + (threadIdx.x & 31);
    const int r = (unsigned)i / (unsigned)per_row, v = i - r * per_row;
    float f[8] = {};
    if (i < end && v < live) unpack<T>(__ldcs(x + (row0 + r) * live + v), f);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(f[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (i >= end) continue;
    const int e = fp8_exponent(top);
    const float inv = fp8_scale(-e);
    codes[(row0 + r) * per_row + v] =
        make_uint2(fp8_pack4(f[0], f[1], f[2], f[3], inv), fp8_pack4(f[4], f[5], f[6], f[7], inv));
    if ((v & 15) == 0) scales[(row0 + r) * groups + (v >> 4)] = fp8_scale(e);
  }
}

__device__ __forceinline__ void restore8(uint2 q, float scale, float (&f)[8]) {
  float a[4], b[4];
  fp8_unpack4(q.x, a);
  fp8_unpack4(q.y, b);
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
    restore_kernel(int rows, int T_, int C, int groups, const uint2* __restrict__ codes,
                   const float* __restrict__ scales, uint4* __restrict__ out) {
  const int per_row = C / 8;
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int left = T_ - row0 < rows ? (int)(T_ - row0) : rows;
  const int end = left * per_row;
#pragma unroll 4
  for (int i = threadIdx.x; i < end; i += kThreads) {
    const int r = (unsigned)i / (unsigned)per_row, v = i - r * per_row;
    const uint2 q = __ldcs(codes + (row0 + r) * groups * 16 + v);
    float f[8];
    restore8(q, __ldg(scales + (row0 + r) * groups + (v >> 4)), f);
    // a value next to the type's largest may have been rounded past it; NaN stays
    constexpr float top = Largest<T>::value;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] > top ? top : (f[j] < -top ? -top : f[j]);
    out[(row0 + r) * per_row + v] = pack<T>(f);
  }
}

// d_pre [T, 2F]: dg = dh u act'(g), du = dh act(g), and h = act(g) u (out, if wanted).
template <typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
    gated_grad_kernel(int rows, int T_, int F, int groups, const uint4* __restrict__ d_out,
                      const uint2* __restrict__ gate, const float* __restrict__ gate_scales,
                      const uint2* __restrict__ up, const float* __restrict__ up_scales,
                      uint4* __restrict__ d_pre, uint4* __restrict__ out) {
  const int per_row = F / 8;
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  const int left = T_ - row0 < rows ? (int)(T_ - row0) : rows;
  const int end = left * per_row;
#pragma unroll 2
  for (int i = threadIdx.x; i < end; i += kThreads) {
    const int r = (unsigned)i / (unsigned)per_row, v = i - r * per_row;
    const int64_t row = row0 + r;
    const uint4 dv = __ldcs(d_out + row * per_row + v);
    const uint2 gv = __ldcs(gate + row * groups * 16 + v);
    const uint2 uv = __ldcs(up + row * groups * 16 + v);
    const float gs = __ldg(gate_scales + row * groups + (v >> 4));
    const float us = __ldg(up_scales + row * groups + (v >> 4));
    float dh[8], g[8], u[8], dg[8], du[8], h[8];
    unpack<T>(dv, dh);
    restore8(gv, gs, g);
    restore8(uv, us, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a, s;
      gate_slope<kAct>(g[j], a, s);
      h[j] = a * u[j];
      dg[j] = dh[j] * u[j] * s;
      du[j] = dh[j] * a;
    }
    d_pre[2 * row * per_row + v] = pack<T>(dg);
    d_pre[(2 * row + 1) * per_row + v] = pack<T>(du);
    if (out) out[row * per_row + v] = pack<T>(h);
  }
}

// A CTA adds 64 columns: eight threads side by side, 32 rows at a time, in an order that depends on
// T alone.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    column_sum_kernel(int T_, int N, int64_t pitch, const T* __restrict__ v, T* __restrict__ sum) {
  __shared__ float part[32][65];
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
cudaError_t launch_blocks(void (*kern)(int, int, KArgs...), int T, int64_t vectors, cudaStream_t s,
                          Args... args) {
  if (T == 0) return cudaSuccess;
  const int rows = rows_per_cta(T, vectors);
  return launch_k(kern, dim3((unsigned)((T - 1) / rows + 1)), dim3(kThreads), 0, s, false, rows, T,
                  args...);
}

template <typename T>
cudaError_t launch_grad(int act, int T_, int F, const void* d_out, CkptIn gate, CkptIn up,
                        void* d_pre, void* out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(F);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T_, F / 8, s, F, groups, static_cast<const uint4*>(d_out),
                         reinterpret_cast<const uint2*>(gate.codes), gate.scales,
                         reinterpret_cast<const uint2*>(up.codes), up.scales,
                         static_cast<uint4*>(d_pre), static_cast<uint4*>(out));
  };
  return act == MOE_ACT_SILU ? go(gated_grad_kernel<T, MOE_ACT_SILU>)
                             : go(gated_grad_kernel<T, MOE_ACT_GELU_TANH>);
}

}  // namespace

cudaError_t launch_checkpoint(int dtype, int T, int C, const void* x, Ckpt out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(C);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T, (int64_t)groups * 16, s, C, groups, static_cast<const uint4*>(x),
                         reinterpret_cast<uint2*>(out.codes), out.scales);
  };
  return dtype == MOE_BF16 ? go(save_kernel<__nv_bfloat16>) : go(save_kernel<__half>);
}

cudaError_t launch_restore(int dtype, int T, int C, CkptIn in, void* out, cudaStream_t s) {
  const int groups = (int)ckpt_groups(C);
  auto go = [&](auto kern) {
    return launch_blocks(kern, T, C / 8, s, C, groups, reinterpret_cast<const uint2*>(in.codes),
                         in.scales, static_cast<uint4*>(out));
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
    return launch_k(column_sum_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, false, T, N, pitch,
                    static_cast<const __nv_bfloat16*>(v), static_cast<__nv_bfloat16*>(sum));
  return launch_k(column_sum_kernel<__half>, grid, dim3(kThreads), 0, s, false, T, N, pitch,
                  static_cast<const __half*>(v), static_cast<__half*>(sum));
}

cudaError_t launch_pad_rows(int dtype, int T, int N, int64_t pitch, const void* v, void* out,
                            cudaStream_t s) {
  (void)dtype;  // 16 bits either way
  return launch_blocks(pad_kernel, T, pitch / 8, s, N, (int)(pitch / 8),
                       static_cast<const uint16_t*>(v), static_cast<uint4*>(out));
}

}  // namespace gb300moe
