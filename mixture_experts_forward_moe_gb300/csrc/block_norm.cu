// block_norm.cu -- the norm, gate and residual between two blocks (include/moe.h:
// moe_block_norm_fwd, moe_block_norm_bwd).
//
//   u = y ry (o + wq), r = a x + g u, h = r rr (o + wp);  ry, rr = 1/sqrt(mean square + eps)
//
// A row is held in registers (16-bit, eight elements per 16-byte vector) by one CTA: both means
// need the whole row, and r needs ry first, so a row is read once and its two reductions run
// over the CTA.  Everything between load and store is f32.
#include "vec16.cuh"

namespace gb300moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// Sums of N values over the CTA, the same bits in every thread: shuffles within a warp, then
// each warp adds the warps' sums in the same butterfly.  One barrier; `buf` may be written again
// only after another one.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float (*buf)[32], int n_warps) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kAll, v[i], off);
  if (n_warps == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i][warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < n_warps ? buf[i][lane] : 0.0f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kAll, v[i], off);
}

struct NormArgs {
  int T, H, n_vec;  // n_vec = H / 8
  int gate, post, pre;
  float a, o, eps, inv_h;
  const uint4 *y, *x, *g, *wq, *wp;
};

// The gate of vector v of row t.
template <typename T>
__device__ __forceinline__ void load_gate(const NormArgs& p, int t, int v, float (&g)[kVec]) {
  if (p.gate == MOE_GATE_CHANNEL) {
    unpack<T>(__ldg(p.g + v), g);
  } else if (p.gate == MOE_GATE_ELEMENT) {
    unpack<T>(__ldg(p.g + (size_t)t * p.n_vec + v), g);
  } else {
    const float s =
        p.gate == MOE_GATE_TOKEN ? DT<T>::to_f(reinterpret_cast<const T*>(p.g)[t]) : 1.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) g[i] = s;
  }
}

// A norm weight's factor o + w (1 without a weight).
template <typename T>
__device__ __forceinline__ void load_weight(const uint4* w, float o, int v, float (&f)[kVec]) {
  if (w) {
    unpack<T>(__ldg(w + v), f);
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] += o;
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = 1.0f;
  }
}

template <typename T, int VPT>
__global__ void __launch_bounds__(512)
    block_norm_fwd_kernel(const NormArgs p, uint4* r_out, uint4* h_out) {
  __shared__ float s_red[2][1][32];
  const int n_warps = blockDim.x >> 5;
  const int t = blockIdx.x;
  const size_t row = (size_t)t * p.n_vec;
  float r[VPT][kVec];
  uint4 xv[VPT];
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    uint4 yv = make_uint4(0, 0, 0, 0);
    xv[i] = make_uint4(0, 0, 0, 0);
    if (v < p.n_vec) {
      yv = p.y[row + v];
      if (p.x) xv[i] = p.x[row + v];
    }
    unpack<T>(yv, r[i]);
  }
  float ry = 1.0f;
  if (p.post) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) ss[0] = fmaf(r[i][j], r[i][j], ss[0]);
    cta_sum<1>(ss, s_red[0], n_warps);
    ry = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
  }
  ss[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < p.n_vec) {
      float f[kVec], x[kVec];
      if (p.post) {
        load_weight<T>(p.wq, p.o, v, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) r[i][j] = r[i][j] * ry * f[j];
      }
      load_gate<T>(p, t, v, f);
      unpack<T>(xv[i], x);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        r[i][j] *= f[j];
        if (p.x) r[i][j] = fmaf(p.a, x[j], r[i][j]);
        ss[0] = fmaf(r[i][j], r[i][j], ss[0]);
      }
      if (r_out) r_out[row + v] = pack<T>(r[i]);
    }
  }
  if (!p.pre) return;
  cta_sum<1>(ss, s_red[1], n_warps);
  const float rr = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < p.n_vec) {
      float f[kVec];
      load_weight<T>(p.wp, p.o, v, f);
#pragma unroll
      for (int j = 0; j < kVec; ++j) f[j] *= r[i][j] * rr;
      h_out[row + v] = pack<T>(f);
    }
  }
}

struct NormGrads {
  const uint4 *dr, *dh;
  uint4 *dy, *dx, *dg;      // dg: element gate only
  void* dg_token;           // token gate
  float* part;              // [gridDim.x][n_cols][H] per-channel partial sums
  int col_g, col_q, col_p;  // which of the n_cols sums is d_gate, d_post_weight, d_pre_weight
  int n_cols;
};

// One row at a time per CTA, grid-strided; the per-channel sums stay in the threads that own the
// channels and go to `part` at the end, one row of partial sums per CTA.
template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512)
    block_norm_bwd_kernel(const NormArgs p, const NormGrads q) {
  __shared__ float s_red[3][2][32];
  const int n_warps = blockDim.x >> 5;
  float acc_g[VPT][kVec] = {}, acc_q[VPT][kVec] = {}, acc_p[VPT][kVec] = {};
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const size_t row = (size_t)t * p.n_vec;
    float y[VPT][kVec], d[VPT][kVec], r[VPT][kVec];
    uint4 dhv[VPT];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float s1[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      const bool in = v < p.n_vec;
      unpack<T>(in ? p.y[row + v] : zero, y[i]);
      unpack<T>(in && q.dr ? q.dr[row + v] : zero, d[i]);
      unpack<T>(in && p.x ? p.x[row + v] : zero, r[i]);
      dhv[i] = in && p.pre ? q.dh[row + v] : zero;
#pragma unroll
      for (int j = 0; j < kVec; ++j) s1[0] = fmaf(y[i][j], y[i][j], s1[0]);
    }
    float ry = 1.0f;
    if (p.post) {
      cta_sum<1>(s1, s_red[0], n_warps);
      ry = rsqrtf(fmaf(s1[0], p.inv_h, p.eps));
    }
    if (p.pre) {
      float s2[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < p.n_vec) {
          float f[kVec], g[kVec], dn[kVec], wp[kVec];
          load_weight<T>(p.post ? p.wq : nullptr, p.o, v, f);
          load_gate<T>(p, t, v, g);
          unpack<T>(dhv[i], dn);
          load_weight<T>(p.wp, p.o, v, wp);
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            r[i][j] = fmaf(p.a, r[i][j], g[j] * (y[i][j] * ry * f[j]));
            s2[0] = fmaf(r[i][j], r[i][j], s2[0]);
            s2[1] = fmaf(r[i][j], dn[j] * wp[j], s2[1]);
          }
        }
      }
      cta_sum<2>(s2, s_red[1], n_warps);
      const float rr = rsqrtf(fmaf(s2[0], p.inv_h, p.eps));
      const float c = s2[1] * rr * rr * p.inv_h;  // mean(dh wp' rhat) rr
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < p.n_vec) {
          float dn[kVec], wp[kVec];
          unpack<T>(dhv[i], dn);
          load_weight<T>(p.wp, p.o, v, wp);
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            d[i][j] = fmaf(rr, dn[j] * wp[j] - c * r[i][j], d[i][j]);
            acc_p[i][j] = fmaf(dn[j], r[i][j] * rr, acc_p[i][j]);
          }
        }
      }
    }
    // d = D; the residual's and the gate's gradients, and the branch's (r holds it from here).
    float s3[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < p.n_vec) {
        float f[kVec], g[kVec], w[kVec];
        load_weight<T>(p.post ? p.wq : nullptr, p.o, v, w);
        load_gate<T>(p, t, v, g);
        if (q.dx) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) f[j] = p.a * d[i][j];
          q.dx[row + v] = pack<T>(f);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float yh = y[i][j] * ry;
          f[j] = d[i][j] * (yh * w[j]);  // D u
          s3[1] += f[j];
          acc_g[i][j] += f[j];
          const float du = d[i][j] * g[j];
          acc_q[i][j] = fmaf(du, yh, acc_q[i][j]);
          r[i][j] = du * w[j];
          s3[0] = fmaf(r[i][j], yh, s3[0]);
          y[i][j] = yh;
        }
        if (q.dg) q.dg[row + v] = pack<T>(f);
      }
    }
    cta_sum<2>(s3, s_red[2], n_warps);
    if (q.dg_token && threadIdx.x == 0)
      reinterpret_cast<T*>(q.dg_token)[t] = DT<T>::from_f(s3[1]);
    const float c = p.post ? s3[0] * p.inv_h : 0.0f;
    if (q.dy) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < p.n_vec) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) r[i][j] = ry * fmaf(-c, y[i][j], r[i][j]);
          q.dy[row + v] = pack<T>(r[i]);
        }
      }
    }
    __syncthreads();  // s_red is written again by the next row
  }
  auto put = [&](int col, const float (&acc)[VPT][kVec]) {
    if (col < 0) return;
    float4* dst =
        reinterpret_cast<float4*>(q.part + ((size_t)blockIdx.x * q.n_cols + col) * p.H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < p.n_vec) {
        dst[2 * v] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        dst[2 * v + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    }
  };
  put(q.col_g, acc_g);
  put(q.col_q, acc_q);
  put(q.col_p, acc_p);
}

// out[col][h] = sum over the CTAs' partial rows, in a fixed order: thread (x, y) adds rows
// y, y + 8, ... of one channel, and the eight sums are added in order.
constexpr int kRedX = 32, kRedY = 8;
struct RedOut {
  void* out[3];
};
template <typename T>
__global__ void __launch_bounds__(kRedX * kRedY)
    block_norm_reduce_kernel(const float* __restrict__ part, int rows, int n_cols, int H,
                             const RedOut o) {
  __shared__ float s[kRedY][kRedX];
  const int h = blockIdx.x * kRedX + threadIdx.x;
  const int col = blockIdx.y;
  float a = 0.0f;
  if (h < H)
#pragma unroll 4
    for (int c = threadIdx.y; c < rows; c += kRedY)
      a += part[((size_t)c * n_cols + col) * H + h];
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && h < H) {
#pragma unroll
    for (int y = 1; y < kRedY; ++y) a += s[y][threadIdx.x];
    reinterpret_cast<T*>(o.out[col])[h] = DT<T>::from_f(a);
  }
}

NormArgs norm_args(const moe_block_norm_t& b, const void* branch, const void* residual,
                   const void* gate, const void* wq, const void* wp) {
  NormArgs p;
  p.T = b.T;
  p.H = b.H;
  p.n_vec = b.H / kVec;
  p.gate = b.gate;
  p.post = b.post_norm != 0;
  p.pre = b.pre_norm != 0;
  p.a = b.residual_scale;
  p.o = b.weight_offset;
  p.eps = b.eps;
  p.inv_h = 1.0f / (float)b.H;
  p.y = static_cast<const uint4*>(branch);
  p.x = static_cast<const uint4*>(residual);
  p.g = static_cast<const uint4*>(gate);
  p.wq = static_cast<const uint4*>(wq);
  p.wp = static_cast<const uint4*>(wp);
  return p;
}

int threads_for(int n_vec, int vpt) {
  const int n = (n_vec + vpt - 1) / vpt;
  return (n + 31) / 32 * 32;
}

template <typename T>
cudaError_t fwd_typed(const NormArgs& p, void* r, void* h, cudaStream_t s) {
  uint4* ro = static_cast<uint4*>(r);
  uint4* ho = static_cast<uint4*>(h);
  const dim3 grid(p.T);
  if (p.n_vec <= 256)
    return launch_k(block_norm_fwd_kernel<T, 1>, grid, dim3(threads_for(p.n_vec, 1)), 0, s,
                    false, p, ro, ho);
  if (p.n_vec <= 1024)
    return launch_k(block_norm_fwd_kernel<T, 2>, grid, dim3(threads_for(p.n_vec, 2)), 0, s,
                    false, p, ro, ho);
  return launch_k(block_norm_fwd_kernel<T, 4>, grid, dim3(threads_for(p.n_vec, 4)), 0, s, false,
                  p, ro, ho);
}

template <typename T>
cudaError_t bwd_typed(const NormArgs& p, const NormGrads& q, int ctas, const RedOut& red,
                      cudaStream_t s) {
  if (p.T > 0) {
    cudaError_t e;
    if (p.n_vec <= 1024)
      e = launch_k(block_norm_bwd_kernel<T, 1>, dim3(ctas), dim3(threads_for(p.n_vec, 1)), 0, s,
                   false, p, q);
    else
      e = launch_k(block_norm_bwd_kernel<T, 4>, dim3(ctas), dim3(threads_for(p.n_vec, 4)), 0, s,
                   false, p, q);
    if (e != cudaSuccess) return e;
  }
  if (q.n_cols == 0) return cudaSuccess;
  return launch_k(block_norm_reduce_kernel<T>, dim3((p.H + kRedX - 1) / kRedX, q.n_cols),
                  dim3(kRedX, kRedY), 0, s, false, (const float*)q.part, ctas, q.n_cols, p.H,
                  red);
}

}  // namespace

int block_norm_bwd_ctas(int T) {
  const int n = num_sms();
  return T < n ? T : n;
}

cudaError_t launch_block_norm_fwd(const moe_block_norm_t& b, const void* branch,
                                  const void* residual, const void* gate, const void* wq,
                                  const void* wp, void* r, void* h, cudaStream_t s) {
  const NormArgs p = norm_args(b, branch, residual, gate, wq, wp);
  return b.dtype == MOE_BF16 ? fwd_typed<__nv_bfloat16>(p, r, h, s) : fwd_typed<__half>(p, r, h, s);
}

cudaError_t launch_block_norm_bwd(const moe_block_norm_t& b, const void* dr, const void* dh,
                                  const void* branch, const void* residual, const void* gate,
                                  const void* wq, const void* wp, void* dy, void* dx, void* dg,
                                  void* dwq, void* dwp, float* part, cudaStream_t s) {
  const NormArgs p = norm_args(b, branch, residual, gate, wq, wp);
  NormGrads q = {};
  q.dr = static_cast<const uint4*>(dr);
  q.dh = static_cast<const uint4*>(dh);
  q.dy = static_cast<uint4*>(dy);
  q.dx = static_cast<uint4*>(dx);
  q.dg = b.gate == MOE_GATE_ELEMENT ? static_cast<uint4*>(dg) : nullptr;
  q.dg_token = b.gate == MOE_GATE_TOKEN ? dg : nullptr;
  q.part = part;
  RedOut red = {};
  auto col = [&](void* out) {
    if (!out) return -1;
    red.out[q.n_cols] = out;
    return q.n_cols++;
  };
  q.col_g = col(b.gate == MOE_GATE_CHANNEL ? dg : nullptr);
  q.col_q = col(dwq);
  q.col_p = col(dwp);
  const int ctas = block_norm_bwd_ctas(b.T);
  return b.dtype == MOE_BF16 ? bwd_typed<__nv_bfloat16>(p, q, ctas, red, s)
                             : bwd_typed<__half>(p, q, ctas, red, s);
}

}  // namespace gb300moe
