// block_norm.cu -- the norm, gate and residual between two blocks (include/moe.h:
// moe_block_norm_fwd, moe_block_norm_bwd).
//
//   u = y ry q, r = a x + g u, h = r rr w;  ry, rr = 1/sqrt(mean square + eps), q = o + wq, w = o + wp
//
// Both means need the whole row, so a row is read once and stays with the threads that read it
// (a "group"); its reductions run over the group.  Everything between load and store is f32.
//   row kernel    forward of few rows, where latency counts: one CTA per row
//   group kernels persistent, one CTA per SM with as many groups as fit: while one group waits
//                 for a reduction or for memory another one computes.  Each thread copies its own
//                 vectors of its next row to shared memory (cp.async) while it works on the
//                 current one: nobody else reads them, so no barrier orders them.  The
//                 per-channel vectors lie in shared memory once per CTA.
//
// The bytes of the rows bound both directions; measured on a GB300 (copy 6.8 TB/s), bf16, gate per
// channel: forward 4096 x 7168 in 39.5-42 us (0.83-0.88 of the copy rate; 4096 x 4096 0.97), one row
// 3.0-3.9 us.  Backward 4096 x 7168 in 80 us (0.65): its warps, 22% of what an SM holds, wait most
// for shared memory (short scoreboard), with no pipe above 53%.
#include <mutex>

#include "block_ops.cuh"
#include "vec16.cuh"
#include "ptx.cuh"

namespace gb300moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kPairs = kVec / 2;

struct NormArgs {
  int T, H, n_vec;  // n_vec = H / 8
  int gate, post, pre;
  float a, o, eps, inv_h;
  const uint4 *y, *x, *g, *wq, *wp;
};

struct NormGrads {
  const uint4 *dr, *dh;
  uint4 *dy, *dx, *dg;  // dg: element gate only
  void* dg_token;       // token gate
  float* part;          // [gridDim.x][n_cols][H] per-channel partial sums
  int col_a, col_p;     // which of the n_cols sums are A and P (below), -1: not wanted
  int n_cols;
};
// Per-channel sums over the rows: P = sum dh rhat, and A = sum c D yhat with c the gate where it
// varies by row and 1 otherwise.  d_pre_weight = P; with a gate per channel d_gate = q A and
// d_post_weight = g A, else d_post_weight = A.

// Sums of N (one or two) values over a group of `warps` warps, the same bits in every thread:
// shuffles within a warp, then each warp adds the warps' sums in the same way.  Consecutive calls of a
// group use the two halves of `buf` in turn: a half is written again only behind the barrier of
// the call between.
template <int N>
struct GroupSum {
  float (*buf)[N][32];  // [2][N][the CTA's warps]
  int warps, warp, lane, bar, threads;
  int base = 0;  // the group's first warp in the CTA
  int turn = 0;
  // Over the warp.  Of two values each half warp takes one after the first exchange, so that they
  // cost one shuffle more than one; lane 0 then holds the first, lane 16 the second.
  __device__ __forceinline__ float over_warp(const float (&v)[N], int n) const {
    float x = v[0];
    if (N == 2 && n == 2) {
      const bool low = lane < 16;
      x = (low ? v[0] : v[N - 1]) + __shfl_xor_sync(kAll, low ? v[N - 1] : v[0], 16);
    } else {
      x += __shfl_xor_sync(kAll, x, 16);
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(kAll, x, off);
    return x;
  }
  __device__ __forceinline__ void operator()(float (&v)[N], int n = N) {
    const float x = over_warp(v, n);
    if (warps == 1) {
      v[0] = __shfl_sync(kAll, x, 0);
      if (N == 2 && n == 2) v[N - 1] = __shfl_sync(kAll, x, 16);
      return;
    }
    if ((lane & 15) == 0 && (lane >> 4) < n) buf[turn][N == 2 ? lane >> 4 : 0][base + warp] = x;
    named_bar_sync(bar, threads);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n && lane < warps ? buf[turn][i][base + lane] : 0.0f;
    const float y = over_warp(v, n);
    v[0] = __shfl_sync(kAll, y, 0);
    if (N == 2 && n == 2) v[N - 1] = __shfl_sync(kAll, y, 16);
    turn ^= 1;
  }
};

__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <typename T>
__device__ __forceinline__ float token_gate(const NormArgs& p, int t) {
  return DT<T>::to_f(reinterpret_cast<const T*>(p.g)[t]);
}

// ---- forward, one CTA per row -----------------------------------------------------------------
template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512)
    norm_row_kernel(const NormArgs p, uint4* r_out, uint4* h_out) {
  __shared__ float s_red[2][1][32];
  const int t = blockIdx.x;
  const size_t row = (size_t)t * p.n_vec;
  GroupSum<1> sum{s_red, (int)blockDim.x >> 5, (int)threadIdx.x >> 5, (int)threadIdx.x & 31, 0,
                  (int)blockDim.x};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 yv[VPT], xv[VPT], gv[VPT], qv[VPT], wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {  // everything is asked for before anything is needed
    const int v = threadIdx.x + i * blockDim.x;
    const bool in = v < p.n_vec;
    yv[i] = in ? p.y[row + v] : zero;
    xv[i] = in && p.x ? p.x[row + v] : zero;
    gv[i] = zero;
    if (in && p.gate == MOE_GATE_CHANNEL) gv[i] = __ldg(p.g + v);
    if (in && p.gate == MOE_GATE_ELEMENT) gv[i] = __ldg(p.g + row + v);
    qv[i] = in && p.wq ? __ldg(p.wq + v) : zero;
    wv[i] = in && p.wp ? __ldg(p.wp + v) : zero;
  }
  const F2 gt = f2(p.gate == MOE_GATE_TOKEN ? token_gate<T>(p, t) : 1.0f);
  const F2 oq = f2(p.wq ? p.o : 1.0f), ow = f2(p.wp ? p.o : 1.0f), a = f2(p.x ? p.a : 0.0f);
  F2 r[VPT][kPairs];
  float ss[1] = {0.0f};
  float ry = 1.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) unpack<T>(yv[i], r[i]);
  if (p.post) {
    F2 s = f2(0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < kPairs; ++j) s = f2_fma(r[i][j], r[i][j], s);
    ss[0] = f2_sum(s);
    sum(ss);
    ry = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
  }
  F2 s = f2(0.0f);
  const F2 ry2 = f2(ry);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    F2 f[kPairs], x[kPairs];
    if (p.post) {
      unpack<T>(qv[i], f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) r[i][j] = r[i][j] * ry2 * (f[j] + oq);
    }
    if (p.gate == MOE_GATE_CHANNEL || p.gate == MOE_GATE_ELEMENT) {
      unpack<T>(gv[i], f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) r[i][j] = r[i][j] * f[j];
    } else {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) r[i][j] = r[i][j] * gt;
    }
    unpack<T>(xv[i], x);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (p.x) r[i][j] = f2_fma(a, x[j], r[i][j]);
      s = f2_fma(r[i][j], r[i][j], s);
    }
    if (r_out && v < p.n_vec) r_out[row + v] = pack<T>(r[i]);
  }
  if (!p.pre) return;
  ss[0] = f2_sum(s);
  sum(ss);
  const F2 rr = f2(rsqrtf(fmaf(ss[0], p.inv_h, p.eps)));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    F2 f[kPairs];
    unpack<T>(wv[i], f);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) f[j] = (f[j] + ow) * (r[i][j] * rr);
    if (v < p.n_vec) h_out[row + v] = pack<T>(f);
  }
}

// ---- group kernels -----------------------------------------------------------------------------
// Shared memory: the per-channel vectors (kChanRows rows of 16-bit values in size), then each
// group's row buffers of n_vec vectors.
constexpr int kChanRows = 4;
struct GroupShape {
  int threads;  // of a group
  int groups;
  size_t smem;
};

// What a group thread knows of its place.
template <int N>
struct Place {
  int g, tid;
  GroupSum<N> sum;
  __device__ __forceinline__ Place(int threads, float (*red)[N][32]) {
    g = threadIdx.x / threads;
    tid = threadIdx.x - g * threads;
    sum.buf = red;
    sum.base = g * (threads >> 5);
    sum.warps = threads >> 5;
    sum.warp = tid >> 5;
    sum.lane = tid & 31;
    sum.bar = 1 + g;
    sum.threads = threads;
  }
};

// What multiplies a row channel by channel: c q (the gate per channel, if it is one, times the
// post weight's factor) and w (the pre weight's), f32.  They are made once per CTA in shared
// memory, [2][H]; kWide: the rows leave no room for that, so they are made where they are needed.
template <typename T, bool kWide>
struct Channels {
  const uint4 *g, *wq, *wp;
  F2 oq, ow;
  const F2* shared;
  int n_vec;
  __device__ __forceinline__ Channels(const NormArgs& p, void* s)
      : g(p.gate == MOE_GATE_CHANNEL ? p.g : nullptr), wq(p.wq), wp(p.wp),
        oq(f2(p.wq ? p.o : 1.0f)), ow(f2(p.wp ? p.o : 1.0f)), shared(static_cast<F2*>(s)),
        n_vec(p.n_vec) {
    if constexpr (kWide) return;
    F2* to = static_cast<F2*>(s);
    for (int v = threadIdx.x; v < n_vec; v += blockDim.x) {
      F2 a[kPairs], b[kPairs];
      make_post(v, a);
      make_pre(v, b);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        to[at(0, v, j)] = a[j];
        to[at(1, v, j)] = b[j];
      }
    }
  }
  __device__ __forceinline__ void make_post(int v, F2 (&f)[kPairs]) const {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) f[j] = oq;
    if (wq) {
      unpack<T>(__ldg(wq + v), f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) f[j] = f[j] + oq;
    }
    if (g) {
      F2 x[kPairs];
      unpack<T>(__ldg(g + v), x);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) f[j] = f[j] * x[j];
    }
  }
  __device__ __forceinline__ void make_pre(int v, F2 (&f)[kPairs]) const {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) f[j] = ow;
    if (wp) {
      unpack<T>(__ldg(wp + v), f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) f[j] = f[j] + ow;
    }
  }
  // The eight values of vector v lie as two halves of 16 bytes, each next to its neighbours': lanes
  // that read consecutive vectors then meet every bank once.
  __device__ __forceinline__ int at(int which, int v, int j) const {
    return ((which * 2 + j / 2) * n_vec + v) * 2 + j % 2;
  }
  __device__ __forceinline__ void read(int which, int v, F2 (&f)[kPairs]) const {
#pragma unroll
    for (int j = 0; j < kPairs; j += 2) {
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(shared + at(which, v, j));
      f[j].v = x.x;
      f[j + 1].v = x.y;
    }
  }
  __device__ __forceinline__ void post(int v, F2 (&f)[kPairs]) const {
    if constexpr (kWide) make_post(v, f); else read(0, v, f);
  }
  __device__ __forceinline__ void pre(int v, F2 (&f)[kPairs]) const {
    if constexpr (kWide) make_pre(v, f); else read(1, v, f);
  }
};

constexpr int kFwdCta = 1024;  // threads of a forward CTA: 64 registers each
constexpr int kBwdCta = 512;   // of a backward CTA: 128 registers, for the per-channel sums
template <typename T, int VPT, int GATE, bool kWide>
__global__ void __launch_bounds__(kWide ? 512 : kFwdCta, 1)
    norm_group_kernel(const NormArgs p, const GroupShape shape, uint4* r_out, uint4* h_out) {
  constexpr int kTensors = GATE == MOE_GATE_ELEMENT ? 3 : 2;  // y, x, gate
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float s_red[2][1][32];
  Place<1> me(shape.threads, s_red);
  // [2 rows][tensor][n_vec] of this group
  uint4* buf = reinterpret_cast<uint4*>(dyn) + (kWide ? 0 : kChanRows * p.n_vec) +
               (size_t)me.g * 2 * kTensors * p.n_vec;
  const Channels<T, kWide> chan(p, dyn);
  __syncthreads();
  const unsigned step = gridDim.x * shape.groups, T_all = p.T;  // t + step may pass 2^31
  auto fetch = [&](unsigned t, int half) {
    if (t < T_all) {
      const size_t row = (size_t)t * p.n_vec;
      uint4* b = buf + half * kTensors * p.n_vec;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = me.tid + i * shape.threads;
        if (v >= p.n_vec) continue;
        copy_async(b + v, p.y + row + v);
        if (p.x) copy_async(b + p.n_vec + v, p.x + row + v);
        if constexpr (GATE == MOE_GATE_ELEMENT)
          copy_async(b + 2 * p.n_vec + v, p.g + row + v);
      }
    }
    copy_commit();
  };
  const F2 a = f2(p.a);
  const unsigned t0 = blockIdx.x + me.g * gridDim.x;
  fetch(t0, 0);
  int half = 0;
  for (unsigned t = t0; t < T_all; t += step, half ^= 1) {
    fetch(t + step, half ^ 1);
    copy_wait<1>();
    const size_t row = (size_t)t * p.n_vec;
    const uint4* b = buf + half * kTensors * p.n_vec;
    F2 r[VPT][kPairs];
    float ss[1];
    float scale = GATE == MOE_GATE_TOKEN ? token_gate<T>(p, t) : 1.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me.tid + i * shape.threads;
      unpack<T>(v < p.n_vec ? b[v] : make_uint4(0, 0, 0, 0), r[i]);
    }
    if (p.post) {
      F2 s = f2(0.0f);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) s = f2_fma(r[i][j], r[i][j], s);
      ss[0] = f2_sum(s);
      me.sum(ss);
      scale *= rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
    }
    F2 s = f2(0.0f);
    const F2 sc = f2(scale);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me.tid + i * shape.threads;
      if (v >= p.n_vec) continue;
      F2 gw[kPairs], x[kPairs];
      chan.post(v, gw);
      if constexpr (GATE == MOE_GATE_ELEMENT) {
        unpack<T>(b[2 * p.n_vec + v], x);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) gw[j] = gw[j] * x[j];
      }
#pragma unroll
      for (int j = 0; j < kPairs; ++j) r[i][j] = r[i][j] * sc * gw[j];
      if (p.x) {
        unpack<T>(b[p.n_vec + v], x);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) r[i][j] = f2_fma(a, x[j], r[i][j]);
      }
#pragma unroll
      for (int j = 0; j < kPairs; ++j) s = f2_fma(r[i][j], r[i][j], s);
      if (r_out) r_out[row + v] = pack<T>(r[i]);
    }
    if (p.pre) {
      ss[0] = f2_sum(s);
      me.sum(ss);
      const F2 rr = f2(rsqrtf(fmaf(ss[0], p.inv_h, p.eps)));
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = me.tid + i * shape.threads;
        if (v >= p.n_vec) continue;
        F2 f[kPairs];
        chan.pre(v, f);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) f[j] = f[j] * (r[i][j] * rr);
        h_out[row + v] = pack<T>(f);
      }
    }
  }
  copy_wait<0>();
}

// D = dr + rr (dh w - rhat mean(dh w rhat));  dx = a D;  dg = D u;
// dy = ry (g D q - yhat mean(g D q yhat)).  r is computed again from y and x.
template <typename T, int VPT, int GATE, bool kWide>
__global__ void __launch_bounds__(kBwdCta, 1)
    norm_group_bwd_kernel(const NormArgs p, const NormGrads q, const GroupShape shape) {
  constexpr int kTensors = GATE == MOE_GATE_ELEMENT ? 5 : 4;  // y, x, dr, dh, gate
  constexpr int kRows = kWide ? 1 : 2;  // rows in shared memory: the next one too, if it fits
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ float s_red[2][2][32];
  pdl_trigger();  // the sums over the CTAs wait for this grid before they read
  Place<2> me(shape.threads, s_red);
  const int n_vec = p.n_vec;
  uint4* rows = reinterpret_cast<uint4*>(dyn) + (kWide ? 0 : kChanRows * n_vec);
  uint4* buf = rows + (size_t)me.g * kRows * kTensors * n_vec;  // [row][tensor][n_vec]
  const Channels<T, kWide> chan(p, dyn);
  if (!p.x || !q.dr || !p.pre)  // what is not there stays zero
    for (int v = threadIdx.x; v < shape.groups * kRows * kTensors * n_vec; v += blockDim.x)
      rows[v] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const unsigned step = gridDim.x * shape.groups, T_all = p.T;  // t + step may pass 2^31
  auto fetch = [&](unsigned t, int half) {
    if (t < T_all) {
      const size_t row = (size_t)t * n_vec;
      uint4* b = buf + half * kTensors * n_vec;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = me.tid + i * shape.threads;
        if (v >= n_vec) continue;
        copy_async(b + v, p.y + row + v);
        if (p.x) copy_async(b + n_vec + v, p.x + row + v);
        if (q.dr) copy_async(b + 2 * n_vec + v, q.dr + row + v);
        if (p.pre) copy_async(b + 3 * n_vec + v, q.dh + row + v);
        if constexpr (GATE == MOE_GATE_ELEMENT) copy_async(b + 4 * n_vec + v, p.g + row + v);
      }
    }
    copy_commit();
  };
  const F2 a = f2(p.a);
  F2 sum_a[VPT][kPairs], sum_p[VPT][kPairs];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < kPairs; ++j) sum_a[i][j] = sum_p[i][j] = f2(0.0f);
  // This thread's part of a row's sum of y^2.
  auto square = [&](const uint4* b) {
    F2 s = f2(0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me.tid + i * shape.threads;
      if (v >= n_vec) continue;
      F2 y[kPairs];
      unpack<T>(b[v], y);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) s = f2_fma(y[j], y[j], s);
    }
    return f2_sum(s);
  };
  const unsigned t0 = blockIdx.x + me.g * gridDim.x;
  float ss[2] = {0.0f, 0.0f};
  float ry = 1.0f;  // of the current row; the next one's is reduced with this row's last sum
  fetch(t0, 0);
  int half = 0;
  if (p.post && t0 < T_all) {
    copy_wait<0>();
    ss[0] = square(buf);
    me.sum(ss, 1);
    ry = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
  }
  for (unsigned t = t0; t < T_all; t += step) {
    if constexpr (!kWide) fetch(t + step, half ^ 1);
    copy_wait<kRows - 1>();
    const size_t row = (size_t)t * n_vec;
    const uint4* b = buf + half * kTensors * n_vec;
    const float gt = GATE == MOE_GATE_TOKEN ? token_gate<T>(p, t) : 1.0f;
    F2 d[VPT][kPairs];  // r, then D, then D c q
    float rr = 0.0f, c = 0.0f;  // D = dr + rr dh w - c r
    if (p.pre) {
      F2 s0 = f2(0.0f), s1 = f2(0.0f);
      const F2 sc = f2(ry * gt);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = me.tid + i * shape.threads;
        if (v >= n_vec) continue;
        F2 y[kPairs], x[kPairs], w[kPairs];
        unpack<T>(b[v], y);
        chan.post(v, w);
        if constexpr (GATE == MOE_GATE_ELEMENT) {
          unpack<T>(b[4 * n_vec + v], x);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) w[j] = w[j] * x[j];
        }
        unpack<T>(b[n_vec + v], x);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) d[i][j] = f2_fma(a, x[j], y[j] * sc * w[j]);
        unpack<T>(b[3 * n_vec + v], x);
        chan.pre(v, w);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          s0 = f2_fma(d[i][j], d[i][j], s0);
          s1 = f2_fma(d[i][j], x[j] * w[j], s1);
        }
      }
      ss[0] = f2_sum(s0);
      ss[1] = f2_sum(s1);
      me.sum(ss);
      rr = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
      c = -ss[1] * rr * rr * rr * p.inv_h;
    }
    const F2 rr2 = f2(rr), c2 = f2(c), ry2 = f2(ry), gt2 = f2(gt);
    F2 s = f2(0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = me.tid + i * shape.threads;
      if (v >= n_vec) continue;
      F2 f[kPairs], y[kPairs], w[kPairs];
      unpack<T>(b[2 * n_vec + v], f);
      if (p.pre) {
        unpack<T>(b[3 * n_vec + v], y);
        chan.pre(v, w);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          sum_p[i][j] = f2_fma(y[j], d[i][j] * rr2, sum_p[i][j]);
          d[i][j] = f2_fma(rr2, y[j] * w[j], f2_fma(c2, d[i][j], f[j]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) d[i][j] = f[j];
      }
      if (q.dx) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) f[j] = a * d[i][j];
        q.dx[row + v] = pack<T>(f);
      }
      unpack<T>(b[v], y);
      chan.post(v, w);
      if constexpr (GATE == MOE_GATE_ELEMENT) {
        F2 g[kPairs];
        unpack<T>(b[4 * n_vec + v], g);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const F2 e = d[i][j] * (y[j] * ry2);
          f[j] = e * w[j];  // D u
          sum_a[i][j] = f2_fma(g[j], e, sum_a[i][j]);
          s = f2_fma(g[j], f[j], s);
          d[i][j] = d[i][j] * (g[j] * w[j]);
        }
        if (q.dg) q.dg[row + v] = pack<T>(f);
      } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const F2 e = d[i][j] * (y[j] * ry2);
          if constexpr (GATE == MOE_GATE_TOKEN)
            sum_a[i][j] = f2_fma(gt2, e, sum_a[i][j]);
          else
            sum_a[i][j] = sum_a[i][j] + e;
          s = f2_fma(e, w[j], s);
          d[i][j] = d[i][j] * w[j];
        }
      }
    }
    ss[0] = ss[1] = 0.0f;
    const bool more = !kWide && p.post && t + step < T_all;
    if (p.post || GATE == MOE_GATE_TOKEN) {
      ss[0] = f2_sum(s);
      if (more) {
        copy_wait<0>();
        ss[1] = square(buf + (half ^ 1) * kTensors * n_vec);
      }
      me.sum(ss);
      if (GATE == MOE_GATE_TOKEN && q.dg_token && me.tid == 0)
        reinterpret_cast<T*>(q.dg_token)[t] = DT<T>::from_f(ss[0]);
    }
    if (q.dy) {
      const F2 k1 = f2(ry * gt);
      const F2 k2 = f2(p.post ? -ss[0] * gt * p.inv_h * ry * ry : 0.0f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = me.tid + i * shape.threads;
        if (v >= n_vec) continue;
        F2 y[kPairs];
        unpack<T>(b[v], y);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) y[j] = f2_fma(k2, y[j], k1 * d[i][j]);
        q.dy[row + v] = pack<T>(y);
      }
    }
    if constexpr (!kWide) {
      half ^= 1;
      if (more) ry = rsqrtf(fmaf(ss[1], p.inv_h, p.eps));
    } else {
      fetch(t + step, 0);
      if (p.post && t + step < T_all) {
        copy_wait<0>();
        ss[0] = square(buf);
        me.sum(ss, 1);
        ry = rsqrtf(fmaf(ss[0], p.inv_h, p.eps));
      }
    }
  }
  copy_wait<0>();
  if (q.n_cols == 0) return;
  // The groups' sums meet in the row buffers (as large as two f32 rows per group) and are added in
  // the order of the groups.
  __syncthreads();
  float4* s_sum = reinterpret_cast<float4*>(rows);  // [groups][2][2 n_vec]
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = me.tid + i * shape.threads;
    if (v >= p.n_vec) continue;
    float4* at = s_sum + (size_t)me.g * 4 * p.n_vec + 2 * v;
    const float2 a0 = f2_get(sum_a[i][0]), a1 = f2_get(sum_a[i][1]), a2 = f2_get(sum_a[i][2]),
                 a3 = f2_get(sum_a[i][3]);
    at[0] = make_float4(a0.x, a0.y, a1.x, a1.y);
    at[1] = make_float4(a2.x, a2.y, a3.x, a3.y);
    at += 2 * p.n_vec;
    const float2 p0 = f2_get(sum_p[i][0]), p1 = f2_get(sum_p[i][1]), p2 = f2_get(sum_p[i][2]),
                 p3 = f2_get(sum_p[i][3]);
    at[0] = make_float4(p0.x, p0.y, p1.x, p1.y);
    at[1] = make_float4(p2.x, p2.y, p3.x, p3.y);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int col = k == 0 ? q.col_a : q.col_p;
    if (col < 0) continue;
    float4* dst = reinterpret_cast<float4*>(q.part + ((size_t)blockIdx.x * q.n_cols + col) * p.H);
    for (int v = threadIdx.x; v < 2 * p.n_vec; v += blockDim.x) {
      float4 s = s_sum[(size_t)k * 2 * p.n_vec + v];
      for (int g = 1; g < shape.groups; ++g) {
        const float4 o = s_sum[(size_t)(2 * g + k) * 2 * p.n_vec + v];
        s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
      }
      dst[v] = s;
    }
  }
}

// Sums over the CTAs' partial rows, in a fixed order: thread (x, y) adds rows y, y + 16, ... of
// one channel, and the sixteen sums are added in order.
constexpr int kRedX = 32, kRedY = 16;
struct RedOut {
  void *g, *q, *p;      // d_gate per channel, d_post_weight, d_pre_weight (or null)
  const void *gate, *wq;  // per-channel gate (or null) and post weight (or null)
  float o;
  int col_a, col_p;
};
template <typename T>
__global__ void __launch_bounds__(kRedX * kRedY)
    norm_reduce_kernel(const float* __restrict__ part, int rows, int n_cols, int H,
                       const RedOut o) {
  __shared__ float s[kRedY][kRedX];
  pdl_wait();
  const int h = blockIdx.x * kRedX + threadIdx.x;
  const int col = blockIdx.y;
  float a = 0.0f;
  if (h < H)
#pragma unroll 8
    for (int c = threadIdx.y; c < rows; c += kRedY)
      a += part[((size_t)c * n_cols + col) * H + h];
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y != 0 || h >= H) return;
#pragma unroll
  for (int y = 1; y < kRedY; ++y) a += s[y][threadIdx.x];
  if (col == o.col_p) {
    static_cast<T*>(o.p)[h] = DT<T>::from_f(a);
    return;
  }
  if (o.g) {
    const float w = o.wq ? o.o + DT<T>::to_f(static_cast<const T*>(o.wq)[h]) : 1.0f;
    static_cast<T*>(o.g)[h] = DT<T>::from_f(a * w);
  }
  if (o.q) {
    const float g = o.gate ? DT<T>::to_f(static_cast<const T*>(o.gate)[h]) : 1.0f;
    static_cast<T*>(o.q)[h] = DT<T>::from_f(a * g);
  }
}

// ---- host side ---------------------------------------------------------------------------------
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

constexpr int kSmemMax = 226 * 1024;  // leaves room for the static arrays

// As many groups as the threads, the barriers and the shared memory allow; `chans` rows'
// worth of per-channel vectors lies beside the groups' `bufs` row buffers.
GroupShape group_shape(const NormArgs& p, int vpt, int most, int chans, int bufs) {
  GroupShape s;
  s.threads = threads_for(p.n_vec, vpt);
  s.groups = most / s.threads;
  // a group of one warp needs no barrier; there are fifteen for the others
  if (s.threads > 32 && s.groups > 15) s.groups = 15;
  const int row = p.n_vec * 16;
  const int fit = (kSmemMax - chans * row) / (bufs * row);
  if (s.groups > fit) s.groups = fit;
  s.smem = (size_t)(chans + s.groups * bufs) * row;
  return s;
}

template <auto Kernel, typename... Args>
cudaError_t launch_group(const GroupShape& s, int ctas, cudaStream_t stream, Args... args) {
  static cudaError_t result[64];
  static std::once_flag once[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (s.groups < 1) return cudaErrorInvalidConfiguration;
  std::call_once(once[dev], [dev] {
    result[dev] =
        cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  });
  if (result[dev] != cudaSuccess) return result[dev];
  return launch_k(Kernel, dim3(ctas), dim3(s.threads * s.groups), s.smem, stream, false, args...);
}

// Forward: two vectors per thread up to rows of 8192, so that the threads make two groups or more;
// four beyond.
bool fwd_wide(const NormArgs& p) { return threads_for(p.n_vec, 2) > kFwdCta / 2; }
GroupShape fwd_shape(const NormArgs& p) {
  const int bufs = p.gate == MOE_GATE_ELEMENT ? 6 : 4;
  return fwd_wide(p) ? group_shape(p, 4, 512, 0, bufs) : group_shape(p, 2, kFwdCta, kChanRows, bufs);
}
template <typename T, int GATE>
cudaError_t fwd_groups(const NormArgs& p, uint4* r, uint4* h, cudaStream_t s) {
  const GroupShape g = fwd_shape(p);
  const int ctas = p.T < num_sms() ? p.T : num_sms();
  return fwd_wide(p)
             ? launch_group<norm_group_kernel<T, 4, GATE, true>>(g, ctas, s, p, g, r, h)
             : launch_group<norm_group_kernel<T, 2, GATE, false>>(g, ctas, s, p, g, r, h);
}

template <typename T>
cudaError_t fwd_typed(const NormArgs& p, void* r, void* h, cudaStream_t s) {
  uint4* ro = static_cast<uint4*>(r);
  uint4* ho = static_cast<uint4*>(h);
  // A row per CTA while every group of the other kernel would get two rows or fewer.
  if ((int64_t)p.T <= 2ll * num_sms() * fwd_shape(p).groups) {
    const dim3 grid(p.T);
    if (p.n_vec <= 1024)
      return launch_k(norm_row_kernel<T, 1>, grid, dim3(threads_for(p.n_vec, 1)), 0, s, false, p,
                      ro, ho);
    return launch_k(norm_row_kernel<T, 4>, grid, dim3(threads_for(p.n_vec, 4)), 0, s, false, p,
                    ro, ho);
  }
  switch (p.gate) {
    case MOE_GATE_CHANNEL: return fwd_groups<T, MOE_GATE_CHANNEL>(p, ro, ho, s);
    case MOE_GATE_TOKEN: return fwd_groups<T, MOE_GATE_TOKEN>(p, ro, ho, s);
    case MOE_GATE_ELEMENT: return fwd_groups<T, MOE_GATE_ELEMENT>(p, ro, ho, s);
    default: return fwd_groups<T, MOE_GATE_NONE>(p, ro, ho, s);
  }
}

// Backward: two vectors per thread up to rows of 8192, four beyond.
template <typename T, int GATE>
cudaError_t bwd_groups(const NormArgs& p, const NormGrads& q, int ctas, cudaStream_t s) {
  const int bufs = GATE == MOE_GATE_ELEMENT ? 5 : 4;
  const GroupShape g = group_shape(p, 2, kBwdCta, kChanRows, 2 * bufs);
  if (g.groups >= 1)
    return launch_group<norm_group_bwd_kernel<T, 2, GATE, false>>(g, ctas, s, p, q, g);
  const GroupShape w = group_shape(p, 4, kBwdCta, 0, bufs);
  return launch_group<norm_group_bwd_kernel<T, 4, GATE, true>>(w, ctas, s, p, q, w);
}

template <typename T>
cudaError_t bwd_typed(const NormArgs& p, const NormGrads& q, int ctas, const RedOut& red,
                      cudaStream_t s) {
  if (p.T > 0) {
    cudaError_t e;
    switch (p.gate) {
      case MOE_GATE_CHANNEL: e = bwd_groups<T, MOE_GATE_CHANNEL>(p, q, ctas, s); break;
      case MOE_GATE_TOKEN: e = bwd_groups<T, MOE_GATE_TOKEN>(p, q, ctas, s); break;
      case MOE_GATE_ELEMENT: e = bwd_groups<T, MOE_GATE_ELEMENT>(p, q, ctas, s); break;
      default: e = bwd_groups<T, MOE_GATE_NONE>(p, q, ctas, s);
    }
    if (e != cudaSuccess) return e;
  }
  if (q.n_cols == 0) return cudaSuccess;
  return launch_k(norm_reduce_kernel<T>, dim3((p.H + kRedX - 1) / kRedX, q.n_cols),
                  dim3(kRedX, kRedY), 0, s, p.T > 0, (const float*)q.part, ctas, q.n_cols, p.H,
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
  red.g = b.gate == MOE_GATE_CHANNEL ? dg : nullptr;
  red.q = dwq;
  red.p = dwp;
  red.gate = b.gate == MOE_GATE_CHANNEL ? gate : nullptr;
  red.wq = wq;
  red.o = b.weight_offset;
  q.col_a = red.g || red.q ? q.n_cols++ : -1;
  q.col_p = red.p ? q.n_cols++ : -1;
  red.col_a = q.col_a;
  red.col_p = q.col_p;
  const int ctas = block_norm_bwd_ctas(b.T);
  return b.dtype == MOE_BF16 ? bwd_typed<__nv_bfloat16>(p, q, ctas, red, s)
                             : bwd_typed<__half>(p, q, ctas, red, s);
}

}  // namespace gb300moe
