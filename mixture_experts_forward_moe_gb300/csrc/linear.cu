// linear.cu -- dense product with bias, activation and residual in its epilogue (include/moe.h:
// moe_linear): out = act(x w^T + b) + residual, 16-bit operands, f32 accumulation.
//
// One row of x (a few, when the product is small) is a stream of the weights and runs on the CUDA
// cores (gemv_kernel).  Everything else runs on tcgen05: the weights are the MMA's M side, the rows
// of x its N side (BN), so that few rows of x cost few columns.  Up to 64 rows, in small products and
// up to 128 columns a CTA has a tile of 128 weight rows (mma_kernel), beyond that a pair of SMs has
// one of 256 (pair_kernel).
//
// What bounds it, and what it measured on a GB300 (bf16; a copy runs at 6.8 TB/s, a
// large library product at 1951 TFLOP/s in a burst and 1718 sustained):
//   one row: the weights' bytes; 7168 x 7168 in 18.6 us, 0.81 of the copy rate
//   16 and 64 rows: the same, and the start and join of a launch; 20.0-20.5 and 22.0-22.4 us
//   4096 x 7168 x 18432 with the residual: the MMAs (tensor pipe 90% active); 549-590 us, 0.94-1.01
//     of the burst rate
//   4096 x 7168 x 2048: the MMAs and the epilogue of the last wave; 82-87 us, 0.71-0.75
//   4096 x 256 x 7168 to f32: the tiles' loads from L2 and the join; 22 us, 0.45
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "block_ops.cuh"
#include "vec16.cuh"
#include "ptx.cuh"

namespace gb300moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// True in one lane of a converged warp.  The producer's and the issuer's loops run in that lane
// alone, so that stage, phase and addresses are those of one thread.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// mbar_try_wait may suspend the thread for a while; this only looks.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A bounded wait (as mbar_wait: false once `limit_ns` has passed or another role gave up, at the
// first look with a limit of 0) that reads the timer every 64 polls.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         uint64_t limit_ns, int* status) {
  if (limit_ns == 0) {
    if (mbar_test_wait(bar, parity)) return true;
  } else {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((it & 63) != 0) continue;
      if (*abort) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0)
        t0 = t;
      else if (t - t0 > limit_ns)
        break;
    }
  }
  *abort = 1;
  if (status) atomicCAS(status, 0, (int)MOE_ERR_TIMEOUT);
  return false;
}

// T, N and K may be anything up to 2^31 - 1: no sum of one of them with a tile's size is taken in 32
// bits.
struct LinArgs {
  int T, N, K;
  int act, out_f32;
  const void* bias;
  const void* res;
  void* out;
  int* status;
  uint64_t limit_ns;
};

// Position in a ring of `stages` barriers.  A look at a barrier takes over a hundred cycles to
// come back even when its phase is over, so the next stage's is looked at (`ready`) before the
// current stage's copies or MMAs are issued; only if it was not over yet is it waited for.
struct Ring {
  uint64_t* bars;
  int stages, stage;
  uint32_t parity;
  bool ready;
  __device__ __forceinline__ Ring(uint64_t* b, int n, uint32_t p)
      : bars(b), stages(n), stage(0), parity(p), ready(false) {}
  __device__ __forceinline__ uint64_t* bar() const { return bars + stage; }
  __device__ __forceinline__ void next() {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
    ready = mbar_test_wait(bars + stage, parity);
  }
};

// After a wait gave up: copies of the last `stages` of `issued` stages, or MMAs, land (one
// bounded budget) before the CTA leaves.  Whether one gave up is asked behind a barrier that all
// roles pass after their last wait: a role may be done with its own work before another gives up.
// (Waiting for them in every case cost 1.3 of 6.0 us at 5 x 256 x 7168: twelve looks at barriers.)
constexpr uint64_t kDrainNs = 1000000000ull;
__device__ __forceinline__ void land_copies(uint64_t* full_bar, int issued, int stages) {
  const uint64_t t = global_timer_ns();
  const int n = issued < stages ? issued : stages;
  for (int i = issued - n; i < issued; ++i)
    while (!mbar_try_wait(&full_bar[i % stages], (uint32_t)((i / stages) & 1)))
      if (global_timer_ns() - t > kDrainNs) break;
}
__device__ __forceinline__ void land_mmas(uint64_t* bar) {
  const uint64_t t = global_timer_ns();
  while (!mbar_try_wait(bar, 0))
    if (global_timer_ns() - t > kDrainNs) break;
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case MOE_LINEAR_SILU:
      return __fdividef(z, 1.0f + expf(-z));
    case MOE_LINEAR_GELU_TANH: {
      // z/2 (1 + tanh u) = z / (1 + e^-2u)
      const float u = 0.7978845608028654f * fmaf(0.044715f * z * z, z, z);
      return __fdividef(z, 1.0f + expf(-2.0f * u));
    }
    case MOE_LINEAR_RELU2: {
      const float r = fmaxf(z, 0.0f);
      return z != z ? z : r * r;
    }
    default:
      return z;
  }
}

// One output from its f32 sum.
template <typename T>
__device__ __forceinline__ void finish(const LinArgs& p, float z, int t, int n) {
  const int64_t o = (int64_t)t * p.N + n;
  if (p.bias) z += DT<T>::to_f(static_cast<const T*>(p.bias)[n]);
  z = activate(z, p.act);
  if (p.out_f32) {
    if (p.res) z += static_cast<const float*>(p.res)[o];
    static_cast<float*>(p.out)[o] = z;
  } else {
    if (p.res) z += DT<T>::to_f(static_cast<const T*>(p.res)[o]);
    static_cast<T*>(p.out)[o] = DT<T>::from_f(z);
  }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float ld_cluster_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Eight consecutive outputs of row t from their f32 sums, as whole vectors: N is a multiple of 8.
template <typename T>
struct Finish {
  const LinArgs& p;
  int n;
  float bias[8];
  __device__ __forceinline__ Finish(const LinArgs& a, int col) : p(a), n(col) {
#pragma unroll
    for (int j = 0; j < 8; ++j) bias[j] = 0.0f;
    if (a.bias && n < a.N)
      unpack<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.bias) + n), bias);
  }
  // The residuals of kCols rows t, t + step, ... below t1, asked for together: a branch or a
  // conversion between two loads would wait for the first.
  template <int kCols>
  __device__ __forceinline__ void residual(int t, int step, int t1, float (&r)[kCols][8]) const {
    if (!p.res || n >= p.N) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = 0.0f;
    } else if (p.out_f32) {
      float4 v[kCols][2];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const float4* src = reinterpret_cast<const float4*>(
            static_cast<const float*>(p.res) + (int64_t)(i * step < t1 - t ? t + i * step : t) * p.N +
            n);
        v[i][0] = src[0];
        v[i][1] = src[1];
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        r[i][0] = v[i][0].x, r[i][1] = v[i][0].y, r[i][2] = v[i][0].z, r[i][3] = v[i][0].w;
        r[i][4] = v[i][1].x, r[i][5] = v[i][1].y, r[i][6] = v[i][1].z, r[i][7] = v[i][1].w;
      }
    } else {
      uint4 v[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        v[i] = *reinterpret_cast<const uint4*>(
            static_cast<const T*>(p.res) + (int64_t)(i * step < t1 - t ? t + i * step : t) * p.N + n);
#pragma unroll
      for (int i = 0; i < kCols; ++i) unpack<T>(v[i], r[i]);
    }
  }
  __device__ __forceinline__ void store(int t, float (&z)[8], const float (&r)[8]) const {
    if (n >= p.N) return;
    const int64_t o = (int64_t)t * p.N + n;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += bias[j];
    if (p.act != MOE_LINEAR_NONE)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = activate(z[j], p.act);
    if (p.res)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] += r[j];
    if (p.out_f32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
      dst[0] = make_float4(z[0], z[1], z[2], z[3]);
      dst[1] = make_float4(z[4], z[5], z[6], z[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + o) = pack<T>(z);
    }
  }
};

// f[k] = from[at(k)], f32 or T, all asked for before the first is converted; 0 without `have`.
template <typename T, int kCount, typename At>
__device__ __forceinline__ void load_raw(float (&f)[kCount], bool have, const void* from, bool f32,
                                         At at) {
#pragma unroll
  for (int k = 0; k < kCount; ++k) f[k] = 0.0f;
  if (!have) return;
  if (f32) {
#pragma unroll
    for (int k = 0; k < kCount; ++k) f[k] = static_cast<const float*>(from)[at(k)];
  } else {
    T raw[kCount];
#pragma unroll
    for (int k = 0; k < kCount; ++k) raw[k] = static_cast<const T*>(from)[at(k)];
#pragma unroll
    for (int k = 0; k < kCount; ++k) f[k] = DT<T>::to_f(raw[k]);
  }
}

// The join below for any N: consecutive threads take consecutive outputs one by one.
template <typename T, int kSplit>
__device__ __forceinline__ void join_scalar(const LinArgs& p, uint32_t base, int c0, int c1,
                                            int n0, int t0, uint32_t stride, uint32_t first) {
  constexpr int kAtOnce = kSplit == 1 ? 16 : (kSplit == 2 ? 8 : (kSplit <= 4 ? 4 : 2));
  const int end = c1 * kSlab;
  for (int i = c0 * kSlab + (int)threadIdx.x; i < end; i += kAtOnce * (int)blockDim.x) {
    // everything is asked for before the first output is written: a store may hide any load
    float v[kAtOnce][kSplit], r[kAtOnce], b[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int at = i + k * (int)blockDim.x < end ? i + k * (int)blockDim.x : i;
#pragma unroll
      for (int s = 0; s < kSplit; ++s)
        v[k][s] = kSplit > 1 ? ld_cluster_f1(cluster_map(base + (uint32_t)at * 4u,
                                                         (uint32_t)s * stride + first))
                             : ld_shared_f1(base + (uint32_t)at * 4u);
    }
    // Bias and residual; an output that is not there stands for the first of the tile.
    auto place = [&](int k, int& n) -> int64_t {
      const int at = i + k * (int)blockDim.x;
      n = n0 + at % kSlab;
      const bool in = at < end && n < p.N;
      if (!in) n = n0;
      return (int64_t)(t0 + (in ? at / kSlab : c0)) * p.N + n;
    };
    load_raw<T, kAtOnce>(b, p.bias && n0 < p.N, p.bias, false, [&](int k) -> int64_t {
      int n;
      place(k, n);
      return n;
    });
    load_raw<T, kAtOnce>(r, p.res && n0 < p.N, p.res, p.out_f32 != 0, [&](int k) {
      int n;
      return place(k, n);
    });
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int at = i + k * (int)blockDim.x;
      const int n = n0 + at % kSlab;
      if (at >= end || n >= p.N) continue;
      float z = v[k][0];
#pragma unroll
      for (int s = 1; s < kSplit; ++s) z += v[k][s];
      z = activate(z + b[k], p.act) + r[k];
      const int64_t o = (int64_t)(t0 + at / kSlab) * p.N + n;
      if (p.out_f32)
        static_cast<float*>(p.out)[o] = z;
      else
        static_cast<T*>(p.out)[o] = DT<T>::from_f(z);
    }
  }
}

// The f32 sums of a tile lie in shared memory as [column][128 weight rows] at `base`, in kSplit
// parts of K that belong to the cluster's CTAs s * stride + first.  This CTA (part `part`) adds
// the parts of its share of the columns [0, cols), in their order, and finishes the outputs of
// the rows t0 ... of x: sixteen threads take the 128 consecutive outputs of a row.  A peer's
// shared memory is slow to answer, so all parts are asked for at once.
template <typename T, int kSplit>
__device__ __forceinline__ void join_parts(const LinArgs& p, uint32_t base, int cols, int n0,
                                           int t0, int part, uint32_t stride, uint32_t first) {
  const int c1 = cols * (part + 1) / kSplit;
  if ((p.N & 7) != 0)
    return join_scalar<T, kSplit>(p, base, cols * part / kSplit, c1, n0, t0, stride, first);
  const int g = threadIdx.x & 15;
  const Finish<T> f(p, n0 + g * 8);
  constexpr int kCols = kSplit <= 2 ? 4 : (kSplit <= 4 ? 2 : 1);  // rows of x at a time
  const int step = (int)blockDim.x / 16;
  for (int c = cols * part / kSplit + (int)(threadIdx.x >> 4); c < c1; c += kCols * step) {
    float4 v[kCols][kSplit][2];
    float r[kCols][8];
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int ci = c + i * step < c1 ? c + i * step : c;
      const uint32_t at = base + (uint32_t)((ci * kSlab + g * 8) * 4);
#pragma unroll
      for (int s = 0; s < kSplit; ++s) {
        if (kSplit > 1) {
          const uint32_t a = cluster_map(at, (uint32_t)s * stride + first);
          v[i][s][0] = ld_cluster_f4(a);
          v[i][s][1] = ld_cluster_f4(a + 16);
        } else {
          v[i][s][0] = ld_shared_f4(at);
          v[i][s][1] = ld_shared_f4(at + 16);
        }
      }
    }
    f.template residual<kCols>(t0 + c, step, t0 + c1, r);
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      if (c + i * step >= c1) break;
      float4 a = v[i][0][0], b = v[i][0][1];
#pragma unroll
      for (int s = 1; s < kSplit; ++s) {
        a.x += v[i][s][0].x, a.y += v[i][s][0].y, a.z += v[i][s][0].z, a.w += v[i][s][0].w;
        b.x += v[i][s][1].x, b.y += v[i][s][1].y, b.z += v[i][s][1].z, b.w += v[i][s][1].w;
      }
      float z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      f.store(t0 + c + i * step, z, r[i]);
    }
  }
}
template <typename T, int kMaxSplit>
__device__ __forceinline__ void join(const LinArgs& p, uint32_t base, int cols, int n0, int t0,
                                     int part, int split, uint32_t stride, uint32_t first) {
  if (split == 1) return join_parts<T, 1>(p, base, cols, n0, t0, part, stride, first);
  if (split == 2) return join_parts<T, 2>(p, base, cols, n0, t0, part, stride, first);
  if (split == 3) return join_parts<T, 3>(p, base, cols, n0, t0, part, stride, first);
  if (split == 4) return join_parts<T, 4>(p, base, cols, n0, t0, part, stride, first);
  if constexpr (kMaxSplit > 4) {
    if (split == 5) return join_parts<T, 5>(p, base, cols, n0, t0, part, stride, first);
    if (split == 6) return join_parts<T, 6>(p, base, cols, n0, t0, part, stride, first);
    if (split == 7) return join_parts<T, 7>(p, base, cols, n0, t0, part, stride, first);
    return join_parts<T, 8>(p, base, cols, n0, t0, part, stride, first);
  }
}

// Cluster barrier after which a CTA may leave: it orders nothing but the peers' finished reads
// (cluster_sync's release would first wait for this CTA's global stores).
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::
                   : "memory");
}

// ---- few rows: weights streamed once through the CUDA cores -----------------------------------
constexpr int kGemvRows = 4;
constexpr int kGemvWarps = 8;

// `wpr` warps (1, 2, 4 or 8) share one weight row; the CTA's 8 warps hold 8 / wpr rows.
template <typename T, int NT>
__global__ void __launch_bounds__(kGemvWarps * 32)
    gemv_kernel(const LinArgs p, const uint4* __restrict__ x, const uint4* __restrict__ w,
                int wpr) {
  __shared__ float s_part[kGemvWarps][NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = kGemvWarps / wpr;
  const int n = blockIdx.x * rows + warp / wpr;
  const int kv = p.K / 8;
  float acc[NT] = {};
  if (n < p.N) {
    const uint4* wr = w + (size_t)n * kv;
#pragma unroll 4
    for (int i = (warp % wpr) * 32 + lane; i < kv; i += wpr * 32) {
      float a[8], b[8];
      unpack<T>(__ldg(wr + i), a);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        unpack<T>(__ldg(x + (size_t)t * kv + i), b);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t] = fmaf(a[j], b[j], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc[t] += __shfl_xor_sync(kAll, acc[t], off);
    if (lane == 0) s_part[warp][t] = acc[t];
  }
  __syncthreads();
  const int i = threadIdx.x;
  if (i < rows * NT) {
    const int r = i % rows, t = i / rows;
    const int no = blockIdx.x * rows + r;
    if (no < p.N) {
      float z = 0.0f;
      for (int s = 0; s < wpr; ++s) z += s_part[r * wpr + s][t];
      finish<T>(p, z, t, no);
    }
  }
}

// ---- tcgen05: one 128 x BN tile per CTA, K split over a cluster -------------------------------
// A cluster of S CTAs shares a tile: CTA r multiplies its part of K, leaves its f32 accumulators
// in its shared memory, and after a cluster barrier each CTA adds all S parts of its share of the
// tile through distributed shared memory, in the order of the parts, and finishes it.
// Roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer, warps 2-5 read TMEM; all warps
// take part in the join.  Every wait is bounded (MOE_ERR_TIMEOUT in the status word); a CTA that
// gave up still meets the barriers and waits, bounded, for its copies and MMAs in flight.
// The tensor cores add to an accumulator with truncation, so its error grows with the number of
// additions: the 64-k blocks go round kAccs accumulators, which the epilogue adds.
// kLong: f32 results of so many blocks that an accumulator would meet more than kDrainKb of them.
// It meets kDrainKb in a row, and the epilogue warps add it to sums in registers while the next ones
// fill.  128 x 128 x 32768: 16.5 us and an error of 4.8e-7 in norms; without it 15.1 us and 1.0e-6; on
// SM pairs, which do the same, 29.7 us.  16 x 19584 x 7168: 49.1 us and 4.8e-7, without 49.2 and 1.8e-6.
constexpr int kMmaThreads = 192;
constexpr int kAccs = 4;
constexpr int kMaxStages = 12;
constexpr int kDrainKb = 8;

template <int BN>
struct Shape {
  static constexpr int kStages = BN == 32 ? 3 : 4;
  static constexpr int kABytes = kSlab * kBlockK * 2;
  static constexpr int kBBytes = BN * kBlockK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kTmemCols = kAccs * BN;
  // CTAs that fit an SM (228 KB of shared memory, 512 TMEM columns)
  static constexpr int kPerSm = BN <= 32 ? 3 : 2;
  static_assert(kPerSm * kTmemCols <= 512, "TMEM");
  static_assert(BN * kSlab * 4 <= kStages * kStageBytes, "the accumulators of a join");
};

template <typename T, int BN, bool kLong>
__global__ void __launch_bounds__(kMmaThreads)
    mma_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const LinArgs p, int split, int stages) {
  using S = Shape<BN>;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kMaxStages];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ __align__(8) uint64_t tfull_bar[kAccs];   // kLong: an accumulator is to be added,
  __shared__ __align__(8) uint64_t tempty_bar[kAccs];  // and was
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  // the same offset in every CTA of the cluster: the join reads the peers' tiles there
  const uint32_t raw = smem_u32(dsmem);
  uint8_t* smem = dsmem + ((1024u - (raw & 1023u)) & 1023u);
  const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = blockIdx.x / split;
  const int slabs = (p.N - 1) / kSlab + 1;
  const int n0 = (tile % slabs) * kSlab;
  const int t0 = (tile / slabs) * BN;
  const int num_kb = (p.K - 1) / kBlockK + 1;
  const int kb0 = (int)((int64_t)num_kb * rank / split);
  const int kb1 = (int)((int64_t)num_kb * (rank + 1) / split);
  const int cols = p.T - t0 < BN ? p.T - t0 : BN;  // live columns

  auto load = [&](int kb, int stage) {
    uint8_t* st = smem + stage * S::kStageBytes;
    mbar_arrive_expect_tx(&full_bar[stage], S::kStageBytes);
    tma_load_2d(st, &tmW, &full_bar[stage], kb * kBlockK, n0);
    tma_load_2d(st + S::kABytes, &tmX, &full_bar[stage], kb * kBlockK, t0);
  };
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < stages; ++s) {
        mbar_init(&full_bar[s], 1);
        mbar_init(&empty_bar[s], 1);
      }
      mbar_init(&done_bar, 1);
      if constexpr (kLong)
        for (int a = 0; a < kAccs; ++a) {
          mbar_init(&tfull_bar[a], 1);
          mbar_init(&tempty_bar[a], 4);  // an arrival per epilogue warp
        }
      s_abort = 0;
      fence_mbar_init();
    }
  } else if (warp == 1) {
    tmem_alloc(&s_tmem, S::kTmemCols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  int issued = 0;       // by the producer: stages asked for
  bool issuer = false;  // the thread that issues the MMAs

  if (warp == 0) {
    if (elect_one()) {
      Ring r(empty_bar, stages, 1u);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!r.ready && !wait_bar(r.bar(), r.parity, abort_flag, p.limit_ns, p.status)) break;
        const int stage = r.stage;
        r.next();
        load(kb, stage);
        ++issued;
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      issuer = true;
      Ring r(full_bar, stages, 0u);
      const uint32_t base = smem_u32(smem);
      const uint32_t idesc = idesc_f16_m128(BN, DT<T>::kIsBF16);
      for (int kb = kb0; kb < kb1; ++kb) {
        const int i = kb - kb0;
        const int pass = i / kDrainKb, acc = kLong ? pass % kAccs : i % kAccs;
        const bool fresh = kLong ? i % kDrainKb == 0 : i < kAccs;  // the accumulator starts over
        if (kLong && fresh && pass >= kAccs &&
            !wait_bar(&tempty_bar[acc], (uint32_t)((pass / kAccs - 1) & 1), abort_flag, p.limit_ns,
                      p.status))
          break;
        if (!r.ready && !wait_bar(r.bar(), r.parity, abort_flag, p.limit_ns, p.status)) break;
        tc_fence_after();
        const uint32_t sa = base + (uint32_t)(r.stage * S::kStageBytes);
        const uint32_t sb = sa + (uint32_t)S::kABytes;
        const uint32_t d = tmem + (uint32_t)(acc * BN);
        uint64_t* empty = &empty_bar[r.stage];
        r.next();
#pragma unroll
        for (int k = 0; k < kBlockK / 16; ++k)
          umma_f16(d, sw128_kmajor_desc(sa + k * 32), sw128_kmajor_desc(sb + k * 32), idesc,
                   (!fresh || k > 0) ? 1u : 0u);
        umma_commit(empty);
        if (kLong && (i % kDrainKb == kDrainKb - 1 || kb + 1 == kb1)) umma_commit(&tfull_bar[acc]);
      }
      // done_bar flips when every MMA issued has completed
      umma_commit(&done_bar);
    }
  } else if constexpr (kLong) {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float sum[BN] = {};
    bool ok = true;
    for (int pass = 0; kb0 + pass * kDrainKb < kb1 && ok; ++pass) {
      const int acc = pass % kAccs;
      ok = __all_sync(kAll, wait_bar(&tfull_bar[acc], (uint32_t)((pass / kAccs) & 1), abort_flag,
                                     p.limit_ns, p.status));
      tc_fence_after();
      if (!ok) break;
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 16) {
        float v[16];
        tmem_ld_x16(tb + (uint32_t)(acc * BN + c0), v);
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[c0 + j] += v[j];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[acc]);
    }
    // the last pass' MMAs have completed, so nothing reads the stages any more
    float* stash = reinterpret_cast<float*>(smem);
    if (ok) {
#pragma unroll
      for (int c = 0; c < BN; ++c)
        if (c < cols) stash[c * kSlab + row] = sum[c];
    }
  } else {
    const bool ok =
        __all_sync(kAll, wait_bar(&done_bar, 0, abort_flag, p.limit_ns, p.status));
    tc_fence_after();
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
    if (ok) {
      float* stash = reinterpret_cast<float*>(smem);
      const int accs = kb1 - kb0 < kAccs ? kb1 - kb0 : kAccs;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        tmem_ld_x16(tb + (uint32_t)c0, v);
        for (int a = 1; a < accs; ++a) {
          float u[16];
          tmem_ld_x16(tb + (uint32_t)(a * BN + c0), u);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += u[j];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) stash[(c0 + j) * kSlab + row] = v[j];
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  join<T, 8>(p, smem_u32(smem), cols, n0, t0, rank, split, 1u, 0u);
  if (*abort_flag) {
    land_copies(full_bar, issued, stages);
    if (issuer) land_mmas(&done_bar);
  }
  __syncwarp();
  if (split > 1) cluster_leave();  // a peer may still read this CTA's part
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// ---- tcgen05 on pairs of SMs: 256 x BN tiles -------------------------------------------------
// One SM's MMA of 128 x BN reads (128 + BN) rows of shared memory per k while TMA writes as many,
// and at BN = 128 that alone asks for twice the 128 bytes a cycle that shared memory gives.  A
// pair of CTAs (cta_group::2) multiplies 256 weight rows by BN rows of x with each CTA holding
// 128 weight rows and half of the rows of x: at BN = 256 half the traffic per MMA.
// A cluster is `split` pairs, each with its part of K; the CTAs of the same side join as above.
// At BN = 256 two CTAs share an SM: one's epilogue and start run under the other's MMAs.  At 128 a
// CTA has its SM alone and four stages of two blocks.
// Roles (192 threads): warp 0 TMA producer; warp 1 issues the MMAs (even CTA) or tells the even
// CTA that a stage of this CTA has landed (odd CTA); warps 2-5 epilogue.
// kF32: f32 results.  Every kDrainKb blocks the MMAs move on to the other of two accumulators
// and the epilogue warps add the finished one to sums in registers, rounded to nearest (the
// tensor cores truncate; a chain over all of K would cost several bits).
constexpr int kJoinCols = 128;  // columns whose sums are in shared memory at a time (64 KB)

// TMEM address of the lanes that an epilogue warp may read.
__device__ __forceinline__ uint32_t tmem_lane(uint32_t tmem, int warp) {
  return tmem + ((uint32_t)((warp & 3) * 32) << 16);
}
// Columns [from, from + min(cols, kJoinCols)) of a warp's accumulator rows, to shared memory.
__device__ __forceinline__ void stash_cols(uint32_t tb, int from, float* stash, int row,
                                           int cols) {
  for (int c0 = 0; c0 < cols && c0 < kJoinCols; c0 += 16) {
    float v[16];
    tmem_ld_x16(tb + (uint32_t)(from + c0), v);
#pragma unroll
    for (int j = 0; j < 16; ++j) stash[(c0 + j) * kSlab + row] = v[j];
  }
}

template <int BN, bool kF32>
struct PairShape {
  // 64-k blocks per stage: at BN = 128 the four MMAs of one block take less time than a stage's
  // waits and arrivals
  static constexpr int kKps = BN == 128 ? 2 : 1;
  static constexpr int kPerSm = BN == 128 ? 1 : 2;
  static constexpr int kABytes = kSlab * kBlockK * 2;
  static constexpr int kBBytes = BN / 2 * kBlockK * 2;
  static constexpr int kBlockBytes = kABytes + kBBytes;
  static constexpr int kStageBytes = kKps * kBlockBytes;
  static constexpr int kStages = BN == 128 ? 4 : 3;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
  static constexpr int kMaxStages = BN == 128 ? 4 : 6;  // of a CTA alone on its SM
  static constexpr int kBufs = kF32 ? 2 : 1;
  static constexpr int kTmemCols = kBufs * BN;
  static_assert(kPerSm * (kSmem + 2048) <= 228 * 1024 && kPerSm * kTmemCols <= 512, "per SM");
  static_assert(kJoinCols * kSlab * 4 <= kStages * kStageBytes, "the sums of a tile");
  static_assert(!kF32 || (BN == 128 && kDrainKb % kKps == 0), "the sums of a row stay in registers");
};

// Arrives on the barrier at this offset of both CTAs of the pair when the MMAs issued so far
// have completed.
__device__ __forceinline__ void umma_commit_both(uint32_t bar, uint32_t even) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)(3u << even))
      : "memory");
}

template <typename T, int BN, bool kF32>
__global__ void __launch_bounds__(kMmaThreads, PairShape<BN, kF32>::kPerSm)
    pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const LinArgs p, int split, int stages) {
  using S = PairShape<BN, kF32>;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[S::kMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[S::kMaxStages];
  __shared__ __align__(8) uint64_t tfull_bar[S::kBufs];
  __shared__ __align__(8) uint64_t tempty_bar[S::kBufs];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t raw = smem_u32(dsmem);
  uint8_t* smem = dsmem + ((1024u - (raw & 1023u)) & 1023u);
  const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  const uint32_t rank = cluster_ctarank();
  const uint32_t side = rank & 1u, even = rank & ~1u;
  const int part = (int)(rank >> 1);
  const int tile = blockIdx.x / (2 * split);
  const int slabs = (p.N - 1) / (2 * kSlab) + 1;
  const int n0 = (tile % slabs) * 2 * kSlab + (int)side * kSlab;  // this CTA's weight rows
  const int t0 = (tile / slabs) * BN;
  const int num_kb = (p.K - 1) / kBlockK + 1;
  const int kb0 = (int)((int64_t)num_kb * part / split);
  const int kb1 = (int)((int64_t)num_kb * (part + 1) / split);
  const int cols = p.T - t0 < BN ? p.T - t0 : BN;
  const int mma_n = (cols + 31) & ~31;  // each CTA holds half of these rows of x
  const int chunk = kF32 ? kDrainKb : kb1 - kb0;  // blocks of one accumulator pass

  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < stages; ++s) {
        // the even CTA's stage is full when its copies and, by the forwarder, the odd CTA's landed
        mbar_init(&full_bar[s], side == 0 ? 2 : 1);
        mbar_init(&empty_bar[s], 1);
      }
      for (int b = 0; b < S::kBufs; ++b) {
        mbar_init(&tfull_bar[b], 1);
        mbar_init(&tempty_bar[b], 8);  // an arrival per epilogue warp of both CTAs
      }
      mbar_init(&drain_bar, 1);
      s_abort = 0;
      fence_mbar_init();
    }
  } else if (warp == 1) {
    tmem_alloc_pair(&s_tmem, S::kTmemCols);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool got = false;  // this epilogue warp saw its accumulator
  int issued = 0;    // by the producer: stages asked for
  const uint32_t peer_abort = cluster_map(smem_u32(&s_abort), rank ^ 1u);
  // by one thread; on giving up the peer CTA is told too
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (wait_bar(bar, parity, abort_flag, p.limit_ns, p.status)) return true;
    st_cluster_u32(peer_abort, 1u);
    return false;
  };

  if (warp == 0) {
    if (elect_one()) {
      Ring r(empty_bar, stages, 1u);
      const int tx = t0 + (int)side * (mma_n / 2);
      for (int kb = kb0; kb < kb1; kb += S::kKps) {
        if (!r.ready && !wait(r.bar(), r.parity)) break;
        uint8_t* st = smem + r.stage * S::kStageBytes;
        uint64_t* full = &full_bar[r.stage];
        r.next();
        const int n = kb1 - kb < S::kKps ? kb1 - kb : S::kKps;
        mbar_arrive_expect_tx(full, (uint32_t)(n * S::kBlockBytes));
#pragma unroll
        for (int j = 0; j < S::kKps; ++j) {
          if (j >= n) break;
          uint8_t* at = st + j * S::kBlockBytes;
          tma_load_2d(at, &tmW, full, (kb + j) * kBlockK, n0);
          tma_load_2d(at + S::kABytes, &tmX, full, (kb + j) * kBlockK, tx);
        }
        ++issued;
      }
    }
  } else if (warp == 1 && side != 0) {
    if (elect_one()) {
      Ring r(full_bar, stages, 0u);
      const uint32_t to = cluster_map(smem_u32(full_bar), even);
      for (int kb = kb0; kb < kb1; kb += S::kKps) {
        if (!r.ready && !wait(r.bar(), r.parity)) break;
        mbar_arrive_cluster(to + (uint32_t)r.stage * 8u);
        r.next();
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      Ring r(full_bar, stages, 0u);
      int buf = 0;
      uint32_t buf_phase = 0;
      bool ok = true;
      const uint32_t base = smem_u32(smem);
      const uint32_t idesc = idesc_f16(256, mma_n, DT<T>::kIsBF16);
      const uint32_t empty_own = smem_u32(empty_bar), tfull_own = smem_u32(tfull_bar);
      for (int kc = kb0; kc < kb1 && ok; kc += chunk) {
        if (kF32 && !wait(&tempty_bar[buf], buf_phase ^ 1u)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * BN);
        const int ke = kc + chunk < kb1 ? kc + chunk : kb1;
        for (int kb = kc; kb < ke; kb += S::kKps) {
          if (!r.ready && !wait(r.bar(), r.parity)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = base + (uint32_t)(r.stage * S::kStageBytes);
          const uint32_t at = (uint32_t)r.stage * 8u;
          r.next();
#pragma unroll
          for (int j = 0; j < S::kKps; ++j) {
            if (kb + j >= ke) break;
            const uint32_t sa = st + (uint32_t)(j * S::kBlockBytes);
            const uint32_t sb = sa + (uint32_t)S::kABytes;
#pragma unroll
            for (int k = 0; k < kBlockK / 16; ++k)
              umma_f16_pair(d, sw128_kmajor_desc(sa + k * 32), sw128_kmajor_desc(sb + k * 32),
                            idesc, (kb > kc || j > 0 || k > 0) ? 1u : 0u);
          }
          umma_commit_both(empty_own + at, even);
        }
        if (!ok) break;
        umma_commit_both(tfull_own + (uint32_t)buf * 8u, even);
        if (++buf == S::kBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      // every MMA issued has completed once drain_bar flips
      umma_commit_pair(smem_u32(&drain_bar));
      land_mmas(&drain_bar);
    }
  } else {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tb = tmem_lane(tmem, warp);
    float* stash = reinterpret_cast<float*>(smem);
    if constexpr (kF32) {
      float acc[BN] = {};
      int buf = 0;
      uint32_t buf_phase = 0;
      bool ok = true;
      for (int kc = kb0; kc < kb1 && ok; kc += chunk) {
        ok = __all_sync(kAll, wait(&tfull_bar[buf], buf_phase));
        tc_fence_after();
        if (ok) {
#pragma unroll
          for (int c0 = 0; c0 < BN; c0 += 16) {
            float v[16];
            tmem_ld_x16(tb + (uint32_t)(buf * BN + c0), v);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c0 + j] += v[j];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_map(smem_u32(&tempty_bar[buf]), even));
        }
        if (++buf == S::kBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      if (ok) {
#pragma unroll
        for (int c = 0; c < BN; ++c)
          if (c < cols) stash[c * kSlab + row] = acc[c];
      }
    } else {
      got = __all_sync(kAll, wait(&tfull_bar[0], 0));
      tc_fence_after();
      if (got) stash_cols(tb, 0, stash, row, cols);
    }
  }
  __syncwarp();
  tc_fence_before();
  // Both CTAs of a pair are past their MMAs here, and the parts of a split are in place.
  cluster_sync();
  tc_fence_after();
  join<T, 4>(p, smem_u32(smem), cols < kJoinCols ? cols : kJoinCols, n0, t0, part, split, 2u, side);
  if constexpr (BN > kJoinCols) {  // not split: the second half by the CTA alone
    if (cols > kJoinCols) {
      __syncthreads();
      if (warp >= 2 && got) stash_cols(tmem_lane(tmem, warp), kJoinCols,
                                       reinterpret_cast<float*>(smem), (warp & 3) * 32 + lane,
                                       cols - kJoinCols);
      __syncwarp();
      tc_fence_before();
      __syncthreads();
      join_parts<T, 1>(p, smem_u32(smem), cols - kJoinCols, n0, t0 + kJoinCols, 0, 2u, side);
    }
  }
  // (the even CTA's stages are full only with the odd CTA's copies told of: else a second passes)
  if (*abort_flag) land_copies(full_bar, issued, stages);
  __syncwarp();
  if (split > 1)
    cluster_leave();  // a peer may still read this CTA's part
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::kTmemCols);
  }
}

// ---- host side ---------------------------------------------------------------------------------
constexpr int kSmemLimit = 226 * 1024;  // dynamic; leaves room for the static variables

// Sets a kernel's shared-memory limit, once per device; `Kernel` names the instance.
template <auto Kernel>
cudaError_t set_smem_limit(int bytes) {
  static cudaError_t result[64];
  static std::once_flag once[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [dev, bytes] {
    result[dev] =
        cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  return result[dev];
}

// Clusters of `cluster` CTAs with `smem` bytes each (one size per kernel) that the device holds at
// once: a cluster stays within one group of SMs, so this can be less than SMs / cluster.
template <auto Kernel>
int max_clusters(int cluster, int smem) {
  static int cached[64][9];
  static std::once_flag once[64][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || cluster > 8) return 0;
  std::call_once(once[dev][cluster], [=] {
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (set_smem_limit<Kernel>(kSmemLimit) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    cached[dev][cluster] = n;
  });
  return cached[dev][cluster];
}

template <auto Kernel, typename... Rest>
cudaError_t launch_tiles(const LinArgs& p, int dtype, const void* x, const void* w, int box_x,
                         int smem, int64_t ctas, int cluster, cudaStream_t s, Rest... rest) {
  const cudaError_t e = set_smem_limit<Kernel>(kSmemLimit);
  if (e != cudaSuccess) return e;
  CUtensorMap tmW, tmX;
  if (!make_map16(&tmW, dtype, w, (uint64_t)p.K, (uint64_t)p.N, kSlab) ||
      !make_map16(&tmX, dtype, x, (uint64_t)p.K, (uint64_t)p.T, (uint32_t)box_x))
    return cudaErrorInvalidValue;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kMmaThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, Kernel, tmW, tmX, p, rest...);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Split K while the SMs take the parts, two each (one of 64-row tiles), and each part keeps at
// least seven 64-k blocks.  16 x 7168 x 7168: 20.0 us in the five parts of this rule, 20.4 in two,
// 21.1 in four, 23.5 in eight.  64 rows: 22.2 in the two parts of this rule, 24.3 in one or five.
// 33 x 4096 x 2048: 7.2 in its four, 8.3 in one, 7.0 in three, 8.5 in eight.  Against two per SM
// 64-row tiles lose most at 826 x 494 x 1808, 10.9 to 10.6.
template <int BN>
int mma_split(const LinArgs& p) {
  const int64_t tiles = ceil_div(p.N, kSlab) * ceil_div(p.T, BN), num_kb = ceil_div(p.K, kBlockK);
  const int64_t sms = num_sms();
  int split = 1;
  while (split < 8 && num_kb >= (split + 1) * 7 &&
         tiles * (split + 1) <= (BN == 64 ? sms : 2 * sms))
    ++split;
  return split;
}

// f32 results of which an accumulator of a one-CTA tile would meet more than kDrainKb blocks: past
// that 2048 x 128 x 18432 was off by 1.1e-6 (norms), and by 4.8e-7 within.
template <int BN>
bool long_sums(const LinArgs& p) {
  return p.out_f32 && ceil_div(p.K, kBlockK) > (int64_t)kAccs * mma_split<BN>(p) * kDrainKb;
}

template <typename T, int BN>
cudaError_t launch_mma(const LinArgs& p, int dtype, const void* x, const void* w,
                       cudaStream_t s) {
  const int64_t tiles = ceil_div(p.N, kSlab) * ceil_div(p.T, BN);
  const int split = mma_split<BN>(p);
  // Alone on its SM a CTA takes all the shared memory for stages.
  int stages = Shape<BN>::kStages;
  if (tiles * split <= num_sms()) stages = (kSmemLimit - 1024) / Shape<BN>::kStageBytes;
  if (stages > kMaxStages) stages = kMaxStages;
  const int smem = stages * Shape<BN>::kStageBytes + 1024;
  return long_sums<BN>(p) ? launch_tiles<mma_kernel<T, BN, true>>(
                                p, dtype, x, w, BN, smem, tiles * split, split, s, split, stages)
                          : launch_tiles<mma_kernel<T, BN, false>>(
                                p, dtype, x, w, BN, smem, tiles * split, split, s, split, stages);
}

template <typename T, int BN, bool kF32>
cudaError_t launch_pair(const LinArgs& p, int dtype, const void* x, const void* w,
                        cudaStream_t s) {
  const int64_t tiles = ceil_div(p.N, 2 * kSlab) * ceil_div(p.T, BN);
  const int num_kb = (p.K - 1) / kBlockK + 1;
  int split = 1;
  if (BN == 128)  // a part of a 256-column tile does not fit beside a second CTA
    while (split < 4 && num_kb >= (split + 1) * 7 &&
           tiles <= max_clusters<pair_kernel<T, BN, kF32>>(2 * (split + 1),
                                                              PairShape<BN, kF32>::kSmem))
      ++split;
  // A CTA alone on its SM needs the stages of two to keep as many bytes on the way.
  const bool alone = tiles * split * 2 <= num_sms();
  const int stages = alone ? PairShape<BN, kF32>::kMaxStages : PairShape<BN, kF32>::kStages;
  return launch_tiles<pair_kernel<T, BN, kF32>>(
      p, dtype, x, w, BN / 2, stages * PairShape<BN, kF32>::kStageBytes + 1024,
      tiles * split * 2, 2 * split, s, split, stages);
}

template <typename T>
cudaError_t launch_gemv(const LinArgs& p, const void* x, const void* w, cudaStream_t s) {
  // Warps per weight row: enough for about sixteen warps per SM.
  int wpr = 1;
  while (wpr < kGemvWarps && (int64_t)p.N * wpr < (int64_t)num_sms() * 16 &&
         p.K / 8 >= wpr * 2 * 32)
    wpr *= 2;
  const int rows = kGemvWarps / wpr;
  const dim3 grid((p.N - 1) / rows + 1), block(kGemvWarps * 32);
  const uint4* xv = static_cast<const uint4*>(x);
  const uint4* wv = static_cast<const uint4*>(w);
  switch (p.T) {
    case 1: return launch_k(gemv_kernel<T, 1>, grid, block, 0, s, false, p, xv, wv, wpr);
    case 2: return launch_k(gemv_kernel<T, 2>, grid, block, 0, s, false, p, xv, wv, wpr);
    case 3: return launch_k(gemv_kernel<T, 3>, grid, block, 0, s, false, p, xv, wv, wpr);
    default: return launch_k(gemv_kernel<T, 4>, grid, block, 0, s, false, p, xv, wv, wpr);
  }
}

// Products of at most this many 128 x 64 x 64 blocks stay with one-CTA tiles: a pair's start and
// cluster barriers cost more than its better use of shared memory gains (905 x 224 x 296, 150
// blocks: 7.0 us against 8.9; 826 x 494 x 1808, 1508: 11.8 against 13.9; 512 x 256 x 7168, 1792:
// 15.9 against 13.3; 128 x 2048 x 4096, 2048: 13.3 against 11.0).
constexpr int64_t kSmallTiles = 1600;

template <typename T>
cudaError_t launch_typed(const LinArgs& p, int dtype, const void* x, const void* w,
                         cudaStream_t s) {
  // Two to four rows cost the CUDA cores two to four times the arithmetic of one, which hides behind
  // the weights' bytes no more: 7168 x 7168 took 18.4, 22.6, 27.9 and 38.8 us against 19.5 on the
  // tensor cores, 256 x 7168 with two to four rows 3.1 to 3.8 against 5.8, and 2048 x 2048 crosses at
  // four rows.
  if (p.T == 1 || (p.T <= kGemvRows && (int64_t)p.T * p.N * p.K <= 1 << 24))
    return launch_gemv<T>(p, x, w, s);
  if (p.T <= 16) return launch_mma<T, 16>(p, dtype, x, w, s);
  if (p.T <= 32) return launch_mma<T, 32>(p, dtype, x, w, s);
  const int64_t kbs = ceil_div(p.K, kBlockK);
  // Up to kSlab columns a pair's second CTA has no column of its own: 4096 x 128 x 2048 took 11.1 us
  // on pairs and 8.3 here, 32768 x 128 x 1024 36.4 and 21.8, 8192 x 32 x 4096 20.1 and 17.0.  (Three
  // slabs lose a quarter of a pair, and less than pairs gain: 8192 x 384 x 7168 41.5 and 72.6.)
  // f32 results of long sums stay on pairs there.
  const bool narrow_out = p.N <= kSlab && !long_sums<64>(p);
  if (p.T <= 64 || narrow_out ||
      ceil_div(p.N, kSlab) * ceil_div(p.T, 64) * kbs <= kSmallTiles)
    return launch_mma<T, 64>(p, dtype, x, w, s);
  if (p.out_f32) return launch_pair<T, 128, true>(p, dtype, x, w, s);
  // The time of the busiest SM, in thirds of a pass over K with a 128-column tile: those run one
  // per SM at a time.  A 256-column tile alone on its SM takes 1.4 of them (512 x 4096 x 7168: 28
  // and 39 us), two that share an SM 2.7 (8192^3: 895 us in 128 columns, 594 in 256).
  const int64_t slabs = ceil_div(p.N, 2 * kSlab), sms = num_sms();
  const int64_t narrow = 3 * ceil_div(slabs * ceil_div(p.T, 128) * 2, sms);
  const int64_t wide_ctas = slabs * ceil_div(p.T, 256) * 2;
  const int64_t wide = wide_ctas <= sms ? 4 : 8 * ceil_div(wide_ctas, 2 * sms);
  return wide <= narrow ? launch_pair<T, 256, false>(p, dtype, x, w, s)
                        : launch_pair<T, 128, false>(p, dtype, x, w, s);
}

}  // namespace

cudaError_t launch_linear(const moe_linear_t& g, const void* x, const void* w, const void* bias,
                          const void* residual, void* out, int* status, cudaStream_t s) {
  LinArgs p;
  p.T = g.T;
  p.N = g.N;
  p.K = g.K;
  p.act = g.activation;
  p.out_f32 = g.out_f32 != 0;
  p.bias = bias;
  p.res = residual;
  p.out = out;
  p.status = status;
  p.limit_ns = wait_limit_ns();
  return g.dtype == MOE_BF16 ? launch_typed<__nv_bfloat16>(p, g.dtype, x, w, s)
                             : launch_typed<__half>(p, g.dtype, x, w, s);
}

}  // namespace gb300moe
