// linear.cu -- dense product with bias, activation and residual in its epilogue (include/moe.h:
// moe_linear): out = act(x w^T + b) + residual, 16-bit operands, f32 accumulation.
//
// Up to kGemvRows rows of x the product is a stream of the weights and runs on the CUDA cores
// (gemv_kernel).  Beyond that it runs on tcgen05 (mma_kernel): the weights are the MMA's M side
// (128 rows), the rows of x its N side (BN), so that few rows of x cost few columns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "vec16.cuh"
#include "ptx.cuh"

namespace gb300moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;

struct LinArgs {
  int T, N, K;
  int act, out_f32;
  const void* bias;
  const void* res;
  void* out;
  int* status;
  uint64_t limit_ns;
};

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

// Sixteen consecutive rows of x (t ... t+15, the first `live` of them) for one output column: all
// residuals are asked for before the first is needed.
template <typename T>
__device__ __forceinline__ void finish16(const LinArgs& p, float (&z)[16], int t, int live,
                                         int n) {
  const float b = p.bias ? DT<T>::to_f(static_cast<const T*>(p.bias)[n]) : 0.0f;
  const int64_t o = (int64_t)t * p.N + n;
  float r[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    r[j] = 0.0f;
    if (p.res && j < live)
      r[j] = p.out_f32 ? static_cast<const float*>(p.res)[o + (int64_t)j * p.N]
                       : DT<T>::to_f(static_cast<const T*>(p.res)[o + (int64_t)j * p.N]);
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (j >= live) break;
    float v = z[j] + b;
    if (p.act != MOE_LINEAR_NONE) v = activate(v, p.act);
    if (p.res) v += r[j];
    if (p.out_f32)
      static_cast<float*>(p.out)[o + (int64_t)j * p.N] = v;
    else
      static_cast<T*>(p.out)[o + (int64_t)j * p.N] = DT<T>::from_f(v);
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

// Adds the `split` parts of a tile of 128 weight rows by `cols` rows of x, in their order, and
// finishes this CTA's share (the `part`-th of `split`).  Part s lies at `base` of the cluster's
// CTA s * stride + first, as [column][128 rows].
template <typename T>
__device__ __forceinline__ void join(const LinArgs& p, uint32_t base, int cols, int n0, int t0,
                                     int part, int split, uint32_t stride, uint32_t first) {
  // four rows of one column per item
  const int items = cols * (kSlab / 4);
  const int i0 = (int)((int64_t)items * part / split);
  const int i1 = (int)((int64_t)items * (part + 1) / split);
  for (int i = i0 + (int)threadIdx.x; i < i1; i += (int)blockDim.x) {
    float4 v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < split)
        v[s] = ld_cluster_f4(cluster_map(base + (uint32_t)i * 16u, (uint32_t)s * stride + first));
    float4 z = v[0];
#pragma unroll
    for (int s = 1; s < 8; ++s)
      if (s < split) {
        z.x += v[s].x;
        z.y += v[s].y;
        z.z += v[s].z;
        z.w += v[s].w;
      }
    const int t = t0 + i / (kSlab / 4);
    const int n = n0 + (i % (kSlab / 4)) * 4;
    if (n < p.N) finish<T>(p, z.x, t, n);
    if (n + 1 < p.N) finish<T>(p, z.y, t, n + 1);
    if (n + 2 < p.N) finish<T>(p, z.z, t, n + 2);
    if (n + 3 < p.N) finish<T>(p, z.w, t, n + 3);
  }
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
// gave up waits, bounded, for its copies and MMAs in flight and still meets the barriers.
// The tensor cores add to an accumulator with truncation, so its error grows with the number of
// additions: the 64-k blocks go round kAccs accumulators, which the epilogue adds.
constexpr int kMmaThreads = 192;
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr int kAccs = 4;

template <int BN>
struct Shape {
  static constexpr int kStages = BN == 32 ? 3 : 4;
  static constexpr int kABytes = kSlab * kBlockK * 2;
  static constexpr int kBBytes = BN * kBlockK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
  static constexpr int kTmemCols = kAccs * BN;
  // CTAs that fit an SM (228 KB of shared memory, 512 TMEM columns)
  static constexpr int kPerSm = BN <= 32 ? 3 : 2;
  static_assert(kPerSm * kTmemCols <= 512, "TMEM");
  static_assert(BN * kSlab * 4 <= kStages * kStageBytes, "the accumulators of a join");
};

template <typename T, int BN>
__global__ void __launch_bounds__(kMmaThreads)
    mma_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const LinArgs p, int split) {
  using S = Shape<BN>;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[S::kStages];
  __shared__ __align__(8) uint64_t empty_bar[S::kStages];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  // the same offset in every CTA of the cluster: the join reads the peers' tiles there
  const uint32_t raw = smem_u32(dsmem);
  uint8_t* smem = dsmem + ((1024u - (raw & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = blockIdx.x / split;
  const int slabs = (p.N + kSlab - 1) / kSlab;
  const int n0 = (tile % slabs) * kSlab;
  const int t0 = (tile / slabs) * BN;
  const int num_kb = (p.K + kBlockK - 1) / kBlockK;
  const int kb0 = (int)((int64_t)num_kb * rank / split);
  const int kb1 = (int)((int64_t)num_kb * (rank + 1) / split);
  const int cols = p.T - t0 < BN ? p.T - t0 : BN;  // live columns

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&done_bar, 1);
    s_abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, p.limit_ns, p.status)) break;
        uint8_t* st = smem + stage * S::kStageBytes;
        mbar_arrive_expect_tx(&full_bar[stage], S::kStageBytes);
        tma_load_2d(st, &tmW, &full_bar[stage], kb * kBlockK, n0);
        tma_load_2d(st + S::kABytes, &tmX, &full_bar[stage], kb * kBlockK, t0);
        ++issued;
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (*abort_flag) {  // let the copies in flight land before the CTA goes away
        const uint64_t t = global_timer_ns();
        const int n = issued < S::kStages ? issued : S::kStages;
        for (int i = issued - n; i < issued; ++i)
          while (!mbar_try_wait(&full_bar[i % S::kStages], (uint32_t)((i / S::kStages) & 1)))
            if (global_timer_ns() - t > kDrainNs) break;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      const uint32_t base = smem_u32(smem);
      const uint32_t idesc = idesc_f16_m128(BN, DT<T>::kIsBF16);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full_bar[stage], phase, abort_flag, p.limit_ns, p.status)) break;
        tc_fence_after();
        const uint32_t sa = base + (uint32_t)(stage * S::kStageBytes);
        const uint32_t sb = sa + (uint32_t)S::kABytes;
#pragma unroll
        for (int k = 0; k < kBlockK / 16; ++k)
          umma_f16(tmem + (uint32_t)((kb - kb0) % kAccs * BN), sw128_kmajor_desc(sa + k * 32),
                   sw128_kmajor_desc(sb + k * 32), idesc, (kb - kb0 >= kAccs || k > 0) ? 1u : 0u);
        umma_commit(&empty_bar[stage]);
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // done_bar flips when every MMA issued has completed; on an abort that is all that is left
      umma_commit(&done_bar);
      if (*abort_flag) {
        const uint64_t t = global_timer_ns();
        while (!mbar_try_wait(&done_bar, 0))
          if (global_timer_ns() - t > kDrainNs) break;
      }
    }
  } else {
    const bool ok = mbar_wait(&done_bar, 0, abort_flag, p.limit_ns, p.status);
    tc_fence_after();
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
    __syncwarp();
    if (__all_sync(kAll, ok)) {
      float* part = reinterpret_cast<float*>(smem);
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
        if (split > 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(c0 + j) * kSlab + row] = v[j];
        } else if (n0 + row < p.N) {
          finish16<T>(p, v, t0 + c0, cols - c0, n0 + row);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (split > 1) {
    cluster_sync();
    join<T>(p, smem_u32(smem), cols, n0, t0, rank, split, 1u, 0u);
    __syncwarp();
    cluster_sync();  // no CTA leaves while a peer may still read its part
  } else {
    __syncthreads();
  }
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
// Two CTAs share an SM: one's epilogue and start run under the other's MMAs.
// Roles (192 threads): warp 0 TMA producer; warp 1 issues the MMAs (even CTA) or tells the even
// CTA that a stage of this CTA has landed (odd CTA); warps 2-5 epilogue.
// kF32: f32 results.  Every kDrainKb blocks the MMAs move on to the other of two accumulators
// and the epilogue warps add the finished one to sums in registers, rounded to nearest (the
// tensor cores truncate; a chain over all of K would cost several bits).
constexpr int kDrainKb = 8;

template <int BN, bool kF32>
struct PairShape {
  static constexpr int kABytes = kSlab * kBlockK * 2;
  static constexpr int kBBytes = BN / 2 * kBlockK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 3 : 4;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
  static constexpr int kBufs = kF32 ? 2 : 1;
  static constexpr int kTmemCols = kBufs * BN;
  static_assert(2 * (kSmem + 2048) <= 228 * 1024 && kTmemCols <= 256, "two CTAs per SM");
  static_assert(!kF32 || BN == 128, "the sums of a row stay in registers");
};

template <typename T, int BN, bool kF32>
__global__ void __launch_bounds__(kMmaThreads, 2)
    pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const LinArgs p, int split) {
  using S = PairShape<BN, kF32>;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[S::kStages];
  __shared__ __align__(8) uint64_t empty_bar[S::kStages];
  __shared__ __align__(8) uint64_t tfull_bar[S::kBufs];
  __shared__ __align__(8) uint64_t tempty_bar[S::kBufs];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t raw = smem_u32(dsmem);
  uint8_t* smem = dsmem + ((1024u - (raw & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  const uint32_t rank = cluster_ctarank();
  const uint32_t side = rank & 1u, even = rank & ~1u;
  const int part = (int)(rank >> 1);
  const int tile = blockIdx.x / (2 * split);
  const int slabs = (p.N + 2 * kSlab - 1) / (2 * kSlab);
  const int n0 = (tile % slabs) * 2 * kSlab + (int)side * kSlab;  // this CTA's weight rows
  const int t0 = (tile / slabs) * BN;
  const int num_kb = (p.K + kBlockK - 1) / kBlockK;
  const int kb0 = (int)((int64_t)num_kb * part / split);
  const int kb1 = (int)((int64_t)num_kb * (part + 1) / split);
  const int cols = p.T - t0 < BN ? p.T - t0 : BN;
  const int chunk = kF32 ? kDrainKb : kb1 - kb0;  // blocks of one accumulator pass

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
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
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(&s_tmem, S::kTmemCols);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t peer_abort = cluster_map(smem_u32(&s_abort), rank ^ 1u);
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait(bar, parity, abort_flag, p.limit_ns, p.status)) return true;
    st_cluster_u32(peer_abort, 1u);
    return false;
  };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      const int tx = t0 + (int)side * (BN / 2);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait(&empty_bar[stage], phase ^ 1u)) break;
        uint8_t* st = smem + stage * S::kStageBytes;
        mbar_arrive_expect_tx(&full_bar[stage], S::kStageBytes);
        tma_load_2d(st, &tmW, &full_bar[stage], kb * kBlockK, n0);
        tma_load_2d(st + S::kABytes, &tmX, &full_bar[stage], kb * kBlockK, tx);
        ++issued;
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (*abort_flag) {  // let the copies in flight land (one budget for all)
        const uint64_t t = global_timer_ns();
        const int n = issued < S::kStages ? issued : S::kStages;
        for (int i = issued - n; i < issued; ++i)
          while (!mbar_try_wait(&full_bar[i % S::kStages], (uint32_t)((i / S::kStages) & 1)))
            if (global_timer_ns() - t > kDrainNs) break;
      }
    }
  } else if (warp == 1 && side != 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait(&full_bar[stage], phase)) break;
        mbar_arrive_cluster(cluster_map(smem_u32(&full_bar[stage]), even));
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      const uint32_t base = smem_u32(smem);
      const uint32_t idesc = idesc_f16(256, BN, DT<T>::kIsBF16);
      const uint32_t odd = even | 1u;
      for (int kc = kb0; kc < kb1 && ok; kc += chunk) {
        if (kF32 && !wait(&tempty_bar[buf], buf_phase ^ 1u)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf * BN);
        const int ke = kc + chunk < kb1 ? kc + chunk : kb1;
        for (int kb = kc; kb < ke; ++kb) {
          if (!wait(&full_bar[stage], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + (uint32_t)(stage * S::kStageBytes);
          const uint32_t sb = sa + (uint32_t)S::kABytes;
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            umma_f16_pair(d, sw128_kmajor_desc(sa + k * 32), sw128_kmajor_desc(sb + k * 32), idesc,
                          (kb > kc || k > 0) ? 1u : 0u);
          umma_commit_pair(smem_u32(&empty_bar[stage]));
          umma_commit_pair(cluster_map(smem_u32(&empty_bar[stage]), odd));
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(smem_u32(&tfull_bar[buf]));
        umma_commit_pair(cluster_map(smem_u32(&tfull_bar[buf]), odd));
        if (++buf == S::kBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      // every MMA issued has completed once drain_bar flips
      umma_commit_pair(smem_u32(&drain_bar));
      const uint64_t t = global_timer_ns();
      while (!mbar_try_wait(&drain_bar, 0))
        if (global_timer_ns() - t > kDrainNs) break;
    }
  } else {
    const int q = warp & 3;
    const int row = q * 32 + lane;
    const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
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
        for (int c = 0; c < BN; ++c) {
          if (c < cols) {
            if (split > 1)
              stash[c * kSlab + row] = acc[c];
            else if (n0 + row < p.N)
              finish<T>(p, acc[c], t0 + c, n0 + row);
          }
        }
      }
    } else {
      const bool ok = wait(&tfull_bar[0], 0);
      tc_fence_after();
      __syncwarp();
      if (__all_sync(kAll, ok)) {
        for (int c0 = 0; c0 < cols; c0 += 16) {
          float v[16];
          tmem_ld_x16(tb + (uint32_t)c0, v);
          if (split > 1) {
#pragma unroll
            for (int j = 0; j < 16; ++j) stash[(c0 + j) * kSlab + row] = v[j];
          } else if (n0 + row < p.N) {
            finish16<T>(p, v, t0 + c0, cols - c0, n0 + row);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (split > 1) {
    join<T>(p, smem_u32(smem), cols, n0, t0, part, split, 2u, side);
    __syncwarp();
    cluster_sync();  // no CTA leaves while a peer may still read its part
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::kTmemCols);
  }
}

// ---- host side ---------------------------------------------------------------------------------
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

template <auto Kernel>
cudaError_t launch_tiles(const LinArgs& p, int dtype, const void* x, const void* w, int box_x,
                         int smem, int64_t ctas, int cluster, int split, cudaStream_t s) {
  const cudaError_t e = set_smem_limit<Kernel>(smem);
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
  return cudaLaunchKernelEx(&cfg, Kernel, tmW, tmX, p, split);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T, int BN>
cudaError_t launch_mma(const LinArgs& p, int dtype, const void* x, const void* w,
                       cudaStream_t s) {
  const int64_t tiles = ceil_div(p.N, kSlab) * ceil_div(p.T, BN);
  const int num_kb = (p.K + kBlockK - 1) / kBlockK;
  // Split K while the tiles leave SM slots empty and each part keeps at least four 64-k blocks.
  int split = 1;
  while (split < 8 && tiles * split * 2 <= (int64_t)num_sms() * Shape<BN>::kPerSm &&
         num_kb >= split * 2 * 4)
    split *= 2;
  return launch_tiles<mma_kernel<T, BN>>(p, dtype, x, w, BN, Shape<BN>::kSmem, tiles * split,
                                         split, split, s);
}

template <typename T, int BN, bool kF32>
cudaError_t launch_pair(const LinArgs& p, int dtype, const void* x, const void* w,
                        cudaStream_t s) {
  const int64_t tiles = ceil_div(p.N, 2 * kSlab) * ceil_div(p.T, BN);
  const int num_kb = (p.K + kBlockK - 1) / kBlockK;
  int split = 1;
  if (BN == 128)  // a part of a 256-column tile does not fit beside a second CTA
    while (split < 4 && tiles * split * 2 <= num_sms() && num_kb >= split * 2 * 4) split *= 2;
  return launch_tiles<pair_kernel<T, BN, kF32>>(p, dtype, x, w, BN / 2,
                                                PairShape<BN, kF32>::kSmem, tiles * split * 2,
                                                2 * split, split, s);
}

template <typename T>
cudaError_t launch_gemv(const LinArgs& p, const void* x, const void* w, cudaStream_t s) {
  // Warps per weight row: enough for about sixteen warps per SM.
  int wpr = 1;
  while (wpr < kGemvWarps && (int64_t)p.N * wpr < (int64_t)num_sms() * 16 &&
         p.K / 8 >= wpr * 2 * 32)
    wpr *= 2;
  const int rows = kGemvWarps / wpr;
  const dim3 grid((p.N + rows - 1) / rows), block(kGemvWarps * 32);
  const uint4* xv = static_cast<const uint4*>(x);
  const uint4* wv = static_cast<const uint4*>(w);
  switch (p.T) {
    case 1: return launch_k(gemv_kernel<T, 1>, grid, block, 0, s, false, p, xv, wv, wpr);
    case 2: return launch_k(gemv_kernel<T, 2>, grid, block, 0, s, false, p, xv, wv, wpr);
    case 3: return launch_k(gemv_kernel<T, 3>, grid, block, 0, s, false, p, xv, wv, wpr);
    default: return launch_k(gemv_kernel<T, 4>, grid, block, 0, s, false, p, xv, wv, wpr);
  }
}

template <typename T>
cudaError_t launch_typed(const LinArgs& p, int dtype, const void* x, const void* w,
                         cudaStream_t s) {
  if (p.T <= kGemvRows) return launch_gemv<T>(p, x, w, s);
  if (p.T <= 16) return launch_mma<T, 16>(p, dtype, x, w, s);
  if (p.T <= 32) return launch_mma<T, 32>(p, dtype, x, w, s);
  if (p.T <= 64) return launch_mma<T, 64>(p, dtype, x, w, s);
  if (p.out_f32) return launch_pair<T, 128, true>(p, dtype, x, w, s);
  // 256 columns once those tiles alone give every SM one
  if (ceil_div(p.N, 2 * kSlab) * ceil_div(p.T, 256) * 2 >= num_sms())
    return launch_pair<T, 256, false>(p, dtype, x, w, s);
  return launch_pair<T, 128, false>(p, dtype, x, w, s);
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
