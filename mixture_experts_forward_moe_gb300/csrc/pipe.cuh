// pipe.cuh -- what the tcgen05 products (linear.cu, dense.cu) share: bounded waits, rings of
// barriers, commits to both CTAs of a pair, and launch limits of kernels.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "ptx.cuh"

namespace gb300moe {

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

// K that one accumulator takes.  The tensor cores add with truncation, always toward zero: a sum of terms
// of one sign loses 4e-7 of itself per 64 k, 5e-5 in kChainK, a fifth of an f16's least half step (1.7e-3
// in 262144, three of its half steps).  Sums of several accumulators are rounded (to nearest).
constexpr int kChainK = 8192;

// TMEM address of the lanes that an epilogue warp may read.
__device__ __forceinline__ uint32_t tmem_lane(uint32_t tmem, int warp) {
  return tmem + ((uint32_t)((warp & 3) * 32) << 16);
}
// Arrives on the barrier at this offset of both CTAs of the pair when the MMAs issued so far
// have completed.
__device__ __forceinline__ void umma_commit_both(uint32_t bar, uint32_t even) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)(3u << even))
      : "memory");
}

// What threads wrote to shared memory (and barriers they set up), to copies and MMAs.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Cluster barrier after which a CTA may leave: it orders nothing but the peers' finished reads
// (cluster_sync's release would first wait for this CTA's global stores).
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::
                   : "memory");
}

// ---- host side ---------------------------------------------------------------------------------
constexpr int kSmemLimit = 226 * 1024;  // dynamic; leaves room for the static variables

// A 2-D map of rows `pitch` bytes apart with the 128-byte swizzle, boxes of 128 bytes x box_rows.
inline bool rows_map(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base,
                     uint64_t inner, uint64_t rows, uint64_t pitch, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {pitch};
  cuuint32_t box[2] = {(cuuint32_t)(128 / size), box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sets a kernel's shared-memory limit, once per device; `Kernel` names the instance.
template <auto Kernel>
inline cudaError_t set_smem_limit(int bytes) {
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

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace gb300moe
