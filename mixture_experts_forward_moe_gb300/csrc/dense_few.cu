// dense_few.cu -- the gated product of two to 32 rows of x, and up to 128 where the weights are few
// (few_rows in dense_api.cu; include/moe.h: moe_gated_linear without checkpoints), on the tensor cores with
// the weights as the M side.
//
// D[r, t] = sum_k W(r, k) x(t, k): a tile is 64 gate rows of the weights and the 64 up rows that go
// with them, against all rows of x (16 to 128 columns of D), so that none of the MMAs' rows are empty
// and every weight is read once.  What bounds it is the weights' bytes: a CTA has up to 200 KB of
// them and of x on their way.  K is split over a cluster, whose sums meet in shared memory and are
// added in the order of the parts.  7168 x 2048 at 2, 16, 64 and 128 rows: 13, 13, 15 and 17.5 us (4.5
// to 3.4 TB/s: the start and the join show); 7168 x 18432 at 2 and 32 rows 80 and 83 us (6.6, 6.3).
#include "rows.cuh"

namespace gb300moe {

namespace {

constexpr int kOuts = 64;          // of a tile: gate rows, and as many up rows
constexpr int kThreads = 6 * 32;   // warp 0 copies, warp 1 issues the MMAs, warps 2-5 read the sums
constexpr int kBlock = 64;         // k of a stage
constexpr int kWBytes = 2 * kOuts * kBlock * 2;

template <int kN>
struct Shape {
  static constexpr int kStageBytes = kWBytes + kN * kBlock * 2;
  static constexpr int kStages = 200 * 1024 / kStageBytes;
  static constexpr int kSmem = 1024 + kStages * kStageBytes;
  static_assert(kSmem <= kSmemLimit, "shared memory");
  static_assert(kStages * kStageBytes >= 2 * kOuts * kN * (int)sizeof(float), "the sums");
};
constexpr int kAccs = 4;  // accumulators of a part of K that is longer than one may take

// grid.x: groups of outputs, each `parts` CTAs side by side (the cluster).  x_rows: rows of x that a
// copy brings; the columns of D behind them hold anything, and nothing reads them.
template <typename T, int kN>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
               const RowsCall p, int parts, int x_rows, uint64_t limit_ns) {
  using S = Shape<kN>;
  constexpr int kStages = S::kStages, kCols = kN < 32 ? 32 : kN;  // of TMEM
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t done_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t raw = smem_u32(dsmem);
  uint8_t* smem = dsmem + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = blockIdx.x % (unsigned)parts;
  const int64_t group = blockIdx.x / (unsigned)parts;
  const int all = (p.K - 1) / kBlock + 1;
  const int first = (int)((int64_t)all * part / parts);
  const int last = (int)((int64_t)all * (part + 1) / parts);
  const int n0 = (int)(group * kOuts);
  const int chain = chain_of<kAccs>(last - first, kChainK / kBlock);  // blocks of an accumulator
  const uint32_t tmem_cols = last - first > chain ? kAccs * kCols : kCols;
  volatile int* abort_flag = &s_abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return wait_bar(bar, parity, abort_flag, limit_ns, p.status);
  };
  int issued = 0;  // by the thread that copies (the same one is elected here and below)

  if (warp == 0) {
    if (elect_one()) {
      prefetch_tensormap(&w_map);
      prefetch_tensormap(&x_map);
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&full_bar[s], 1);
        mbar_init(&empty_bar[s], 1);
      }
      mbar_init(&done_bar, 1);
      s_abort = 0;
      fence_mbar_init();
      fence_async_shared();  // the barriers, to the copies
      // the first weights come into L2 while the kernel before this one ends
      for (int b = first; b < last && b < first + kStages; ++b) {
        tma_prefetch_l2_2d(&w_map, b * kBlock, n0);
        tma_prefetch_l2_2d(&w_map, b * kBlock, p.N + n0);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(&s_tmem, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  if (warp == 1) pdl_trigger();

  if (warp == 0) {
    if (elect_one()) {
      Ring r(empty_bar, kStages, 1u);
      for (int b = first; b < last; ++b) {
        if (!r.ready && !wait(r.bar(), r.parity)) break;
        uint8_t* to = smem + r.stage * S::kStageBytes;
        uint64_t* full = &full_bar[r.stage];
        r.next();
        mbar_arrive_expect_tx(full, (uint32_t)(kWBytes + x_rows * kBlock * 2));
        // gate rows past N are rows of up, whose outputs are left out
        tma_load_2d(to, &w_map, full, b * kBlock, n0);
        tma_load_2d(to + kWBytes / 2, &w_map, full, b * kBlock, p.N + n0);
        tma_load_2d(to + kWBytes, &x_map, full, b * kBlock, 0);
        ++issued;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      Ring r(full_bar, kStages, 0u);
      const uint32_t idesc = idesc_f16_m128(kN, DT<T>::kIsBF16);
      uint32_t d = tmem;
      for (int b = first, in = 0; b < last; ++b, ++in) {
        if (in == chain) in = 0, d += (uint32_t)kCols;
        if (!r.ready && !wait(r.bar(), r.parity)) break;
        tc_fence_after();
        uint64_t* empty = &empty_bar[r.stage];
        const uint32_t a = base + (uint32_t)(r.stage * S::kStageBytes), x = a + (uint32_t)kWBytes;
        r.next();
#pragma unroll
        for (int k = 0; k < kBlock / 16; ++k)
          umma_f16(d, sw128_kmajor_desc(a + (uint32_t)(k * 32)),
                   sw128_kmajor_desc(x + (uint32_t)(k * 32)), idesc, in > 0 || k > 0 ? 1u : 0u);
        umma_commit(empty);
      }
      umma_commit(&done_bar);  // also where a wait gave up: the MMAs in flight
    }
    __syncwarp();
  }

  // Sums [columns][rows of the tile], where the stages were.
  float* sums = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const bool got = __all_sync(kAll, wait(&done_bar, 0u));
    tc_fence_after();
    if (got) {
      const uint32_t ta = tmem_lane(tmem, warp);
      const int row = (warp & 3) * 32 + lane;
#pragma unroll
      for (int c0 = 0; c0 < kN; c0 += 16) {
        if (c0 >= p.T) break;
        float v[16];
        tmem_ld_x16(ta + (uint32_t)c0, v);
        add_accumulators(ta + (uint32_t)c0, kCols, (last - first - 1) / chain, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) sums[(c0 + c) * 2 * kOuts + row] = v[c];
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag) {
    if (issued > 0) land_copies(full_bar, issued, kStages);
    if (warp == 1 && lane == 0) land_mmas(&done_bar);
  }
  if (parts > 1)
    cluster_sync();
  else
    __syncthreads();
  finish_tile<T, true, kOuts, kThreads>(p, base, sums, 2 * kOuts, group, part, parts, 0, p.T, 1.0f,
                                           nullptr);
  if (parts > 1) cluster_leave();  // a peer may still read this CTA's sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

template <typename T, int kN>
cudaError_t go(const RowsCall& c, cudaStream_t s) {
  constexpr auto kern = few_kernel<T, kN>;
  constexpr int kSmem = Shape<kN>::kSmem;
  const cudaError_t e = set_smem_limit<kern>(kSmem);
  if (e != cudaSuccess) return e;
  const int64_t groups = (c.N - 1) / kOuts + 1;
  const int parts = parts_of<kern>(groups, (c.K - 1) / kBlock + 1, 10, kThreads, kSmem);
  if (parts == 0) return cudaErrorInvalidConfiguration;
  const int x_rows = (c.T + 7) / 8 * 8;
  const CUtensorMapDataType type =
      DT<T>::kIsBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap w_map, x_map;
  if (!rows_map(&w_map, type, 2, c.w, (uint64_t)c.K, 2 * (uint64_t)c.N, (uint64_t)c.K * 2, kOuts) ||
      !rows_map(&x_map, type, 2, c.x, (uint64_t)c.K, (uint64_t)c.T, (uint64_t)c.K * 2,
                (uint32_t)x_rows))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)kSmem;
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
  return cudaLaunchKernelEx(&cfg, kern, w_map, x_map, c, parts, x_rows, wait_limit_ns());
}

template <typename T>
cudaError_t pick(const RowsCall& c, cudaStream_t s) {
  if (c.T <= 16) return go<T, 16>(c, s);
  if (c.T <= 32) return go<T, 32>(c, s);
  if (c.T <= 64) return go<T, 64>(c, s);
  return go<T, 128>(c, s);
}

}  // namespace

cudaError_t launch_few(const RowsCall& c, cudaStream_t s) {
  return c.dtype == MOE_BF16 ? pick<__nv_bfloat16>(c, s) : pick<__half>(c, s);
}

}  // namespace gb300moe
