// dense_w4.cu -- 4-bit weights against more rows of x than dense_rows.cu streams well, on the tensor
// cores with TMEM accumulators (include/moe.h: moe_linear_w4a16, moe_gated_linear_w4a16).
//
// D[r, t] = sum_k W(r, k) x(t, k): 128 weight rows are the M side, 32 to 128 rows of x the N side.  The
// weights are decoded once for all of them, as they come: E2M1 codes times their E4M3 scale are exact
// f16, written into the swizzled tile that the MMAs read.  x is taken in f16, bf16 x times a power of two
// per row where it needs one (rows.cuh).
// bf16 x is converted by a small kernel before: done in this one, by every CTA for itself, it cost
// more than the decoding (64 rows of 7168 x 7168: 51 us, now 23).
// What bounds it is the issue of the decoding, about three instructions of a lane per weight with the
// stores and waits, on as many SMs as the tiles and parts of K fill.  7168 x 7168 at 17, 32, 64, 128
// and 256 rows: 20, 21, 23, 29 and 45 us.
// Gated: 64 gate rows and the 64 up rows that go with them.
// A cluster is parts of K of the same rows, whose sums meet in shared memory and are added in the
// order of the parts.
#include "rows.cuh"

namespace gb300moe {

namespace {

constexpr int kRows = 128;                     // of a tile
constexpr int kDecodeWarps = 16;               // then one copies x, and one issues the MMAs
constexpr int kThreads = (kDecodeWarps + 2) * 32;
constexpr int kBlock = 256;                    // k of which a part of K has a whole number
constexpr int kStageK = 128;                   // k of a stage: two 64-k tiles of each operand
constexpr int kWBytes = kRows * kStageK * 2;
constexpr int kSlots = 3;                      // stages of a warp's 16 rows on their way
constexpr int kSlotBytes = 16 * 64 + 16 * 32;  // codes, and 32 bytes that hold a row's 8 scales

template <int kN>
struct Shape {
  static constexpr int kStages = kN <= 64 ? 3 : 2;
  static constexpr int kStageBytes = kWBytes + kN * kStageK * 2;
  static constexpr int kSmem =
      1024 + kStages * kStageBytes + kDecodeWarps * kSlots * kSlotBytes;
  static_assert(kSmem <= kSmemLimit, "shared memory");
  static_assert(kStages * kStageBytes >= kRows * kN * (int)sizeof(float), "the sums");
};
constexpr int kAccs = 4;  // accumulators of a part of K that is longer than one may take

// grid.x: groups of weight rows, each `parts` CTAs side by side (the cluster); grid.y: kN rows of x.
// x_rows: rows of x that a copy brings; x_scale: of its rows, not null where the kernel before this one
// made x16 and it and nothing else.
template <typename T, bool kGated, int kN>
__global__ void __launch_bounds__(kThreads, 1)
    w4_kernel(const __grid_constant__ CUtensorMap x16, const RowsCall p, const float* x_scale,
              int parts, int x_rows, uint64_t limit_ns) {
  using S = Shape<kN>;
  constexpr int kStages = S::kStages;
  constexpr int kOuts = kGated ? kRows / 2 : kRows;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kStages];  // of weights
  __shared__ __align__(8) uint64_t x_bar[kStages];
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
  const int64_t t0 = (int64_t)blockIdx.y * kN;
  const int cols = p.T - t0 < kN ? (int)(p.T - t0) : kN;
  const int all = (p.K - 1) / kBlock + 1;
  const int first = (int)((int64_t)all * part / parts);
  const int last = (int)((int64_t)all * (part + 1) / parts);
  const int steps = 2 * (last - first);
  const int chain = chain_of<kAccs>(steps, kChainK / kStageK);  // steps of an accumulator
  const uint32_t tmem_cols = steps > chain ? kAccs * kN : kN;
  volatile int* abort_flag = &s_abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return wait_bar(bar, parity, abort_flag, limit_ns, p.status);
  };

  if (warp == kDecodeWarps + 1) {
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&full_bar[s], kDecodeWarps / 2);
        mbar_init(&x_bar[s], 1);
        mbar_init(&empty_bar[s], 1);
      }
      mbar_init(&done_bar, 1);
      s_abort = 0;
      fence_mbar_init();
      fence_async_shared();  // the barriers, to the copies
    }
    __syncwarp();
    tmem_alloc(&s_tmem, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  int issued = 0;  // by the thread that copies x: stages asked for

  if (warp < kDecodeWarps) {
    // Warps 0-7 decode even stages, 8-15 odd ones, each 16 rows.
    const int g = lane >> 2, t = lane & 3, odd = warp >> 3, w16 = (warp & 7) * 16;
    const uint32_t ring =
        base + (uint32_t)(kStages * S::kStageBytes + warp * kSlots * kSlotBytes);
    // A weight row of the warp's: rows past the end stand for the last one.
    auto row_of = [&](int i) -> int64_t {
      const int r = w16 + i;
      int64_t n = group * kOuts + (kGated ? r & (kOuts - 1) : r);
      n = n < p.N ? n : p.N - 1;
      return kGated && r >= kOuts ? n + p.N : n;
    };
    const int64_t pitch = p.K / 2, scales = p.K / 16;
    const uint8_t* from[2];
    uint32_t scale_at[2];  // this lane's scales in its slot, the same in every one
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = row_of(h * 8 + g);
      from[h] = p.codes + row * pitch + (int64_t)first * 128 + odd * 64 + t * 16;
      scale_at[h] = (uint32_t)(1024 + (h * 8 + g) * 32) +
                    (uint32_t)(((int)((row * scales + odd * 8) & 15) + t * 2) ^ ((g & 4) << 2));
    }
    // Lanes 0-15 copy the first half of a row's 32 bytes of scales, lanes 16-31 the other; rows 4-7
    // and 12-15 have their halves swapped, so that eight rows' reads touch different banks.
    const uint8_t* const scale_end = p.scales + (kGated ? 2 * (int64_t)p.N : p.N) * scales;
    const uint8_t* scale_from =
        p.scales + ((row_of(lane & 15) * scales + (int64_t)first * 16 + odd * 8) & ~int64_t(15)) +
        (lane >> 4) * 16;
    const uint32_t scale_to =
        ring + (uint32_t)(1024 + (lane & 15) * 32 + ((lane >> 4) ^ ((lane >> 2) & 1)) * 16);
    // K is a multiple of 32, a lane's vector.
    int left = p.K - first * kBlock - odd * kStageK - t * 32;  // k from this lane's next vector on
    if (t == 0 && odd == 0)  // into L2 while the kernel before this one ends
      for (int b = 0; b < kSlots - 1 && first + b < last; ++b)
        for (int h = 0; h < 2; ++h) prefetch_l2(from[h] + b * 128);
    if (!x_scale) pdl_wait();
    // Vector h of a lane at h * 512 of its slot, 16 bytes a lane.
    const int blocks = last - first;
    auto load = [&](int b, int slot) {
      if (b < blocks) {
        const uint32_t to = ring + (uint32_t)(slot * kSlotBytes + lane * 16);
        const int bytes = left > 0 ? 16 : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          copy16_part(to + (uint32_t)(h * 512), bytes ? from[h] : p.codes, bytes);
        // the tensor may end inside a vector of scales, or before it
        const int64_t rest = scale_end - scale_from;
        const int some = rest >= 16 ? 16 : rest > 0 ? (int)rest : 0;
        copy16_part(scale_to + (uint32_t)(slot * kSlotBytes), some ? scale_from : p.scales, some);
        from[0] += 128;
        from[1] += 128;
        scale_from += 16;
        left -= kBlock;
      }
      copy_commit();
    };
    int ahead_left = left;  // of the vector that is decoded
    bool ok = true;
#pragma unroll
    for (int s = 0; s < kSlots - 1; ++s) load(s, s);
    int slot = 0, stage = odd % kStages, round = odd / kStages;
    for (int b = 0; b < blocks; ++b) {
      copy_wait<kSlots - 2>();
      __syncwarp();  // the scales are other lanes' copies; and the slot before this one has been read
      load(b + kSlots - 1, slot == 0 ? kSlots - 1 : slot - 1);
      const uint32_t at = ring + (uint32_t)(slot * kSlotBytes);
      uint4 w[2];
      uint32_t s[2][2];  // scales of the lane's first and second 16 k, in both halves
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[h] = lds16(at + (uint32_t)(h * 512 + lane * 16));
        // behind K lie the next row's scales, which could be NaN
        two_scales(ahead_left > 0 ? lds2(at + scale_at[h]) : 0u, s[h]);
        if (t & 2) {  // in another order: eight lanes' stores touch every bank once
          w[h] = make_uint4(w[h].z, w[h].w, w[h].x, w[h].y);
          const uint32_t s0 = s[h][0];
          s[h][0] = s[h][1];
          s[h][1] = s0;
        }
      }
      ahead_left -= kBlock;
      ok = __all_sync(kAll, wait(&empty_bar[stage], (uint32_t)(round & 1) ^ 1u));
      if (!ok) break;
      // a lane's 32 k: half of a row of 64-k tile t / 2
      const uint32_t to = base + (uint32_t)(stage * S::kStageBytes + (t >> 1) * (kWBytes / 2) +
                                            (w16 + g) * 128);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t chunk = (uint32_t)((((t & 1) * 4 + (c ^ (t & 2))) ^ g) * 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t q[4];
          nvfp4_decode8(word_of(w[h], c), s[h][c >> 1], q);
          sts16(to + (uint32_t)(h * 1024) + chunk, make_uint4(q[0], q[1], q[2], q[3]));
        }
      }
      fence_async_shared();  // to the MMAs
      __syncwarp();
      if (lane == 0) mbar_arrive(&full_bar[stage]);
      stage += 2;
      if (stage >= kStages) stage -= kStages, ++round;
      slot = slot + 1 == kSlots ? 0 : slot + 1;
    }
    copy_wait<0>();
  } else if (warp == kDecodeWarps) {
    if (elect_one()) {
      prefetch_tensormap(&x16);
      pdl_wait();
      int stage = 0, round = 0;
      for (; issued < steps; ++issued) {
        if (!wait(&empty_bar[stage], (uint32_t)(round & 1) ^ 1u)) break;
        const int k = first * kBlock + issued * kStageK;
        uint8_t* to = smem + stage * S::kStageBytes + kWBytes;
        // columns of D past the rows that are copied hold anything, and nothing reads them
        mbar_arrive_expect_tx(&x_bar[stage], (uint32_t)(x_rows * kStageK * 2));
        tma_load_2d(to, &x16, &x_bar[stage], k, (int)t0);
        tma_load_2d(to + kN * 128, &x16, &x_bar[stage], k + 64, (int)t0);
        if (++stage == kStages) stage = 0, ++round;
      }
    }
    __syncwarp();
  } else {
    pdl_wait();
    pdl_trigger();
    if (elect_one()) {
      Ring r(full_bar, kStages, 0u);
      const uint32_t idesc = idesc_f16_m128(kN, 0);
      uint32_t d = tmem;
      for (int i = 0, in = 0; i < steps; ++i, ++in) {
        if (in == chain) in = 0, d += (uint32_t)kN;
        if (!r.ready && !wait(r.bar(), r.parity)) break;
        if (!wait(&x_bar[r.stage], r.parity)) break;
        tc_fence_after();
        const int stage = r.stage;
        const uint32_t a = base + (uint32_t)(stage * S::kStageBytes), b = a + (uint32_t)kWBytes;
        r.next();
#pragma unroll
        for (int k = 0; k < kStageK / 16; ++k)
          umma_f16(d,
                   sw128_kmajor_desc(a + (uint32_t)((k >> 2) * (kWBytes / 2) + (k & 3) * 32)),
                   sw128_kmajor_desc(b + (uint32_t)((k >> 2) * (kN * 128) + (k & 3) * 32)), idesc,
                   in > 0 || k > 0 ? 1u : 0u);
        umma_commit(&empty_bar[stage]);
      }
      umma_commit(&done_bar);  // also where a wait gave up: the MMAs in flight
    }
    __syncwarp();
  }

  // Sums [columns][rows of the tile], where the stages were.
  float* sums = reinterpret_cast<float*>(smem);
  if (warp < 4) {
    const bool got = __all_sync(kAll, wait(&done_bar, 0u));
    tc_fence_after();
    if (got) {
      const uint32_t ta = tmem_lane(tmem, warp);
#pragma unroll
      for (int c0 = 0; c0 < kN; c0 += 16) {
        if (c0 >= cols) break;
        float v[16];
        tmem_ld_x16(ta + (uint32_t)c0, v);
        add_accumulators(ta + (uint32_t)c0, kN, (steps - 1) / chain, v);
#pragma unroll
        for (int c = 0; c < 16; ++c) sums[(c0 + c) * kRows + warp * 32 + lane] = v[c];
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag) {
    if (issued > 0) land_copies(x_bar, issued, kStages);
    if (threadIdx.x == 0) land_mmas(&done_bar);
  }
  pdl_wait();  // the decoders have not waited for x_scale
  const float alpha = *p.alpha;
  if (parts > 1)
    cluster_sync();
  else
    __syncthreads();
  finish_tile<T, kGated, kOuts, kThreads>(p, base, sums, kRows, group, part, parts, t0, cols, alpha,
                                           x_scale);
  if (parts > 1) cluster_leave();  // a peer may still read this CTA's sums
  if (warp == kDecodeWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// bf16 -> f16, a CTA a row of `vecs` vectors: its largest magnitude first, with up to kHold vectors of a
// thread kept for the second step.
constexpr int kRowThreads = 512, kHold = 4;  // at most
__global__ void __launch_bounds__(kRowThreads)
    to_f16_kernel(const uint4* x, uint4* out, float* scales, int vecs, int* status) {
  __shared__ uint32_t s_top[kRowThreads / 32];
  const int threads = blockDim.x;
  pdl_wait();
  pdl_trigger();
  const uint4* const from = x + (int64_t)blockIdx.x * vecs;
  uint4* const to = out + (int64_t)blockIdx.x * vecs;
  const int lane = threadIdx.x & 31;
  uint4 v[kHold];
  uint32_t top = 0u;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = threadIdx.x + k * threads;
    v[k] = i < vecs ? from[i] : zero4();
  }
#pragma unroll
  for (int k = 0; k < kHold; ++k) top = max(top, top_bits(v[k]));
  for (int i = threadIdx.x + kHold * threads; i < vecs; i += threads)
    top = max(top, top_bits(from[i]));
  top = __reduce_max_sync(kAll, top);
  if (lane == 0) s_top[threadIdx.x >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(kAll, lane < threads / 32 ? s_top[lane] : 0u);
  const RowScale s = row_scale(top);
  if (threadIdx.x == 0) {
    scales[blockIdx.x] = s.up;
    if (past_f16(top)) set_status(status, MOE_ERR_F16_RANGE);
  }
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = threadIdx.x + k * threads;
    if (i < vecs) to[i] = bf16x8_times(v[k], s.down);
  }
  for (int i = threadIdx.x + kHold * threads; i < vecs; i += threads)
    to[i] = bf16x8_times(from[i], s.down);
}

template <typename T, bool kGated, int kN>
cudaError_t go(const RowsCall& c, void* x16, cudaStream_t s) {
  constexpr auto kern = w4_kernel<T, kGated, kN>;
  constexpr int kSmem = Shape<kN>::kSmem, kOuts = kGated ? kRows / 2 : kRows;
  const cudaError_t e = set_smem_limit<kern>(kSmem);
  if (e != cudaSuccess) return e;
  const int64_t groups = (c.N - 1) / kOuts + 1, tall = (c.T - 1) / kN + 1;
  const int all = (c.K - 1) / kBlock + 1;
  const int parts = parts_of<kern>(groups * tall, all, 6, kThreads, kSmem);
  if (parts == 0) return cudaErrorInvalidConfiguration;
  const bool prepare = c.dtype == MOE_BF16;
  const int x_rows = c.T < kN ? (c.T + 7) / 8 * 8 : kN;
  CUtensorMap map;
  if (!rows_map(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, prepare ? x16 : c.x,
                (uint64_t)c.K, (uint64_t)c.T, (uint64_t)c.K * 2, (uint32_t)x_rows))
    return cudaErrorInvalidValue;
  float* const x_scale =
      prepare ? reinterpret_cast<float*>(static_cast<char*>(x16) + (size_t)c.T * c.K * 2) : nullptr;
  if (prepare) {
    const int vecs = c.K / 8, warps = (vecs - 1) / (kHold * 32) + 1;
    const cudaError_t f = launch_k(
        to_f16_kernel, dim3((unsigned)c.T), dim3(warps * 32 < kRowThreads ? warps * 32 : kRowThreads), 0,
        s, true, static_cast<const uint4*>(c.x), static_cast<uint4*>(x16), x_scale, vecs, c.status);
    if (f != cudaSuccess) return f;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * parts), (unsigned)tall);
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
  return cudaLaunchKernelEx(&cfg, kern, map, c, (const float*)x_scale, parts, x_rows,
                            wait_limit_ns());
}

template <typename T, bool kGated>
cudaError_t pick(const RowsCall& c, void* x16, cudaStream_t s) {
  if (c.T <= 32) return go<T, kGated, 32>(c, x16, s);
  if (c.T <= 64) return go<T, kGated, 64>(c, x16, s);
  return go<T, kGated, 128>(c, x16, s);
}

}  // namespace

size_t w4_bytes(int dtype, int64_t T, int64_t K) {
  return dtype == MOE_BF16 && T > kFewW4Rows ? (size_t)T * ((size_t)K * 2 + sizeof(float)) : 0;
}

cudaError_t launch_w4(const RowsCall& c, void* x16, cudaStream_t s) {
  if (c.dtype == MOE_BF16)
    return c.gated ? pick<__nv_bfloat16, true>(c, x16, s) : pick<__nv_bfloat16, false>(c, x16, s);
  return c.gated ? pick<__half, true>(c, x16, s) : pick<__half, false>(c, x16, s);
}

}  // namespace gb300moe
