// dense.cu -- the dense products of a feed-forward block and of its training, on pairs of SMs
// (tcgen05, cta_group::2), with the gated product, its gradient and 8-bit checkpoints in the
// epilogue (include/moe.h: moe_gated_linear, moe_gated_linear_bwd, moe_linear_bwd).
//
// D[m, n] = sum_k A(m, k) B(n, k), f32 accumulation.  The operands lie in memory as they are:
//   x w^T       A = x [M, K], B = w [N, K]           both with k contiguous ("K-major")
//   dy w        A = dy [M, K], B = w [K, N]          B with n contiguous ("MN-major")
//   dy^T x      A = dy [K, M], B = x [K, N]          both MN-major
// so nothing is transposed: the tensor cores read a 128-byte-swizzled tile in either order.
//
// A pair of CTAs has a tile of 256 x 256: each CTA 128 rows of A and of B, and its 128 rows of
// the accumulator (two of 256 TMEM columns, so that one tile's epilogue runs under the next one's
// MMAs).  The grid is persistent, one CTA per SM.  Rows of D are TMEM lanes, so a thread of the
// epilogue holds consecutive columns of one row: the gated product, whose tile holds 128 gate columns
// (the even CTA's rows of B) and the 128 up columns that go with them (the odd CTA's), needs no
// exchange, and the largest value of a checkpoint's 128 channels one between two threads.  Outputs go
// through shared memory to TMA stores, which cut what lies outside the tensor.
// Where the last tiles would leave most pairs idle they are split along K: their f32 sums go to the
// workspace, and join_kernel adds them in order and finishes the outputs.
#include "activation.cuh"
#include "dense_ops.cuh"
#include "fp8.cuh"
#include "pipe.cuh"
#include "vec16.cuh"

namespace gb300moe {

namespace {

enum Epi { kPlain, kGated, kGatedSave, kGradient };

constexpr int kTile = 256;
constexpr int kThreads = 320;
constexpr int kOperandBytes = kSlab * kBlockK * 2;  // 128 rows of an operand, 64 k
constexpr int kBoxBytes = 128 * 128;  // an epilogue box: 128 rows of 128 bytes
constexpr int kAllEpilogue = 3;       // named barriers: 1 and 2 of a half, 3 of both

constexpr bool gated(int epi) { return epi != kPlain; }

// A tile is 256 rows by kBN columns.  Boxes of each half of the epilogue warps, and stages in what is
// left of shared memory.  (Two boxes and five stages everywhere: 4096 x 4096 x 7168 in 124 us, 117
// with six stages.)
template <int kEpi, int kBN>
struct Plan {
  static constexpr int kStageBytes = kOperandBytes + kBN / 2 * kBlockK * 2;
  static constexpr int kBoxes = kEpi == kGradient ? 2 : 1;
  // a gated tile's 64 columns share boxes between the halves
  static constexpr bool kShared = gated(kEpi) && kBN != kTile;
  static constexpr int kStages = kBN != kTile ? 8 : kEpi == kGradient ? 5 : 6;
  static constexpr int kSmem = kStages * kStageBytes + (kShared ? 1 : 2) * kBoxes * kBoxBytes + 1024;
};

// The tensor cores add to an accumulator with truncation, and 448 additions (K = 7168) move a sum by
// 1e-5 of its terms: nothing in 16 bits, but one value in a thousand of a checkpoint becomes its
// neighbour.  Where pre-activations are saved the accumulators are added, rounded, to sums in
// registers after as many 64-k blocks; 0: never.
template <int kEpi>
constexpr int kDrainBlocks = kEpi == kGatedSave ? 8 : 0;

struct Maps {
  CUtensorMap a, b;
  CUtensorMap o0, o1, o2;  // outputs: h | gate and up codes, or the two halves of d_pre
  CUtensorMap in;          // kGradient: d_out
  CUtensorMap parts;       // sums of the tiles that are split
};

struct Args {
  int M, N, K;    // outputs (gated: N of 2 N rows of b)
  int mt, nt;     // tiles
  int64_t whole;  // tiles that are not split; then
  int rest;       // the others, each
  int split;      // in as many parts of K
  int a_rows;     // of a K-major a that a copy brings
  int want_out;   // kGradient: h too
  Ckpt gate, up;  // kGatedSave (codes by TMA)
  int* status;
  uint64_t limit_ns;
};

// Descriptor of an MN-major operand with the 128-byte swizzle: boxes of 64 (mn) x 64 (k), a k row
// 128 bytes; eight k rows further 1024 bytes (stride offset), 64 mn further a box (leading offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBlockK * 128 >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <bool kMn>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, int k16) {
  return kMn ? sw128_mnmajor_desc(saddr + (uint32_t)k16 * 2048u)
             : sw128_kmajor_desc(saddr + (uint32_t)k16 * 32u);
}

template <bool kMn, int kRows>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                             int mn, int k) {
  if constexpr (kMn) {
    tma_load_2d(dst, map, bar, mn, k);
    if (kRows > 64) tma_load_2d(dst + kBlockK * 128, map, bar, mn + 64, k);
  } else {
    tma_load_2d(dst, map, bar, k, mn);
  }
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the last N groups of this thread have read their shared memory.
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 16 bytes at byte 16 j of row `row` of a box, where the 128-byte swizzle has them.
__device__ __forceinline__ uint4* box_at(uint8_t* box, int row, int j) {
  return reinterpret_cast<uint4*>(box + row * 128 + ((j ^ (row & 7)) << 4));
}

// 32 columns of two places of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld_x32(uint32_t t, float (&a)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) a[i] = __uint_as_float(r[i]);
}

// Tiles in an order that keeps those of one time close: bands of kBand rows of tiles, column by
// column.  (All of one row of tiles first would read all of b for every 256 rows of a.)
constexpr int kBand = 8;
struct Place {
  int m, n;  // first row of the tile; its column of tiles
};
__device__ __forceinline__ Place place_of(int mt, int nt, int64_t tile) {
  const int64_t band = (int64_t)kBand * nt;
  const int b = (int)(tile / band);
  const int in = (int)(tile % band);
  const int left = mt - b * kBand;
  const int rows = left < kBand ? left : kBand;
  return Place{(b * kBand + in % rows) * kTile, in / rows};
}

// A unit of work: a tile, or a part of one; its 64-k blocks, and where its sums go (-1: finished).
struct Unit {
  Place at;
  int kb0, kb1, row;
};
__device__ __forceinline__ Unit unit_of(const Args& p, int num_kb, int64_t u) {
  Unit r;
  if (u < p.whole) {
    r.at = place_of(p.mt, p.nt, u);
    r.kb0 = 0;
    r.kb1 = num_kb;
    r.row = -1;
  } else {
    const int i = (int)(u - p.whole), part = i / p.rest;
    r.at = place_of(p.mt, p.nt, p.whole + i % p.rest);
    r.kb0 = (int)((int64_t)num_kb * part / p.split);
    r.kb1 = (int)((int64_t)num_kb * (part + 1) / p.split);
    r.row = i * kTile;
  }
  return r;
}

// Roles (320 threads): warp 0 TMA producer; warp 1 issues the MMAs (even CTA) or tells the even CTA
// that a stage of this CTA has landed (odd CTA); warps 2-5 and 6-9 epilogue, each four half of the
// columns.  (One half for all: 4096 x 2048 x 7168 saved in 145 us.)  Every wait is bounded
// (MOE_ERR_TIMEOUT in the status word); a pair in which one gave up waits for its copies, MMAs and
// stores in flight before it leaves.
template <typename T, bool kAMn, bool kBMn, int kEpi, int kAct, int kBN>
__global__ void __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ Maps maps, const Args p) {
  using P = Plan<kEpi, kBN>;
  constexpr int kStages = P::kStages, kStageBytes = P::kStageBytes;
  constexpr int kHalf = kBN / 2;  // columns of a half of the warps; gated: gate columns of a tile
  constexpr int kDrain = kDrainBlocks<kEpi>;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ __align__(8) uint64_t empty_bar[kStages];
  __shared__ __align__(8) uint64_t tfull_bar[2];
  __shared__ __align__(8) uint64_t tempty_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ __align__(8) uint64_t in_bar[2];
  // kGatedSave: the exponents of a half's largest gate and up of each row
  __shared__ int8_t s_exp[2][2][kEpi == kGatedSave ? 128 : 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t raw = smem_u32(dsmem);
  uint8_t* smem = dsmem + ((1024u - (raw & 1023u)) & 1023u);
  const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  const uint32_t rank = cluster_ctarank();  // in the pair
  const int side = (int)rank;
  const int num_kb = (p.K - 1) / kBlockK + 1;
  const int64_t units = p.whole + (int64_t)p.rest * p.split;
  const int64_t step = num_clusters_x();
  // Fewer than 128 rows of a: the others of its operand hold anything, and make rows of D that nothing
  // reads.
  const bool some = kAMn || side == 0 || p.M > kSlab;
  const int bytes = kStageBytes - (kAMn ? 0 : (kSlab - (some ? p.a_rows : 0)) * kBlockK * 2);
  auto load_block = [&](const Unit& q, int kb, int stage) {
    uint8_t* st = smem + stage * kStageBytes;
    uint64_t* full = &full_bar[stage];
    // gated: the even CTA has the gate rows of b, the odd one the up rows; gate rows past N are rows
    // of up, whose columns the epilogue leaves out
    const int nb = gated(kEpi) ? side * p.N + q.at.n * kHalf : q.at.n * kBN + side * kHalf;
    mbar_arrive_expect_tx(full, (uint32_t)bytes);
    if (some) load_operand<kAMn, kSlab>(st, &maps.a, full, q.at.m + side * kSlab, kb * kBlockK);
    load_operand<kBMn, kHalf>(st + kOperandBytes, &maps.b, full, nb, kb * kBlockK);
  };
  int issued = 0;  // by the producer (the same thread is elected here and below): stages asked for

  if (warp == 0) {
    if (elect_one()) {
      prefetch_tensormap(&maps.a);
      prefetch_tensormap(&maps.b);
      for (int s = 0; s < kStages; ++s) {
        // the even CTA's stage is full when its copies and, by the forwarder, the odd CTA's landed
        mbar_init(&full_bar[s], side == 0 ? 2 : 1);
        mbar_init(&empty_bar[s], 1);
      }
      for (int b = 0; b < 2; ++b) {
        mbar_init(&tfull_bar[b], 1);
        mbar_init(&tempty_bar[b], 16);  // an arrival per epilogue warp of both CTAs
        mbar_init(&in_bar[b], 1);
      }
      mbar_init(&drain_bar, 1);
      s_abort = 0;
      fence_mbar_init();
      fence_async_shared();  // the barriers, to the copies
      // the first stages are on their way while the pair starts
      pdl_wait();
      const Unit q = unit_of(p, num_kb, cluster_id_x());
      for (; issued < kStages && q.kb0 + issued < q.kb1; ++issued)
        load_block(q, q.kb0 + issued, issued);
    }
  } else if (warp == 1) {
    tmem_alloc_pair(&s_tmem, 2 * kBN);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_leave();  // the peer's barriers are there (fence_mbar_init released them)
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_trigger();
  const uint32_t peer_abort = cluster_map(smem_u32(&s_abort), rank ^ 1u);
  // by one thread, or by all of a warp; on giving up the peer CTA is told too
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (wait_bar(bar, parity, abort_flag, p.limit_ns, p.status)) return true;
    st_cluster_u32(peer_abort, 1u);
    return false;
  };

  if (warp == 0) {
    if (elect_one()) {
      Ring r(empty_bar, kStages, 1u);
      bool ok = true;
      const int early = issued;
      for (int i = 0; i < early; ++i) r.next();
      for (int64_t u = cluster_id_x(); u < units && ok; u += step) {
        const Unit q = unit_of(p, num_kb, u);
        for (int kb = u < step ? q.kb0 + early : q.kb0; kb < q.kb1; ++kb) {
          if (!r.ready && !wait(r.bar(), r.parity)) {
            ok = false;
            break;
          }
          const int stage = r.stage;
          r.next();
          load_block(q, kb, stage);
          ++issued;
        }
      }
    }
  } else if (warp == 1 && side != 0) {
    if (elect_one()) {
      Ring r(full_bar, kStages, 0u);
      const uint32_t to = cluster_map(smem_u32(full_bar), 0u);
      bool ok = true;
      for (int64_t u = cluster_id_x(); u < units && ok; u += step) {
        const Unit q = unit_of(p, num_kb, u);
        for (int kb = q.kb0; kb < q.kb1; ++kb) {
          if (!r.ready && !wait(r.bar(), r.parity)) {
            ok = false;
            break;
          }
          mbar_arrive_cluster(to + (uint32_t)r.stage * 8u);
          r.next();
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      Ring r(full_bar, kStages, 0u);
      int buf = 0;
      uint32_t buf_phase = 0;
      bool ok = true;
      const uint32_t base = smem_u32(smem);
      const uint32_t idesc = idesc_f16(256, kBN, DT<T>::kIsBF16) | (kAMn ? 1u << 15 : 0u) |
                             (kBMn ? 1u << 16 : 0u);
      const uint32_t empty_own = smem_u32(empty_bar), tfull_own = smem_u32(tfull_bar);
      for (int64_t u = cluster_id_x(); u < units && ok; u += step) {
        const Unit q = unit_of(p, num_kb, u);
        const int pass = kDrain > 0 ? kDrain : q.kb1 - q.kb0;  // blocks of one accumulator
        for (int kc = q.kb0; kc < q.kb1 && ok; kc += pass) {
          if (!wait(&tempty_bar[buf], buf_phase ^ 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(buf * kBN);
          const int ke = kc + pass < q.kb1 ? kc + pass : q.kb1;
          for (int kb = kc; kb < ke; ++kb) {
            if (!r.ready && !wait(r.bar(), r.parity)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = base + (uint32_t)(r.stage * kStageBytes);
            const uint32_t sb = sa + (uint32_t)kOperandBytes;
            const uint32_t at = (uint32_t)r.stage * 8u;
            r.next();
#pragma unroll
            for (int k = 0; k < kBlockK / 16; ++k)
              umma_f16_pair(d, operand_desc<kAMn>(sa, k), operand_desc<kBMn>(sb, k), idesc,
                            (kb > kc || k > 0) ? 1u : 0u);
            umma_commit_both(empty_own + at, 0u);
          }
          if (!ok) break;
          umma_commit_both(tfull_own + (uint32_t)buf * 8u, 0u);
          buf ^= 1;
          if (buf == 0) buf_phase ^= 1u;
        }
      }
      // every MMA issued has completed once drain_bar flips
      umma_commit_pair(smem_u32(&drain_bar));
      land_mmas(&drain_bar);
    }
  } else {
    // ---- epilogue ----
    const int half = (warp - 2) >> 2;  // of the columns
    const int row = (warp & 3) * 32 + lane;
    // issues the half's stores, or those of both
    const bool leader = ((threadIdx.x - 64) & (P::kShared ? 255 : 127)) == 0;
    const uint32_t tb = tmem_lane(tmem, warp);
    uint8_t* boxes =
        smem + kStages * kStageBytes + (P::kShared ? 0 : half * P::kBoxes * kBoxBytes);
    uint64_t* in = &in_bar[P::kShared ? 0 : half];
    int buf = 0;
    uint32_t buf_phase = 0, in_phase = 0;
    auto sync = [&] {
      if (P::kShared)
        named_bar_sync(kAllEpilogue, 256);
      else
        named_bar_sync(1 + half, 128);
    };
    // The half's (first) box, once no store reads it any more.
    auto next_box = [&]() -> uint8_t* {
      if (leader) store_wait_read<0>();
      sync();
      return boxes;
    };
    // Written boxes to the stores' view; then `issue` by the leader.
    auto publish = [&](auto issue) {
      fence_async_shared();
      sync();
      if (leader) {
        issue();
        store_commit();
      }
    };
    // Passes of an accumulator over `blocks` k blocks.
    auto passes = [&](int blocks) { return kDrain > 0 ? (blocks - 1) / kDrain + 1 : 1; };
    // The accumulator has been read; `left` passes of unit u follow.  Where no later pass takes this
    // buffer nobody waits for the arrival, and the even CTA may leave before it comes.
    auto free_buffer = [&](int left, int64_t u) {
      if (left < 2 && u + step < units) {
        const Unit n = unit_of(p, num_kb, u + step);
        left += passes(n.kb1 - n.kb0) + (u + 2 * step < units ? 1 : 0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && left >= 2)
        mbar_arrive_cluster(cluster_map(smem_u32(&tempty_bar[buf]), 0u));
      buf ^= 1;
      if (buf == 0) buf_phase ^= 1u;
    };
    for (int64_t u = cluster_id_x(); u < units; u += step) {
      const Unit q = unit_of(p, num_kb, u);
      const int m = q.at.m + side * kSlab;
      const bool live = m < p.M;  // a row of this CTA is one of D's (uniform)
      const bool part = q.row >= 0;
      const int n0 = q.at.n * kHalf + (P::kShared ? 0 : half * 64);  // gated: the box's first column
      const bool input = kEpi == kGradient && live && !part;
      if constexpr (kEpi == kGradient) {
        if (leader && input) {
          store_wait_read<0>();
          mbar_arrive_expect_tx(in, kBoxBytes);
          tma_load_2d(boxes, &maps.in, in, n0, m);
        }
      }
      bool got = true;
      float sums[kDrain > 0 ? 2 : 1][kDrain > 0 ? 64 : 1];  // gate and up
      if constexpr (kDrain > 0) {
#pragma unroll
        for (int i = 0; i < 64; ++i) sums[0][i] = sums[1][i] = 0.0f;
        for (int kc = q.kb0; kc < q.kb1 && got; kc += kDrain) {
          got = __all_sync(kAll, wait(&tfull_bar[buf], buf_phase));
          tc_fence_after();
          if (!got) break;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            float v[32];
            tmem_ld_x32(tb + (uint32_t)(buf * kBN + (h >> 1) * kHalf + half * 64 + (h & 1) * 32), v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sums[h >> 1][(h & 1) * 32 + i] += v[i];
          }
          free_buffer(passes(q.kb1 - kc) - 1, u);
        }
      } else {
        got = __all_sync(kAll, wait(&tfull_bar[buf], buf_phase));
        tc_fence_after();
      }
      if (input) {
        got = __all_sync(kAll, got && wait(in, in_phase));
        if (got) in_phase ^= 1u;
      }
      // the eight warps leave together: named barriers are between them
      if (!named_bar_and(kAllEpilogue, 256, got)) break;
      const uint32_t d = tb + (uint32_t)(buf * kBN);
      // gated: this warp's 32-column pieces of the gate columns, and where they lie in the box
      constexpr int kPieces = kHalf / 64;
      const int col0 = half * (kHalf / 2), piece0 = P::kShared ? half : 0;
      if (kBN == kTile && part) {
        for (int c = 0; c < 4 && live; ++c) {
          int col = half * 128 + c * 32;
          float v[32];
          if constexpr (kDrain > 0) {
            col = (c >> 1) * kHalf + half * 64 + (c & 1) * 32;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = c < 2 ? (c == 0 ? sums[0][i] : sums[0][32 + i])
                           : (c == 2 ? sums[kDrain > 0][i] : sums[kDrain > 0][32 + i]);
          } else {
            tmem_ld_x32(d + (uint32_t)col, v);
          }
          uint8_t* b = next_box();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(box_at(b, row, j)) =
                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          publish([&] { tma_store_2d(&maps.parts, b, col, q.row + side * kSlab); });
        }
      } else if constexpr (kEpi == kPlain) {
        for (int c = 0; c < kHalf / 64 && live; ++c) {
          const int col = half * kHalf + c * 64, to = q.at.n * kBN + col;
          if (to >= p.N) break;
          float v[64];
          tmem_ld_x64(d + (uint32_t)col, v);
          uint8_t* b = next_box();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = v[j * 8 + i];
            *box_at(b, row, j) = pack<T>(w);
          }
          publish([&] { tma_store_2d(&maps.o0, b, to, m); });
        }
      } else if constexpr (kEpi == kGated) {
        if (live && n0 < p.N) {
          uint8_t* b = next_box();
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            float g[32], v[32];
            tmem_ld_x32(d + (uint32_t)(col0 + h * 32), g);
            tmem_ld_x32(d + (uint32_t)(kHalf + col0 + h * 32), v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = gate_value<kAct>(g[j * 8 + i]) * v[j * 8 + i];
              *box_at(b, row, (piece0 + h) * 4 + j) = pack<T>(w);
            }
          }
          publish([&] { tma_store_2d(&maps.o0, b, n0, m); });
        }
      } else if constexpr (kEpi == kGatedSave) {
        // columns behind N are gate rows that belong to up, or nothing
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (n0 + (i & ~7) >= p.N) sums[0][i] = sums[1][i] = 0.0f;  // N is a multiple of 8
        if (live && n0 < p.N) {
          uint8_t* b = next_box();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = gate_value<kAct>(sums[0][j * 8 + i]) * sums[1][j * 8 + i];
            *box_at(b, row, j) = pack<T>(w);
          }
          publish([&] { tma_store_2d(&maps.o0, b, n0, m); });
        }
        // Both halves write the codes of gate (first box) and up (second).
        if (leader) store_wait_read<0>();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 64; ++i) top = fmaxf(top, finite_abs(sums[k][i]));
          s_exp[half][k][row] = (int8_t)(top == 0.0f ? -128 : fp8_exponent(top));
        }
        named_bar_sync(kAllEpilogue, 256);
        uint8_t* first = smem + kStages * kStageBytes;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // the larger value's exponent; a group of zeros has a scale of 1
          const int most = max((int)s_exp[0][k][row], (int)s_exp[1][k][row]);
          const int e = most == -128 ? 0 : most;
          if (k == half && live && m + row < p.M)
            (k == 0 ? p.gate : p.up).scales[(int64_t)(m + row) * p.nt + q.at.n] = fp8_scale(e);
          const float inv = fp8_scale(-e);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              c[i] = fp8_pack4(sums[k][j * 16 + 4 * i], sums[k][j * 16 + 4 * i + 1],
                               sums[k][j * 16 + 4 * i + 2], sums[k][j * 16 + 4 * i + 3], inv);
            *box_at(first + k * kBoxBytes, row, half * 4 + j) = make_uint4(c[0], c[1], c[2], c[3]);
          }
        }
        fence_async_shared();
        named_bar_sync(kAllEpilogue, 256);
        if (leader && live) {
          tma_store_2d(half == 0 ? &maps.o1 : &maps.o2, boxes, q.at.n * kSlab, m);
          store_commit();
        }
      } else {
        if (live && n0 < p.N) {
          // d_out lies in the first box, where its place takes d_gate; h waits in registers until
          // the store of d_up has read the second one
          uint8_t *bg = boxes, *bu = boxes + kBoxBytes;
          uint4 hold[kPieces * 4];
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            float g[32], v[32];
            tmem_ld_x32(d + (uint32_t)(col0 + h * 32), g);
            tmem_ld_x32(d + (uint32_t)(kHalf + col0 + h * 32), v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float dh[8], dg[8], du[8], hv[8];
              unpack<T>(*box_at(bg, row, (piece0 + h) * 4 + j), dh);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float a, s;
                gate_slope<kAct>(g[j * 8 + i], a, s);
                hv[i] = a * v[j * 8 + i];
                dg[i] = dh[i] * v[j * 8 + i] * s;
                du[i] = dh[i] * a;
              }
              hold[h * 4 + j] = pack<T>(hv);
              *box_at(bg, row, (piece0 + h) * 4 + j) = pack<T>(dg);
              *box_at(bu, row, (piece0 + h) * 4 + j) = pack<T>(du);
            }
          }
          publish([&] {
            tma_store_2d(&maps.o1, bg, n0, m);
            tma_store_2d(&maps.o2, bu, n0, m);
          });
          if (p.want_out) {
            if (leader) store_wait_read<0>();
            sync();
#pragma unroll
            for (int j = 0; j < kPieces * 4; ++j) *box_at(bu, row, piece0 * 4 + j) = hold[j];
            publish([&] { tma_store_2d(&maps.o0, bu, n0, m); });
          }
        }
      }
      if constexpr (kDrain == 0) free_buffer(0, u);
    }
    if (leader) {
      store_wait_read<0>();  // the writes themselves end with the kernel
      // d_out of a tile that gave up may still be on its way
      if (kEpi == kGradient && *abort_flag) {
        const uint64_t t = global_timer_ns();
        while (!mbar_try_wait(in, in_phase))
          if (global_timer_ns() - t > kDrainNs / 100) break;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  // Every arrival sent to the peer has been waited for there, unless one gave up: then what was sent
  // is released first.  (A release in every case costs 0.6 us: it waits for the stores to memory.)
  __syncthreads();
  if (*abort_flag)
    cluster_sync();
  else
    cluster_leave();
  tc_fence_after();
  // (the even CTA's stages are full only with the odd CTA's copies told of: else a second passes)
  if (*abort_flag) land_copies(full_bar, issued, kStages);
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kBN);
  }
}

// ---- tiles split along K: the parts' sums, and the epilogue on them ----------------------------
// A warp takes a row of a tile and 128 columns (gated: 128 gate and 128 up columns), a lane four of
// them; the parts are added in their order.  They were written just before and lie in L2.
struct JoinArgs {
  int M, N, mt, nt, rows;  // rows of a tile that may be any
  int64_t whole;
  int rest, split, want_out;
  const float* sums;  // [split][rest][kTile][kTile]
  void *o0, *o1;      // as Maps; d_pre
  const void* in;
  Ckpt gate, up;
};

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <typename T>
__device__ __forceinline__ void put4(void* base, int64_t at, const float (&v)[4]) {
  T h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = DT<T>::from_f(v[i]);
  *reinterpret_cast<uint2*>(static_cast<T*>(base) + at) = *reinterpret_cast<uint2*>(h);
}

template <typename T, int kEpi, int kAct>
__global__ void __launch_bounds__(256) join_kernel(const JoinArgs p) {
  pdl_wait();
  pdl_trigger();
  constexpr int kGroups = gated(kEpi) ? 1 : 2;
  const int lane = threadIdx.x & 31;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int g = (int)(at % kGroups);
  const int row = (int)(at / kGroups % p.rows);
  const int64_t tile = at / kGroups / p.rows;
  if (tile >= p.rest) return;
  const Place q = place_of(p.mt, p.nt, p.whole + tile);
  const int64_t m = (int64_t)q.m + row;
  const int n = gated(kEpi) ? q.n * kSlab + lane * 4 : q.n * kTile + g * kSlab + lane * 4;
  if (m >= p.M) return;
  const int64_t part = (int64_t)p.rest * kTile * kTile;
  auto sum = [&](int col) {
    const float* from = p.sums + (tile * kTile + row) * kTile + col;
    float4 s = *reinterpret_cast<const float4*>(from);
    int i = 1;
    for (; i + 3 <= p.split; i += 3) {  // three on their way at a time
      const float4 a = *reinterpret_cast<const float4*>(from + i * part);
      const float4 b = *reinterpret_cast<const float4*>(from + (i + 1) * part);
      const float4 c = *reinterpret_cast<const float4*>(from + (i + 2) * part);
      s = add4(add4(add4(s, a), b), c);
    }
    for (; i < p.split; ++i) s = add4(s, *reinterpret_cast<const float4*>(from + i * part));
    return s;
  };
  const bool live = n < p.N;  // N is a multiple of 8
  if constexpr (!gated(kEpi)) {
    if (!live) return;
    const float4 s = sum(g * kSlab + lane * 4);
    const float v[4] = {s.x, s.y, s.z, s.w};
    put4<T>(p.o0, m * p.N + n, v);
  } else {
    float4 sg = make_float4(0.0f, 0.0f, 0.0f, 0.0f), su = sg;
    if (live) {
      sg = sum(lane * 4);
      su = sum(kSlab + lane * 4);
    }
    const float gv[4] = {sg.x, sg.y, sg.z, sg.w}, uv[4] = {su.x, su.y, su.z, su.w};
    if constexpr (kEpi == kGradient) {
      if (!live) return;
      float dh[4], h[4], dg[4], du[4];
      const uint2 raw = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.in) + m * p.N + n);
      const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, s;
        dh[i] = DT<T>::to_f(t[i]);
        gate_slope<kAct>(gv[i], a, s);
        h[i] = a * uv[i];
        dg[i] = dh[i] * uv[i] * s;
        du[i] = dh[i] * a;
      }
      if (p.want_out) put4<T>(p.o0, m * p.N + n, h);
      put4<T>(p.o1, m * 2 * p.N + n, dg);
      put4<T>(p.o1, (m * 2 + 1) * p.N + n, du);
    } else {
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = gate_value<kAct>(gv[i]) * uv[i];
      if (live) put4<T>(p.o0, m * p.N + n, h);
      if constexpr (kEpi == kGatedSave) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float(&v)[4] = half == 0 ? gv : uv;
          const Ckpt& to = half == 0 ? p.gate : p.up;
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, finite_abs(v[i]));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
          const int e = fp8_exponent(top);
          if (lane == 0) to.scales[m * p.nt + q.n] = fp8_scale(e);
          *reinterpret_cast<uint32_t*>(to.codes + (m * p.nt + q.n) * kCkptGroup + lane * 4) =
              live ? fp8_pack4(v[0], v[1], v[2], v[3], fp8_scale(-e)) : 0u;
        }
      }
    }
  }
}

// ---- host side ---------------------------------------------------------------------------------
// Pairs of CTAs that the device holds at once with the shared memory of `Kernel`: a pair stays
// within one group of SMs, so this can be less than half the SMs.
template <auto Kernel>
int max_pairs(int smem) {
  static int cached[64];
  static std::once_flag once[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::call_once(once[dev], [=] {
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (set_smem_limit<Kernel>(smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    cached[dev] = n;
  });
  return cached[dev];
}

// A 2-D map of rows `pitch` bytes apart with the 128-byte swizzle, boxes of 128 bytes x box_rows.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, int size, const void* base, uint64_t inner,
              uint64_t rows, uint64_t pitch, uint32_t box_rows) {
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
CUtensorMapDataType type16(int dtype) {
  return dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}
bool map16(CUtensorMap* m, int dtype, const void* base, int64_t inner, int64_t rows, int64_t pitch,
           int box_rows) {
  return make_map(m, type16(dtype), 2, base, (uint64_t)inner, (uint64_t)rows, (uint64_t)pitch * 2,
                  (uint32_t)box_rows);
}

// Which tiles are split, and in how many parts of K.  `pairs` take their tiles in turn; the last
// `rest` of them, which would leave most pairs idle, are split so that all have a part.  A part has
// at least eight 64-k blocks, and splitting has to gain more blocks than joining costs.
struct Split {
  int64_t whole;
  int rest, split;
};
constexpr int kMaxSplit = 16, kPartBlocks = 8, kJoinBlocks = 16;
Split split_of(int64_t tiles, int64_t K) {
  const int64_t pairs = num_sms() / 2, num_kb = ceil_div(K, kBlockK);
  const int64_t rest = tiles % pairs;
  int64_t split = rest > 0 ? pairs / rest : 1;
  if (split > num_kb / kPartBlocks) split = num_kb / kPartBlocks;
  if (split > kMaxSplit) split = kMaxSplit;
  if (split < 2 || num_kb - ceil_div(num_kb, split) <= kJoinBlocks) return Split{tiles, 0, 1};
  return Split{tiles - rest, (int)rest, (int)split};
}
int64_t tiles_n(int64_t N, bool gate, int bn) { return ceil_div(N, gate ? bn / 2 : bn); }

// Tiles of 128 columns where those of 256 leave pairs idle.  In units of a 64-k block of a 256-column
// tile: a narrow one costs 0.65 (the loads of a, which it shares with fewer columns), a tile's start
// and epilogue about 16 and 12.
bool narrow(int64_t M, int64_t N, int64_t K, bool gate) {
  const int64_t pairs = num_sms() / 2, mt = ceil_div(M, kTile), num_kb = ceil_div(K, kBlockK);
  const int64_t wide_tiles = mt * tiles_n(N, gate, kTile);
  const Split sp = split_of(wide_tiles, K);
  double wide = (double)(sp.whole / pairs) * (num_kb + 16);
  if (sp.rest > 0)
    wide += ceil_div(num_kb, sp.split) + 16 + kJoinBlocks;
  else if (sp.whole % pairs)
    wide += num_kb + 16;
  const double thin = (double)ceil_div(mt * tiles_n(N, gate, 128), pairs) * (0.65 * num_kb + 12);
  return thin < wide;
}

struct Problem {
  int dtype, M, N, K;
  const void *a, *b;
  int64_t a_pitch;
  void *o0, *o1;  // h or the product; d_pre
  const void* in;
  Ckpt gate, up;
  float* parts;
  int* status;
};

template <typename T, bool kAMn, bool kBMn, int kEpi, int kAct, int kBN>
cudaError_t run_tiles(const Problem& q, cudaStream_t s) {
  constexpr bool kGate = gated(kEpi);
  using P = Plan<kEpi, kBN>;
  constexpr auto kern = dense_kernel<T, kAMn, kBMn, kEpi, kAct, kBN>;
  Args p = {};
  p.M = q.M;
  p.N = q.N;
  p.K = q.K;
  p.mt = (int)ceil_div(q.M, kTile);
  p.nt = (int)tiles_n(q.N, kGate, kBN);
  const int64_t tiles = (int64_t)p.mt * p.nt;
  const Split sp = kBN == kTile ? split_of(tiles, q.K) : Split{tiles, 0, 1};
  p.whole = sp.whole;
  p.rest = sp.rest;
  p.split = sp.split;
  p.a_rows = q.M < kSlab ? (q.M + 7) / 8 * 8 : kSlab;
  p.want_out = q.o0 != nullptr;
  p.gate = q.gate;
  p.up = q.up;
  p.status = q.status;
  p.limit_ns = wait_limit_ns();
  Maps maps;
  const int64_t N = q.N, rows_b = kGate ? 2 * N : N;
  bool ok = kAMn ? map16(&maps.a, q.dtype, q.a, q.M, q.K, q.a_pitch, kBlockK)
                 : map16(&maps.a, q.dtype, q.a, q.K, q.M, q.a_pitch, p.a_rows);
  ok = ok && (kBMn ? map16(&maps.b, q.dtype, q.b, rows_b, q.K, rows_b, kBlockK)
                   : map16(&maps.b, q.dtype, q.b, q.K, rows_b, q.K, kBN / 2));
  maps.o0 = maps.o1 = maps.o2 = maps.in = maps.parts = maps.a;  // those that are not used
  if (q.o0) ok = ok && map16(&maps.o0, q.dtype, q.o0, N, q.M, N, kSlab);
  if constexpr (kEpi == kGradient) {
    ok = ok && map16(&maps.o1, q.dtype, q.o1, N, q.M, 2 * N, kSlab) &&
         map16(&maps.o2, q.dtype, static_cast<T*>(q.o1) + N, N, q.M, 2 * N, kSlab) &&
         map16(&maps.in, q.dtype, q.in, N, q.M, N, kSlab);
  } else if constexpr (kEpi == kGatedSave) {
    const uint64_t width = (uint64_t)ckpt_width(N);
    ok = ok &&
         make_map(&maps.o1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.gate.codes, width, (uint64_t)q.M,
                  width, kSlab) &&
         make_map(&maps.o2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.up.codes, width, (uint64_t)q.M,
                  width, kSlab);
  }
  if (p.rest > 0)
    ok = ok && make_map(&maps.parts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, q.parts, kTile,
                        (uint64_t)p.rest * p.split * kTile, kTile * 4, kSlab);
  if (!ok) return cudaErrorInvalidValue;
  const int pairs = max_pairs<kern>(P::kSmem);
  if (pairs <= 0) return cudaErrorInvalidConfiguration;
  const int64_t units = p.whole + (int64_t)p.rest * p.split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (units < pairs ? units : pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)P::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, maps, p);
  if (e != cudaSuccess || p.rest == 0) return e;
  JoinArgs j = {};
  j.M = q.M;
  j.N = q.N;
  j.mt = p.mt;
  j.nt = p.nt;
  j.rows = q.M < kTile ? q.M : kTile;
  j.whole = p.whole;
  j.rest = p.rest;
  j.split = p.split;
  j.want_out = p.want_out;
  j.sums = q.parts;
  j.o0 = q.o0;
  j.o1 = q.o1;
  j.in = q.in;
  j.gate = q.gate;
  j.up = q.up;
  const int64_t warps = (int64_t)p.rest * j.rows * (kGate ? 1 : 2);
  return launch_k(join_kernel<T, kEpi, kAct>, dim3((unsigned)ceil_div(warps, 8)), dim3(256), 0, s,
                  true, j);
}

template <typename T, bool kAMn, bool kBMn, int kEpi, int kAct>
cudaError_t run(const Problem& q, cudaStream_t s) {
  if constexpr (kEpi != kGatedSave) {  // whose checkpoints have 128 channels to a scale
    if (narrow(q.M, q.N, q.K, gated(kEpi))) return run_tiles<T, kAMn, kBMn, kEpi, kAct, 128>(q, s);
  }
  return run_tiles<T, kAMn, kBMn, kEpi, kAct, kTile>(q, s);
}

template <int kEpi>
cudaError_t run_gated(int act, const Problem& q, cudaStream_t s) {
  if (q.dtype == MOE_BF16)
    return act == MOE_ACT_SILU
               ? run<__nv_bfloat16, false, false, kEpi, MOE_ACT_SILU>(q, s)
               : run<__nv_bfloat16, false, false, kEpi, MOE_ACT_GELU_TANH>(q, s);
  return act == MOE_ACT_SILU ? run<__half, false, false, kEpi, MOE_ACT_SILU>(q, s)
                             : run<__half, false, false, kEpi, MOE_ACT_GELU_TANH>(q, s);
}

}  // namespace

size_t dense_split_bytes(int64_t M, int64_t N, int64_t K, bool gate) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const Split sp = split_of(ceil_div(M, kTile) * tiles_n(N, gate, kTile), K);
  return (size_t)sp.rest * sp.split * kTile * kTile * sizeof(float);
}

cudaError_t launch_dense_nn(int dtype, int M, int N, int K, const void* a, int64_t a_pitch,
                            const void* b, void* out, float* parts, int* status, cudaStream_t s) {
  Problem q = {};
  q.dtype = dtype, q.M = M, q.N = N, q.K = K, q.a = a, q.a_pitch = a_pitch, q.b = b, q.o0 = out;
  q.parts = parts, q.status = status;
  return dtype == MOE_BF16 ? run<__nv_bfloat16, false, true, kPlain, 0>(q, s)
                           : run<__half, false, true, kPlain, 0>(q, s);
}

cudaError_t launch_dense_tn(int dtype, int M, int N, int K, const void* a, int64_t a_pitch,
                            const void* b, void* out, float* parts, int* status, cudaStream_t s) {
  Problem q = {};
  q.dtype = dtype, q.M = M, q.N = N, q.K = K, q.a = a, q.a_pitch = a_pitch, q.b = b, q.o0 = out;
  q.parts = parts, q.status = status;
  return dtype == MOE_BF16 ? run<__nv_bfloat16, true, true, kPlain, 0>(q, s)
                           : run<__half, true, true, kPlain, 0>(q, s);
}

cudaError_t launch_gated(int dtype, int act, int T, int F, int H, const void* x, const void* w,
                         void* out, Ckpt gate, Ckpt up, float* parts, int* status,
                         cudaStream_t s) {
  Problem q = {};
  q.dtype = dtype, q.M = T, q.N = F, q.K = H, q.a = x, q.a_pitch = H, q.b = w, q.o0 = out;
  q.gate = gate, q.up = up, q.parts = parts, q.status = status;
  return gate.codes ? run_gated<kGatedSave>(act, q, s) : run_gated<kGated>(act, q, s);
}

cudaError_t launch_gated_grad(int dtype, int act, int T, int F, int H, const void* x, const void* w,
                              const void* d_out, void* d_pre, void* out, float* parts, int* status,
                              cudaStream_t s) {
  Problem q = {};
  q.dtype = dtype, q.M = T, q.N = F, q.K = H, q.a = x, q.a_pitch = H, q.b = w, q.o0 = out, q.o1 = d_pre;
  q.in = d_out, q.parts = parts, q.status = status;
  return run_gated<kGradient>(act, q, s);
}

}  // namespace gb300moe
