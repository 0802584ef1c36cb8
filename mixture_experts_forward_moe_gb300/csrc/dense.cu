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
// A call's two gradients (dy w and dy^T x) are one launch, whose pairs share out the tiles of both.
#include "activation.cuh"
#include "dense_ops.cuh"
#include "fp8.cuh"
#include "pipe.cuh"
#include "vec16.cuh"

#include <math.h>

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
// registers after every few 64-k blocks.
// What truncation takes off grows with K, which is the rows of x where d_w is made: past kChainK of it
// (kLong) accumulators are added to sums in registers as well.  4096 x 7168 x 18432, both gradients: 1257
// us, 1234 in one accumulator.
constexpr int kChainBlocks = kChainK / kBlockK;
// A sum of f32 on the CUDA cores is off by less the shorter K is, so a short K is drained more often:
// no more codes fall on their neighbours than those of an f32 product.  That has 518 of 168 million there
// at K = 136, 358 and 505 of 84 million at 264 and 512, 532 and 1245 of 42 million at 2056 and 7168.
// Drained every block 483, 258, 322, 239 and 364, every two 652, 313, 445, 247 and 307, every four 659,
// 560, 712, 398 and 441, every eight 659, 564, 1240, 784 and 825.  A pass costs time where the products
// are short: 16384 x 5120 x 512 takes 129 us with two blocks, 108 with four.
inline int drain_blocks(int64_t K) {
  const int64_t blocks = ceil_div(K, kBlockK);
  return blocks <= 4 ? 1 : blocks <= 12 ? 2 : blocks <= 64 ? 4 : 8;
}

struct Maps {
  CUtensorMap a[2], b[2], o0[2];  // of each product; o0: h, gated
  CUtensorMap o1, o2;             // gate and up codes, or the two halves of d_pre
  CUtensorMap in;                 // kGradient: d_out
  CUtensorMap parts;              // sums of the tiles that are split
};

// A product.
struct Prod {
  int M, N, num_kb;  // outputs (gated: N of 2 N rows of b), 64-k blocks
  int mt, nt;        // tiles
  int64_t whole;     // tiles that are not split; then
  int rest;          // the others, each
  int split;         // in as many parts of K,
  int part_row;      // whose sums begin there
  int a_mn;          // a is MN-major (kPlain)
  int a_rows;        // of a K-major a that a copy brings
};
struct Args {
  Prod q[2];
  int64_t units[2];  // tiles and parts of each; a unit of the first costs no less
  // kPlain (see unit_at): every pair takes `own` of the first's units, the first `more` pairs one
  // more, and all take `rounds` of the second's
  int64_t own, more, rounds;
  int want_out;      // kGradient: h too
  int drain;         // kGatedSave, kLong: blocks between two roundings of the sums
  Ckpt gate, up;     // kGatedSave (codes by TMA)
  int* status;
  uint64_t limit_ns;
};

// Descriptor of an MN-major operand with the 128-byte swizzle: boxes of 64 (mn) x 64 (k), a k row
// 128 bytes; eight k rows further 1024 bytes (stride offset), 64 mn further a box (leading offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBlockK * 128 >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Of an operand in either order, and what 16 k further add to it (in units of 16 bytes).
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, bool mn) {
  return mn ? sw128_mnmajor_desc(saddr) : sw128_kmajor_desc(saddr);
}
__device__ __forceinline__ uint64_t k16_step(bool mn) { return mn ? 2048 / 16 : 32 / 16; }

template <int kRows>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                             int mn, int k, bool is_mn) {
  if (is_mn) {
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
  int prod;
  Place at;
  int kb0, kb1, row;
};
template <int kEpi>
__device__ __forceinline__ Unit unit_of(const Args& p, int64_t u) {
  Unit r;
  r.prod = kEpi == kPlain && u >= p.units[0] ? 1 : 0;
  const Prod& q = p.q[r.prod];
  if (r.prod) u -= p.units[0];
  if (u < q.whole) {
    r.at = place_of(q.mt, q.nt, u);
    r.kb0 = 0;
    r.kb1 = q.num_kb;
    r.row = -1;
  } else {
    const int i = (int)(u - q.whole), part = i / q.rest;
    r.at = place_of(q.mt, q.nt, q.whole + i % q.rest);
    r.kb0 = (int)((int64_t)q.num_kb * part / q.split);
    r.kb1 = (int)((int64_t)q.num_kb * (part + 1) / q.split);
    r.row = q.part_row + i * kTile;
  }
  return r;
}

// The s-th unit of this pair, -1 past its last.  Pairs take the first product's units in turn, which
// leaves some with one more of them; of the second's all take as many, and the others the rest.
template <int kEpi>
__device__ __forceinline__ int64_t unit_at(const Args& p, int64_t s) {
  const int64_t pairs = num_clusters_x(), i = cluster_id_x();
  if constexpr (kEpi == kPlain) {
    const int64_t own = p.own + (i < p.more ? 1 : 0);
    if (s >= own) {
      s -= own;
      if (s >= p.rounds && i < p.more) return -1;
      const int64_t v = s < p.rounds ? s * pairs + i
                                     : p.rounds * pairs + (s - p.rounds) * (pairs - p.more) +
                                           (i - p.more);
      return v < p.units[1] ? p.units[0] + v : -1;
    }
  }
  const int64_t u = i + s * pairs;
  return u < p.units[0] ? u : -1;
}

// Roles (320 threads): warp 0 TMA producer; warp 1 issues the MMAs (even CTA) or tells the even CTA
// that a stage of this CTA has landed (odd CTA); warps 2-5 and 6-9 epilogue, each four half of the
// columns.  (One half for all: 4096 x 2048 x 7168 saved in 145 us.)  Every wait is bounded
// (MOE_ERR_TIMEOUT in the status word); a pair in which one gave up waits for its copies, MMAs and
// stores in flight before it leaves.
template <typename T, int kEpi, int kAct, int kBN, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ Maps maps, const Args p) {
  using P = Plan<kEpi, kBN>;
  constexpr int kStages = P::kStages, kStageBytes = P::kStageBytes;
  constexpr int kHalf = kBN / 2;  // columns of a half of the warps; gated: gate columns of a tile
  constexpr bool kDrain = kEpi == kGatedSave || kLong;
  static_assert(!kDrain || kBN == kTile, "a thread's 128 sums");
  constexpr bool kBMn = kEpi == kPlain;
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
  auto load_block = [&](const Unit& q, int kb, int stage) {
    const Prod& d = p.q[q.prod];
    uint8_t* st = smem + stage * kStageBytes;
    uint64_t* full = &full_bar[stage];
    const bool a_mn = kEpi == kPlain && d.a_mn;
    // Fewer than 128 rows of a: the others of its operand hold anything, and make rows of D that
    // nothing reads.
    const bool some = a_mn || side == 0 || d.M > kSlab;
    const int left_out = a_mn ? 0 : (kSlab - (some ? d.a_rows : 0)) * kBlockK * 2;
    // gated: the even CTA has the gate rows of b, the odd one the up rows; gate rows past N are rows
    // of up, whose columns the epilogue leaves out
    const int nb = gated(kEpi) ? side * d.N + q.at.n * kHalf : q.at.n * kBN + side * kHalf;
    mbar_arrive_expect_tx(full, (uint32_t)(kStageBytes - left_out));
    if (some)
      load_operand<kSlab>(st, &maps.a[q.prod], full, q.at.m + side * kSlab, kb * kBlockK, a_mn);
    load_operand<kHalf>(st + kOperandBytes, &maps.b[q.prod], full, nb, kb * kBlockK, kBMn);
  };
  int issued = 0;  // by the producer (the same thread is elected here and below): stages asked for

  if (warp == 0) {
    if (elect_one()) {
      prefetch_tensormap(&maps.a[0]);
      prefetch_tensormap(&maps.b[0]);
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
      const int64_t u = unit_at<kEpi>(p, 0);
      if (u >= 0) {
        const Unit q = unit_of<kEpi>(p, u);
        for (; issued < kStages && q.kb0 + issued < q.kb1; ++issued)
          load_block(q, q.kb0 + issued, issued);
      }
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
      int64_t u;
      for (int64_t s = 0; ok && (u = unit_at<kEpi>(p, s)) >= 0; ++s) {
        const Unit q = unit_of<kEpi>(p, u);
        for (int kb = s == 0 ? q.kb0 + early : q.kb0; kb < q.kb1; ++kb) {
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
      int64_t u;
      for (int64_t s = 0; ok && (u = unit_at<kEpi>(p, s)) >= 0; ++s) {
        const Unit q = unit_of<kEpi>(p, u);
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
      const uint32_t idesc_b = idesc_f16(256, kBN, DT<T>::kIsBF16) | (kBMn ? 1u << 16 : 0u);
      const uint32_t empty_own = smem_u32(empty_bar), tfull_own = smem_u32(tfull_bar);
      int64_t u;
      for (int64_t s = 0; ok && (u = unit_at<kEpi>(p, s)) >= 0; ++s) {
        const Unit q = unit_of<kEpi>(p, u);
        const int pass = kDrain ? p.drain : q.kb1 - q.kb0;  // blocks of one accumulator
        const bool a_mn = kEpi == kPlain && p.q[q.prod].a_mn;
        const uint32_t idesc = idesc_b | (a_mn ? 1u << 15 : 0u);
        const uint64_t a_step = k16_step(a_mn);
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
            const uint64_t da = operand_desc(sa, a_mn), db = operand_desc(sb, kBMn);
            const uint32_t at = (uint32_t)r.stage * 8u;
            r.next();
#pragma unroll
            for (int k = 0; k < kBlockK / 16; ++k)
              umma_f16_pair(d, da + k * a_step, db + k * k16_step(kBMn), idesc,
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
    auto passes = [&](int blocks) { return kDrain ? (blocks - 1) / p.drain + 1 : 1; };
    // The accumulator has been read; `left` passes of the s-th unit follow.  Where no later pass takes
    // this buffer nobody waits for the arrival, and the even CTA may leave before it comes.
    auto free_buffer = [&](int left, int64_t s) {
      const int64_t next = left < 2 ? unit_at<kEpi>(p, s + 1) : -1;
      if (next >= 0) {
        const Unit n = unit_of<kEpi>(p, next);
        left += passes(n.kb1 - n.kb0) + (unit_at<kEpi>(p, s + 2) >= 0 ? 1 : 0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && left >= 2)
        mbar_arrive_cluster(cluster_map(smem_u32(&tempty_bar[buf]), 0u));
      buf ^= 1;
      if (buf == 0) buf_phase ^= 1u;
    };
    int64_t u;
    for (int64_t s = 0; (u = unit_at<kEpi>(p, s)) >= 0; ++s) {
      const Unit q = unit_of<kEpi>(p, u);
      const int M = p.q[q.prod].M, N = p.q[q.prod].N;
      const int m = q.at.m + side * kSlab;
      const bool live = m < M;  // a row of this CTA is one of D's (uniform)
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
      float sums[kDrain ? 2 : 1][kDrain ? 64 : 1];  // gate and up, or the half's 128 columns
      auto sum_col = [&](int h) {  // where 32 of them lie in an accumulator
        return gated(kEpi) ? (h >> 1) * kHalf + half * 64 + (h & 1) * 32 : half * kHalf + h * 32;
      };
      if constexpr (kDrain) {
#pragma unroll
        for (int i = 0; i < 64; ++i) sums[0][i] = sums[1][i] = 0.0f;
        for (int kc = q.kb0; kc < q.kb1 && got; kc += p.drain) {
          got = __all_sync(kAll, wait(&tfull_bar[buf], buf_phase));
          tc_fence_after();
          if (!got) break;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            float v[32];
            tmem_ld_x32(tb + (uint32_t)(buf * kBN + sum_col(h)), v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sums[h >> 1][(h & 1) * 32 + i] += v[i];
          }
          free_buffer(passes(q.kb1 - kc) - 1, s);
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
      auto pre_activations = [&](int h, float(&g)[32], float(&v)[32]) {
        if constexpr (kDrain) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            g[i] = h == 0 ? sums[0][i] : sums[0][32 + i];
            v[i] = h == 0 ? sums[1][i] : sums[1][32 + i];
          }
        } else {
          tmem_ld_x32(d + (uint32_t)(col0 + h * 32), g);
          tmem_ld_x32(d + (uint32_t)(kHalf + col0 + h * 32), v);
        }
      };
      if (kBN == kTile && part) {
        for (int c = 0; c < 4 && live; ++c) {
          int col = half * 128 + c * 32;
          float v[32];
          if constexpr (kDrain) {
            col = sum_col(c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = c < 2 ? (c == 0 ? sums[0][i] : sums[0][32 + i])
                           : (c == 2 ? sums[kDrain ? 1 : 0][i] : sums[kDrain ? 1 : 0][32 + i]);
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
          if (to >= N) break;
          float v[64];
          if constexpr (kDrain) {
#pragma unroll
            for (int i = 0; i < 64; ++i) v[i] = c == 0 ? sums[0][i] : sums[1][i];
          } else {
            tmem_ld_x64(d + (uint32_t)col, v);
          }
          uint8_t* b = next_box();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = v[j * 8 + i];
            *box_at(b, row, j) = pack<T>(w);
          }
          publish([&] { tma_store_2d(&maps.o0[q.prod], b, to, m); });
        }
      } else if constexpr (kEpi == kGated) {
        if (live && n0 < N) {
          uint8_t* b = next_box();
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            float g[32], v[32];
            pre_activations(h, g, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = gate_value<kAct>(g[j * 8 + i]) * v[j * 8 + i];
              *box_at(b, row, (piece0 + h) * 4 + j) = pack<T>(w);
            }
          }
          publish([&] { tma_store_2d(&maps.o0[q.prod], b, n0, m); });
        }
      } else if constexpr (kEpi == kGatedSave) {
        // columns behind N are gate rows that belong to up, or nothing
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (n0 + (i & ~7) >= N) sums[0][i] = sums[1][i] = 0.0f;  // N is a multiple of 8
        if (live && n0 < N) {
          uint8_t* b = next_box();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = gate_value<kAct>(sums[0][j * 8 + i]) * sums[1][j * 8 + i];
            *box_at(b, row, j) = pack<T>(w);
          }
          publish([&] { tma_store_2d(&maps.o0[q.prod], b, n0, m); });
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
          if (k == half && live && m + row < M)
            (k == 0 ? p.gate : p.up).scales[(int64_t)(m + row) * p.q[0].nt + q.at.n] = fp8_scale(e);
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
        if (live && n0 < N) {
          // d_out lies in the first box, where its place takes d_gate; h waits in registers until
          // the store of d_up has read the second one
          uint8_t *bg = boxes, *bu = boxes + kBoxBytes;
          uint4 hold[kPieces * 4];
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            float g[32], v[32];
            pre_activations(h, g, v);
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
            publish([&] { tma_store_2d(&maps.o0[q.prod], bu, n0, m); });
          }
        }
      }
      if constexpr (!kDrain) free_buffer(0, s);
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

CUtensorMapDataType type16(int dtype) {
  return dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}
bool map16(CUtensorMap* m, int dtype, const void* base, int64_t inner, int64_t rows, int64_t pitch,
           int box_rows) {
  return rows_map(m, type16(dtype), 2, base, (uint64_t)inner, (uint64_t)rows, (uint64_t)pitch * 2,
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
// and epilogue about 16 and 12.  (More than kChainBlocks are added up in tiles of 256 alone.)
bool narrow(int64_t M, int64_t N, int64_t K, bool gate) {
  const int64_t pairs = num_sms() / 2, mt = ceil_div(M, kTile), num_kb = ceil_div(K, kBlockK);
  if (num_kb > kChainBlocks) return false;
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

// The units and parts of a product in tiles of `bn` columns.
Prod prod_of(int M, int N, int K, bool gate, int bn, Split sp) {
  Prod q = {};
  q.M = M;
  q.N = N;
  q.num_kb = (int)ceil_div(K, kBlockK);
  q.mt = (int)ceil_div(M, kTile);
  q.nt = (int)tiles_n(N, gate, bn);
  q.whole = sp.whole;
  q.rest = sp.rest;
  q.split = sp.split;
  q.a_rows = M < kSlab ? (M + 7) / 8 * 8 : kSlab;
  return q;
}
int64_t units_of(const Prod& q) { return q.whole + (int64_t)q.rest * q.split; }

struct Problem {
  int dtype;
  float* parts;
  int* status;
  // gated
  int M, N, K;
  const void *x, *w, *in;
  void *h, *d_pre;
  Ckpt gate, up;
  // kPlain: one or two products, the one with the longer units first
  const Product* list[2];
  int n;
};

// The products of a call: tiles of 256 columns, some split, or of 128.
struct Choice {
  int bn;
  int first;  // the product with the longer units
  Split sp[2];
  bool apart;  // a launch for each
};

// What the busiest pair does, in 64-k blocks of a 256-column tile, where n[0] units of c[0] are shared
// out before n[1] of c[1] as unit_at does it; `rounds` as there.
double busiest(const int64_t (&n)[2], const double (&c)[2], int64_t pairs, int64_t* rounds) {
  const int64_t more = n[0] % pairs, own = n[0] / pairs;
  int64_t most = 0, all = 0;  // units of the second that a pair takes, and that all take
  if (n[1] > 0) {
    const int64_t behind = (int64_t)ceil(c[0] / c[1]);
    most = (pairs - more) * behind >= n[1] ? ceil_div(n[1], pairs - more)
                                           : ceil_div(n[1] + more * behind, pairs);
    all = more == 0 ? most : most > behind ? most - behind : 0;
  }
  if (rounds) *rounds = all;
  const double late = more > 0 ? (own + 1) * c[0] + all * c[1] : 0.0;
  const double rest = own * c[0] + most * c[1];
  return late > rest ? late : rest;
}

// A unit costs its blocks, or its epilogue where that takes longer.
double unit_cost(int64_t blocks, int bn) {
  const double mma = bn == kTile ? (double)blocks : 0.65 * blocks;
  const double epilogue = bn == kTile ? 8.0 : 5.0;
  return mma > epilogue ? mma : epilogue;
}

// Two gradients share a launch, which fills the pairs that the first one's last tiles leave idle and
// starts once: 243 rows of 416 x 1784 take 9 us, in two launches 17, and 4096 rows of 4096 x 4096
// 155, in two 181.  Its units are whole, though, where a launch for each splits its last tiles: 6943
// rows of 12360 x 680 take 237 us in one and 210 in two.  The busiest pairs' blocks foretell that to
// about a tenth (3051 rows of 2960 x 6136: two should gain 7% and lose 4%), which is what a gain has
// to be.
constexpr int kStartBlocks = 16;  // what a launch costs

Choice choose(const Product* q, int n) {
  const int64_t pairs = num_sms() / 2;
  Choice r = {};
  if (n == 1) {
    r.bn = narrow(q[0].M, q[0].N, q[0].K, false) ? 128 : kTile;
    const int64_t tiles = ceil_div(q[0].M, kTile) * tiles_n(q[0].N, false, r.bn);
    r.sp[0] = r.bn == kTile ? split_of(tiles, q[0].K) : Split{tiles, 0, 1};
    return r;
  }
  double best = 0.0;
  const bool may_narrow = ceil_div(q[0].K > q[1].K ? q[0].K : q[1].K, kBlockK) <= kChainBlocks;
  for (const int bn : {kTile, 128}) {
    if (bn != kTile && !may_narrow) break;
    Choice t = {};
    t.bn = bn;
    int64_t tiles[2], kb[2];
    double work = 0.0;
    for (int i = 0; i < 2; ++i) {
      tiles[i] = ceil_div(q[i].M, kTile) * tiles_n(q[i].N, false, bn);
      kb[i] = ceil_div(q[i].K, kBlockK);
      work += tiles[i] * unit_cost(kb[i], bn);
    }
    const double share = work / pairs;
    double join = 0.0;
    for (int i = 0; i < 2; ++i) {
      t.sp[i] = Split{tiles[i], 0, 1};
      // A tile that takes longer than a pair's share is split, in parts of at least eight blocks.
      int64_t split = share > 1.0 ? (int64_t)ceil(kb[i] / share) : kMaxSplit;
      if (split > kb[i] / kPartBlocks) split = kb[i] / kPartBlocks;
      if (split > kMaxSplit) split = kMaxSplit;
      if (split * tiles[i] > 2 * pairs) split = 2 * pairs / tiles[i];
      if (bn == kTile && split > 1 && kb[i] - ceil_div(kb[i], split) > kJoinBlocks) {
        t.sp[i] = Split{0, (int)tiles[i], (int)split};
        join = kJoinBlocks;
      }
    }
    int64_t units[2];
    double cost[2];
    for (int i = 0; i < 2; ++i) {
      units[i] = t.sp[i].whole + (int64_t)t.sp[i].rest * t.sp[i].split;
      cost[i] = unit_cost(ceil_div(kb[i], t.sp[i].split), bn);
    }
    t.first = cost[1] > cost[0];
    const double total =
        join + busiest({units[t.first], units[1 - t.first]}, {cost[t.first], cost[1 - t.first]},
                       pairs, nullptr);
    if (bn == kTile || total < best) best = total, r = t;
  }
  double two = kStartBlocks;
  for (int i = 0; i < 2; ++i) {
    const Choice c = choose(q + i, 1);
    const int64_t kb = ceil_div(q[i].K, kBlockK);
    const Split& sp = c.sp[0];
    two += sp.whole / pairs * unit_cost(kb, c.bn);
    if (sp.rest > 0)
      two += unit_cost(ceil_div(kb, sp.split), c.bn) + kJoinBlocks;
    else if (sp.whole % pairs)
      two += unit_cost(kb, c.bn);
  }
  r.apart = two < 0.9 * best;
  return r;
}

template <typename T, int kEpi, int kAct, int kBN, bool kLong>
cudaError_t run_tiles(const Problem& q, const Choice& ch, cudaStream_t s) {
  constexpr bool kGate = gated(kEpi);
  using P = Plan<kEpi, kBN>;
  constexpr auto kern = dense_kernel<T, kEpi, kAct, kBN, kLong>;
  Args p = {};
  Maps maps = {};
  bool ok = true;
  const int n = kGate ? 1 : q.n;
  int part_rows = 0;
  for (int i = 0; i < n; ++i) {
    const int from = i == 0 ? ch.first : 1 - ch.first;
    const Product* l = kGate ? nullptr : q.list[from];
    const int M = kGate ? q.M : l->M, N = kGate ? q.N : l->N, K = kGate ? q.K : l->K;
    Prod& d = p.q[i];
    d = prod_of(M, N, K, kGate, kBN, ch.sp[kGate ? 0 : from]);
    d.a_mn = !kGate && l->tn;
    d.part_row = part_rows;
    part_rows += d.rest * d.split * kTile;
    p.units[i] = units_of(d);
    if constexpr (kGate) {
      ok = ok && map16(&maps.a[0], q.dtype, q.x, K, M, K, d.a_rows) &&
           map16(&maps.b[0], q.dtype, q.w, K, 2 * (int64_t)N, K, kBN / 2);
    } else {
      ok = ok &&
           (l->tn ? map16(&maps.a[i], q.dtype, l->a, M, K, l->a_pitch, kBlockK)
                  : map16(&maps.a[i], q.dtype, l->a, K, M, l->a_pitch, d.a_rows)) &&
           map16(&maps.b[i], q.dtype, l->b, N, K, N, kBlockK);
    }
    void* out = kGate ? q.h : l->out;
    if (out)
      ok = ok && map16(&maps.o0[i], q.dtype, out, N, M, N, kSlab);
    else
      maps.o0[i] = maps.a[0];
  }
  if (n == 1) maps.a[1] = maps.b[1] = maps.o0[1] = maps.a[0];  // those that are not used
  maps.o1 = maps.o2 = maps.in = maps.parts = maps.a[0];
  if constexpr (kEpi == kGradient) {
    const int64_t N = q.N;
    ok = ok && map16(&maps.o1, q.dtype, q.d_pre, N, q.M, 2 * N, kSlab) &&
         map16(&maps.o2, q.dtype, static_cast<T*>(q.d_pre) + N, N, q.M, 2 * N, kSlab) &&
         map16(&maps.in, q.dtype, q.in, N, q.M, N, kSlab);
  } else if constexpr (kEpi == kGatedSave) {
    const uint64_t width = (uint64_t)ckpt_width(q.N);
    ok = ok &&
         rows_map(&maps.o1, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.gate.codes, width, (uint64_t)q.M,
                  width, kSlab) &&
         rows_map(&maps.o2, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.up.codes, width, (uint64_t)q.M,
                  width, kSlab);
  }
  if (part_rows > 0)
    ok = ok && rows_map(&maps.parts, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, q.parts, kTile,
                        (uint64_t)part_rows, kTile * 4, kSlab);
  if (!ok) return cudaErrorInvalidValue;
  const int pairs = max_pairs<kern>(P::kSmem);
  if (pairs <= 0) return cudaErrorInvalidConfiguration;
  const int64_t units = p.units[0] + p.units[1];
  const int64_t grid = units < pairs ? units : pairs;
  p.own = p.units[0] / grid;
  p.more = p.units[0] % grid;
  if (n == 2)
    busiest({p.units[0], p.units[1]},
            {unit_cost(ceil_div(p.q[0].num_kb, p.q[0].split), kBN),
             unit_cost(ceil_div(p.q[1].num_kb, p.q[1].split), kBN)},
            grid, &p.rounds);
  p.want_out = q.h != nullptr;
  p.drain = kLong ? kChainBlocks : drain_blocks(q.K);
  p.gate = q.gate;
  p.up = q.up;
  p.status = q.status;
  p.limit_ns = wait_limit_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * grid));
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, maps, p);
  for (int i = 0; i < n && e == cudaSuccess; ++i) {
    const Prod& d = p.q[i];
    if (d.rest == 0) continue;
    JoinArgs j = {};
    j.M = d.M;
    j.N = d.N;
    j.mt = d.mt;
    j.nt = d.nt;
    j.rows = d.M < kTile ? d.M : kTile;
    j.whole = d.whole;
    j.rest = d.rest;
    j.split = d.split;
    j.want_out = p.want_out;
    j.sums = q.parts + (int64_t)d.part_row * kTile;
    j.o0 = kGate ? q.h : q.list[i == 0 ? ch.first : 1 - ch.first]->out;
    j.o1 = q.d_pre;
    j.in = q.in;
    j.gate = q.gate;
    j.up = q.up;
    const int64_t warps = (int64_t)d.rest * j.rows * (kGate ? 1 : 2);
    e = launch_k(join_kernel<T, kEpi, kAct>, dim3((unsigned)ceil_div(warps, 8)), dim3(256), 0, s,
                 true, j);
  }
  return e;
}

// Whether a unit has more blocks than an accumulator may take.
bool long_units(int64_t K, const Split& sp) {
  const int64_t blocks = ceil_div(K, kBlockK);
  return (sp.whole > 0 ? blocks : ceil_div(blocks, sp.split)) > kChainBlocks;
}

template <typename T, int kEpi, int kAct>
cudaError_t run(const Problem& q, cudaStream_t s) {
  Choice ch = {};
  const int64_t mt = ceil_div(q.M, kTile);
  if constexpr (kEpi != kGatedSave) {  // whose checkpoints have 128 channels to a scale
    if (narrow(q.M, q.N, q.K, true)) {
      ch.sp[0] = Split{mt * tiles_n(q.N, true, 128), 0, 1};
      return run_tiles<T, kEpi, kAct, 128, false>(q, ch, s);
    }
  }
  ch.sp[0] = split_of(mt * tiles_n(q.N, true, kTile), q.K);
  if constexpr (kEpi != kGatedSave) {
    if (long_units(q.K, ch.sp[0])) return run_tiles<T, kEpi, kAct, kTile, true>(q, ch, s);
  }
  return run_tiles<T, kEpi, kAct, kTile, false>(q, ch, s);
}

template <typename T>
cudaError_t run_products(const Problem& q, const Choice& ch, cudaStream_t s) {
  bool any = false;
  for (int i = 0; i < q.n; ++i) any = any || long_units(q.list[i]->K, ch.sp[i]);
  if (any) return run_tiles<T, kPlain, 0, kTile, true>(q, ch, s);
  return ch.bn == kTile ? run_tiles<T, kPlain, 0, kTile, false>(q, ch, s)
                        : run_tiles<T, kPlain, 0, 128, false>(q, ch, s);
}

template <int kEpi>
cudaError_t run_gated(int act, const Problem& q, cudaStream_t s) {
  if (q.dtype == MOE_BF16)
    return act == MOE_ACT_SILU
               ? run<__nv_bfloat16, kEpi, MOE_ACT_SILU>(q, s)
               : run<__nv_bfloat16, kEpi, MOE_ACT_GELU_TANH>(q, s);
  return act == MOE_ACT_SILU ? run<__half, kEpi, MOE_ACT_SILU>(q, s)
                             : run<__half, kEpi, MOE_ACT_GELU_TANH>(q, s);
}

}  // namespace

size_t gated_split_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const Split sp = split_of(ceil_div(M, kTile) * tiles_n(N, true, kTile), K);
  return (size_t)sp.rest * sp.split * kTile * kTile * sizeof(float);
}

size_t products_split_bytes(const Product* list, int n) {
  for (int i = 0; i < n; ++i)
    if (list[i].M <= 0 || list[i].N <= 0 || list[i].K <= 0) return 0;
  const Choice ch = choose(list, n);
  if (ch.apart) {
    const size_t a = products_split_bytes(list, 1), b = products_split_bytes(list + 1, 1);
    return a > b ? a : b;
  }
  size_t tiles = 0;
  for (int i = 0; i < n; ++i) tiles += (size_t)ch.sp[i].rest * ch.sp[i].split;
  return tiles * kTile * kTile * sizeof(float);
}

cudaError_t launch_products(int dtype, const Product* list, int n, float* parts, int* status,
                            cudaStream_t s) {
  Problem q = {};
  q.dtype = dtype, q.parts = parts, q.status = status, q.n = n;
  const Choice ch = choose(list, n);
  if (ch.apart) {
    const cudaError_t e = launch_products(dtype, list, 1, parts, status, s);
    return e == cudaSuccess ? launch_products(dtype, list + 1, 1, parts, status, s) : e;
  }
  for (int i = 0; i < n; ++i) q.list[i] = list + i;
  return dtype == MOE_BF16 ? run_products<__nv_bfloat16>(q, ch, s)
                           : run_products<__half>(q, ch, s);
}

cudaError_t launch_gated(int dtype, int act, int T, int F, int H, const void* x, const void* w,
                         void* out, Ckpt gate, Ckpt up, float* parts, int* status,
                         cudaStream_t s) {
  Problem q = {};
  q.dtype = dtype, q.M = T, q.N = F, q.K = H, q.x = x, q.w = w, q.h = out;
  q.gate = gate, q.up = up, q.parts = parts, q.status = status;
  return gate.codes ? run_gated<kGatedSave>(act, q, s) : run_gated<kGated>(act, q, s);
}

cudaError_t launch_gated_grad(int dtype, int act, int T, int F, int H, const void* x, const void* w,
                              const void* d_out, void* d_pre, void* out, float* parts, int* status,
                              cudaStream_t s) {
  Problem q = {};
  q.dtype = dtype, q.M = T, q.N = F, q.K = H, q.x = x, q.w = w, q.h = out, q.d_pre = d_pre;
  q.in = d_out, q.parts = parts, q.status = status;
  return run_gated<kGradient>(act, q, s);
}

}  // namespace gb300moe
