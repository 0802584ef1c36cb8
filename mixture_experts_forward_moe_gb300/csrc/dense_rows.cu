// dense_rows.cu -- up to sixteen rows of x against 4-bit weights, which are streamed once
// (include/moe.h: moe_linear_w4a16, moe_gated_linear_w4a16), and the 16-bit gated product of one row
// (moe_gated_linear).  4 bits, 7168 x 7168 at 1, 4, 8 and 16 rows of bf16 x: 12, 11, 12 and 16 us;
// 16 bits, 4096 weight rows of 7168: 11.5 us.
//
// What bounds it is the weights' bytes, and for 4 bits as much the instructions that decode them.
// They go into the operand layout of mma.sync m16n8k16 as they lie: 16 weight rows are its M side,
// eight rows of x its N side.  (One row of x leaves seven of eight columns empty; on the CUDA cores
// every weight would cost an f32 multiply-add per row of x beside its decoding.)  A lane's 16 bytes of
// a row are 32 consecutive k, eight MMAs, whose k are assigned to lanes as they lie there: the order
// of k within a sum is free as long as x follows it.  E2M1 codes times their E4M3 scale are exact f16,
// so x is taken in f16, bf16 x times a power of two per row and chunk of K where it needs one (rows.cuh).
// A CTA of four warps has 64 or 128 weight rows, a warp 16 or 32, and a part of K: its x is staged once
// and read by all warps.  A cluster is the parts of the same rows, whose sums meet in shared memory
// and are added in the order of the parts.
// A lane copies the bytes that it will use itself (cp.async) into a ring of stages, several blocks
// ahead and without any barrier.
// Gated: an MMA's rows 0-7 are gate rows and 8-15 the up rows that go with them.
#include "rows.cuh"

namespace gb300moe {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kLaneK = 32;           // k of 16 bytes
constexpr int kBlock = 8 * kLaneK;   // k of a block: two vectors of four lanes, 128 bytes of a row
constexpr int kUnits = kLaneK / 8;   // 16-byte units of x that go with a vector
// How scales lie: a block's 16 of a row on 16 bytes (K a multiple of 256), or from any even byte.
enum Kind { kBits4, kBits4Any };
// Bytes of a row that hold a block's scales, and a warp's stage: two vectors of 16 rows per lane, and
// the scales.
template <Kind kKind>
constexpr int scale_bytes() {
  return kKind == kBits4 ? 16 : 32;
}
template <Kind kKind, int kMT>
constexpr int stage_bytes() {
  return kMT * (2 * 2 * 32 * 16 + 16 * scale_bytes<kKind>());
}

// The grid: groups of weight rows, each `parts` CTAs side by side (the cluster).
// chunk: blocks of K whose x is staged at a time.  Shared memory: x, rows of chunk * kK values and 64
// bytes more (two rows' reads then touch every bank once), then the rings.
template <typename T, Kind kKind, int kMT, int kNT, bool kGated, int kStages>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const RowsCall p, int parts, int chunk) {
  constexpr int kScaleBytes = scale_bytes<kKind>();
  constexpr int kCols = 8 * kNT;
  constexpr int kStageBytes = stage_bytes<kKind, kMT>();
  constexpr int kScaleAt = kMT * 4 * 512;           // in a stage
  constexpr int kOuts = kGated ? 8 * kMT : 16 * kMT;  // outputs of a warp
  constexpr bool kBf16 = DT<T>::kIsBF16;
  extern __shared__ __align__(16) uint8_t smem[];
  // bf16 x: the largest of each row, of up to four warps that staged it
  __shared__ uint32_t s_top[kWarps][kBf16 ? 16 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int part = blockIdx.x % (unsigned)parts;
  const int64_t group = blockIdx.x / (unsigned)parts;
  const int64_t out0 = (group * kWarps + warp) * kOuts;
  const int cols = p.T;  // at most kCols
  const int all = (p.K - 1) / kBlock + 1;
  const int first = (int)((int64_t)all * part / parts);
  const int last = (int)((int64_t)all * (part + 1) / parts);
  const int x_pitch = chunk * kBlock * 2 + 64;
  const uint32_t xs = smem_u32(smem);
  const uint32_t ring = xs + (uint32_t)(cols * x_pitch) + (uint32_t)(warp * kStages * kStageBytes);

  // A weight row of a 16 (0-7 and 8-15): rows past the end stand for the last one.
  auto row_of = [&](int i, int r) -> int64_t {
    int64_t n = out0 + (kGated ? i * 8 + (r & 7) : i * 16 + r);
    n = n < p.N ? n : p.N - 1;
    return kGated && r >= 8 ? n + p.N : n;
  };
  // This lane's place in its two rows, of the block that is loaded next.
  const uint8_t* from[kMT][2];
  const int64_t pitch = p.K / 2;
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      from[i][h] = p.codes + row_of(i, h * 8 + g) * pitch +
                   (int64_t)first * 128 + t * 16;
  // 4 bits: lanes 0-15 copy a row's 16 bytes each, or the first half of its 32 and lanes 16-31 the
  // other; `scale_in` is where this lane's first scale lies in them, which is the same in every
  // block.  (Rows 4-7 and 12-15 have their halves swapped: eight rows' reads touch different banks.)
  const uint8_t* scale_from[kMT];
  int scale_in[kMT][2];
  const uint8_t* const scale_end = p.scales + (kGated ? 2 * (int64_t)p.N : p.N) * (p.K / 16);
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const int64_t at = row_of(i, lane & 15) * (p.K / 16) + (int64_t)first * 16;
    scale_from[i] = p.scales + (at & ~int64_t(15)) + (lane >> 4) * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      scale_in[i][h] =
          (kKind == kBits4 ? 0 : (int)(row_of(i, h * 8 + g) * (p.K / 16) & 15)) + t * 2;
  }

  // Vector (i, h, v) of a lane at ((i * 2 + h) * 2 + v) * 512 of its stage, 16 bytes a lane.
  auto load = [&](int b, int stage) {
    if (b < last) {
      const uint32_t to = ring + (uint32_t)(stage * kStageBytes) + (uint32_t)lane * 16u;
      const int64_t left = p.K - (int64_t)b * kBlock;  // K is a multiple of a lane's
      if (kKind == kBits4 || left >= kBlock) {
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int v = 0; v < 2; ++v)
              copy16(to + (uint32_t)(((i * 2 + h) * 2 + v) * 512), from[i][h] + v * 64);
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const bool in = (v * 4 + t) * kLaneK < left;
#pragma unroll
          for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              copy16_part(to + (uint32_t)(((i * 2 + h) * 2 + v) * 512),
                          in ? from[i][h] + v * 64 : from[i][h] - t * 16, in ? 16 : 0);
        }
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) from[i][h] += 128;
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        const uint32_t dst = ring + (uint32_t)(stage * kStageBytes + kScaleAt +
                                               (i * 16 + (lane & 15)) * kScaleBytes);
        if constexpr (kKind == kBits4) {
          if (lane < 16) copy16(dst, scale_from[i]);
        } else {
          // the tensor may end inside the vector, or before it
          const int64_t rest = scale_end - scale_from[i];
          const int bytes = rest >= 16 ? 16 : rest > 0 ? (int)rest : 0;
          copy16_part(dst + (uint32_t)(((lane >> 4) ^ ((lane >> 2) & 1)) * 16),
                      bytes > 0 ? scale_from[i] : p.scales, bytes);
        }
        scale_from[i] += 16;
      }
    }
    copy_commit();
  };

  // x of one chunk: unit u of a block's vector (8 k) of lane t lies at u * 4 + t.  Eight threads or more
  // have a row, x_per of them, so that its largest value stays in registers until they meet.  bf16 x is
  // staged as it is first, and `again` times a power of two where a row needs one.
  const int x_per = kWarps * 32 / (cols <= 1 ? 1 : cols <= 2 ? 2 : cols <= 4 ? 4 : cols <= 8 ? 8 : 16);
  const int x_row = threadIdx.x / (unsigned)x_per, x_first = threadIdx.x % (unsigned)x_per;
  auto stage_x = [&](int b0, bool again, float scale) {
    const uint4* const from = static_cast<const uint4*>(p.x) + ((int64_t)x_row * p.K + (int64_t)b0 * kBlock) / 8;
    const int64_t left = (p.K - (int64_t)b0 * kBlock) / 8;
    const int units = x_row < cols ? chunk * kBlock / 8 : 0;
    const uint32_t to = xs + (uint32_t)(x_row * x_pitch);
    uint32_t top = 0u;
    constexpr int kAhead = 4;  // loads that a thread has on their way
    for (int u0 = x_first; u0 < units; u0 += kAhead * x_per) {
      uint4 v[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int u = u0 + a * x_per;
        v[a] = u < units && u < left ? from[u] : zero4();
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int u = u0 + a * x_per;
        if (u >= units) break;
        if constexpr (kBf16) {
          top = max(top, top_bits(v[a]));
          v[a] = bf16x8_times(v[a], scale);
        }
        sts16(to + (uint32_t)((u & ~15) | ((u & 3) << 2) | ((u >> 2) & 3)) * 16u, v[a]);
      }
    }
    if (kBf16 && !again) {
      if (x_per >= 32) {
        top = __reduce_max_sync(0xffffffffu, top);
      } else {
        for (int o = x_per / 2; o > 0; o >>= 1)
          top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      if (x_first % 32 == 0) s_top[x_first / 32][x_row] = top;
    }
  };

  // Consecutive MMAs of one accumulator wait for one another: a single tile has two.
  constexpr int kAccs = kMT * kNT == 1 ? 2 : 1;
  float acc[kAccs][kMT][kNT][4];
  // Times alpha, of the chunks before this one: an accumulator takes no more than a chunk (kChainK at
  // most), which has its own scales of x.
  float total[kMT][kNT][4] = {};
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) f(i, j, c);
  };
  // `xb`: this lane's first unit of the block's x, for row g
  auto multiply = [&](int stage, uint32_t xb, int left) {
    const uint32_t at = ring + (uint32_t)(stage * kStageBytes) + (uint32_t)lane * 16u;
    const uint32_t at_s = ring + (uint32_t)(stage * kStageBytes + kScaleAt);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint4 xv[kNT][kUnits];
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int c = 0; c < kUnits; ++c)
          xv[j][c] = j * 8 + g < cols
                         ? lds16(xb + (uint32_t)(j * 8 * x_pitch + (v * kUnits + c) * 64))
                         : zero4();
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        uint4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) w[h] = lds16(at + (uint32_t)(((i * 2 + h) * 2 + v) * 512));
        uint32_t s[2][2];  // scales of the lane's first and second 16 k, in both halves
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t row = at_s + (uint32_t)((i * 16 + h * 8 + g) * kScaleBytes);
          uint32_t two;
          if constexpr (kKind == kBits4)
            two = lds2(row + (uint32_t)(t * 2 + v * 8));
          else  // behind K lie the next row's, which could be NaN
            two = (v * 4 + t) * kLaneK < left
                      ? lds2(row + (uint32_t)((scale_in[i][h] + v * 8) ^ ((g & 4) << 2)))
                      : 0u;
          two_scales(two, s[h]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t q0[4], q1[4];
          nvfp4_decode8(word_of(w[0], c), s[0][c >> 1], q0);
          nvfp4_decode8(word_of(w[1], c), s[1][c >> 1], q1);
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            mma_16816(acc[0][i][j], q0[0], q1[0], q0[1], q1[1], xv[j][c].x, xv[j][c].y);
            mma_16816(acc[kAccs - 1][i][j], q0[2], q1[2], q0[3], q1[3], xv[j][c].z, xv[j][c].w);
          }
        }
      }
    }
  };

  // The first blocks come into L2 while the kernel before this one ends.
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
    if (t == 0 && first + s < last)
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) prefetch_l2(from[i][h] + s * 128);
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(first + s, s);
  const float alpha = *p.alpha;
  int stage = 0;
  for (int b0 = first; b0 < last; b0 += chunk) {
    if (b0 > first) __syncthreads();  // the last chunk's x has been read
    each([&](int i, int j, int c) { acc[0][i][j][c] = acc[kAccs - 1][i][j][c] = 0.0f; });
    RowScale scale = {1.0f, 1.0f};  // lane c's: of row c
    bool scaled = false;            // the same in all warps
    for (;;) {
      stage_x(b0, scaled, kBf16 ? __shfl_sync(0xffffffffu, scale.down, x_row) : 1.0f);
      __syncthreads();
      if (!kBf16 || scaled) break;
      uint32_t top = 0u;
      if (lane < cols)
        for (int q = 0; q < x_per; q += 32) top = max(top, s_top[q / 32][lane]);
      scaled = __any_sync(0xffffffffu, needs_scale(top));
      if (!scaled) break;
      scale = row_scale(top);
      if (past_f16(top)) set_status(p.status, MOE_ERR_F16_RANGE);
    }
    const int end = last - b0 < chunk ? last - b0 : chunk;
    for (int b = 0; b < end; ++b) {
      copy_wait<kStages - 2>();
      __syncwarp();  // the scales are other lanes' copies
      // into the stage that the block before this one has left
      load(b0 + b + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      multiply(stage, xs + (uint32_t)(g * x_pitch + b * kBlock * 2 + t * 16),
               b0 + b + 1 < all ? kBlock : p.K - (all - 1) * kBlock);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    each([&](int i, int j, int c) {
      float z = kAccs == 1 ? acc[0][i][j][c] : acc[0][i][j][c] + acc[kAccs - 1][i][j][c];
      z *= alpha;
      if (kBf16 && scaled) z *= __shfl_sync(0xffffffffu, scale.up, j * 8 + 2 * t + (c & 1));
      total[i][j][c] += z;
    });
  }
  copy_wait<0>();

  // Sums [cols][kAll]: the weight rows of the CTA, a gated product's gate rows before its up rows.
  constexpr int kAll = kWarps * 16 * kMT, kUp = kWarps * kOuts;
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
  each([&](int i, int j, int c) {
    const int w = warp * kOuts;
    const int r = kGated ? (c >> 1) * kUp + w + i * 8 + g : w + i * 16 + (c >> 1) * 8 + g;
    sums[(j * 8 + 2 * t + (c & 1)) * kAll + r] = total[i][j][c];
  });
  if (parts > 1)
    cluster_sync();
  else
    __syncthreads();
  finish_tile<T, kGated, kUp, kWarps * 32>(p, xs, sums, kAll, group, part, parts, 0, cols, 1.0f, nullptr);
  if (parts > 1) cluster_leave();  // a peer may still read this CTA's sums
}

// ---- 16-bit weights, one row of x: on the CUDA cores --------------------------------------------
// A gate row and its up row by `wpr` warps (a power of two) of the CTA's.  2 x 2048 rows of 7168 with 128
// bytes of a lane on their way: 11.5 us in CTAs of four warps or eight, 11.9 of two; 64 bytes 13.2.
constexpr int kGemvWarps = 4;
template <typename T>
__global__ void __launch_bounds__(kGemvWarps * 32) gated_gemv_kernel(const RowsCall p, int wpr) {
  __shared__ float s_part[kGemvWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int outs = kGemvWarps / wpr;
  const int64_t n = (int64_t)blockIdx.x * outs + warp / wpr;
  const int kv = p.K / 8;
  F2 gate = f2(0.0f), up = f2(0.0f);
  if (n < p.N) {
    const uint4* wg = static_cast<const uint4*>(p.w) + n * kv;
    const uint4* wu = wg + (int64_t)p.N * kv;
    const uint4* x = static_cast<const uint4*>(p.x);
    constexpr int kAhead = 4;
    const int i1 = warp % wpr * 32 + lane;
    for (int a = 0; a < kAhead; ++a)
      if (lane % 8 == 0 && i1 + a * wpr * 32 < kv) {
        prefetch_l2(wg + i1 + a * wpr * 32);
        prefetch_l2(wu + i1 + a * wpr * 32);
      }
    pdl_wait();
    pdl_trigger();
    for (int i0 = i1; i0 < kv; i0 += kAhead * wpr * 32) {
      uint4 g[kAhead], u[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int i = i0 + a * wpr * 32;
        g[a] = i < kv ? __ldcs(wg + i) : zero4();
        u[a] = i < kv ? __ldcs(wu + i) : zero4();
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int i = i0 + a * wpr * 32;
        if (i >= kv) break;
        F2 fg[4], fu[4], fx[4];
        unpack<T>(g[a], fg);
        unpack<T>(u[a], fu);
        unpack<T>(x[i], fx);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          gate = f2_fma(fg[j], fx[j], gate);
          up = f2_fma(fu[j], fx[j], up);
        }
      }
    }
  }
  float z[2] = {f2_sum(gate), f2_sum(up)};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z[h] += __shfl_xor_sync(0xffffffffu, z[h], o);
    if (lane == 0) s_part[warp][h] = z[h];
  }
  __syncthreads();
  const int r = threadIdx.x;
  const int64_t no = (int64_t)blockIdx.x * outs + r;
  if (r < outs && no < p.N) {
    float a = 0.0f, b = 0.0f;
    for (int q = 0; q < wpr; ++q) {
      a += s_part[r * wpr + q][0];
      b += s_part[r * wpr + q][1];
    }
    finish<T, true>(p, 0, no, a, b);
  }
}

// Parts of K: those that leave the busiest SM the least time, in blocks.  A CTA costs about four
// blocks beside its own, and one alone on its SM has too few bytes on their way.
int even_parts(int64_t groups, int blocks) {
  const int64_t sms = num_sms();
  int64_t best = 0;
  int parts = 1;
  for (int q = 1; q <= kMaxParts && q <= blocks; ++q) {
    const int64_t waves = (groups * q + sms - 1) / sms;
    const int64_t busiest = (waves == 1 ? 2 : waves) * ((blocks + q - 1) / q + 4);
    if (q == 1 || busiest < best) best = busiest, parts = q;
  }
  return parts;
}

template <typename T, Kind kKind, bool kGated, int kMT, int kNT>
cudaError_t go(const RowsCall& c, cudaStream_t s) {
  constexpr int kStages = kMT == 1 ? 4 : 3;
  constexpr auto kern = rows_kernel<T, kKind, kMT, kNT, kGated, kStages>;
  constexpr int kRing = kWarps * kStages * stage_bytes<kKind, kMT>();
  static_assert(kRing >= kWarps * 16 * kMT * 8 * kNT * (int)sizeof(float), "the sums");
  const cudaError_t e = set_smem_limit<kern>(kSmemLimit);
  if (e != cudaSuccess) return e;
  const int64_t outs = (kGated ? 8 : 16) * kMT * kWarps;
  const int64_t groups = (c.N + outs - 1) / outs;
  const int all = (c.K - 1) / kBlock + 1;
  const int parts = even_parts(groups, all), cols = c.T;
  // All of a part's x, or as much at a time as leaves room for three CTAs per SM (two).
  int chunk = (all + parts - 1) / parts;
  constexpr int kMost = (kMT * kNT == 1 ? 2 : 1) * kChainK / kBlock;  // two accumulators share a chunk
  if (chunk > kMost) chunk = kMost;
  const int fit = (((kMT == 1 ? 75 : 112) * 1024 - kRing) / cols - 64) / (kBlock * 2);
  if (chunk > fit) chunk = fit > 0 ? fit : 1;
  const int smem = kRing + cols * (chunk * kBlock * 2 + 64);
  if (smem > kSmemLimit) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * parts));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = (size_t)smem;
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
  return cudaLaunchKernelEx(&cfg, kern, c, parts, chunk);
}

template <typename T, Kind kKind, bool kGated>
cudaError_t pick(const RowsCall& c, cudaStream_t s) {
  // Past four rows the reads of x from shared memory cost more than those of the weights, unless a
  // warp has 32 weight rows (eight rows of 7168 x 7168: 15.9 us against 21.6).
  if (c.T <= 4) return go<T, kKind, kGated, 1, 1>(c, s);
  if (c.T <= 8) return go<T, kKind, kGated, 2, 1>(c, s);
  return go<T, kKind, kGated, 2, 2>(c, s);
}

template <typename T>
cudaError_t typed(const RowsCall& c, cudaStream_t s) {
  if (!c.codes) {
    int wpr = 1;  // enough for about sixteen warps per SM
    while (wpr < kGemvWarps && (int64_t)c.N * wpr < (int64_t)num_sms() * 16 && c.K / 8 >= wpr * 2 * 32)
      wpr *= 2;
    return launch_k(gated_gemv_kernel<T>, dim3((unsigned)((c.N - 1) / (kGemvWarps / wpr) + 1)),
                    dim3(kGemvWarps * 32), 0, s, true, c, wpr);
  }
  if (c.T > kFewW4Rows) return cudaErrorInvalidValue;
  if (c.K % 256 == 0)
    return c.gated ? pick<T, kBits4, true>(c, s) : pick<T, kBits4, false>(c, s);
  return c.gated ? pick<T, kBits4Any, true>(c, s) : pick<T, kBits4Any, false>(c, s);
}

}  // namespace

cudaError_t launch_rows(const RowsCall& c, cudaStream_t s) {
  return c.dtype == MOE_BF16 ? typed<__nv_bfloat16>(c, s) : typed<__half>(c, s);
}

}  // namespace gb300moe
