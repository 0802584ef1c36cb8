// dense_rows.cu -- few rows of x against many weight rows, which are streamed once: 4-bit weights
// (include/moe.h: moe_linear_w4a16, moe_gated_linear_w4a16) and the 16-bit gated product of a few
// tokens (moe_gated_linear).
//
// What bounds it is the weights' bytes, so weights go from memory to registers, straight into the
// operand layout of mma.sync m16n8k16: 16 weight rows are its M side, eight rows of x its N side.  (One row of x leaves seven of eight columns
// empty; on the CUDA cores every weight would cost an f32 multiply-add per row of x beside its
// decoding.)  A lane's 16 bytes of a row are consecutive k, and the k of an MMA are assigned to
// lanes as they lie there: the order of k within a sum is free as long as x follows it.
//   16 bits: 8 k of 16 bytes, two MMAs; four lanes 64 bytes of a row
//   4 bits: 32 k of 16 bytes, eight MMAs; E2M1 codes times their E4M3 scale are exact f16, so x is
//     taken in f16 (bf16 x is exact there between 2^-14 and 65504; larger values are reported)
// The CTA's eight warps split K; their sums are added in the order of the warps.
// Gated: an MMA's rows 0-7 are gate rows and 8-15 the up rows that go with them.
#include "activation.cuh"
#include "dense_ops.cuh"
#include "nvfp4.cuh"
#include "vec16.cuh"

#include <type_traits>

namespace gb300moe {

namespace {

constexpr int kWarps = 8;

template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT<T>::kIsBF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// A lane's weights of one block of K: kVec vectors of two rows, and for 4 bits their scales.
template <bool kW4, int kMT>
struct Block {
  static constexpr int kVecs = kW4 ? 1 : 2;
  static constexpr int kLaneK = kW4 ? 32 : 8;       // k of a vector
  static constexpr int kK = 4 * kLaneK * kVecs;     // k of a block
  uint4 a[kMT][2][kVecs];
  uint32_t sc[kMT][2];
};

template <typename T, bool kW4, int kMT, int kNT, bool kGated>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const RowsCall p) {
  using B = Block<kW4, kMT>;
  using X = typename std::conditional<kW4, __half, T>::type;  // what the MMAs take
  constexpr int kRows = 16 * kMT, kCols = 8 * kNT;
  constexpr int kXVecs = B::kVecs * B::kLaneK / 8;  // 16-byte vectors of a lane's x
  __shared__ float part[kWarps][kRows][kCols + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int64_t out0 = (int64_t)blockIdx.x * (kGated ? kRows / 2 : kRows);
  const int t0 = blockIdx.y * kCols;
  const int blocks = (p.K - 1) / B::kK + 1;
  const int b0 = (int)((int64_t)blocks * warp / kWarps);
  const int b1 = (int)((int64_t)blocks * (warp + 1) / kWarps);

  // This lane's two weight rows of each 16: rows past the end stand for the last one.
  const uint8_t* rows[kMT][2];
  const uint8_t* scales[kMT][2];
  const int64_t pitch = kW4 ? p.K / 2 : (int64_t)p.K * 2;
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int64_t n = out0 + (kGated ? i * 8 + g : i * 16 + h * 8 + g);
      n = n < p.N ? n : p.N - 1;
      if (kGated && h == 1) n += p.N;
      rows[i][h] = (kW4 ? p.codes : static_cast<const uint8_t*>(p.w)) + n * pitch;
      scales[i][h] = kW4 ? p.scales + n * (p.K / 16) : nullptr;
    }
  const T* x[kNT];
  bool live[kNT];
#pragma unroll
  for (int j = 0; j < kNT; ++j) {
    const int64_t row = (int64_t)t0 + j * 8 + g;
    live[j] = row < p.T;
    x[j] = static_cast<const T*>(p.x) + (live[j] ? row : 0) * p.K;
  }

  auto lane_k = [&](int b, int v) { return (int64_t)b * B::kK + (v * 4 + t) * B::kLaneK; };
  auto load = [&](int b, B& w) {
#pragma unroll
    for (int v = 0; v < B::kVecs; ++v) {
      const int64_t k = lane_k(b, v);
      const bool in = k < p.K;  // K is a multiple of the lane's
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w.a[i][h][v] =
              in ? __ldcs(reinterpret_cast<const uint4*>(rows[i][h] + (kW4 ? k / 2 : k * 2)))
                 : zero4();
          if (kW4)
            w.sc[i][h] =
                in ? __ldg(reinterpret_cast<const unsigned short*>(scales[i][h] + k / 16)) : 0u;
        }
    }
  };
  bool over = false;
  auto load_x = [&](int b, int j, uint4 (&xv)[kXVecs]) {
#pragma unroll
    for (int v = 0; v < B::kVecs; ++v) {
      const int64_t k = lane_k(b, v);
      const bool in = live[j] && k < p.K;
#pragma unroll
      for (int c = 0; c < B::kLaneK / 8; ++c)
        xv[v * (B::kLaneK / 8) + c] =
            in ? __ldg(reinterpret_cast<const uint4*>(x[j] + k + c * 8)) : zero4();
    }
  };

  float acc[kMT][kNT][4] = {};
  auto multiply = [&](int b, const B& w, const uint4 (&x0)[kXVecs]) {
    uint4 xv[kNT][kXVecs];
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
      if (j == 0) {
#pragma unroll
        for (int c = 0; c < kXVecs; ++c) xv[0][c] = x0[c];
      } else {
        load_x(b, j, xv[j]);
      }
      if constexpr (kW4 && DT<T>::kIsBF16) {
#pragma unroll
        for (int c = 0; c < kXVecs; ++c) xv[j][c] = bf16x8_to_f16x8(xv[j][c], over);
      }
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
      if constexpr (kW4) {
        uint32_t s[2][2];  // scale of the lane's first and second 16 k, in both halves
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s4[4];
          nvfp4_scales(w.sc[i][h], s4);
          s[h][0] = s4[0];
          s[h][1] = s4[1];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t w0 = c == 0 ? w.a[i][0][0].x : c == 1 ? w.a[i][0][0].y
                              : c == 2 ? w.a[i][0][0].z : w.a[i][0][0].w;
          const uint32_t w1 = c == 0 ? w.a[i][1][0].x : c == 1 ? w.a[i][1][0].y
                              : c == 2 ? w.a[i][1][0].z : w.a[i][1][0].w;
          uint32_t q0[4], q1[4];
          nvfp4_decode8(w0, s[0][c >> 1], q0);
          nvfp4_decode8(w1, s[1][c >> 1], q1);
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            mma_16816<X>(acc[i][j], q0[0], q1[0], q0[1], q1[1], xv[j][c].x, xv[j][c].y);
            mma_16816<X>(acc[i][j], q0[2], q1[2], q0[3], q1[3], xv[j][c].z, xv[j][c].w);
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < B::kVecs; ++v) {
          const uint4 &w0 = w.a[i][0][v], &w1 = w.a[i][1][v];
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            mma_16816<X>(acc[i][j], w0.x, w1.x, w0.y, w1.y, xv[j][v].x, xv[j][v].y);
            mma_16816<X>(acc[i][j], w0.z, w1.z, w0.w, w1.w, xv[j][v].z, xv[j][v].w);
          }
        }
      }
    }
  };

  // The next block's weights, and x of the first eight rows, are on their way during this one's MMAs.
  B cur, next;
  uint4 xc[kXVecs], xn[kXVecs];
  if (b0 < b1) {
    load(b0, cur);
    load_x(b0, 0, xc);
  }
#pragma unroll 2
  for (int b = b0; b < b1; ++b) {
    if (b + 1 < b1) {
      load(b + 1, next);
      load_x(b + 1, 0, xn);
    }
    multiply(b, cur, xc);
    cur = next;
#pragma unroll
    for (int c = 0; c < kXVecs; ++c) xc[c] = xn[c];
  }
  if (kW4 && over) set_status(p.status, MOE_ERR_F16_RANGE);

#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        part[warp][i * 16 + (c >> 1) * 8 + g][j * 8 + 2 * t + (c & 1)] = acc[i][j][c];
  __syncthreads();

  const float alpha = kW4 ? __ldg(p.alpha) : 1.0f;
  auto total = [&](int row, int col) {
    float s = part[0][row][col];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += part[w][row][col];
    return s * alpha;
  };
  constexpr int kOuts = kGated ? kRows / 2 : kRows;
  for (int i = threadIdx.x; i < kOuts * kCols; i += kWarps * 32) {
    const int r = i % kOuts, c = i / kOuts;
    const int64_t n = out0 + r, row = (int64_t)t0 + c;
    if (n >= p.N || row >= p.T) continue;
    const int64_t o = row * p.N + n;
    float z;
    if constexpr (kGated) {
      const int at = r / 8 * 16 + r % 8;
      const float gate = total(at, c), up = total(at + 8, c);
      z = (p.act == MOE_ACT_SILU ? gate_value<MOE_ACT_SILU>(gate)
                                 : gate_value<MOE_ACT_GELU_TANH>(gate)) * up;
    } else {
      z = total(r, c);
      if (p.bias) z += DT<T>::to_f(static_cast<const T*>(p.bias)[n]);
      z = activate(z, p.act);
      if (p.res) z += DT<T>::to_f(static_cast<const T*>(p.res)[o]);
    }
    static_cast<T*>(p.out)[o] = DT<T>::from_f(z);
  }
}

template <typename T, bool kW4, bool kGated, int kMT, int kNT>
cudaError_t go(const RowsCall& c, cudaStream_t s) {
  const int64_t outs = kGated ? 8 * kMT : 16 * kMT;
  const dim3 grid((unsigned)((c.N + outs - 1) / outs), (unsigned)((c.T - 1) / (8 * kNT) + 1));
  return launch_k(rows_kernel<T, kW4, kMT, kNT, kGated>, grid, dim3(kWarps * 32), 0, s, false, c);
}

template <typename T, bool kW4, bool kGated>
cudaError_t pick(const RowsCall& c, cudaStream_t s) {
  if (c.T <= 8) return go<T, kW4, kGated, 1, 1>(c, s);
  if (c.T <= 16) return go<T, kW4, kGated, 1, 2>(c, s);
  return go<T, kW4, kGated, 2, 4>(c, s);
}

template <typename T>
cudaError_t typed(const RowsCall& c, cudaStream_t s) {
  if (!c.codes) return pick<T, false, true>(c, s);
  return c.gated ? pick<T, true, true>(c, s) : pick<T, true, false>(c, s);
}

}  // namespace

cudaError_t launch_rows(const RowsCall& c, cudaStream_t s) {
  return c.dtype == MOE_BF16 ? typed<__nv_bfloat16>(c, s) : typed<__half>(c, s);
}

}  // namespace gb300moe
