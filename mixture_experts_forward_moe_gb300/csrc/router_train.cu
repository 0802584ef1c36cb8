// router_train.cu -- training of the router (include/moe.h: moe_balance_loss_fwd,
// moe_router_bwd): per-expert counts, the balance loss over ragged sequences, and the gradient of
// the logits from that loss and from the route weights.
//
// One warp per token, its row of logits spread over the lanes, as in the router itself.  A token is
// a chain of a load, an exponential per expert and two to five warp reductions, so the kernels are
// bound by that chain and the warps that hide it before they are by memory.  Measured on a GB300:
// loss of 32768 tokens, 256 experts, 11 sequences 17.6 us (5.1 us at the copy rate),
// of 512 tokens 6.6; gradient of 32768 tokens, 384 experts 25.5 us (0.59 of the copy rate), of 512
// tokens 2.8.
#include <limits.h>
#include <math.h>

#include "block_ops.cuh"
#include "vec16.cuh"
#include "ptx.cuh"

namespace gb300moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
  return v;
}

// A row of E logits (or coefficients) in a warp: lane l holds the VEC consecutive experts from
// (l + 32 i) VEC on, i < N.  VEC is 4 when E is a multiple of 4 (rows are then whole 16-byte
// vectors), else 1.
template <int VEC, int N>
struct Row {
  float v[N][VEC];
  __device__ __forceinline__ void load(const float* row, int E, int lane, float fill) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = (lane + 32 * i) * VEC;
      if constexpr (VEC == 4) {
        float4 x = make_float4(fill, fill, fill, fill);
        if (e < E) x = *reinterpret_cast<const float4*>(row + e);
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
      } else {
        v[i][0] = e < E ? row[e] : fill;
      }
    }
  }
  __device__ __forceinline__ void store(float* row, int E, int lane) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = (lane + 32 * i) * VEC;
      if (e >= E) continue;
      if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(row + e) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
      else
        row[e] = v[i][0];
    }
  }
};
#define EACH(i, j)                  \
  _Pragma("unroll") for (int i = 0; i < N; ++i) _Pragma("unroll") for (int j = 0; j < VEC; ++j)

// e^x and 1/x by the special-function unit alone, tiny results flushed to 0.  The error of e^x
// relative to itself grows with |x|, 2^-24 of it, while e^x (x <= 0 here) falls faster, so a row's
// sum is off by a few 2^-24.
__device__ __forceinline__ float exp_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Sigmoid s and 1 - s, each good relative to itself at either end.
__device__ __forceinline__ void sigmoid2(float x, float& s, float& om) {
  const float t = exp_fast(-fabsf(x));
  const float d = rcp_fast(1.0f + t), td = t * d;
  s = x >= 0.0f ? d : td;
  om = x >= 0.0f ? td : d;
}
// Sums and the gradient over a row, two values per instruction where there are pairs.
template <int VEC, int N>
__device__ __forceinline__ float row_sum(const Row<VEC, N>& x) {
  if constexpr (VEC == 4) {
    F2 s = f2(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i)
      s = s + (f2(x.v[i][0], x.v[i][1]) + f2(x.v[i][2], x.v[i][3]));
    return f2_sum(s);
  } else {
    float s = 0.0f;
    EACH(i, j) s += x.v[i][j];
    return s;
  }
}
template <int VEC, int N>
__device__ __forceinline__ float row_dot(const Row<VEC, N>& x, const Row<VEC, N>& y) {
  if constexpr (VEC == 4) {
    F2 s = f2(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        s = f2_fma(f2(x.v[i][j], x.v[i][j + 1]), f2(y.v[i][j], y.v[i][j + 1]), s);
    return f2_sum(s);
  } else {
    float s = 0.0f;
    EACH(i, j) s = fmaf(x.v[i][j], y.v[i][j], s);
    return s;
  }
}
// v = (v inv (c scale - b) + q) om
template <int VEC, int N>
__device__ __forceinline__ void row_gradient(Row<VEC, N>& v, float inv, const Row<VEC, N>& c,
                                             float scale, float b, const Row<VEC, N>& q,
                                             const Row<VEC, N>& om) {
  if constexpr (VEC == 4) {
    const F2 i2 = f2(inv), s2 = f2(scale), b2 = f2(-b);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const F2 g = f2_fma(f2(v.v[i][j], v.v[i][j + 1]) * i2,
                            f2_fma(f2(c.v[i][j], c.v[i][j + 1]), s2, b2),
                            f2(q.v[i][j], q.v[i][j + 1])) *
                     f2(om.v[i][j], om.v[i][j + 1]);
        const float2 r = f2_get(g);
        v.v[i][j] = r.x;
        v.v[i][j + 1] = r.y;
      }
  } else {
    EACH(i, j) v.v[i][j] =
        fmaf(v.v[i][j] * inv, fmaf(c.v[i][j], scale, -b), q.v[i][j]) * om.v[i][j];
  }
}
// Below this sum of sigmoids every logit is under -57, where sigmoid(x) is e^x to all of f32's
// digits: the row (or selection) is then shifted by its largest logit, as a softmax is, instead
// of underflowing.
constexpr float kTinySum = 1e-25f;

// Scores of a row, proportional to its probabilities: e^(x - max), or sigmoid(x) (shifted as said
// above); `om` is 1 - sigmoid (1 for softmax).  Returns 1 / the row's sum, 0 for a row of -inf
// alone (a sum of NaN stays one).  `shift`, if wanted: the max, or infinity for plain sigmoids.
template <int VEC, int N>
__device__ __forceinline__ float row_scores(Row<VEC, N>& x, Row<VEC, N>& om, int scoring,
                                            float* shift = nullptr) {
  float sum = 0.0f;
  if (scoring == MOE_SIGMOID) {
    Row<VEC, N> s;
    EACH(i, j) sigmoid2(x.v[i][j], s.v[i][j], om.v[i][j]);
    sum = warp_sum(row_sum(s));
    if (!__any_sync(kAll, sum < kTinySum)) {
      x = s;
      if (shift) *shift = INFINITY;
      return __fdividef(1.0f, sum);
    }
  }
  float m = -INFINITY;
  EACH(i, j) m = fmaxf(m, x.v[i][j]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;
  if (shift) *shift = m;
  EACH(i, j) {
    x.v[i][j] = exp_fast(x.v[i][j] - m);
    om.v[i][j] = 1.0f;
  }
  sum = warp_sum(row_sum(x));
  return sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
}

// First sequence s with seq_offsets[s + 1] > t (n_seq when there is none).  Lane l holds
// `mine` = seq_offsets[l + 1] (or INT_MAX past the end), which answers for the first 32.
__device__ __forceinline__ int seq_of(const int32_t* off, int n_seq, int t, int mine) {
  const int first = __popc(__ballot_sync(kAll, mine <= t));
  if (first < 32 || n_seq <= 32) return first < n_seq ? first : n_seq;
  int lo = 32, hi = n_seq;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}
__device__ __forceinline__ int my_offset(const int32_t* off, int n_seq, int lane) {
  return off && lane < n_seq ? off[lane + 1] : INT_MAX;
}
__device__ __forceinline__ int clamp_i(int v, int lo, int hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}

// ---- balance loss, first pass ----------------------------------------------------------------
// CTA c takes the tokens [c*chunk, (c+1)*chunk) and writes one record per sequence that it
// meets: the sums of p, the counts and the live tokens.  Along the tokens each next (chunk,
// sequence) pair has a larger c + s, so record c + s is its own: n_chunks + n_seq records hold
// all pairs, and no float is added in an order that depends on scheduling.
struct Records {
  float* prob;     // [n_rec][E]
  int32_t* count;  // [n_rec][E]
  int32_t* live;   // [n_rec]
};

template <int VEC, int N>
__global__ void __launch_bounds__(kWarps * 32)
    balance_chunk_kernel(int T, int E, int K, int n_seq, int scoring, int chunk,
                         const float* __restrict__ x, const int32_t* __restrict__ ids,
                         const int32_t* __restrict__ off, const Records rec, int* ticket,
                         int* status) {
  extern __shared__ __align__(16) uint8_t dyn[];
  const int pitch = (E + 3) & ~3;
  float* s_prob = reinterpret_cast<float*>(dyn);                   // [kWarps][pitch]
  int* s_count = reinterpret_cast<int*>(s_prob + kWarps * pitch);  // [E]
  __shared__ int s_live;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;  // the second pass' count of its CTAs
  pdl_trigger();  // the second pass waits for this grid before it reads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * chunk;
  const int c1 = T - c0 < chunk ? T : c0 + chunk;
  bool bad = false;
  int t0 = c0;
  for (int s = off ? seq_of(off, n_seq, c0, my_offset(off, n_seq, lane)) : 0;
       s < n_seq && t0 < c1; ++s) {
    if (off) t0 = max(t0, off[s]);
    const int t1 = off ? min(c1, off[s + 1]) : c1;
    if (t1 <= t0) continue;
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = 0;
    if (threadIdx.x == 0) s_live = 0;
    __syncthreads();
    Row<VEC, N> acc = {};
    int live = 0;
    // the next token's row and ids are on their way while this one's are worked on
    Row<VEC, N> next;
    int next_id = -1;
    auto fetch = [&](int t) {
      if (t >= t1) return;
      next.load(x + (size_t)t * E, E, lane, -INFINITY);
      next_id = lane < K ? ids[(size_t)t * K + lane] : -1;
    };
    fetch(t0 + warp);
    for (int t = t0 + warp; t < t1; t += kWarps) {
      Row<VEC, N> v = next, om;
      const int id = next_id;
      fetch(t + kWarps);
      const bool on = id >= 0 && id < E;
      bad |= id < -1 || id >= E;
      if (!__any_sync(kAll, on)) continue;
      ++live;
      if (on) atomicAdd(&s_count[id], 1);
      const float inv = row_scores(v, om, scoring);
      EACH(i, j) acc.v[i][j] = fmaf(v.v[i][j], inv, acc.v[i][j]);
    }
    if (lane == 0 && live) atomicAdd(&s_live, live);
    acc.store(s_prob + warp * pitch, E, lane);
    __syncthreads();
    const size_t r = (size_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) p += s_prob[w * pitch + e];
      rec.prob[r * E + e] = p;
      rec.count[r * E + e] = s_count[e];
    }
    if (threadIdx.x == 0) rec.live[r] = s_live;
    t0 = t1;
    __syncthreads();
  }
  if (bad) set_status(status, MOE_ERR_BAD_EXPERT_ID);
}

// ---- balance loss, second pass ---------------------------------------------------------------
// A unit is 32 experts of a sequence.  A CTA takes `per_cta` units, each by 32 / per_cta warps (a
// power of two; by one warp, in turns, past 32): warp r of R adds the chunks r, r + R, ..., and the
// warps' sums are added in order.  The CTA that finishes last, by `ticket` (0 at the start of the
// launch), adds the CTAs' parts of the loss, again in a fixed order.
constexpr int kFinWarps = 32;

__global__ void __launch_bounds__(kFinWarps * 32)
    balance_final_kernel(int T, int E, int K, int n_seq, int chunk, int per_cta, float coeff,
                         const int32_t* __restrict__ off, const Records rec,
                         float* __restrict__ loss, int32_t* __restrict__ counts,
                         int32_t* __restrict__ live_out, float* __restrict__ prob_sum,
                         float* __restrict__ coef, float* part, int* ticket, int* status) {
  __shared__ float s_p[kFinWarps][32];
  __shared__ int s_c[kFinWarps][32];
  __shared__ int s_seqs[kFinWarps];
  __shared__ float s_loss[kFinWarps];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (E + 31) / 32;
  const int64_t units = (int64_t)n_seq * tiles;
  int rows = 1;
  while (rows * 2 * per_cta <= kFinWarps) rows *= 2;
  const int at_once = kFinWarps / rows;  // units of the CTA at a time
  // The chunks of sequence s are [first, last]; empty when it has no tokens.
  auto range = [&](int s, int& first, int& last) {
    const int a = off ? clamp_i(off[s], 0, T) : 0;
    const int b = off ? clamp_i(off[s + 1], 0, T) : T;
    first = a / chunk;
    last = b > a ? (b - 1) / chunk : first - 1;
  };
  pdl_wait();
  // Sequences with live tokens.
  int seqs = 0;
  for (int s = tid; s < n_seq; s += kFinWarps * 32) {
    int c, last;
    range(s, c, last);
    bool any = false;
    for (; c <= last && !any; ++c) any = rec.live[(size_t)c + s] > 0;
    seqs += any;
    if (off && blockIdx.x == 0 && (off[s] < 0 || off[s + 1] < off[s] || off[s + 1] > T))
      set_status(status, MOE_ERR_INVALID_ARG);
  }
  seqs = __reduce_add_sync(kAll, seqs);
  if (lane == 0) s_seqs[warp] = seqs;
  float loss_part = 0.0f;
  for (int u0 = 0; u0 < per_cta; u0 += at_once) {
    const int k = u0 + warp / rows, row = warp % rows;
    const int64_t unit = (int64_t)blockIdx.x * per_cta + k;
    const bool mine = k < per_cta && unit < units;  // the same for the warp
    const int s = mine ? (int)(unit / tiles) : 0;
    const int tile = mine ? (int)(unit - (int64_t)s * tiles) : 0;
    const int e = tile * 32 + lane;
    float p = 0.0f;
    int cnt = 0, live = 0;
    if (mine) {
      int first, last;
      range(s, first, last);
      if (row == 0)
        for (int c = first + lane; c <= last; c += 32) live += rec.live[(size_t)c + s];
      if (e < E)
#pragma unroll 8
        for (int c = first + row; c <= last; c += rows) {
          const size_t r = ((size_t)c + s) * E + e;
          p += rec.prob[r];
          cnt += rec.count[r];
        }
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = cnt;
    __syncthreads();
    if (mine && row == 0) {
      const int T_all = __reduce_add_sync(kAll, live);
      const int n_all = __reduce_add_sync(kAll, s_seqs[lane]);
      for (int r = 1; r < rows; ++r) {
        p += s_p[warp + r][lane];
        cnt += s_c[warp + r][lane];
      }
      if (e < E) {
        const float T_s = (float)max(T_all, 1);
        const float w =
            (float)cnt * (coeff * (float)E) / ((float)max(n_all, 1) * (float)K) / T_s / T_s;
        const size_t o = (size_t)s * E + e;
        counts[o] = cnt;
        prob_sum[o] = p;
        coef[o] = w;
        loss_part = fmaf(w, p, loss_part);
      }
      if (tile == 0 && lane == 0) live_out[s] = T_all;
    }
    __syncthreads();
  }
  loss_part = warp_sum(loss_part);
  if (lane == 0) s_loss[warp] = loss_part;
  __syncthreads();
  if (warp != 0) return;
  loss_part = warp_sum(s_loss[lane]);
  if (gridDim.x == 1) {
    if (lane == 0) *loss = loss_part;
    return;
  }
  if (lane == 0) {
    part[blockIdx.x] = loss_part;
    __threadfence();
    s_last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
  }
  __syncwarp();
  if (s_last) {
    __threadfence();
    float l = 0.0f;
    for (int i = lane; i < (int)gridDim.x; i += 32) l += __ldcg(part + i);
    l = warp_sum(l);
    if (lane == 0) *loss = l;
  }
}

// ---- balance loss of few tokens in one launch --------------------------------------------------
// One CTA.  First each warp reduces its tokens' rows to the shift and the inverse of their sum,
// and adds their routes to the counts (integers, in global memory); then thread (group, expert)
// takes every groups-th sequence and adds its tokens' probabilities in their order.
constexpr int kSmallTokens = 64, kSmallSeqs = 128, kSmallThreads = 1024;

template <int VEC, int N>
__global__ void __launch_bounds__(kSmallThreads)
    balance_small_kernel(int T, int E, int K, int n_seq, int scoring, float coeff,
                         const float* __restrict__ x, const int32_t* __restrict__ ids,
                         const int32_t* __restrict__ off, float* __restrict__ loss,
                         int32_t* __restrict__ counts, int32_t* __restrict__ live_out,
                         float* __restrict__ prob_sum, float* __restrict__ coef, int* status) {
  __shared__ float s_inv[kSmallTokens], s_max[kSmallTokens];  // s_inv < 0: not live
  __shared__ int s_live[kSmallSeqs];
  __shared__ float s_loss[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < n_seq * E; i += kSmallThreads) __stcg(counts + i, 0);
  for (int i = tid; i < n_seq; i += kSmallThreads) s_live[i] = 0;
  const int mine = my_offset(off, n_seq, lane);
  __threadfence_block();
  __syncthreads();
  bool bad = false;
  for (int t = warp; t < T; t += kSmallThreads / 32) {
    Row<VEC, N> v, om;
    v.load(x + (size_t)t * E, E, lane, -INFINITY);
    const int id = lane < K ? ids[(size_t)t * K + lane] : -1;
    const bool on = id >= 0 && id < E;
    int s = 0;
    bool in = true;
    if (off) {
      s = seq_of(off, n_seq, t, mine);
      in = s < n_seq && off[s] <= t;
    }
    const bool live = __any_sync(kAll, on) && in;
    bad |= in && (id < -1 || id >= E);
    float inv = -1.0f, m = 0.0f;
    if (live) {
      inv = row_scores(v, om, scoring, &m);
      if (on) atomicAdd(counts + s * E + id, 1);
    }
    if (lane == 0) {
      s_inv[t] = inv;
      s_max[t] = m;
      if (live) atomicAdd(&s_live[s], 1);
    }
  }
  if (bad) set_status(status, MOE_ERR_BAD_EXPERT_ID);
  if (off)
    for (int s = tid; s < n_seq; s += kSmallThreads)
      if (off[s] < 0 || off[s + 1] < off[s] || off[s + 1] > T)
        set_status(status, MOE_ERR_INVALID_ARG);
  __threadfence();  // the counts, before other threads read them below
  __syncthreads();
  int n_live = 0;
  for (int s = 0; s < n_seq; ++s) n_live += s_live[s] > 0;
  const int pitch = (E + 31) & ~31;
  const int groups = kSmallThreads / pitch;  // at least one: E <= 1024
  const int group = tid / pitch, e = tid - group * pitch;
  float loss_part = 0.0f;
  if (group < groups && e < E) {
    for (int s = group; s < n_seq; s += groups) {
      const int a = off ? clamp_i(off[s], 0, T) : 0;
      const int b = off ? clamp_i(off[s + 1], 0, T) : T;
      float p = 0.0f;
      // no branch between the rows' loads: they are all on their way together
      if (scoring == MOE_SOFTMAX) {
#pragma unroll 8
        for (int t = a; t < b; ++t) {
          const float q = exp_fast(x[(size_t)t * E + e] - s_max[t]) * s_inv[t];
          p += s_inv[t] < 0.0f ? 0.0f : q;
        }
      } else {
#pragma unroll 8
        for (int t = a; t < b; ++t) {
          const float v = x[(size_t)t * E + e];
          float score, om;
          sigmoid2(v, score, om);
          if (s_max[t] != INFINITY) score = exp_fast(v - s_max[t]);
          p += s_inv[t] < 0.0f ? 0.0f : score * s_inv[t];
        }
      }
      const int cnt = __ldcg(counts + s * E + e);
      const float T_s = (float)max(s_live[s], 1);
      const float w =
          (float)cnt * (coeff * (float)E) / ((float)max(n_live, 1) * (float)K) / T_s / T_s;
      prob_sum[s * E + e] = p;
      coef[s * E + e] = w;
      loss_part = fmaf(w, p, loss_part);
    }
  }
  for (int s = tid; s < n_seq; s += kSmallThreads) live_out[s] = s_live[s];
  loss_part = warp_sum(loss_part);
  if (lane == 0) s_loss[warp] = loss_part;
  __syncthreads();
  if (warp == 0) {
    loss_part = warp_sum(s_loss[lane]);
    if (lane == 0) *loss = loss_part;
  }
}

// ---- gradient of the logits --------------------------------------------------------------------
//   d x_j = (1 - s_j) (p_j (c_j - sum_i c_i p_i - A) + q_j)
// with c the loss' coefficients, q the route weights' terms of the selected experts and A what
// softmax weights without renormalisation take from every expert (1 - s_j is 1 for softmax).
// The q of a token meet the row in shared memory.
// Four CTAs per SM up to 384 experts (64 registers): a token is a chain of loads and reductions, and
// only other warps hide it (384 experts, 32768 tokens: 31.5 us with three, 27 with four).
template <int VEC, int N>
__global__ void __launch_bounds__(kWarps * 32, N * VEC <= 12 ? 4 : 1)
    router_bwd_kernel(int T, int E, int K, int n_seq, int scoring, int renorm, float rsf,
                      const float* x, const int32_t* __restrict__ ids,
                      const float* __restrict__ dw, const float* __restrict__ coef,
                      const int32_t* __restrict__ off, const float* __restrict__ d_loss,
                      float* out) {
  extern __shared__ __align__(16) uint8_t dyn[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pitch = (E + 3) & ~3;
  float* s_row = reinterpret_cast<float*>(dyn) + warp * pitch;  // this warp's q, by expert
  for (int e = lane; e < pitch; e += 32) s_row[e] = 0.0f;
  __syncwarp();
  const float scale = d_loss ? *d_loss : 1.0f;
  const int mine = my_offset(off, n_seq, lane);
  const int stride = gridDim.x * kWarps;
  for (int t = blockIdx.x * kWarps + warp; t < T; t += stride) {
    const float* row = x + (size_t)t * E;
    float* dst = out + (size_t)t * E;
    Row<VEC, N> v, om;
    v.load(row, E, lane, -INFINITY);
    const int id = lane < K ? ids[(size_t)t * K + lane] : -1;
    const bool on = id >= 0 && id < E;
    float g = 0.0f, xs = -INFINITY;
    if (dw && on) {
      g = dw[(size_t)t * K + lane] * rsf;
      xs = row[id];
    }
    if (!__any_sync(kAll, on)) {
      const Row<VEC, N> zero = {};
      zero.store(dst, E, lane);
      continue;
    }
    const float* c = nullptr;
    if (coef) {
      if (!off) {
        c = coef;
      } else {
        const int s = seq_of(off, n_seq, t, mine);
        if (s < n_seq && off[s] <= t) c = coef + (size_t)s * E;
      }
    }
    Row<VEC, N> cc = {};
    if (c) cc.load(c, E, lane, 0.0f);
    const float inv = row_scores(v, om, scoring);
    float mean_c = 0.0f;
    if (c) mean_c = warp_sum(row_dot(cc, v)) * inv;
    float all = 0.0f;
    Row<VEC, N> q_row = {};
    if (dw) {
      float q;
      if (!renorm && scoring == MOE_SOFTMAX) {
        // the row's scores are in their owners' registers
        v.store(s_row, E, lane);
        __syncwarp();
        q = on ? s_row[id] * inv * g : 0.0f;
        all = warp_sum(q);
        __syncwarp();
        for (int e = lane; e < pitch; e += 32) s_row[e] = 0.0f;
        __syncwarp();
      } else {
        float s, unused;
        bool shift = scoring == MOE_SOFTMAX;
        if (!shift) sigmoid2(xs, s, unused);
        if (!renorm) {
          q = s * g;
        } else {
          float sum = 0.0f;
          if (!shift) {
            sum = warp_sum(s);
            shift = __any_sync(kAll, sum < kTinySum);
          }
          if (shift) {  // by the selection's own largest logit: it may lie far below the row's
            const float m = warp_max(xs);
            s = m == -INFINITY ? 0.0f : exp_fast(xs - m);
            sum = warp_sum(s);
          }
          const float w = sum == 0.0f ? 0.0f : __fdividef(s, sum);
          q = w * (g - warp_sum(w * g));
        }
      }
      // An expert named twice gets the sum of its routes, in route order, from the first.  Whether
      // there is one shows when every route leaves its number at its expert: one gets lost.
      if (on) s_row[id] = __int_as_float(lane);
      __syncwarp();
      const bool lost = on && __float_as_int(s_row[id]) != lane;
      __syncwarp();
      bool first = on;
      float tot = q;
      if (__any_sync(kAll, lost)) {
        const unsigned same = __match_any_sync(kAll, on ? id : -1 - lane);
        first = on && (int)__ffs(same) - 1 == lane;
        tot = 0.0f;
        for (int j = 0; j < K; ++j) {
          const float qj = __shfl_sync(kAll, q, j);
          if ((same >> j) & 1u) tot += qj;
        }
      }
      if (first) s_row[id] = tot;
      __syncwarp();
      q_row.load(s_row, E, lane, 0.0f);
      __syncwarp();
      if (on) s_row[id] = 0.0f;
      __syncwarp();
    }
    row_gradient(v, inv, cc, scale, mean_c * scale + all, q_row, om);
    v.store(dst, E, lane);
  }
}

// CTAs of the first pass: four on each of a GB300's 152 SMs (32768 tokens of 256 experts, both
// passes: 17.3 us, with two on each 19.5).  Part of the order of the sums, so the same on every
// device.
constexpr int kChunkCtas = 608;
constexpr int kFinCtas = 304;

// Workspace of the balance loss past its header (whose words other calls own): the records, the
// parts of the loss and the ticket, all of them written by the call that reads them.
struct BalanceLayout {
  int chunk, n_chunks, per_cta, fin_ctas;
  size_t prob, count, live, part, ticket, total;
};
BalanceLayout balance_layout(int T, int E, int n_seq) {
  BalanceLayout L;
  // a token per warp at least
  L.chunk = ((T + kChunkCtas - 1) / kChunkCtas + kWarps - 1) / kWarps * kWarps;
  if (L.chunk < kWarps) L.chunk = kWarps;
  L.n_chunks = (T + L.chunk - 1) / L.chunk;
  // Second pass: one CTA spares the join of the CTAs' parts of the loss, as long as its warps have
  // few records to read (t512 of 128 experts: 6.9 us against 7.6); else two CTAs per SM at most.
  const int64_t tiles = (E + 31) / 32, units = n_seq * tiles;
  const bool one = (L.n_chunks + (int64_t)n_seq) * tiles <= 16 * kFinWarps;
  L.per_cta = (int)(one ? units : (units + kFinCtas - 1) / kFinCtas);
  L.fin_ctas = (int)((units + L.per_cta - 1) / L.per_cta);
  size_t o = kHeaderBytes;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t n_rec = (size_t)L.n_chunks + n_seq;
  L.prob = take(n_rec * E * sizeof(float));
  L.count = take(n_rec * E * sizeof(int32_t));
  L.live = take(n_rec * sizeof(int32_t));
  L.part = take((size_t)L.fin_ctas * sizeof(float));
  L.ticket = take(sizeof(int));
  L.total = o;
  return L;
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int n_seq) { return balance_layout(T, E, n_seq).total; }

// CALL(VEC, N) for rows of E values.
#define ROUTER_ROW(E, CALL)                     \
  [&]() -> cudaError_t {                        \
    const int e_ = (E);                         \
    if (e_ % 4 == 0) {                          \
      if (e_ <= 128) return CALL(4, 1);         \
      if (e_ <= 256) return CALL(4, 2);         \
      if (e_ <= 384) return CALL(4, 3);         \
      if (e_ <= 512) return CALL(4, 4);         \
      return CALL(4, 8);                        \
    }                                           \
    if (e_ <= 32) return CALL(1, 1);            \
    if (e_ <= 64) return CALL(1, 2);            \
    if (e_ <= 128) return CALL(1, 4);           \
    if (e_ <= 192) return CALL(1, 6);           \
    if (e_ <= 256) return CALL(1, 8);           \
    if (e_ <= 384) return CALL(1, 12);          \
    if (e_ <= 512) return CALL(1, 16);          \
    return CALL(1, 32);                         \
  }()

cudaError_t launch_balance_loss(const moe_problem_t& p, int n_seq, float coeff, const float* x,
                                const int32_t* ids, const int32_t* off, float* loss,
                                int32_t* counts, int32_t* live, float* prob_sum, float* coef,
                                void* workspace, cudaStream_t s) {
  const BalanceLayout L = balance_layout(p.T, p.E, n_seq);
  char* ws = static_cast<char*>(workspace);
  Records rec;
  rec.prob = reinterpret_cast<float*>(ws + L.prob);
  rec.count = reinterpret_cast<int32_t*>(ws + L.count);
  rec.live = reinterpret_cast<int32_t*>(ws + L.live);
  int* status = reinterpret_cast<int*>(ws);
  int* ticket = reinterpret_cast<int*>(ws + L.ticket);
  // Few tokens: one launch of one CTA, whose second step takes a sequence's tokens one after the
  // other, while that costs less than a second launch (26 tokens of 370 experts 6.1 us against 6.2,
  // 64 of 128 8.4 against 5.8; 13 tokens in 18 sequences 6.5 against 12.9).
  const int groups = kSmallThreads / ((p.E + 31) / 32 * 32);
  if (p.T <= kSmallTokens && p.T <= 32 + 8 * (n_seq - 1) && n_seq <= kSmallSeqs &&
      (int64_t)p.T * p.E <= 16384 && (int64_t)n_seq * p.E <= 32768 && (n_seq + groups - 1) / groups <= 16) {
#define SMALL_(V, N)                                                                          \
  launch_k(balance_small_kernel<V, N>, dim3(1), dim3(kSmallThreads), 0, s, false, p.T, p.E,   \
           p.top_k, n_seq, p.scoring, coeff, x, ids, off, loss, counts, live, prob_sum, coef, \
           status)
    return ROUTER_ROW(p.E, SMALL_);
#undef SMALL_
  }
  if (p.T > 0) {
    const size_t smem = (size_t)(kWarps + 1) * (p.E + 3) * 4;
#define CHUNK_(V, N)                                                                             \
  launch_k(balance_chunk_kernel<V, N>, dim3(L.n_chunks), dim3(kWarps * 32), smem, s, false, p.T, \
           p.E, p.top_k, n_seq, p.scoring, L.chunk, x, ids, off, rec, ticket, status)
    const cudaError_t e = ROUTER_ROW(p.E, CHUNK_);
#undef CHUNK_
    if (e != cudaSuccess) return e;
  } else {  // no first pass
    const cudaError_t e = cudaMemsetAsync(ticket, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
  }
  return launch_k(balance_final_kernel, dim3(L.fin_ctas), dim3(kFinWarps * 32), 0, s,
                  p.T > 0, p.T, p.E, p.top_k, n_seq, L.chunk, L.per_cta, coeff, off, rec, loss, counts,
                  live, prob_sum, coef, reinterpret_cast<float*>(ws + L.part), ticket, status);
}

cudaError_t launch_router_bwd(const moe_problem_t& p, int n_seq, const float* x,
                              const int32_t* ids, const float* dw, const float* coef,
                              const int32_t* off, const float* d_loss, float* out,
                              cudaStream_t s) {
  if (p.T == 0) return cudaSuccess;
  const int need = (p.T + kWarps - 1) / kWarps;
  const int most = num_sms() * 4;  // what is resident: a second wave would start over
  const size_t smem = (size_t)kWarps * (p.E + 3) * 4;
#define BWD_(V, N)                                                                                \
  launch_k(router_bwd_kernel<V, N>, dim3(need < most ? need : most), dim3(kWarps * 32), smem, s, \
           false, p.T, p.E, p.top_k, n_seq, p.scoring, p.renormalize, p.routed_scaling_factor, \
           x, ids, dw, coef, off, d_loss, out)
  return ROUTER_ROW(p.E, BWD_);
#undef BWD_
}

}  // namespace gb300moe
