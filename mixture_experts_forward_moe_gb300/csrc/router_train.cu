// router_train.cu -- training of the router (include/moe.h: moe_balance_loss_fwd,
// moe_router_bwd): per-expert counts, the balance loss over ragged sequences, and the gradient of
// the logits from that loss and from the route weights.
//
// One warp per token, expert e in lane e % 32, as in the router itself.
#include <math.h>

#include "common.cuh"

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

// A token's unnormalised probabilities, safe at both ends of the range: softmax shifts by the
// largest logit m.  sigmoid(x) / sum sigmoid is unchanged when every sigmoid is multiplied by
// e^-b; with b = min(m, 0) the largest stays near 1 where plain sigmoids would underflow.
// A row of -inf alone gives zeros.
struct Shift {
  float b;   // subtracted in the exponent
  float eb;  // e^b (sigmoid)
};
__device__ __forceinline__ Shift row_shift(float m, int scoring) {
  Shift s;
  s.b = m == -INFINITY ? 0.0f : (scoring == MOE_SOFTMAX ? m : fminf(m, 0.0f));
  s.eb = scoring == MOE_SOFTMAX ? 1.0f : expf(s.b);
  return s;
}
// e: the shifted score; om: 1 - sigmoid(x) (1 for softmax).
__device__ __forceinline__ void score(float x, const Shift& s, int scoring, float& e, float& om) {
  if (scoring == MOE_SOFTMAX) {
    e = expf(x - s.b);
    om = 1.0f;
  } else if (x >= 0.0f) {
    const float t = expf(-x);
    e = __frcp_rn(1.0f + t);
    om = t * e;
  } else {
    const float t = expf(x - s.b);
    om = __frcp_rn(fmaf(t, s.eb, 1.0f));
    e = t * om;
  }
}
__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

// First sequence s with seq_offsets[s + 1] > t (n_seq when there is none).
__device__ __forceinline__ int seq_of(const int32_t* off, int n_seq, int t) {
  int lo = 0, hi = n_seq;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
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

template <int VPL>
__global__ void __launch_bounds__(kWarps * 32)
    balance_chunk_kernel(int T, int E, int K, int n_seq, int scoring, int chunk,
                         const float* __restrict__ x, const int32_t* __restrict__ ids,
                         const int32_t* __restrict__ off, const Records rec, int* status) {
  extern __shared__ uint8_t dyn[];
  float* s_prob = reinterpret_cast<float*>(dyn);                // [kWarps][E]
  int* s_count = reinterpret_cast<int*>(s_prob + kWarps * E);   // [E]
  __shared__ int s_live;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * chunk;
  const int c1 = T - c0 < chunk ? T : c0 + chunk;
  bool bad = false;
  int t0 = c0;
  for (int s = off ? seq_of(off, n_seq, c0) : 0; s < n_seq && t0 < c1; ++s) {
    if (off) t0 = max(t0, off[s]);
    const int t1 = off ? min(c1, off[s + 1]) : c1;
    if (t1 <= t0) continue;
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = 0;
    if (threadIdx.x == 0) s_live = 0;
    __syncthreads();
    float acc[VPL] = {};
    int live = 0;
    for (int t = t0 + warp; t < t1; t += kWarps) {
      const int id = lane < K ? ids[(size_t)t * K + lane] : -1;
      const bool on = id >= 0 && id < E;
      bad |= id < -1 || id >= E;
      if (!__any_sync(kAll, on)) continue;
      ++live;
      if (on) atomicAdd(&s_count[id], 1);
      const float* row = x + (size_t)t * E;
      float v[VPL];
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < E ? row[e] : -INFINITY;
        m = fmaxf(m, v[i]);
      }
      const Shift sh = row_shift(warp_max(m), scoring);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float om;
        score(v[i], sh, scoring, v[i], om);
        sum += v[i];
      }
      const float inv = inverse(warp_sum(sum));
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
    }
    if (lane == 0 && live) atomicAdd(&s_live, live);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) s_prob[warp * E + e] = acc[i];
    }
    __syncthreads();
    const size_t r = (size_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) p += s_prob[w * E + e];
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
// One CTA per (32 experts, sequence): 32 lanes of chunks per expert, joined in a fixed order.
// The CTA that finishes last adds the CTAs' parts of the loss, again in a fixed order.
constexpr int kFinE = 32, kFinC = 32;

__global__ void __launch_bounds__(kFinE * kFinC)
    balance_final_kernel(int T, int E, int K, int n_seq, int chunk, float coeff,
                         const int32_t* __restrict__ off, const Records rec,
                         float* __restrict__ loss, int32_t* __restrict__ counts,
                         int32_t* __restrict__ live_out, float* __restrict__ prob_sum,
                         float* __restrict__ coef, float* part, int* ticket, int* status) {
  __shared__ float s_p[kFinC][kFinE];
  __shared__ int s_c[kFinC][kFinE];
  __shared__ int s_live, s_nlive, s_last;
  const int tid = threadIdx.y * kFinE + threadIdx.x;
  if (tid == 0) s_live = s_nlive = 0;
  __syncthreads();
  // The chunks of sequence s are [first, last]; empty when it has no tokens.
  auto range = [&](int s, int& first, int& last) {
    const int a = off ? clamp_i(off[s], 0, T) : 0;
    const int b = off ? clamp_i(off[s + 1], 0, T) : T;
    first = a / chunk;
    last = b > a ? (b - 1) / chunk : first - 1;
  };
  int n = 0;
  for (int s = tid; s < n_seq; s += kFinE * kFinC) {
    int c, last;
    range(s, c, last);
    bool any = false;
    for (; c <= last && !any; ++c) any = rec.live[(size_t)c + s] > 0;
    n += any;
    if (off && blockIdx.x == 0 && blockIdx.y == 0 &&
        (off[s] < 0 || off[s + 1] < off[s] || off[s + 1] > T))
      set_status(status, MOE_ERR_INVALID_ARG);
  }
  if (n) atomicAdd(&s_nlive, n);
  float loss_part = 0.0f;
  const int e = blockIdx.x * kFinE + threadIdx.x;
  for (int s = blockIdx.y; s < n_seq; s += gridDim.y) {
    int first, last;
    range(s, first, last);
    int live = 0;
    for (int c = first + tid; c <= last; c += kFinE * kFinC) live += rec.live[(size_t)c + s];
    if (live) atomicAdd(&s_live, live);
    float p = 0.0f;
    int cnt = 0;
    if (e < E)
#pragma unroll 4
      for (int c = first + threadIdx.y; c <= last; c += kFinC) {
        const size_t r = ((size_t)c + s) * E + e;
        p += rec.prob[r];
        cnt += rec.count[r];
      }
    s_p[threadIdx.y][threadIdx.x] = p;
    s_c[threadIdx.y][threadIdx.x] = cnt;
    __syncthreads();
    if (threadIdx.y == 0 && e < E) {
#pragma unroll
      for (int y = 1; y < kFinC; ++y) {
        p += s_p[y][threadIdx.x];
        cnt += s_c[y][threadIdx.x];
      }
      const float T_s = (float)max(s_live, 1);
      const float w = (float)cnt * (coeff * (float)E) / ((float)max(s_nlive, 1) * (float)K) / T_s /
                      T_s;
      const size_t o = (size_t)s * E + e;
      counts[o] = cnt;
      prob_sum[o] = p;
      coef[o] = w;
      loss_part = fmaf(w, p, loss_part);
      if (blockIdx.x == 0 && threadIdx.x == 0) live_out[s] = s_live;
    }
    __syncthreads();
    if (tid == 0) s_live = 0;
    __syncthreads();
  }
  const int n_parts = gridDim.x * gridDim.y;
  if (threadIdx.y == 0) {
    loss_part = warp_sum(loss_part);
    if (threadIdx.x == 0) {
      part[blockIdx.y * gridDim.x + blockIdx.x] = loss_part;
      __threadfence();
      s_last = atomicAdd(ticket, 1) == n_parts - 1;
    }
    __syncwarp();
    if (s_last) {
      __threadfence();
      float l = 0.0f;
      for (int i = threadIdx.x; i < n_parts; i += kFinE) l += __ldcg(part + i);
      l = warp_sum(l);
      if (threadIdx.x == 0) {
        *loss = l;
        *ticket = 0;
      }
    }
  }
}

// ---- gradient of the logits --------------------------------------------------------------------
template <int VPL>
__global__ void __launch_bounds__(kWarps * 32)
    router_bwd_kernel(int T, int E, int K, int n_seq, int scoring, int renorm, float rsf,
                      const float* x, const int32_t* __restrict__ ids,
                      const float* __restrict__ dw, const float* __restrict__ coef,
                      const int32_t* __restrict__ off, const float* __restrict__ d_loss,
                      float* out) {
  extern __shared__ uint8_t dyn[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* s_row = reinterpret_cast<float*>(dyn) + warp * E;  // this warp's route terms, by expert
  for (int e = lane; e < E; e += 32) s_row[e] = 0.0f;
  __syncwarp();
  const float scale = d_loss ? *d_loss : 1.0f;
  for (int t = blockIdx.x * kWarps + warp; t < T; t += gridDim.x * kWarps) {
    const int id = lane < K ? ids[(size_t)t * K + lane] : -1;
    const bool on = id >= 0 && id < E;
    const float* row = x + (size_t)t * E;
    float* dst = out + (size_t)t * E;
    if (!__any_sync(kAll, on)) {
      for (int e = lane; e < E; e += 32) dst[e] = 0.0f;
      continue;
    }
    float v[VPL], om[VPL];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < E ? row[e] : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    const Shift sh = row_shift(warp_max(m), scoring);
    const float* c = nullptr;
    if (coef) {
      if (!off) {
        c = coef;
      } else {
        const int s = seq_of(off, n_seq, t);
        if (s < n_seq && off[s] <= t) c = coef + (size_t)s * E;
      }
    }
    float sum = 0.0f, csum = 0.0f, cc[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      score(v[i], sh, scoring, v[i], om[i]);
      cc[i] = c && e < E ? c[e] * scale : 0.0f;
      sum += v[i];
      csum = fmaf(cc[i], v[i], csum);
    }
    const float inv = inverse(warp_sum(sum));
    const float mean_c = warp_sum(csum) * inv;
    // The route weights' term of each selected expert, up to the factor 1 - sigmoid.
    float all = 0.0f;  // softmax over all experts: p_j times this is subtracted
    if (dw) {
      const float xs = on ? row[id] : -INFINITY;
      const float g = on ? dw[(size_t)t * K + lane] * rsf : 0.0f;
      float es, oms, q;
      if (renorm) {
        // shifted by the selection's own largest logit: it may lie far below the row's
        score(xs, row_shift(warp_max(xs), scoring), scoring, es, oms);
        const float w = es * inverse(warp_sum(es));
        q = w * (g - warp_sum(w * g));
      } else {
        score(xs, sh, scoring, es, oms);
        if (scoring == MOE_SOFTMAX) {
          q = es * inv * g;
          all = warp_sum(q);
        } else {
          q = es * sh.eb * g;  // the sigmoid itself: the shift undone
        }
      }
      // An expert named twice gets the sum of its routes, in route order, from the first.
      const unsigned same = __match_any_sync(kAll, on ? id : -1 - lane);
      float tot = q;
      if (__any_sync(kAll, on && __popc(same) > 1)) {
        tot = 0.0f;
        for (int j = 0; j < K; ++j) {
          const float qj = __shfl_sync(kAll, q, j);
          if ((same >> j) & 1u) tot += qj;
        }
      }
      if (on && (int)__ffs(same) - 1 == lane) s_row[id] = tot;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) {
        const float p = v[i] * inv;
        float d = p * (cc[i] - mean_c - all);
        if (dw) d += s_row[e];
        dst[e] = d * om[i];
      }
    }
    __syncwarp();
    if (dw && on) s_row[id] = 0.0f;
    __syncwarp();
  }
}

constexpr int kBalanceChunk = 64;

// Workspace of the balance loss past its header: the records and the parts of the loss.
struct BalanceLayout {
  int n_chunks, e_tiles, seq_ctas;
  size_t prob, count, live, part, total;
};
BalanceLayout balance_layout(int T, int E, int n_seq) {
  BalanceLayout L;
  L.n_chunks = (T + kBalanceChunk - 1) / kBalanceChunk;
  L.e_tiles = (E + kFinE - 1) / kFinE;
  L.seq_ctas = n_seq < 512 ? n_seq : 512;
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
  L.part = take((size_t)L.e_tiles * L.seq_ctas * sizeof(float));
  L.total = o;
  return L;
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int n_seq) { return balance_layout(T, E, n_seq).total; }

// CALL(values per lane) for E experts.
#define ROUTER_VPL(E, CALL)            \
  [&]() -> cudaError_t {               \
    const int need_ = ((E) + 31) / 32; \
    if (need_ <= 1) return CALL(1);    \
    if (need_ <= 2) return CALL(2);    \
    if (need_ <= 4) return CALL(4);    \
    if (need_ <= 8) return CALL(8);    \
    if (need_ <= 12) return CALL(12);  \
    if (need_ <= 16) return CALL(16);  \
    return CALL(32);                   \
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
  int* ticket = reinterpret_cast<int*>(ws + kTicketOffset);
  if (p.T > 0) {
    const size_t smem = (size_t)(kWarps + 1) * p.E * 4;
#define CHUNK_(V)                                                                             \
  launch_k(balance_chunk_kernel<V>, dim3(L.n_chunks), dim3(kWarps * 32), smem, s, false, p.T, \
           p.E, p.top_k, n_seq, p.scoring, kBalanceChunk, x, ids, off, rec, status)
    const cudaError_t e = ROUTER_VPL(p.E, CHUNK_);
#undef CHUNK_
    if (e != cudaSuccess) return e;
  }
  return launch_k(balance_final_kernel, dim3(L.e_tiles, L.seq_ctas), dim3(kFinE, kFinC), 0, s,
                  false, p.T, p.E, p.top_k, n_seq, kBalanceChunk, coeff, off, rec, loss, counts,
                  live, prob_sum, coef, reinterpret_cast<float*>(ws + L.part), ticket, status);
}

cudaError_t launch_router_bwd(const moe_problem_t& p, int n_seq, const float* x,
                              const int32_t* ids, const float* dw, const float* coef,
                              const int32_t* off, const float* d_loss, float* out,
                              cudaStream_t s) {
  if (p.T == 0) return cudaSuccess;
  const int need = (p.T + kWarps - 1) / kWarps;
  const int most = num_sms() * 8;
  const size_t smem = (size_t)kWarps * p.E * 4;
#define BWD_(V)                                                                                \
  launch_k(router_bwd_kernel<V>, dim3(need < most ? need : most), dim3(kWarps * 32), smem, s, \
           false, p.T, p.E, p.top_k, n_seq, p.scoring, p.renormalize, p.routed_scaling_factor, \
           x, ids, dw, coef, off, d_loss, out)
  return ROUTER_VPL(p.E, BWD_);
#undef BWD_
}

}  // namespace gb300moe
