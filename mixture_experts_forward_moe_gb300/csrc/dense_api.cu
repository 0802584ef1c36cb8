// dense_api.cu -- the C entry points of the dense feed-forward block declared in include/moe.h:
// argument checks and workspace carving of moe_gated_linear(_bwd), moe_linear_bwd, moe_checkpoint,
// moe_checkpoint_restore, moe_linear_w4a16 and moe_gated_linear_w4a16.
#include "dense_ops.cuh"

using namespace gb300moe;

namespace {

moe_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
template <typename... P>
bool aligned(const void* p, P... rest) {
  return aligned(p) && aligned(rest...);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
size_t larger(size_t a, size_t b) { return a > b ? a : b; }

bool dtype_ok(int32_t d) { return d == MOE_BF16 || d == MOE_F16; }

moe_status_t check_gated(const moe_gated_linear_t* p) {
  if (!p || p->T < 0 || p->H <= 0 || p->F <= 0 || !dtype_ok(p->dtype)) return MOE_ERR_INVALID_ARG;
  if (p->activation < MOE_ACT_SILU || p->activation > MOE_ACT_RELU2) return MOE_ERR_INVALID_ARG;
  if (p->activation == MOE_ACT_RELU2) return MOE_ERR_UNSUPPORTED;  // has no up projection
  if (p->H % 8 != 0 || p->F % 8 != 0 || p->F > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Both parts of a checkpoint, or neither.
bool both(const void* codes, const void* scales) { return (codes != nullptr) == (scales != nullptr); }

// Few tokens that save nothing have the weights as the M side (dense_few.cu), where reading them takes
// longest: 16 x 2048 x 7168 in 15.5 us against 21, 32 x 18432 x 7168 in 85 against 90, but 128 x 18432 x
// 7168 in 103 against 92 and 64 x 4096 x 4096 in 21 against 20.
bool few_rows(const moe_gated_linear_t& p, bool save) {
  return !save && (p.T <= 32 || (p.T <= kFewRows && 2 * (int64_t)p.F * p.H < 1 << 25));
}

size_t gated_bytes(const moe_gated_linear_t& p) {
  return kHeaderBytes + align256(gated_split_bytes(p.T, p.F, p.H));
}

// The gradients of a product [T, N] of x [T, K] and w [N, K]: d_x and d_w.
struct Gradients {
  Product list[2];
  Gradients(int T, int N, int K, const void* dy, int64_t pitch, const void* x, const void* w,
            void* d_x, void* d_w)
      : list{{false, T, K, N, dy, pitch, w, d_x}, {true, N, K, T, dy, pitch, x, d_w}} {}
};
// Bytes of their sums, whichever are wanted.
size_t gradient_bytes(int T, int N, int K) {
  const Gradients g(T, N, K, nullptr, 0, nullptr, nullptr, nullptr, nullptr);
  return larger(larger(products_split_bytes(g.list, 1), products_split_bytes(g.list + 1, 1)),
                products_split_bytes(g.list, 2));
}
cudaError_t launch_gradients(int dtype, const Gradients& g, float* parts, int* status,
                             cudaStream_t s) {
  const bool x = g.list[0].out != nullptr, w = g.list[1].out != nullptr;
  if (!x && !w) return cudaSuccess;
  return launch_products(dtype, g.list + (x ? 0 : 1), x && w ? 2 : 1, parts, status, s);
}

// The last part of a workspace, x restored from its checkpoint: needed where it is one, and up to a
// megabyte always, so that small calls have one size.
constexpr size_t kSmallX = 1 << 20;
struct Restored {
  size_t x, bytes;  // where it begins, and the whole workspace
  Restored(size_t at, size_t size) : x(at), bytes(at + align256(size)) {}
  size_t without() const { return bytes - x <= kSmallX ? bytes : x; }
  size_t need(bool restored) const { return restored ? bytes : without(); }
};

// moe_gated_linear_bwd: status | d_pre [T, 2F] | parts of K | x [T, H]
struct GatedBwd {
  size_t d_pre, parts;
  Restored x;
  explicit GatedBwd(const moe_gated_linear_t& p)
      : d_pre(kHeaderBytes), parts(d_pre + align256((size_t)p.T * 2 * p.F * 2)),
        x(parts + align256(larger(gated_split_bytes(p.T, p.F, p.H),
                                  gradient_bytes(p.T, 2 * p.F, p.H))),
          (size_t)p.T * p.H * 2) {}
};

moe_status_t check_linear_bwd(const moe_linear_t* g) {
  if (!g || g->T < 0 || g->N <= 0 || g->K <= 0 || !dtype_ok(g->dtype)) return MOE_ERR_INVALID_ARG;
  if (g->activation < MOE_LINEAR_NONE || g->activation > MOE_LINEAR_RELU2)
    return MOE_ERR_INVALID_ARG;
  if (g->activation != MOE_LINEAR_NONE || g->out_f32 || g->K % 8 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// moe_linear_bwd: status | d_out with rows of a multiple of 8 | parts of K | x [T, K]
struct LinearBwd {
  int64_t pitch;
  size_t d_out, parts;
  Restored x;
  explicit LinearBwd(const moe_linear_t& g)
      : pitch(((int64_t)g.N + 7) / 8 * 8), d_out(kHeaderBytes),
        parts(d_out + (pitch != g.N ? align256((size_t)g.T * (size_t)pitch * 2) : 0)),
        x(parts + align256(gradient_bytes(g.T, g.N, g.K)), (size_t)g.T * g.K * 2) {}
};

constexpr int32_t kMaxW4Rows = 1 << 20;

// status | x in f16, its rows' scales
size_t w4_workspace(int dtype, int64_t T, int64_t K) {
  return kHeaderBytes + align256(w4_bytes(dtype, T, K));
}
// Past sixteen rows the weights are decoded once for all on the tensor cores.
cudaError_t launch_rows4(const RowsCall& c, void* workspace, cudaStream_t s) {
  return c.T > kFewW4Rows ? launch_w4(c, static_cast<char*>(workspace) + kHeaderBytes, s)
                          : launch_rows(c, s);
}

moe_status_t check_w4(int32_t T, int32_t N, int32_t K) {
  if (T < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  return K % 32 != 0 || T > kMaxW4Rows ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
moe_status_t check_linear_w4(const moe_linear_t* g) {
  if (!g || !dtype_ok(g->dtype)) return MOE_ERR_INVALID_ARG;
  if (g->activation < MOE_LINEAR_NONE || g->activation > MOE_LINEAR_RELU2)
    return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_w4(g->T, g->N, g->K);
  return st == MOE_OK && g->out_f32 ? MOE_ERR_UNSUPPORTED : st;
}
moe_status_t check_gated_w4(const moe_gated_linear_t* p) {
  if (!p || !dtype_ok(p->dtype)) return MOE_ERR_INVALID_ARG;
  if (p->activation < MOE_ACT_SILU || p->activation > MOE_ACT_RELU2) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_w4(p->T, p->F, p->H);
  if (st != MOE_OK) return st;
  return p->activation == MOE_ACT_RELU2 || p->F > INT32_MAX / 2 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_gated_linear_workspace_size(const moe_gated_linear_t* p) {
  return check_gated(p) == MOE_OK ? gated_bytes(*p) : 0;
}

moe_status_t moe_gated_linear(const moe_gated_linear_t* p, const void* x, const void* w_gate_up,
                              void* out, uint8_t* gate_codes, float* gate_scales,
                              uint8_t* up_codes, float* up_scales, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const moe_status_t st = check_gated(p);
  if (st != MOE_OK) return st;
  const bool save = gate_codes != nullptr;
  if (!both(gate_codes, gate_scales) || !both(up_codes, up_scales) || !both(gate_codes, up_codes))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !w_gate_up || (p->T > 0 && (!x || !out))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, w_gate_up, out, gate_codes, gate_scales, up_codes, up_scales, workspace))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < gated_bytes(*p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (p->T == 0) return MOE_OK;
  const cudaStream_t s = (cudaStream_t)stream;
  if (few_rows(*p, save)) {
    RowsCall c = {};
    c.T = p->T, c.N = p->F, c.K = p->H, c.dtype = p->dtype, c.gated = 1, c.act = p->activation;
    c.x = x, c.w = w_gate_up, c.out = out, c.status = static_cast<int*>(workspace);
    return from_cuda(p->T == 1 ? launch_rows(c, s) : launch_few(c, s));
  }
  return from_cuda(launch_gated(
      p->dtype, p->activation, p->T, p->F, p->H, x, w_gate_up, out, Ckpt{gate_codes, gate_scales},
      Ckpt{up_codes, up_scales},
      reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeaderBytes),
      static_cast<int*>(workspace), s));
}

size_t moe_gated_linear_bwd_workspace_size(const moe_gated_linear_t* p) {
  return check_gated(p) == MOE_OK ? GatedBwd(*p).x.bytes : 0;
}
size_t moe_gated_linear_bwd_workspace_size_x16(const moe_gated_linear_t* p) {
  return check_gated(p) == MOE_OK ? GatedBwd(*p).x.without() : 0;
}

moe_status_t moe_gated_linear_bwd(const moe_gated_linear_t* p, const void* d_out, const void* x,
                                  const uint8_t* x_codes, const float* x_scales,
                                  const void* w_gate_up, const uint8_t* gate_codes,
                                  const float* gate_scales, const uint8_t* up_codes,
                                  const float* up_scales, void* d_x, void* d_w, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status_t st = check_gated(p);
  if (st != MOE_OK) return st;
  const bool saved = gate_codes != nullptr;
  if (!both(gate_codes, gate_scales) || !both(up_codes, up_scales) || !both(gate_codes, up_codes) ||
      !both(x_codes, x_scales) || (x && x_codes))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !w_gate_up || (p->T > 0 && !d_out)) return MOE_ERR_INVALID_ARG;
  const bool need_x = !saved || d_w != nullptr;  // to compute the pre-activations, or for d_w
  if (p->T > 0 && need_x && !x && !x_codes) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_out, x, x_codes, x_scales, w_gate_up, gate_codes, gate_scales, up_codes, up_scales,
               d_x, d_w, out, workspace))
    return MOE_ERR_INVALID_ARG;
  const GatedBwd at(*p);
  const bool restored = need_x && x_codes;
  if (workspace_bytes < at.x.need(restored)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (p->T == 0)
    return d_w ? from_cuda(cudaMemsetAsync(d_w, 0, (size_t)2 * p->F * p->H * 2, s)) : MOE_OK;
  if (!d_x && !d_w && !out) return MOE_OK;
  char* ws = static_cast<char*>(workspace);
  int* status = static_cast<int*>(workspace);
  float* parts = reinterpret_cast<float*>(ws + at.parts);
  void* d_pre = ws + at.d_pre;
  if (restored) {
    if (const cudaError_t e = launch_restore(p->dtype, p->T, p->H, CkptIn{x_codes, x_scales},
                                             ws + at.x.x, s))
      return from_cuda(e);
    x = ws + at.x.x;
  }
  const cudaError_t e =
      saved ? launch_gated_grad_saved(p->dtype, p->activation, p->T, p->F, d_out,
                                      CkptIn{gate_codes, gate_scales}, CkptIn{up_codes, up_scales},
                                      d_pre, out, s)
            : launch_gated_grad(p->dtype, p->activation, p->T, p->F, p->H, x, w_gate_up, d_out,
                                d_pre, out, parts, status, s);
  if (e != cudaSuccess) return from_cuda(e);
  return from_cuda(launch_gradients(
      p->dtype, Gradients(p->T, 2 * p->F, p->H, d_pre, 2 * (int64_t)p->F, x, w_gate_up, d_x, d_w),
      parts, status, s));
}

size_t moe_linear_bwd_workspace_size(const moe_linear_t* g) {
  return check_linear_bwd(g) == MOE_OK ? LinearBwd(*g).x.bytes : 0;
}
size_t moe_linear_bwd_workspace_size_x16(const moe_linear_t* g) {
  return check_linear_bwd(g) == MOE_OK ? LinearBwd(*g).x.without() : 0;
}

moe_status_t moe_linear_bwd(const moe_linear_t* g, const void* d_out, const void* x,
                            const uint8_t* x_codes, const float* x_scales, const void* w, void* d_x,
                            void* d_w, void* d_bias, void* workspace, size_t workspace_bytes,
                            void* stream) {
  const moe_status_t st = check_linear_bwd(g);
  if (st != MOE_OK) return st;
  if (!both(x_codes, x_scales) || (x && x_codes) || !workspace) return MOE_ERR_INVALID_ARG;
  if (g->T > 0 && (!d_out || (d_x && !w) || (d_w && !x && !x_codes))) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_out, x, x_codes, x_scales, w, d_x, d_w, d_bias, workspace))
    return MOE_ERR_INVALID_ARG;
  const LinearBwd at(*g);
  const bool restored = d_w && x_codes;
  if (workspace_bytes < at.x.need(restored)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const cudaStream_t s = (cudaStream_t)stream;
  if (g->T == 0) {
    cudaError_t e = cudaSuccess;
    if (d_w) e = cudaMemsetAsync(d_w, 0, (size_t)g->N * g->K * 2, s);
    if (e == cudaSuccess && d_bias) e = cudaMemsetAsync(d_bias, 0, (size_t)g->N * 2, s);
    return from_cuda(e);
  }
  if (!d_x && !d_w && !d_bias) return MOE_OK;
  char* ws = static_cast<char*>(workspace);
  int* status = static_cast<int*>(workspace);
  float* parts = reinterpret_cast<float*>(ws + at.parts);
  // Rows of d_out that do not start on 16 bytes are copied, in the pass that adds them if there is one.
  const bool pad = at.pitch != g->N;
  if (d_bias) {
    if (const cudaError_t e = launch_column_sum(g->dtype, g->T, g->N, at.pitch, d_out,
                                                pad ? ws + at.d_out : nullptr, d_bias, s))
      return from_cuda(e);
  } else if (pad) {
    if (const cudaError_t e = launch_pad_rows(g->T, g->N, at.pitch, d_out, ws + at.d_out, s))
      return from_cuda(e);
  }
  if (pad) d_out = ws + at.d_out;
  if (restored) {
    if (const cudaError_t e = launch_restore(g->dtype, g->T, g->K, CkptIn{x_codes, x_scales},
                                             ws + at.x.x, s))
      return from_cuda(e);
    x = ws + at.x.x;
  }
  return from_cuda(launch_gradients(
      g->dtype, Gradients(g->T, g->N, g->K, d_out, at.pitch, x, w, d_x, d_w), parts, status, s));
}

moe_status_t moe_checkpoint(int32_t T, int32_t C, int32_t dtype, const void* x, uint8_t* codes,
                            float* scales, void* stream) {
  if (T < 0 || C <= 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x || !codes || !scales)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, codes, scales)) return MOE_ERR_INVALID_ARG;
  if (C % 8 != 0) return MOE_ERR_UNSUPPORTED;
  return from_cuda(launch_checkpoint(dtype, T, C, x, Ckpt{codes, scales}, (cudaStream_t)stream));
}

moe_status_t moe_checkpoint_restore(int32_t T, int32_t C, int32_t dtype, const uint8_t* codes,
                                    const float* scales, void* out, void* stream) {
  if (T < 0 || C <= 0 || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!codes || !scales || !out)) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, scales, out)) return MOE_ERR_INVALID_ARG;
  if (C % 8 != 0) return MOE_ERR_UNSUPPORTED;
  return from_cuda(
      launch_restore(dtype, T, C, CkptIn{codes, scales}, out, (cudaStream_t)stream));
}

size_t moe_linear_w4a16_workspace_size(const moe_linear_t* g) {
  return check_linear_w4(g) == MOE_OK ? w4_workspace(g->dtype, g->T, g->K) : 0;
}

moe_status_t moe_linear_w4a16(const moe_linear_t* g, const void* x, const uint8_t* codes,
                              const uint8_t* scales, const float* alpha, const void* bias,
                              const void* residual, void* out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const moe_status_t st = check_linear_w4(g);
  if (st != MOE_OK) return st;
  if (!workspace || !codes || !scales || !alpha || (g->T > 0 && (!x || !out)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, codes, scales, bias, residual, out, workspace)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < w4_workspace(g->dtype, g->T, g->K)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (g->T == 0) return MOE_OK;
  RowsCall c = {};
  c.T = g->T, c.N = g->N, c.K = g->K, c.dtype = g->dtype, c.act = g->activation;
  c.x = x, c.codes = codes, c.scales = scales, c.alpha = alpha, c.bias = bias, c.res = residual;
  c.out = out, c.status = static_cast<int*>(workspace);
  return from_cuda(launch_rows4(c, workspace, (cudaStream_t)stream));
}

size_t moe_gated_linear_w4a16_workspace_size(const moe_gated_linear_t* p) {
  return check_gated_w4(p) == MOE_OK ? w4_workspace(p->dtype, p->T, p->H) : 0;
}

moe_status_t moe_gated_linear_w4a16(const moe_gated_linear_t* p, const void* x,
                                    const uint8_t* codes, const uint8_t* scales, const float* alpha,
                                    void* out, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  const moe_status_t st = check_gated_w4(p);
  if (st != MOE_OK) return st;
  if (!workspace || !codes || !scales || !alpha || (p->T > 0 && (!x || !out)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, codes, scales, out, workspace)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < w4_workspace(p->dtype, p->T, p->H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (p->T == 0) return MOE_OK;
  RowsCall c = {};
  c.T = p->T, c.N = p->F, c.K = p->H, c.dtype = p->dtype, c.gated = 1, c.act = p->activation;
  c.x = x, c.codes = codes, c.scales = scales, c.alpha = alpha, c.out = out;
  c.status = static_cast<int*>(workspace);
  return from_cuda(launch_rows4(c, workspace, (cudaStream_t)stream));
}

}  // extern "C"
