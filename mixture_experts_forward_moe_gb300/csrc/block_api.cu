// block_api.cu -- the C entry points around the routed experts declared in include/moe.h:
// argument checks and workspace carving of moe_linear, moe_block_norm_fwd/bwd,
// moe_balance_loss_fwd and moe_router_bwd.
#include <math.h>

#include "block_ops.cuh"

using namespace gb300moe;

namespace {

moe_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// NULL, or on a 16-byte boundary (every kernel here moves 16-byte vectors).
bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
template <typename... P>
bool aligned(const void* p, P... rest) {
  return aligned(p) && aligned(rest...);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

moe_status_t check_linear(const moe_linear_t* g) {
  if (!g || g->T < 0 || g->N <= 0 || g->K <= 0) return MOE_ERR_INVALID_ARG;
  if (g->dtype != MOE_BF16 && g->dtype != MOE_F16) return MOE_ERR_INVALID_ARG;
  if (g->activation < MOE_LINEAR_NONE || g->activation > MOE_LINEAR_RELU2)
    return MOE_ERR_INVALID_ARG;
  if (g->K % 8 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

constexpr int kNormMaxH = 16384;

moe_status_t check_norm(const moe_block_norm_t* p) {
  if (!p || p->T < 0 || p->H <= 0) return MOE_ERR_INVALID_ARG;
  if (p->dtype != MOE_BF16 && p->dtype != MOE_F16) return MOE_ERR_INVALID_ARG;
  if (p->gate < MOE_GATE_NONE || p->gate > MOE_GATE_ELEMENT) return MOE_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || !isfinite(p->eps) || !isfinite(p->residual_scale) ||
      !isfinite(p->weight_offset))
    return MOE_ERR_INVALID_ARG;
  if (p->H % 8 != 0 || p->H > kNormMaxH) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// What the forward and the backward take alike.
moe_status_t check_norm_inputs(const moe_block_norm_t& p, const void* branch,
                               const void* residual, const void* gate, const void* wq,
                               const void* wp) {
  // a gate per token or element of no rows has no elements, and may have no address
  const bool empty = p.T == 0 && (p.gate == MOE_GATE_TOKEN || p.gate == MOE_GATE_ELEMENT);
  if (p.gate == MOE_GATE_NONE ? gate != nullptr : !gate && !empty) return MOE_ERR_INVALID_ARG;
  if (p.T > 0 && !branch) return MOE_ERR_INVALID_ARG;
  if ((wq && !p.post_norm) || (wp && !p.pre_norm)) return MOE_ERR_INVALID_ARG;
  if (!aligned(branch, residual, gate, wq, wp)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// The router's training takes the whole expert set: ids of all E experts.
moe_status_t check_router(const moe_problem_t* p, int32_t n_seq, const int32_t* off) {
  const moe_status_t st = check_problem(p);
  if (st != MOE_OK) return st;
  if (p->ep_num_local > 0) return MOE_ERR_UNSUPPORTED;
  if (n_seq < 1 || (!off && n_seq != 1)) return MOE_ERR_INVALID_ARG;
  if (n_seq > 1 << 20) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(const moe_linear_t* g) {
  return check_linear(g) == MOE_OK ? kHeaderBytes : 0;
}

moe_status_t moe_linear(const moe_linear_t* g, const void* x, const void* w, const void* bias,
                        const void* residual, void* out, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const moe_status_t st = check_linear(g);
  if (st != MOE_OK) return st;
  if (!workspace || !w || (g->T > 0 && (!x || !out))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, w, bias, residual, out, workspace)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < kHeaderBytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (g->T == 0) return MOE_OK;
  return from_cuda(launch_linear(*g, x, w, bias, residual, out, static_cast<int*>(workspace),
                                 (cudaStream_t)stream));
}

moe_status_t moe_block_norm_fwd(const moe_block_norm_t* p, const void* branch,
                                const void* residual, const void* gate, const void* post_weight,
                                const void* pre_weight, void* stream_out, void* normed_out,
                                void* stream) {
  moe_status_t st = check_norm(p);
  if (st != MOE_OK) return st;
  st = check_norm_inputs(*p, branch, residual, gate, post_weight, pre_weight);
  if (st != MOE_OK) return st;
  if (!p->pre_norm && normed_out) return MOE_ERR_INVALID_ARG;
  if (p->T > 0 && p->pre_norm && !normed_out) return MOE_ERR_INVALID_ARG;
  if (!aligned(stream_out, normed_out)) return MOE_ERR_INVALID_ARG;
  if (p->T == 0 || (!stream_out && !normed_out)) return MOE_OK;
  return from_cuda(launch_block_norm_fwd(*p, branch, residual, gate, post_weight, pre_weight,
                                         stream_out, normed_out, (cudaStream_t)stream));
}

size_t moe_block_norm_bwd_workspace_size(const moe_block_norm_t* p) {
  if (check_norm(p) != MOE_OK) return 0;
  return kHeaderBytes + align256((size_t)block_norm_bwd_ctas(p->T) * 3 * p->H * sizeof(float));
}

moe_status_t moe_block_norm_bwd(const moe_block_norm_t* p, const void* d_stream,
                                const void* d_normed, const void* branch, const void* residual,
                                const void* gate, const void* post_weight,
                                const void* pre_weight, void* d_branch, void* d_residual,
                                void* d_gate, void* d_post_weight, void* d_pre_weight,
                                void* workspace, size_t workspace_bytes, void* stream) {
  moe_status_t st = check_norm(p);
  if (st != MOE_OK) return st;
  st = check_norm_inputs(*p, branch, residual, gate, post_weight, pre_weight);
  if (st != MOE_OK) return st;
  if (!workspace) return MOE_ERR_INVALID_ARG;
  if (!p->pre_norm && d_normed) return MOE_ERR_INVALID_ARG;
  if (p->T > 0 && p->pre_norm && !d_normed) return MOE_ERR_INVALID_ARG;
  if ((d_gate && p->gate == MOE_GATE_NONE) || (d_post_weight && !post_weight) ||
      (d_pre_weight && !pre_weight))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(d_stream, d_normed, d_branch, d_residual, d_gate, d_post_weight, d_pre_weight,
               workspace))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_block_norm_bwd_workspace_size(p)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return from_cuda(launch_block_norm_bwd(
      *p, d_stream, d_normed, branch, residual, gate, post_weight, pre_weight, d_branch,
      d_residual, d_gate, d_post_weight, d_pre_weight,
      reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeaderBytes),
      (cudaStream_t)stream));
}

size_t moe_balance_loss_workspace_size(const moe_problem_t* p, int32_t n_seq) {
  if (check_problem(p) != MOE_OK || n_seq < 1 || n_seq > 1 << 20) return 0;
  return balance_workspace_bytes(p->T, p->E, n_seq);
}

moe_status_t moe_balance_loss_fwd(const moe_problem_t* p, int32_t n_seq, float coeff,
                                  const float* gating_output, const int32_t* topk_ids,
                                  const int32_t* seq_offsets, float* loss, int32_t* counts,
                                  int32_t* live_tokens, float* prob_sum, float* coef,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status_t st = check_router(p, n_seq, seq_offsets);
  if (st != MOE_OK) return st;
  if (!isfinite(coeff)) return MOE_ERR_INVALID_ARG;
  if (!loss || !counts || !live_tokens || !prob_sum || !coef || !workspace)
    return MOE_ERR_INVALID_ARG;
  if (p->T > 0 && (!gating_output || !topk_ids)) return MOE_ERR_INVALID_ARG;
  if (!aligned(gating_output, topk_ids, counts, prob_sum, coef, workspace))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < balance_workspace_bytes(p->T, p->E, n_seq))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  return from_cuda(launch_balance_loss(*p, n_seq, coeff, gating_output, topk_ids, seq_offsets,
                                       loss, counts, live_tokens, prob_sum, coef, workspace,
                                       (cudaStream_t)stream));
}

moe_status_t moe_router_bwd(const moe_problem_t* p, int32_t n_seq, const float* gating_output,
                            const int32_t* topk_ids, const float* d_topk_weights,
                            const float* coef, const int32_t* seq_offsets, const float* d_loss,
                            float* d_gating_output, void* stream) {
  const moe_status_t st = check_router(p, n_seq, seq_offsets);
  if (st != MOE_OK) return st;
  if (p->T > 0 && (!gating_output || !topk_ids || !d_gating_output)) return MOE_ERR_INVALID_ARG;
  if (!aligned(gating_output, topk_ids, d_topk_weights, coef, d_gating_output))
    return MOE_ERR_INVALID_ARG;
  return from_cuda(launch_router_bwd(*p, n_seq, gating_output, topk_ids, d_topk_weights, coef,
                                     seq_offsets, d_loss, d_gating_output,
                                     (cudaStream_t)stream));
}

}  // extern "C"
