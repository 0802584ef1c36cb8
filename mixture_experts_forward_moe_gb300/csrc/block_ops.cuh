// block_ops.cuh -- launchers of the operators around the routed experts (linear.cu, block_norm.cu,
// router_train.cu), called by block_api.cu with checked arguments.  Apart from common.cuh, which the
// recorded DRAM traffic of the grouped GEMMs is tied to.
#pragma once

#include "common.cuh"

namespace gb300moe {

cudaError_t launch_linear(const moe_linear_t& g, const void* x, const void* w, const void* bias,
                          const void* residual, void* out, int* status, cudaStream_t s);
int block_norm_bwd_ctas(int T);
cudaError_t launch_block_norm_fwd(const moe_block_norm_t& b, const void* branch,
                                  const void* residual, const void* gate, const void* wq,
                                  const void* wp, void* r, void* h, cudaStream_t s);
cudaError_t launch_block_norm_bwd(const moe_block_norm_t& b, const void* dr, const void* dh,
                                  const void* branch, const void* residual, const void* gate,
                                  const void* wq, const void* wp, void* dy, void* dx, void* dg,
                                  void* dwq, void* dwp, float* part, cudaStream_t s);
size_t balance_workspace_bytes(int T, int E, int n_seq);
cudaError_t launch_balance_loss(const moe_problem_t& p, int n_seq, float coeff, const float* x,
                                const int32_t* ids, const int32_t* off, float* loss,
                                int32_t* counts, int32_t* live, float* prob_sum, float* coef,
                                void* workspace, cudaStream_t s);
cudaError_t launch_router_bwd(const moe_problem_t& p, int n_seq, const float* x,
                              const int32_t* ids, const float* dw, const float* coef,
                              const int32_t* off, const float* d_loss, float* out,
                              cudaStream_t s);

}  // namespace gb300moe
