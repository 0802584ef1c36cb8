// dense_ops.cuh -- launchers of the dense feed-forward block and its training (dense.cu,
// dense_rows.cu, checkpoint.cu), called by dense_api.cu with checked arguments.
#pragma once

#include "common.cuh"

namespace gb300moe {

// Channels that share a scale of a checkpoint; a row of codes is a whole number of such groups.
constexpr int kCkptGroup = 128;
inline int64_t ckpt_groups(int64_t C) { return (C + kCkptGroup - 1) / kCkptGroup; }
inline int64_t ckpt_width(int64_t C) { return ckpt_groups(C) * kCkptGroup; }

// E4M3 codes [T, ckpt_width(C)] and f32 scales [T, ckpt_groups(C)].
struct Ckpt {
  uint8_t* codes;
  float* scales;
};
struct CkptIn {
  const uint8_t* codes;
  const float* scales;
};

// A gradient's product: out[M, N] = sum_k a(m, k) b(k, n); a [M, K], or [K, M] (tn), with rows
// a_pitch elements apart (a multiple of 8), b [K, N].
struct Product {
  bool tn;
  int M, N, K;
  const void* a;
  int64_t a_pitch;
  const void* b;
  void* out;
};
// One or two of them, of which neither reads the other's result, in one launch.
cudaError_t launch_products(int dtype, const Product* list, int n, float* parts, int* status,
                            cudaStream_t s);
// Bytes of the f32 sums that a launch leaves in the workspace where it splits K: of the same
// products (the sizes alone), and of a gated product of M x N outputs.
size_t products_split_bytes(const Product* list, int n);
size_t gated_split_bytes(int64_t M, int64_t N, int64_t K);

cudaError_t launch_gated(int dtype, int act, int T, int F, int H, const void* x, const void* w,
                         void* out, Ckpt gate, Ckpt up, float* parts, int* status, cudaStream_t s);
cudaError_t launch_gated_grad(int dtype, int act, int T, int F, int H, const void* x, const void* w,
                              const void* d_out, void* d_pre, void* out, float* parts, int* status,
                              cudaStream_t s);

// Few rows of x against 4-bit weights, or one against the 16-bit weights of a gated product
// (dense_rows.cu).
struct RowsCall {
  int T, N, K;  // gated: N outputs of 2 N weight rows
  int dtype;
  int gated;
  int act;              // moe_linear_act_t, or moe_activation_t when gated
  const void* x;
  const void* w;        // 16-bit weights [rows, K], or
  const uint8_t* codes; // E2M1 codes [rows, K/2] and
  const uint8_t* scales;  // E4M3 scales [rows, K/16]
  const float* alpha;
  const void* bias;
  const void* res;
  void* out;
  int* status;
};
cudaError_t launch_rows(const RowsCall& c, cudaStream_t s);
// The 16-bit gated product of up to kFewRows rows of x (dense_few.cu).
constexpr int kFewRows = 128;
cudaError_t launch_few(const RowsCall& c, cudaStream_t s);
// The same of 4-bit weights, for more rows of x (dense_w4.cu); x16: w4_bytes of workspace, for x in f16
// and a scale per row.
constexpr int kFewW4Rows = 16;
size_t w4_bytes(int dtype, int64_t T, int64_t K);
cudaError_t launch_w4(const RowsCall& c, void* x16, cudaStream_t s);

cudaError_t launch_checkpoint(int dtype, int T, int C, const void* x, Ckpt out, cudaStream_t s);
cudaError_t launch_restore(int dtype, int T, int C, CkptIn in, void* out, cudaStream_t s);
cudaError_t launch_gated_grad_saved(int dtype, int act, int T, int F, const void* d_out, CkptIn gate,
                                    CkptIn up, void* d_pre, void* out, cudaStream_t s);
// sum[n] = sum_t v[t, n] of [T, N] rows that lie `pitch` (a multiple of 8) elements apart; with
// `padded` rows that lie N apart, which are copied there, `pitch` apart.
cudaError_t launch_column_sum(int dtype, int T, int N, int64_t pitch, const void* v, void* padded,
                              void* sum, cudaStream_t s);
// [T, N] -> [T, pitch], anything behind N.
cudaError_t launch_pad_rows(int T, int N, int64_t pitch, const void* v, void* out, cudaStream_t s);

}  // namespace gb300moe
