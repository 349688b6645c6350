// Launchers of the token-wise operators (norm.cu, linear_sm100.cu,
// linear_loss_sm100.cu), shared with their C ABI (tokenwise.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ulysses.h"

namespace uly {

// dst[k][c] = sum over i < parts of src[k][i][c], k < rows, in a fixed order.
uly_status fold_columns_launch(const float *src, int rows, long long parts, int cols, float *dst, cudaStream_t);

bool residual_norm_supported(int vecs);
uly_status residual_norm_launch(int32_t B, int32_t n, int32_t P, int32_t hidden, int32_t dtype, const void *x,
                                const void *h, const void *gate, int32_t gate_mode, const void *w_post,
                                const void *w_pre, float res_scale, float eps, void *r, void *u, cudaStream_t);
size_t residual_norm_bwd_workspace_bytes(int32_t B, int32_t n, int32_t hidden, int32_t dtype, int32_t gate_mode);
uly_status residual_norm_bwd_launch(int32_t B, int32_t n, int32_t P, int32_t hidden, int32_t dtype, const void *r,
                                    const void *h, const void *dr, const void *du, const void *gate,
                                    int32_t gate_mode, const void *w_post, const void *w_pre, float res_scale,
                                    float eps, void *dx, void *dh, float *dw_post, float *dw_pre, void *dgate,
                                    void *workspace, cudaStream_t);

size_t linear_workspace_bytes(int64_t tokens, int32_t in, int32_t out, int32_t activation);
uly_status linear_launch(int64_t tokens, int32_t in, int32_t out, int32_t activation, const void *x, const void *w,
                         const void *bias, const void *residual, void *y, void *pre, void *workspace, cudaStream_t);
size_t linear_bwd_workspace_bytes(int64_t tokens, int32_t in, int32_t out, int32_t activation);
uly_status linear_bwd_launch(int64_t tokens, int32_t in, int32_t out, int32_t activation, const void *x,
                             const void *w, const void *pre, const void *dy, void *dx, void *dw, int32_t dw_dtype,
                             float *dbias, void *workspace, cudaStream_t);

size_t linear_loss_workspace_bytes(int32_t P, int64_t tokens, int32_t hidden, int32_t vocab);
uly_status linear_loss_launch(int32_t P, int64_t tokens, int32_t hidden, int32_t vocab, const void *x, const void *w,
                              const int32_t *labels, int32_t ignore_index, float *shard_sum, int64_t *shard_count,
                              float *loss, void *workspace, cudaStream_t);
size_t linear_loss_bwd_workspace_bytes(int32_t P, int64_t tokens, int32_t hidden, int32_t vocab, int32_t dw_dtype,
                                       int64_t piece_tokens);
uly_status linear_loss_bwd_launch(int32_t P, int64_t tokens, int32_t hidden, int32_t vocab, const void *x,
                                  const void *w, const int32_t *labels, int32_t ignore_index, void *dx, void *dw,
                                  int32_t dw_dtype, int64_t piece_tokens, float *shard_sum, int64_t *shard_count,
                                  float *loss, void *workspace, cudaStream_t);

// loss.cu: the count of valid labels, and the fold of per-shard partials
// (psum, pcnt [P][nb]) into S_r, C_r and L.
void loss_count_launch(const int32_t *labels, long long tokens, int vocab, int ignore_index, long long *count,
                       cudaStream_t);
void loss_finalize_launch(const double *psum, const long long *pcnt, int P, int nb, float *shard_sum,
                          int64_t *shard_count, float *loss, cudaStream_t);

}  // namespace uly
