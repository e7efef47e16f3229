// Host-side interfaces of the many-token and 8-bit kernels.
#pragma once

#include "internal.h"

namespace smoe {

// Many tokens (tokens.cu): the k largest logits of T rows and their gradient.
cudaError_t launch_topk_rows(const float *logits, int T, int n, int ld, int k, int *idx, float *w, cudaStream_t stream);
cudaError_t launch_topk_rows_grad(const int *idx, const float *w, const float *dw, int T, int n, int k, float *dl,
                                  cudaStream_t stream);
// The stable sort of R = T k slots by expert, the gather of the tokens' rows
// into that order, their weighted sum back (w null: plain sum) and its
// gradient.  dtype: SMOE_F32 or SMOE_BF16.
size_t dispatch_workspace(int T, int k, int n);
cudaError_t launch_dispatch(const int *top_idx, int tokens, int k, int n, const void *x, int dtype, int d, int *offsets,
                            int *order, int *place, void *xs, void *workspace, cudaStream_t stream);
cudaError_t launch_sum_tokens(const void *ys, int dtype, const int *place, const float *w, int tokens, int k, int d,
                              void *out, cudaStream_t stream);
cudaError_t launch_combine_tokens_grad(const void *d_out, const void *ys, int dtype, const int *place, const float *w,
                                       int tokens, int k, int d, void *d_ys, float *d_w, cudaStream_t stream);

// n 32-bit words set to zero.
cudaError_t launch_zero_words(int *p, int n, cudaStream_t stream);

// 8-bit rows and products (q8.cu).  offsets null: one matrix (n == 1);
// order null: row r of the batch is row r of xq.
cudaError_t launch_quantize_rows(const void *x, int dtype, bool act, int rows, int cols, int8_t *q, float *scales,
                                 cudaStream_t stream);
size_t q8_workspace(int nsrc, int R, int n, int K);
cudaError_t launch_q8(const int8_t *xq, const float *xs, int nsrc, const int *order, int k, const int *offsets, int R,
                      int n, const int8_t *wq, const float *ws, int N, int K, void *y, int dtype, void *workspace,
                      cudaStream_t stream);

}  // namespace smoe
