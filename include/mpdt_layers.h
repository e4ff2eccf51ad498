/*
 * mpdt_layers.h -- C ABI of the operators that a decoder layer has around its
 * linear layers and its cache, in libmpdt.so: the root-mean-square norm with the
 * residual's addition and an output in 8 bits (and the norm's gradient), new keys
 * rotated on their way into a paged cache with the queries beside them, and
 * products grouped by expert.
 *
 * The conventions of mpdt.h and mpdt_serving.h hold: device pointers, arguments
 * checked on the host before anything is launched, no allocation, no
 * synchronisation, no state between calls, stream order, mpdt_last_error();
 * strides in ELEMENTS; numbers that only the device knows are cut to the buffers.
 * A workspace may be shared by calls on one stream.
 */
#ifndef MPDT_LAYERS_H
#define MPDT_LAYERS_H

#include <stdint.h>

#include "mpdt.h"
#include "mpdt_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a norm writes. */
typedef enum {
    MPDT_NORM_PLAIN = 0,        /* y in the type of x */
    MPDT_NORM_I8_ROWS = 1,      /* INT8 and a scale a row: the X, x_scale of gemm_w8a8 */
    MPDT_NORM_E4M3_ROWS = 2,    /* E4M3 and a scale a row: the A, scale_a of gemm_fp8_rowscaled */
    MPDT_NORM_E4M3_BLOCKS = 3   /* E4M3 and a scale for 1 x 128: the A, scale_a of gemm_fp8_blockscaled */
} mpdt_norm_out;

/* Root-mean-square norm of rows [rows, dim], dim at most 32768 and rows at most
 * 4194303 (more in several calls: rows do not know of each other), of BF16, FP16 or
 * FP32 (dtype); weight [dim] in w_dtype (x's type or MPDT_F32).  For each row
 *   h = x + residual      (residual not NULL: one FP32 addition, rounded once to
 *                          x's type; else h = x)
 *   rstd = 1 / sqrt(mean(h^2) + eps)   (sum in FP64, rounded once to FP32)
 *   y = (h * rstd) * weight            (two FP32 products)
 * and y is rounded once to x's type, or taken from FP32 to 8 bits: with qmax 127
 * (INT8) or 448 (E4M3) and amax the largest |y| of the row or block,
 *   scale = amax / qmax   (FP32 division; 1 where that is 0)
 *   code = round to nearest even of y / scale, cut to [-qmax, qmax].
 * A row or block that holds a NaN has scale NaN (INT8 codes 0, E4M3 codes NaN); an
 * infinite x makes y NaN in its place and 0 elsewhere.  A row of root mean square below
 * 2.9e-39 with eps 0 has an infinite rstd: its y are infinite or NaN, and its scales one or
 * the other (the values that its codes stand for are NaN either way).
 * h is written where h_out is not NULL (it needs a residual); h_out may be exactly
 * x or residual, and with MPDT_NORM_PLAIN out may be exactly x or residual: the
 * same pointer and leading dimension.  scales: [rows] (ld_scales 1 is tight), or
 * [rows, ceil(dim / 128)] with leading dimension ld_scales.  rstd [rows] or NULL. */
mpdt_status rms_norm(int dtype, int64_t rows, int64_t dim, const void* x, int64_t ldx, const void* residual,
                     int64_t ld_res, int w_dtype, const void* weight, double eps, int norm_out, void* out,
                     int64_t ld_out, float* scales, int64_t ld_scales, void* h_out, int64_t ld_h, float* rstd,
                     void* stream);

/* The gradient of a plain rms_norm in h and weight, with grad the one in y, and
 * with the rstd [rows] that it gave:
 *   grad_h = grad_residual + rstd * (g - n * mean(g * n)),  g = grad * weight, n = h * rstd
 *   grad_weight[j] = sum over rows of grad * n      (FP32, in a fixed order)
 * grad_residual, the gradient in h_out, may be NULL (0).  grad_h may be exactly
 * grad or grad_residual.  All [rows, dim] in dtype, rows at most 2^30. */
int64_t rms_norm_backward_workspace(int64_t rows, int64_t dim);
mpdt_status rms_norm_backward(int dtype, int64_t rows, int64_t dim, const void* grad, int64_t ld_grad,
                              const void* h, int64_t ld_h, int w_dtype, const void* weight, const float* rstd,
                              const void* grad_residual, int64_t ld_gres, void* grad_h, int64_t ld_gh,
                              float* grad_weight, void* workspace, int64_t workspace_bytes, void* stream);

/* paged_kv_append with the position's rotation on the way: the first 2 * pairs
 * dimensions of every new key, and of every head of q, are turned in pairs,
 *   a' = a cos t - b sin t,  b' = b cos t + a sin t,  t = p * inv_freq[i],
 * where p = lens - (cu_q[b + 1] - row) is the token's position in its sequence and
 * pair i is (i, i + pairs), or (2 i, 2 i + 1) with interleaved.  The angle is
 * formed, and cos and sin taken of it, in FP64, each rounded once to FP32; the two
 * products are FP32 ones, and a', b' are rounded once to their type (E4M3: divided by
 * the head's scale and cut first, as in paged_kv_append).  Values are stored as they
 * are.  inv_freq [pairs] FP32, 2 * pairs at most dim.  q [tokens, heads, dim] in the
 * type of the new keys, or NULL with heads 0; q_out may be exactly q.  Rows of q that
 * belong to no sequence are not written; a token without a place in the cache is
 * dropped there, and its q turned all the same. */
mpdt_status paged_kv_append_rope(const mpdt_paged_kv* kv, const mpdt_sequences* seq, int dtype,
                                 const void* k_new, int64_t k_token, int64_t k_head,
                                 const void* v_new, int64_t v_token, int64_t v_head,
                                 const float* inv_freq, int64_t pairs, int interleaved, int64_t heads,
                                 const void* q, int64_t q_token, int64_t q_head,
                                 void* q_out, int64_t qo_token, int64_t qo_head, void* stream);

/* Products grouped by expert.  The rows offsets[e] to offsets[e + 1] of A
 * [rows, K] belong to group e (INT32 [groups + 1], ascending: a smaller one than
 * an earlier one counts as that, and all are cut to [0, rows]).  FP32 sums, rounded
 * once; rows that belong to no group are not written. */

/* D[i] = A[i] . B[e], rows i of group e.  A, B BF16 or FP16 (dtype); B[e] at
 * B + e * stride_b is K x N (ldb >= N), or with trans_b N x K (ldb >= K): the
 * other trans_b gives the gradient in A from the one in D.  D [rows, N]: FP32, or
 * the type of A with d16. */
mpdt_status gemm_grouped(int dtype, int64_t groups, int64_t rows, int64_t N, int64_t K, const void* A, int64_t lda,
                         const void* B, int64_t ldb, int64_t stride_b, int trans_b, const int32_t* offsets,
                         void* D, int64_t ldd, int d16, void* stream);

/* D[e] = sum over rows i of group e of A[i]^T G[i]: the gradient in B[e] (K x N),
 * from A [rows, K] and the gradient G [rows, N] in D.  D[e] at D + e * stride_d is
 * K x N: FP32, or the type of A with d16; 0 for a group without rows. */
mpdt_status gemm_grouped_wgrad(int dtype, int64_t groups, int64_t rows, int64_t N, int64_t K, const void* A,
                               int64_t lda, const void* G, int64_t ldg, const int32_t* offsets, void* D,
                               int64_t ldd, int64_t stride_d, int d16, void* stream);

/* The W8A8 layer of gemm_w8a8 by groups: for the rows m of group e
 *   Y[m][o] = bf16(((float(sum_k X[m][k] * W[e][o][k]) * x_scale[m]) * w_scale[e][o]) + bias[e][o])
 * each step one FP32 operation, the sum exact while K * 128^2 < 2^31.  X [rows, K]
 * INT8, x_scale [rows] FP32, W[e] at W + e * stride_w N x K INT8 (ldw >= K),
 * w_scale [groups, N] FP32 (leading dimension ld_ws), bias like it (ld_bias) or
 * NULL (no addition), Y [rows, N] BF16. */
mpdt_status gemm_grouped_w8a8(int64_t groups, int64_t rows, int64_t N, int64_t K, const int8_t* X, int64_t ldx,
                              const float* x_scale, const int8_t* W, int64_t ldw, int64_t stride_w,
                              const float* w_scale, int64_t ld_ws, const float* bias, int64_t ld_bias,
                              const int32_t* offsets, uint16_t* Y, int64_t ldy, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MPDT_LAYERS_H */
