/*
 * mxq_act.h -- C ABI of libmxq.so, third part: the products of mxq.h (MXFP8)
 * and mxq_routed.h (8-bit integers) with bias, activation and residual applied
 * to their sums before the only rounding, and the gradient of that epilogue.
 *
 *   x[m][n] = sum + bias[n]
 *   y[m][n] = act(x[m][n])               (+ residual[m][n])      gated == 0
 *   y[m][n] = act(x[m][n]) x[m][n + N]   (+ residual[m][n])      gated != 0
 *
 * N counts results.  B (and its scales, bias, and the values kept) has W
 * channels: N, or 2 N where gated, the gates first.  Everything up to y is
 * fp32; y, and x where it is kept, are rounded once to the output's type
 * (nearest-even).
 *
 * act: MX_ACT_NONE x; MX_ACT_RELU max(x, 0); MX_ACT_SILU x / (1 + e^-x);
 * MX_ACT_GELU x Phi(x) with the normal distribution's Phi; MX_ACT_GELU_TANH
 * x / (1 + e^(-2 sqrt(2/pi) (x + 0.044715 x^3))).  A NaN gives NaN.  In fp32
 * whatever y's type is (a bf16 y is the fp32 one, rounded): SILU and GELU within
 * 2^-20 of the value; GELU_TANH, whose argument t = 2 sqrt(2/pi) (x + 0.044715
 * x^3) is rounded on the way, within 2^-20 + 4 |t| 2^-24; values below 2^-118 may
 * be 0.
 *
 * The conventions of mxq.h and mxq_routed.h hold.  bias f32 [W] or NULL; by
 * expert, group g's is bias + g * bias_gs.  residual [M, N] of the output's
 * type, pitch ld_res, or NULL; it may be C itself (same pointer and pitch:
 * y is added to it in place), else it must not overlap C.  pre [M, W] of the
 * output's type, pitch ld_pre, or NULL: receives x.
 */
#ifndef MXQ_ACT_H
#define MXQ_ACT_H

#include "mxq_routed.h"

#ifdef __cplusplus
extern "C" {
#endif

enum mx_act {
    MX_ACT_NONE = 0,
    MX_ACT_RELU = 1,
    MX_ACT_SILU = 2,
    MX_ACT_GELU = 3,
    MX_ACT_GELU_TANH = 4
};

/*
 * i8_gemm_nt_act, i8_linear_act, i8_grouped_gemm_rows_act -- i8_gemm_nt,
 * i8_linear and i8_grouped_gemm_rows with the epilogue: B int8 [W, K], sB [W].
 * Rows from offs[G-1] on give 0.  Errors as of those calls, plus MX_E_MODE
 * (act), MX_E_STRIDE (ld_res below N, a negative bias_gs), MX_E_ALIGN (bias or
 * residual not aligned to its element).  i8_linear_act takes
 * i8_linear_workspace(M, K) bytes.
 */
int i8_gemm_nt_act(const int8_t *A, int64_t lda, const float *sA, const int8_t *B, int64_t ldb, const float *sB,
                   int64_t M, int64_t N, int64_t K, int32_t act, int32_t gated, const float *bias,
                   const void *residual, int64_t ld_res, void *C, int64_t ldc, int32_t out_dtype, void *stream);
int i8_linear_act(const void *x, int32_t dtype, int64_t ld_x, const int8_t *B, int64_t ldb, const float *sB,
                  int64_t M, int64_t N, int64_t K, int32_t act, int32_t gated, const float *bias,
                  const void *residual, int64_t ld_res, void *C, int64_t ldc, int32_t out_dtype, void *workspace,
                  int64_t workspace_bytes, void *stream);
int i8_grouped_gemm_rows_act(const int8_t *A, int64_t lda, const float *sA, const int8_t *B, int64_t ldb,
                             int64_t b_gs, const float *sB, int64_t sb_gs, const int32_t *offs, int32_t G,
                             int64_t M, int64_t N, int64_t K, int32_t act, int32_t gated, const float *bias,
                             int64_t bias_gs, void *C, int64_t ldc, int32_t out_dtype, void *stream);

/*
 * mx_gemm_nt_act, mx_grouped_gemm_rows_act -- mx_gemm_nt and
 * mx_grouped_gemm_rows with the epilogue: B [W, K], sB its scales; N a multiple
 * of 128.  The sums are the matrix cores' and, as theirs, differ from exact ones
 * by more than fp32's roundings.  Their order depends on M, W, K, the groups and
 * the layout of the scales: the same call gives the same bits, but a row's bits,
 * of y and of pre, may differ between calls of other sizes, and from
 * mx_gemm_nt's.  (The 8-bit sums are exact: a row's bits there are its own.)
 * The tail (rows from offs[G-1] on) gives 0 in C and in pre.  The
 * _mfma forms take both operands' scales in the matrix-core layout.  Errors as
 * of those calls, plus those above, MX_E_STRIDE for ld_pre below W and
 * MX_E_OVERLAP for pre with anything.  The pipelined kernel needs the scales
 * as there, and takes any C, residual and pre.
 */
int mx_gemm_nt_act(const uint8_t *A, int64_t lda, const uint8_t *sA, int64_t sa_rs, int64_t sa_bs, const uint8_t *B,
                   int64_t ldb, const uint8_t *sB, int64_t sb_rs, int64_t sb_bs, int64_t M, int64_t N, int64_t K,
                   int32_t act, int32_t gated, const float *bias, const void *residual, int64_t ld_res, void *C,
                   int64_t ldc, void *pre, int64_t ld_pre, int32_t out_dtype, void *stream);
int mx_gemm_nt_act_mfma(const uint8_t *A, int64_t lda, const uint8_t *sA, const uint8_t *B, int64_t ldb,
                        const uint8_t *sB, int64_t M, int64_t N, int64_t K, int32_t act, int32_t gated,
                        const float *bias, const void *residual, int64_t ld_res, void *C, int64_t ldc, void *pre,
                        int64_t ld_pre, int32_t out_dtype, void *stream);
int mx_grouped_gemm_rows_act(const uint8_t *A, int64_t lda, const uint8_t *sA, int64_t sa_rs, int64_t sa_bs,
                             const uint8_t *B, int64_t ldb, int64_t b_gs, const uint8_t *sB, int64_t sb_rs,
                             int64_t sb_bs, int64_t sb_gs, const int32_t *offs, int32_t G, int64_t M, int64_t N,
                             int64_t K, int32_t act, int32_t gated, const float *bias, int64_t bias_gs, void *C,
                             int64_t ldc, void *pre, int64_t ld_pre, int32_t out_dtype, void *stream);
int mx_grouped_gemm_rows_act_mfma(const uint8_t *A, int64_t lda, const uint8_t *sA, const uint8_t *B, int64_t ldb,
                                  int64_t b_gs, const uint8_t *sB, int64_t sb_gs, const int32_t *offs, int32_t G,
                                  int64_t M, int64_t N, int64_t K, int32_t act, int32_t gated, const float *bias,
                                  int64_t bias_gs, void *C, int64_t ldc, void *pre, int64_t ld_pre,
                                  int32_t out_dtype, void *stream);

/*
 * mx_act_grad -- the gradient of the epilogue: dy [M, N] and pre [M, W] of
 * dtype to dpre [M, W] of dtype,
 *
 *   dpre[n] = dy[n] act'(pre[n])                             gated == 0
 *   dpre[n] = dy[n] act'(pre[n]) pre[n + N],
 *   dpre[n + N] = dy[n] act(pre[n])                          gated != 0
 *
 * and, where dbias is not NULL, the sums of the unrounded dpre over all rows
 * (offs NULL: dbias f32 [W]) or over each group's rows offs[g-1] <= m <
 * offs[g] (dbias f32 [G, W]; groups of any size, empty ones give 0), in a
 * fixed order.  Rows from offs[G-1] on give 0 and are not read.  The
 * residual's gradient is dy.  act'(0) of MX_ACT_RELU is 0.  Infinite values of
 * pre have the slope's limit there.  Slopes p + x p' (p what act(x) multiplies x
 * by) are as accurate as the values, relative to |p| + |x p'|.
 *
 * workspace: mx_act_grad_workspace bytes, 4-byte aligned, where dbias is wanted
 * (-1 for arguments that mx_act_grad refuses).  Errors: MX_E_NULL, MX_E_DTYPE,
 * MX_E_MODE, MX_E_SHAPE (a negative size, M or N above 2^30, G outside [1,
 * 65535] with offs, more than 2^32 threads, N of more than 65535 blocks of 512
 * bytes, workspace too small), MX_E_STRIDE, MX_E_ALIGN, MX_E_OVERLAP (dpre may
 * not be pre or dy).  N == 0 is a no-op; M == 0 writes dbias (0).
 */
int64_t mx_act_grad_workspace(int64_t M, int64_t N, int32_t dtype, int32_t gated, int32_t groups);
int mx_act_grad(const void *dy, int64_t ld_dy, const void *pre, int64_t ld_pre, int32_t dtype, int64_t M, int64_t N,
                int32_t act, int32_t gated, const int32_t *offs, int32_t G, void *dpre, int64_t ld_d, float *dbias,
                void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_ACT_H */
