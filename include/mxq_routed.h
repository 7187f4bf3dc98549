/*
 * mxq_routed.h -- C ABI of libmxq.so, second part: what stands between the
 * tokens of a routed-expert layer and the casts and contractions of mxq.h,
 * and the matrix product in 8-bit integers.
 *
 *   routing    scores to picks, counts, padded group ends and a row map;
 *              balance loss; gradient                        (mx_route*)
 *   dispatch   token rows to their experts' rows             (mx_dispatch*)
 *   product    int8 codes with a scale for each token and each output
 *              channel, dense and by expert                  (i8_*)
 *   combine    expert rows back to tokens; gradient          (mx_combine*)
 *
 * The conventions of mxq.h hold: device pointers that the caller owns, work
 * on the given stream only, arguments checked on the host before anything is
 * enqueued (a nonzero mx_status means that no output byte was written),
 * nothing allocated, kept or waited for.  Outputs must be disjoint from each
 * other and from the inputs (MX_E_OVERLAP).  Pitches and sizes are in
 * elements.  dtype is MX_DTYPE_F32 or MX_DTYPE_BF16.  The same inputs give
 * the same bits: no floating sum depends on the order in which blocks run.
 *
 * The padded buffer.  E groups of rows, one for each expert: group e holds the
 * rows of the tokens that picked e, in token order, and ends at offs[e], a
 * multiple of `align` (128 for the MXFP8 grouped calls; any size for the
 * 8-bit product).  slot[t][j] is the row of token t's j-th pick, or -1;
 * src[r] = t k + j for that row, or -1 for a row without a token.  Rows at or
 * after offs[E-1] are the tail.  Device data is not trusted: a slot outside
 * [0, M) is skipped and group ends are clamped to an ascending sequence in
 * [0, M], so that no access leaves the operands.
 */
#ifndef MXQ_ROUTED_H
#define MXQ_ROUTED_H

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows that hold any routing of T tokens to k of E experts each, groups
 * padded to `align`: T k + min(E, T k) (align - 1), rounded up to align.
 * -1 for arguments that mx_route refuses. */
int64_t mx_route_rows(int64_t T, int32_t E, int32_t k, int32_t align);

/* Bytes of mx_route's workspace (0 for a batch that one workgroup takes);
 * -1 for arguments that mx_route refuses. */
int64_t mx_route_workspace(int64_t T, int32_t E);

/*
 * mx_route -- softmax routing of T tokens over E experts.
 *
 *   logits [T, E] of dtype, row pitch ld.  valid uint8 [T] or NULL: a token
 *   with valid 0 takes no part, whatever its logits hold.  A logit of -inf
 *   bars the token from that expert; a token with no other logit takes no
 *   part.  Let p be the softmax over the experts and "live" the tokens that
 *   take part.
 *
 *   idx    int32 [T, k]  the k largest logits above -inf, descending, equal
 *                        ones lowest expert first; -1 when none is left
 *   weight f32 [T, k]    p of the pick, divided by the sum over the token's
 *                        picks when normalize != 0; 0 where idx is -1
 *   slot   int32 [T, k], src int32 [M], offs int32 [E]: the padded buffer
 *   counts int32 [E]     picks of each expert (without padding)
 *   live   int32 [1]     live tokens
 *   prob   f32 [E]       mean of p over the live tokens
 *   loss   f32 [1]       E sum_e counts[e] / (k live) prob[e]  (1 when both
 *                        are even; 0 when nothing is live)
 *
 *   A valid token with NaN or +inf among its logits is live, picks nothing,
 *   and has NaN weights; prob and loss are NaN then.
 *
 * Errors: MX_E_NULL, MX_E_DTYPE, MX_E_SHAPE (T < 0 or T k > 2^30, E outside
 * [1, 1024], k outside [1, min(E, 16)], align outside [1, 2^16], M below
 * mx_route_rows or above 2^30, workspace_bytes too small), MX_E_STRIDE
 * (ld < E), MX_E_ALIGN (a pointer not aligned to its element),
 * MX_E_OVERLAP.  T == 0 writes empty groups.  Up to 64 tokens one kernel,
 * otherwise two, or three where the blocks' counts are much to add.
 */
int mx_route(const void *logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t *valid,
             int32_t k, int32_t normalize, int32_t align, int64_t M, int32_t *idx, float *weight, int32_t *slot,
             int32_t *src, int32_t *counts, int32_t *offs, int32_t *live, float *prob, float *loss,
             void *workspace, int64_t workspace_bytes, void *stream);

/*
 * mx_route_grad -- gradient of weight and loss with respect to the logits.
 * dweight f32 [T, k] (NULL: none) is the gradient of mx_route's weight, dloss
 * f32 [1] (NULL: none) that of its loss; idx, weight, counts and live are
 * mx_route's outputs.  counts are constants, as they are in the loss; where
 * ranks share a batch, counts and live may be their sums.  dlogits
 * [T, E] of dtype, pitch ld_d; 0 for tokens that are not live and for barred
 * experts, NaN for a live token with NaN or +inf.  Errors as for mx_route.
 */
int mx_route_grad(const void *logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t *valid,
                  int32_t k, int32_t normalize, const int32_t *idx, const float *weight, const float *dweight,
                  const int32_t *counts, const int32_t *live, const float *dloss, void *dlogits, int64_t ld_d,
                  void *stream);

/*
 * mx_dispatch -- out[slot[t][j]] = x[t] for every pick; rows r with
 * src[r] < 0 are 0.  x [T, N], out [M, N] of dtype, any pitches.  Its
 * gradient is mx_combine with weight NULL.
 *
 * mx_dispatch_i8 -- the same with each row quantized: q int8 [M, K] (pitch
 * ld_q >= K), s f32 [M].  With a = max(max |x|, 127 2^-126):
 * q = round-half-even(x (127 (1 / a))), s = a / 127 (each operation rounded to
 * fp32).  A row with Inf or NaN: q = 0, s = NaN.
 *
 * i8_quantize_rows -- mx_dispatch_i8 without a map: q [T, K], s [T] (rows are
 * tokens, or the output channels of a weight).
 *
 * Errors: MX_E_NULL, MX_E_DTYPE, MX_E_SHAPE (a negative size, T k or M above
 * 2^30, rows above 2^30 elements, k outside [1, 64], a grid above 2^32
 * threads), MX_E_STRIDE (a pitch below its row, a span above 2^48 bytes),
 * MX_E_ALIGN, MX_E_OVERLAP.  Rows of no elements: mx_dispatch is a no-op,
 * the quantizing calls still write s (2^-126).
 */
int mx_dispatch(const void *x, int32_t dtype, int64_t T, int64_t N, int64_t ld_x, const int32_t *slot,
                const int32_t *src, int32_t k, int64_t M, void *out, int64_t ld_out, void *stream);
int mx_dispatch_i8(const void *x, int32_t dtype, int64_t T, int64_t K, int64_t ld_x, const int32_t *slot,
                   const int32_t *src, int32_t k, int64_t M, int8_t *q, int64_t ld_q, float *s, void *stream);
int i8_quantize_rows(const void *x, int32_t dtype, int64_t T, int64_t K, int64_t ld_x, int8_t *q, int64_t ld_q,
                     float *s, void *stream);

/*
 * i8_gemm_nt -- C[m][n] = (float(sum_k A[m][k] B[n][k]) sA[m]) sB[n]
 * (+ bias[n]): A int8 [M, K] pitch lda, B int8 [N, K] pitch ldb, sA f32 [M],
 * sB f32 [N], bias f32 [N] or NULL, C [M, N] of out_dtype, pitch ldc.  The sum
 * is exact (any codes, -128 too); its conversion and each product round to
 * fp32 (with a bias, the last product and the addition in one rounding), then
 * the result to out_dtype (nearest-even).  Any sizes, pitches and alignments of A
 * and B; 16-byte aligned rows are faster.
 *
 * i8_linear -- i8_quantize_rows of x [M, K] (of dtype, pitch ld_x) and
 * i8_gemm_nt in one call.  workspace: i8_linear_workspace(M, K) bytes,
 * 16-byte aligned.
 *
 * i8_grouped_gemm_rows -- rows offs[g-1] <= m < offs[g] (offs[-1] = 0) take
 * B + g b_gs and sB + g sb_gs; rows from offs[G-1] on give 0.  Groups of any
 * size, empty ones too.
 *
 * Errors: MX_E_NULL, MX_E_DTYPE, MX_E_SHAPE (a negative size, M or N above
 * 2^30, K above 131071, G < 1, a grid above 2^32 threads, workspace too
 * small), MX_E_STRIDE (a pitch below its row, a negative group stride, a span
 * above 2^48 bytes), MX_E_ALIGN (a scale, bias, x or C not aligned to its
 * element, the workspace not to 16 bytes), MX_E_OVERLAP (C or the workspace
 * with anything else).  M == 0 or N == 0 is a no-op; K == 0 gives the bias.
 */
int i8_gemm_nt(const int8_t *A, int64_t lda, const float *sA, const int8_t *B, int64_t ldb, const float *sB,
               const float *bias, int64_t M, int64_t N, int64_t K, void *C, int64_t ldc, int32_t out_dtype,
               void *stream);
int64_t i8_linear_workspace(int64_t M, int64_t K);
int i8_linear(const void *x, int32_t dtype, int64_t ld_x, const int8_t *B, int64_t ldb, const float *sB,
              const float *bias, int64_t M, int64_t N, int64_t K, void *C, int64_t ldc, int32_t out_dtype,
              void *workspace, int64_t workspace_bytes, void *stream);
int i8_grouped_gemm_rows(const int8_t *A, int64_t lda, const float *sA, const int8_t *B, int64_t ldb, int64_t b_gs,
                         const float *sB, int64_t sb_gs, const int32_t *offs, int32_t G, int64_t M, int64_t N,
                         int64_t K, void *C, int64_t ldc, int32_t out_dtype, void *stream);

/*
 * mx_combine -- y[t] = sum_j weight[t][j] rows[slot[t][j]] over the picks with
 * a slot (0 when there is none), fp32 in the order of j, rounded once.  rows
 * [M, N], y [T, N] of dtype; weight f32 [T, k], or NULL for 1.
 *
 * mx_combine_grad -- drows[slot[t][j]] = weight[t][j] dy[t], rows with
 * src[r] < 0 are 0; dweight[t][j] = <dy[t], rows[slot[t][j]]> in fp32, 0 for a
 * pick without a slot.  dweight NULL: not computed (rows may be NULL then).
 *
 * Errors as for mx_dispatch.  N == 0: mx_combine is a no-op, mx_combine_grad
 * still writes dweight (0).
 */
int mx_combine(const void *rows, int32_t dtype, int64_t M, int64_t N, int64_t ld_r, const int32_t *slot,
               const float *weight, int32_t k, int64_t T, void *y, int64_t ld_y, void *stream);
int mx_combine_grad(const void *dy, int32_t dtype, int64_t T, int64_t N, int64_t ld_dy, const void *rows,
                    int64_t ld_r, const int32_t *slot, const float *weight, const int32_t *src, int32_t k, int64_t M,
                    void *drows, int64_t ld_d, float *dweight, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_ROUTED_H */
