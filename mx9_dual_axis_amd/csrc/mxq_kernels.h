// Internal launch interface between the C-ABI layer (mxq_abi.cpp) and the
// HIP kernels.  Arguments arrive already validated; each launcher enqueues
// on the given stream and returns the launch's hipError_t.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

// Fused dual-axis MXFP8 cast of a bf16 [M, N] matrix (M, N > 0, multiples
// of 128).  offs == nullptr selects the dense cast; otherwise G >= 0 group
// ends drive the uncovered-tail rule and *err (when non-null) receives the
// offset validation code.
hipError_t launch_dual_axis(const uint16_t* x, int64_t M, int64_t N, int64_t ld_x,
                            uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                            const int32_t* offs, int32_t G, int32_t* err, bool grouped,
                            bool mfma_scales, hipStream_t stream);

// Offset validation alone, for a grouped call on an empty matrix.
hipError_t launch_offs_validate(const int32_t* offs, int32_t G, int64_t M, int32_t* err,
                                hipStream_t stream);

// MX9 pack of [rows, cols] (rows, cols > 0); dtype 0 = fp32, 1 = bf16.
// Row r's blocks go to q + r * ld_q (bytes, a multiple of 16), max_exp +
// r * ld_e and prime + r * ld_pr; the three-part form passes ld_q = 16 *
// ceil(cols/16) and ld_e = ld_pr = ceil(cols/16).
hipError_t launch_mx9_pack(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x,
                           int8_t* q, int64_t ld_q, uint8_t* max_exp, int64_t ld_e, uint8_t* prime,
                           int64_t ld_pr, hipStream_t stream);

// MX9 unpack to [rows, cols] (rows, cols > 0); out_dtype 0 = fp32, 1 = bf16;
// the parts are read with the pitches of launch_mx9_pack.
hipError_t launch_mx9_unpack(const int8_t* q, int64_t ld_q, const uint8_t* max_exp, int64_t ld_e,
                             const uint8_t* prime, int64_t ld_pr, int64_t rows, int64_t cols, int out_dtype,
                             void* y, int64_t ld_y, hipStream_t stream);

// MX9 in blocks of 16 along the middle axis of a contiguous [outer, len,
// inner] array (all > 0), blocks numbered (o * inner + i) * ceil(len/16) + j.
hipError_t launch_mx9_pack_axis(const void* x, int dtype, int64_t outer, int64_t len, int64_t inner,
                                int8_t* q, uint8_t* max_exp, uint8_t* prime, hipStream_t stream);
hipError_t launch_mx9_unpack_axis(const int8_t* q, const uint8_t* max_exp, const uint8_t* prime,
                                  int64_t outer, int64_t len, int64_t inner, int out_dtype, void* y,
                                  hipStream_t stream);

// The largest grid, in threads, that the axis and record calls may launch
// for an [outer, len, inner] view with inner > 1 (tile kernels), over both
// lane layouts; the caller rejects views whose grid would not fit 32 bits.
uint64_t mx9_axis_grid_threads(int64_t outer, int64_t len, int64_t inner);

// The same blocks as 18-byte records (exponent byte, q[16], prime byte); the
// records of one (o, i) form a row, rows at a pitch of ld_p bytes.
hipError_t launch_mx9_pack_records(const void* x, int dtype, int64_t outer, int64_t len, int64_t inner,
                                   uint8_t* packed, int64_t ld_p, hipStream_t stream);
hipError_t launch_mx9_unpack_records(const uint8_t* packed, int64_t ld_p, int64_t outer, int64_t len,
                                     int64_t inner, int out_dtype, void* y, hipStream_t stream);

// MXFP8 block-scaled contraction C = A B^T (codes with the contraction
// contiguous, E8M0 scales per 32 through strided views).  mode 0: dense
// (offs == nullptr) or row groups (group g's rows use B + g * b_gs, rows past
// offs[G-1] give 0); mode 1: contraction groups (group g writes C + g * c_gs
// from its contraction range).  M, N, K are multiples of 128.
hipError_t launch_mx_gemm(const uint8_t* A, int64_t lda, const uint8_t* sA, int64_t sa_rs, int64_t sa_bs,
                          const uint8_t* B, int64_t ldb, int64_t b_gs, const uint8_t* sB, int64_t sb_rs,
                          int64_t sb_bs, int64_t sb_gs, void* C, int64_t ldc, int64_t c_gs, int64_t M, int64_t N,
                          int64_t K, const int32_t* offs, int32_t G, int mode, int out_dtype, bool mfma_scales,
                          hipStream_t stream);

hipError_t launch_scales_to_mfma(const uint8_t* s, int64_t rs, int64_t bs, int64_t rows, int64_t blocks, uint8_t* out,
                                 hipStream_t stream);
hipError_t launch_scales_from_mfma(const uint8_t* in, int64_t rows, int64_t blocks, uint8_t* s, int64_t rs, int64_t bs,
                                   hipStream_t stream);

// Expert routing of T tokens over E <= 1024 experts, k <= 16 picks each, and
// the gradient of its weights and balance loss (route.hip).  M is at least
// T k + min(E, T k) (align - 1).  workspace: route_workspace bytes, 4-byte
// aligned.  dweight and dloss may be null.
int64_t route_workspace(int64_t T, int32_t E);
hipError_t launch_route(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                        int32_t k, bool normalize, int32_t align, int64_t M, int32_t* idx, float* weight,
                        int32_t* slot, int32_t* src, int32_t* counts, int32_t* offs, int32_t* live, float* prob,
                        float* loss, void* workspace, hipStream_t stream);
hipError_t launch_route_grad(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                             int32_t k, bool normalize, const int32_t* idx, const float* weight, const float* dweight,
                             const int32_t* counts, const int32_t* live, const float* dloss, void* dlogits,
                             int64_t ld_d, hipStream_t stream);

// Token rows to and from their experts' rows (routed_rows.hip); pitches in
// elements.  launch_dispatch and launch_combine need N > 0; the others take
// rows of no elements too, and write their scales or dweight.
// launch_quantize_rows with src == nullptr sends row t to row t (M = T > 0);
// with a map M > 0, and T may be 0 (slot null then).  combine and
// combine_grad: weight null means 1; dweight may be null.  The *_blocks
// functions give the grids.
uint64_t dispatch_blocks(int64_t T, int64_t M, int64_t row_bytes);
uint64_t combine_blocks(int64_t T, int64_t row_bytes);
uint64_t token_blocks(int64_t T, int64_t M);
hipError_t launch_dispatch(const void* x, int dtype, int64_t T, int64_t N, int64_t ld_x, const int32_t* slot,
                           const int32_t* src, int32_t k, int64_t M, void* out, int64_t ld_out, hipStream_t stream);
hipError_t launch_quantize_rows(const void* x, int dtype, int64_t T, int64_t K, int64_t ld_x, const int32_t* slot,
                                const int32_t* src, int32_t k, int64_t M, int8_t* q, int64_t ld_q, float* s,
                                hipStream_t stream);
hipError_t launch_combine(const void* rows, int dtype, int64_t M, int64_t N, int64_t ld_r, const int32_t* slot,
                          const float* weight, int32_t k, int64_t T, void* y, int64_t ld_y, hipStream_t stream);
hipError_t launch_combine_grad(const void* dy, int dtype, int64_t T, int64_t N, int64_t ld_dy, const void* rows,
                               int64_t ld_r, const int32_t* slot, const float* weight, const int32_t* src, int32_t k,
                               int64_t M, void* drows, int64_t ld_d, float* dweight, hipStream_t stream);

// Product of 8-bit codes, C = A B^T with row scales (i8_gemm.hip); offs null:
// dense.  M, N > 0, K <= 131071.
uint64_t i8_gemm_threads(int64_t lda, int64_t ldb, int64_t M, int64_t N, int64_t K, bool groups, int32_t G);
hipError_t launch_i8_gemm(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs,
                          const float* sB, int64_t sb_gs, const float* bias, void* C, int64_t ldc, int64_t M,
                          int64_t N, int64_t K, const int32_t* offs, int32_t G, int out_dtype, hipStream_t stream);
// The product of activations that are quantized by the product's own kernel,
// where i8_linear_fuses says so (few rows of whole 16-code pieces, or few tiles).
bool i8_linear_fuses(const void* x, int dtype, int64_t ld_x, const int8_t* B, int64_t ldb, int64_t M, int64_t N, int64_t K);
hipError_t launch_i8_linear_fused(const void* x, int dtype, int64_t ld_x, const int8_t* B, int64_t ldb, const float* sB,
                                  const float* bias, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                  int out_dtype, hipStream_t stream);

}  // namespace mxq
