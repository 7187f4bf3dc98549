// act_abi.cpp -- the C ABI declared in include/mxq_act.h.
//
// As in mxq_abi.cpp: arguments are checked on the host, in the order the
// header lists the errors, before anything is enqueued.
#include "../../include/mxq_act.h"

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mxq_host.h"
#include "mxq_kernels.h"

namespace {

bool act_ok(int32_t act) { return act >= MX_ACT_NONE && act <= MX_ACT_GELU_TANH; }

// What the epilogue adds to a product's arguments.
struct Extra {
    int32_t act, gated;
    const float* bias;
    int64_t bias_gs;
    const void* residual;
    int64_t ld_res;
    void* pre;
    int64_t ld_pre;

    mxq::Epilogue at(int64_t N) const { return {act, bias, bias_gs, gated ? N : 0, residual, ld_res, pre, ld_pre}; }
};

// Its checks, after the product's own.  C first among the spans, then pre; the
// residual may be C itself.  Returns how many spans there are in *n.
int check_extra(const Extra& x, int64_t M, int64_t N, int32_t G, const void* C, int64_t ldc, int32_t out_dtype, Span* sp,
                int* n) {
    if (!act_ok(x.act)) return MX_E_MODE;
    const int64_t esz = elem(out_dtype), W = x.gated ? 2 * N : N;
    const uint64_t cb = matrix_bytes(M, N, ldc, esz), rb = x.residual ? matrix_bytes(M, N, x.ld_res, esz) : 0;
    const uint64_t pb = x.pre ? matrix_bytes(M, W, x.ld_pre, esz) : 0, bg = matrix_bytes(G, 1, x.bias_gs, 4);
    if ((x.residual && x.ld_res < N) || (x.pre && x.ld_pre < W) || x.bias_gs < 0 || cb == kTooLarge || rb == kTooLarge ||
        pb == kTooLarge || bg == kTooLarge)
        return MX_E_STRIDE;
    if (!aligned(x.bias, 4) || !aligned(x.residual, uintptr_t(esz)) || !aligned(x.pre, uintptr_t(esz))) return MX_E_ALIGN;
    const bool in_place = x.residual == C && x.ld_res == ldc;
    sp[0] = {addr(C), cb};
    sp[1] = {addr(x.pre), pb};
    sp[2] = {addr(x.residual), in_place ? 0 : rb};
    sp[3] = {addr(x.bias), x.bias && W > 0 ? uint64_t(W) * 4 - 4 + bg : 0};
    *n = 4;
    return MX_OK;
}

// ---- 8-bit integers ----

// Everything of a product but its left operand, whose rows are lda apart.
int check_i8(int64_t lda, const int8_t* B, int64_t ldb, int64_t b_gs, const float* sB, int64_t sb_gs, const int32_t* offs,
             int32_t G, bool groups, int64_t M, int64_t N, int64_t K, const Extra& x, const void* C, int64_t ldc,
             int32_t out_dtype, Span* sp, int* n) {
    const bool some = M > 0 && N > 0;
    if (some && ((!B && K > 0) || !sB || !C || (groups && !offs))) return MX_E_NULL;
    if (!dtype_ok(out_dtype)) return MX_E_DTYPE;
    if (M < 0 || N < 0 || K < 0 || M > kMaxRows || N > kMaxRows || K > kMaxCodes || G < 1) return MX_E_SHAPE;
    const int64_t W = x.gated ? 2 * N : N;
    if (mxq::i8_gemm_threads(lda, ldb, M, W, K, groups, G) > kMaxThreads) return MX_E_SHAPE;
    if (ldb < K || ldc < N || b_gs < 0 || sb_gs < 0) return MX_E_STRIDE;
    const uint64_t bb = matrix_bytes(W, K, ldb, 1);
    const uint64_t bg = matrix_bytes(G, 1, b_gs, 1), sg = matrix_bytes(G, 1, sb_gs, 4);
    if (bb == kTooLarge || bg == kTooLarge || sg == kTooLarge || bb + bg > kMaxSpan) return MX_E_STRIDE;
    if (!aligned(sB, 4) || !aligned(offs, 4) || !aligned(C, uintptr_t(elem(out_dtype)))) return MX_E_ALIGN;
    const int rc = check_extra(x, M, N, G, C, ldc, out_dtype, sp, n);
    if (rc != MX_OK) return rc;
    sp[(*n)++] = {addr(B), bb ? bb - 1 + bg : 0};
    sp[(*n)++] = {addr(sB), W > 0 ? uint64_t(W) * 4 - 4 + sg : 0};
    sp[(*n)++] = {addr(offs), offs ? uint64_t(G) * 4 : 0};
    return MX_OK;
}

int i8_call(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs, const float* sB,
            int64_t sb_gs, const int32_t* offs, int32_t G, bool groups, int64_t M, int64_t N, int64_t K, const Extra& x,
            void* C, int64_t ldc, int32_t out_dtype, void* stream) {
    if (M > 0 && N > 0 && ((!A && K > 0) || !sA)) return MX_E_NULL;
    Span sp[10];
    int n = 0;
    const int rc = check_i8(lda, B, ldb, b_gs, sB, sb_gs, offs, G, groups, M, N, K, x, C, ldc, out_dtype, sp, &n);
    if (rc != MX_OK) return rc;
    const uint64_t ab = matrix_bytes(M, K, lda, 1);
    if (lda < K || ab == kTooLarge) return MX_E_STRIDE;
    if (!aligned(sA, 4)) return MX_E_ALIGN;
    sp[n++] = {addr(A), ab};
    sp[n++] = {addr(sA), uint64_t(M) * 4};
    if (outputs_clash(sp, 2, n)) return MX_E_OVERLAP;
    if (M == 0 || N == 0) return MX_OK;
    const auto launch = x.gated ? mxq::launch_i8_gemm_act_gated : mxq::launch_i8_gemm_act;
    return status(launch(A, lda, sA, B, ldb, b_gs, sB, sb_gs, x.at(N), C, ldc, M, N, K, groups ? offs : nullptr,
                         groups ? G : 0, out_dtype, hip(stream)));
}

// ---- MXFP8 ----

int mx_call(const uint8_t* A, int64_t lda, const uint8_t* sA, int64_t sa_rs, int64_t sa_bs, const uint8_t* B, int64_t ldb,
            int64_t b_gs, const uint8_t* sB, int64_t sb_rs, int64_t sb_bs, int64_t sb_gs, const int32_t* offs, int32_t G,
            bool groups, int64_t M, int64_t N, int64_t K, const Extra& x, void* C, int64_t ldc, int32_t out_dtype,
            bool mfma, void* stream) {
    if (N < 0 || N > kMaxGemm) return MX_E_SHAPE;
    const int64_t W = x.gated ? 2 * N : N;
    // The products' own checks, of W channels: a pitch of C that holds its N results
    // stands for one that holds W, and an N that is not whole tiles is refused as
    // such a W.
    int rc = check_gemm(A, lda, sA, sa_rs, sa_bs, B, ldb, sB, sb_rs, sb_bs, M, N % 128 == 0 ? W : 1, K, C,
                        ldc < N ? -1 : ldc < W ? W : ldc, out_dtype, mfma);
    if (rc != MX_OK) return rc;
    if (groups && (G < 1 || G > (1 << 20))) return MX_E_SHAPE;
    if (!gemm_grid_fits(M, W, G, groups, false)) return MX_E_SHAPE;     // (smaller tiles are taken where they are few)
    if (groups && !offs) return MX_E_NULL;
    if (!aligned(offs, 4)) return MX_E_ALIGN;
    if (b_gs < 0 || sb_gs < 0) return MX_E_STRIDE;
    Span sp[9];
    int n = 0;
    rc = check_extra(x, M, N, G, C, ldc, out_dtype, sp, &n);
    if (rc != MX_OK) return rc;
    sp[n++] = {addr(A), matrix_bytes(M, K, lda, 1)};
    sp[n++] = {addr(B), uint64_t(G - 1) * uint64_t(b_gs) + matrix_bytes(W, K, ldb, 1)};
    sp[n++] = {addr(sA), scale_bytes(mfma, M, K, sa_rs, sa_bs)};
    sp[n++] = {addr(sB), uint64_t(G - 1) * uint64_t(sb_gs) + scale_bytes(mfma, W, K, sb_rs, sb_bs)};
    sp[n++] = {addr(offs), offs ? uint64_t(G) * 4 : 0};
    if (outputs_clash(sp, 2, n)) return MX_E_OVERLAP;
    if (M == 0 || N == 0) return MX_OK;
    const auto launch = x.gated ? mxq::launch_mx_act_gated : mxq::launch_mx_act;
    return status(launch(A, lda, sA, sa_rs, sa_bs, B, ldb, b_gs, sB, sb_rs, sb_bs, sb_gs, x.at(N), C, ldc, M, N, K,
                         groups ? offs : nullptr, G, out_dtype, mfma, hip(stream)));
}

constexpr int32_t kMaxGradGroups = 65535;      // a grid's second extent

bool grad_shape(int64_t M, int64_t N, int32_t dtype, bool groups, int32_t G) {
    return M >= 0 && N >= 0 && M <= kMaxRows && N <= kMaxRows && G >= 1 && G <= kMaxGradGroups &&
           (N * elem(dtype) + 511) / 512 <= 65535 &&
           (M == 0 || N == 0 || mxq::act_grad_threads(M, N, dtype, groups, G) <= kMaxThreads);
}

}  // namespace

extern "C" {

int i8_gemm_nt_act(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, const float* sB, int64_t M,
                   int64_t N, int64_t K, int32_t act, int32_t gated, const float* bias, const void* residual,
                   int64_t ld_res, void* C, int64_t ldc, int32_t out_dtype, void* stream) {
    return i8_call(A, lda, sA, B, ldb, 0, sB, 0, nullptr, 1, false, M, N, K,
                   {act, gated, bias, 0, residual, ld_res, nullptr, 0}, C, ldc, out_dtype, stream);
}

int i8_grouped_gemm_rows_act(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs,
                             const float* sB, int64_t sb_gs, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                             int64_t K, int32_t act, int32_t gated, const float* bias, int64_t bias_gs, void* C,
                             int64_t ldc, int32_t out_dtype, void* stream) {
    return i8_call(A, lda, sA, B, ldb, b_gs, sB, sb_gs, offs, G, true, M, N, K,
                   {act, gated, bias, bias_gs, nullptr, 0, nullptr, 0}, C, ldc, out_dtype, stream);
}

int i8_linear_act(const void* x, int32_t dtype, int64_t ld_x, const int8_t* B, int64_t ldb, const float* sB, int64_t M,
                  int64_t N, int64_t K, int32_t act, int32_t gated, const float* bias, const void* residual,
                  int64_t ld_res, void* C, int64_t ldc, int32_t out_dtype, void* workspace, int64_t workspace_bytes,
                  void* stream) {
    const bool some = M > 0 && N > 0;
    if (some && ((!x && K > 0) || !workspace)) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    const Extra e{act, gated, bias, 0, residual, ld_res, nullptr, 0};
    const int64_t ld_q = (K + 15) / 16 * 16;
    Span sp[10];
    int n = 0;
    const int rc = check_i8(ld_q, B, ldb, 0, sB, 0, nullptr, 1, false, M, N, K, e, C, ldc, out_dtype, sp, &n);
    if (rc != MX_OK) return rc;
    const int64_t need = i8_linear_workspace(M, K);
    if (some && workspace_bytes < need) return MX_E_SHAPE;
    if (mxq::token_blocks(M, M) * 256 > kMaxThreads) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t xb = matrix_bytes(M, K, ld_x, esz);
    if (ld_x < K || xb == kTooLarge) return MX_E_STRIDE;
    if (!aligned(x, uintptr_t(esz)) || !aligned(workspace, 16)) return MX_E_ALIGN;
    sp[1] = {addr(workspace), some ? uint64_t(need) : 0};        // in the place of pre: C and the workspace are the outputs
    sp[n++] = {addr(x), xb};
    if (outputs_clash(sp, 2, n)) return MX_E_OVERLAP;
    if (some && residual && overlap(sp[1], {addr(residual), matrix_bytes(M, N, ld_res, elem(out_dtype))})) return MX_E_OVERLAP;
    if (!some) return MX_OK;
    const int64_t W = gated ? 2 * N : N;
    if (mxq::i8_linear_fuses(x, dtype, ld_x, B, ldb, M, W, K)) {
        const auto launch = gated ? mxq::launch_i8_linear_fused_act_gated : mxq::launch_i8_linear_fused_act;
        return status(launch(x, dtype, ld_x, B, ldb, sB, e.at(N), C, ldc, M, N, K, out_dtype, hip(stream)));
    }
    int8_t* q = static_cast<int8_t*>(workspace);
    float* s = reinterpret_cast<float*>(q + M * ld_q);
    hipError_t err = mxq::launch_quantize_rows(x, dtype, M, K, ld_x, nullptr, nullptr, 1, M, q, ld_q, s, hip(stream));
    if (err != hipSuccess) return MX_E_LAUNCH;
    const auto launch = gated ? mxq::launch_i8_gemm_act_gated : mxq::launch_i8_gemm_act;
    return status(launch(q, ld_q, s, B, ldb, 0, sB, 0, e.at(N), C, ldc, M, N, K, nullptr, 0, out_dtype, hip(stream)));
}

int mx_gemm_nt_act(const uint8_t* A, int64_t lda, const uint8_t* sA, int64_t sa_rs, int64_t sa_bs, const uint8_t* B,
                   int64_t ldb, const uint8_t* sB, int64_t sb_rs, int64_t sb_bs, int64_t M, int64_t N, int64_t K,
                   int32_t act, int32_t gated, const float* bias, const void* residual, int64_t ld_res, void* C,
                   int64_t ldc, void* pre, int64_t ld_pre, int32_t out_dtype, void* stream) {
    return mx_call(A, lda, sA, sa_rs, sa_bs, B, ldb, 0, sB, sb_rs, sb_bs, 0, nullptr, 1, false, M, N, K,
                   {act, gated, bias, 0, residual, ld_res, pre, ld_pre}, C, ldc, out_dtype, false, stream);
}

int mx_gemm_nt_act_mfma(const uint8_t* A, int64_t lda, const uint8_t* sA, const uint8_t* B, int64_t ldb, const uint8_t* sB,
                        int64_t M, int64_t N, int64_t K, int32_t act, int32_t gated, const float* bias,
                        const void* residual, int64_t ld_res, void* C, int64_t ldc, void* pre, int64_t ld_pre,
                        int32_t out_dtype, void* stream) {
    return mx_call(A, lda, sA, 0, 0, B, ldb, 0, sB, 0, 0, 0, nullptr, 1, false, M, N, K,
                   {act, gated, bias, 0, residual, ld_res, pre, ld_pre}, C, ldc, out_dtype, true, stream);
}

int mx_grouped_gemm_rows_act(const uint8_t* A, int64_t lda, const uint8_t* sA, int64_t sa_rs, int64_t sa_bs,
                             const uint8_t* B, int64_t ldb, int64_t b_gs, const uint8_t* sB, int64_t sb_rs, int64_t sb_bs,
                             int64_t sb_gs, const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K, int32_t act,
                             int32_t gated, const float* bias, int64_t bias_gs, void* C, int64_t ldc, void* pre,
                             int64_t ld_pre, int32_t out_dtype, void* stream) {
    return mx_call(A, lda, sA, sa_rs, sa_bs, B, ldb, b_gs, sB, sb_rs, sb_bs, sb_gs, offs, G, true, M, N, K,
                   {act, gated, bias, bias_gs, nullptr, 0, pre, ld_pre}, C, ldc, out_dtype, false, stream);
}

int mx_grouped_gemm_rows_act_mfma(const uint8_t* A, int64_t lda, const uint8_t* sA, const uint8_t* B, int64_t ldb,
                                  int64_t b_gs, const uint8_t* sB, int64_t sb_gs, const int32_t* offs, int32_t G,
                                  int64_t M, int64_t N, int64_t K, int32_t act, int32_t gated, const float* bias,
                                  int64_t bias_gs, void* C, int64_t ldc, void* pre, int64_t ld_pre, int32_t out_dtype,
                                  void* stream) {
    return mx_call(A, lda, sA, 0, 0, B, ldb, b_gs, sB, 0, 0, sb_gs, offs, G, true, M, N, K,
                   {act, gated, bias, bias_gs, nullptr, 0, pre, ld_pre}, C, ldc, out_dtype, true, stream);
}

int64_t mx_act_grad_workspace(int64_t M, int64_t N, int32_t dtype, int32_t gated, int32_t groups) {
    if (!dtype_ok(dtype) || groups < 0 || !grad_shape(M, N, dtype, groups > 0, groups > 0 ? groups : 1)) return -1;
    return mxq::act_grad_workspace(M, N, dtype, gated != 0, groups > 0, groups);
}

int mx_act_grad(const void* dy, int64_t ld_dy, const void* pre, int64_t ld_pre, int32_t dtype, int64_t M, int64_t N,
                int32_t act, int32_t gated, const int32_t* offs, int32_t G, void* dpre, int64_t ld_d, float* dbias,
                void* workspace, int64_t workspace_bytes, void* stream) {
    if (M > 0 && N > 0 && (!dy || !pre || !dpre)) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    if (!act_ok(act)) return MX_E_MODE;
    const bool groups = offs != nullptr;
    if (!grad_shape(M, N, dtype, groups, groups ? G : 1)) return MX_E_SHAPE;
    const int64_t esz = elem(dtype), W = gated ? 2 * N : N;
    const int64_t need = dbias ? mxq::act_grad_workspace(M, N, dtype, gated != 0, groups, G) : 0;
    if (need > 0 && !workspace) return MX_E_NULL;
    if (need > 0 && workspace_bytes < need) return MX_E_SHAPE;
    const uint64_t yb = matrix_bytes(M, N, ld_dy, esz), xb = matrix_bytes(M, W, ld_pre, esz), db = matrix_bytes(M, W, ld_d, esz);
    if (ld_dy < N || ld_pre < W || ld_d < W || yb == kTooLarge || xb == kTooLarge || db == kTooLarge) return MX_E_STRIDE;
    if (!aligned(dy, uintptr_t(esz)) || !aligned(pre, uintptr_t(esz)) || !aligned(dpre, uintptr_t(esz)) ||
        !aligned(offs, 4) || !aligned(dbias, 4) || !aligned(workspace, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(dpre), db}, {addr(dbias), dbias ? uint64_t(groups ? G : 1) * uint64_t(W) * 4 : 0},
                       {addr(workspace), uint64_t(need)}, {addr(dy), yb}, {addr(pre), xb},
                       {addr(offs), groups ? uint64_t(G) * 4 : 0}};
    if (outputs_clash(sp, 3, 6)) return MX_E_OVERLAP;
    if (N == 0 || (M == 0 && !dbias)) return MX_OK;
    return status(mxq::launch_act_grad(dy, ld_dy, pre, ld_pre, dtype, M, N, act, gated != 0, offs, G, dpre, ld_d, dbias,
                                       static_cast<float*>(workspace), hip(stream)));
}

}  // extern "C"
