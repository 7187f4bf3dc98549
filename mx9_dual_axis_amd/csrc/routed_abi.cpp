// routed_abi.cpp -- the C ABI declared in include/mxq_routed.h.
//
// As in mxq_abi.cpp: arguments are checked on the host, in the order the
// header lists the errors, before anything is enqueued.
#include "../../include/mxq_routed.h"

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mxq_host.h"
#include "mxq_kernels.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxCodes = 131071;     // 131071 * 128 * 128 < 2^31

hipStream_t hip(void* stream) { return static_cast<hipStream_t>(stream); }
int status(hipError_t e) { return e == hipSuccess ? MX_OK : MX_E_LAUNCH; }

bool dtype_ok(int32_t d) { return d == MX_DTYPE_F32 || d == MX_DTYPE_BF16; }
int64_t elem(int32_t d) { return d == MX_DTYPE_F32 ? 4 : 2; }

// The first n_out spans are outputs: disjoint from each other and from the
// inputs that follow; inputs may overlap each other.
bool outputs_clash(const Span* s, int n_out, int n) {
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(s[i], s[j])) return true;
    return false;
}

bool route_shape(int64_t T, int32_t E, int32_t k) {
    return T >= 0 && E >= 1 && E <= 1024 && k >= 1 && k <= 16 && k <= E && T <= kMaxRows / k;
}

// Shapes and the map shared by dispatch and combine.
int check_map(int64_t T, int64_t N, int32_t k, int64_t M) {
    if (T < 0 || N < 0 || M < 0 || k < 1 || k > 64 || N > kMaxRows || M > kMaxRows || T > kMaxRows / k)
        return MX_E_SHAPE;
    return MX_OK;
}

int quantize(const void* x, int32_t dtype, int64_t T, int64_t K, int64_t ld_x, const int32_t* slot,
             const int32_t* src, int32_t k, int64_t M, int8_t* q, int64_t ld_q, float* s, bool mapped, void* stream) {
    const bool some = M > 0;
    if (T > 0 && ((!x && K > 0) || (mapped && !slot))) return MX_E_NULL;
    if (some && ((!q && K > 0) || !s || (mapped && !src))) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    int rc = check_map(T, K, k, M);
    if (rc != MX_OK) return rc;
    if (mxq::token_blocks(T, M) * 256 > kMaxThreads) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t xb = matrix_bytes(T, K, ld_x, esz), qb = matrix_bytes(M, K, ld_q, 1);
    if (ld_x < K || ld_q < K || xb == kTooLarge || qb == kTooLarge) return MX_E_STRIDE;
    if (!aligned(x, uintptr_t(esz)) || !aligned(s, 4) || !aligned(slot, 4) || !aligned(src, 4)) return MX_E_ALIGN;
    const Span sp[] = {{addr(q), qb}, {addr(s), uint64_t(M) * 4}, {addr(x), xb},
                       {addr(slot), slot ? uint64_t(T) * uint64_t(k) * 4 : 0}, {addr(src), src ? uint64_t(M) * 4 : 0}};
    if (outputs_clash(sp, 2, 5)) return MX_E_OVERLAP;
    if (!some) return MX_OK;
    return status(mxq::launch_quantize_rows(x, dtype, T, K, ld_x, slot, src, k, M, q, ld_q, s, hip(stream)));
}

int64_t code_pitch(int64_t K) { return (K + 15) / 16 * 16; }

// Everything of a product but its left operand, whose rows are lda apart.
int check_product(int64_t lda, const int8_t* B, int64_t ldb, int64_t b_gs, const float* sB, int64_t sb_gs, const float* bias,
                  const int32_t* offs, int32_t G, bool groups, int64_t M, int64_t N, int64_t K, const void* C,
                  int64_t ldc, int32_t out_dtype, Span* sp) {
    const bool some = M > 0 && N > 0;
    if (some && ((!B && K > 0) || !sB || !C || (groups && !offs))) return MX_E_NULL;
    if (!dtype_ok(out_dtype)) return MX_E_DTYPE;
    if (M < 0 || N < 0 || K < 0 || M > kMaxRows || N > kMaxRows || K > kMaxCodes || G < 1) return MX_E_SHAPE;
    if (mxq::i8_gemm_threads(lda, ldb, M, N, K, groups, G) > kMaxThreads) return MX_E_SHAPE;
    if (ldb < K || ldc < N || b_gs < 0 || sb_gs < 0) return MX_E_STRIDE;
    const int64_t esz = elem(out_dtype);
    const uint64_t bb = matrix_bytes(N, K, ldb, 1), cb = matrix_bytes(M, N, ldc, esz);
    const uint64_t bg = matrix_bytes(G, 1, b_gs, 1), sg = matrix_bytes(G, 1, sb_gs, 4);
    if (bb == kTooLarge || cb == kTooLarge || bg == kTooLarge || sg == kTooLarge || bb + bg > kMaxSpan)
        return MX_E_STRIDE;
    if (!aligned(sB, 4) || !aligned(bias, 4) || !aligned(offs, 4) || !aligned(C, uintptr_t(esz))) return MX_E_ALIGN;
    sp[0] = {addr(C), cb};
    sp[1] = {addr(B), bb ? bb - 1 + bg : 0};
    sp[2] = {addr(sB), N > 0 ? uint64_t(N) * 4 - 4 + sg : 0};
    sp[3] = {addr(bias), bias ? uint64_t(N) * 4 : 0};
    sp[4] = {addr(offs), offs ? uint64_t(G) * 4 : 0};
    return MX_OK;
}

int gemm(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs, const float* sB,
         int64_t sb_gs, const float* bias, const int32_t* offs, int32_t G, bool groups, int64_t M, int64_t N,
         int64_t K, void* C, int64_t ldc, int32_t out_dtype, void* stream) {
    if (M > 0 && N > 0 && ((!A && K > 0) || !sA)) return MX_E_NULL;
    Span sp[7];
    int rc = check_product(lda, B, ldb, b_gs, sB, sb_gs, bias, offs, G, groups, M, N, K, C, ldc, out_dtype, sp);
    if (rc != MX_OK) return rc;
    const uint64_t ab = matrix_bytes(M, K, lda, 1);
    if (lda < K || ab == kTooLarge) return MX_E_STRIDE;
    if (!aligned(sA, 4)) return MX_E_ALIGN;
    sp[5] = {addr(A), ab};
    sp[6] = {addr(sA), uint64_t(M) * 4};
    if (outputs_clash(sp, 1, 7)) return MX_E_OVERLAP;
    if (M == 0 || N == 0) return MX_OK;
    return status(mxq::launch_i8_gemm(A, lda, sA, B, ldb, b_gs, sB, sb_gs, bias, C, ldc, M, N, K,
                                      groups ? offs : nullptr, groups ? G : 0, out_dtype, hip(stream)));
}

}  // namespace

extern "C" {

int64_t mx_route_rows(int64_t T, int32_t E, int32_t k, int32_t align) {
    if (!route_shape(T, E, k) || align < 1 || align > 65536) return -1;
    const int64_t picks = T * k, groups = picks < E ? picks : E;
    return (picks + groups * (align - 1) + align - 1) / align * align;
}

int64_t mx_route_workspace(int64_t T, int32_t E) {
    if (!route_shape(T, E, 1)) return -1;
    return mxq::route_workspace(T, E);
}

int mx_route(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid, int32_t k,
             int32_t normalize, int32_t align, int64_t M, int32_t* idx, float* weight, int32_t* slot, int32_t* src,
             int32_t* counts, int32_t* offs, int32_t* live, float* prob, float* loss, void* workspace,
             int64_t workspace_bytes, void* stream) {
    if (T > 0 && (!logits || !idx || !weight || !slot)) return MX_E_NULL;
    if (!counts || !offs || !live || !prob || !loss || (M > 0 && !src)) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    const int64_t rows = mx_route_rows(T, E, k, align);
    if (rows < 0 || M < rows || M > kMaxRows) return MX_E_SHAPE;
    const int64_t need = mxq::route_workspace(T, E);
    if (need > 0 && !workspace) return MX_E_NULL;
    if (workspace_bytes < need) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t lb = matrix_bytes(T, E, ld, esz), pk = uint64_t(T) * uint64_t(k) * 4, eb = uint64_t(E) * 4;
    if (ld < E || lb == kTooLarge) return MX_E_STRIDE;
    if (!aligned(logits, uintptr_t(esz)) || !aligned(idx, 4) || !aligned(weight, 4) || !aligned(slot, 4) ||
        !aligned(src, 4) || !aligned(counts, 4) || !aligned(offs, 4) || !aligned(live, 4) || !aligned(prob, 4) ||
        !aligned(loss, 4) || !aligned(workspace, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(idx), pk}, {addr(weight), pk}, {addr(slot), pk}, {addr(src), uint64_t(M) * 4},
                       {addr(counts), eb}, {addr(offs), eb}, {addr(live), 4}, {addr(prob), eb}, {addr(loss), 4},
                       {addr(workspace), uint64_t(need)}, {addr(logits), lb}, {addr(valid), valid ? uint64_t(T) : 0}};
    if (outputs_clash(sp, 10, 12)) return MX_E_OVERLAP;
    return status(mxq::launch_route(logits, dtype, T, E, ld, valid, k, normalize != 0, align, M, idx, weight, slot,
                                    src, counts, offs, live, prob, loss, workspace, hip(stream)));
}

int mx_route_grad(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                  int32_t k, int32_t normalize, const int32_t* idx, const float* weight, const float* dweight,
                  const int32_t* counts, const int32_t* live, const float* dloss, void* dlogits, int64_t ld_d,
                  void* stream) {
    if (T > 0 && (!logits || !counts || !live || !dlogits || (dweight && (!idx || !weight)))) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    if (!route_shape(T, E, k)) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t lb = matrix_bytes(T, E, ld, esz), db = matrix_bytes(T, E, ld_d, esz);
    const uint64_t pk = dweight ? uint64_t(T) * uint64_t(k) * 4 : 0;
    if (ld < E || ld_d < E || lb == kTooLarge || db == kTooLarge) return MX_E_STRIDE;
    if (!aligned(logits, uintptr_t(esz)) || !aligned(dlogits, uintptr_t(esz)) || !aligned(idx, 4) ||
        !aligned(weight, 4) || !aligned(dweight, 4) || !aligned(counts, 4) || !aligned(live, 4) || !aligned(dloss, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(dlogits), db}, {addr(logits), lb}, {addr(valid), valid ? uint64_t(T) : 0},
                       {addr(idx), pk}, {addr(weight), pk}, {addr(dweight), pk}, {addr(counts), uint64_t(E) * 4},
                       {addr(live), 4}, {addr(dloss), dloss ? 4u : 0u}};
    if (outputs_clash(sp, 1, 9)) return MX_E_OVERLAP;
    if (T == 0) return MX_OK;
    return status(mxq::launch_route_grad(logits, dtype, T, E, ld, valid, k, normalize != 0, idx, weight, dweight,
                                         counts, live, dloss, dlogits, ld_d, hip(stream)));
}

int mx_dispatch(const void* x, int32_t dtype, int64_t T, int64_t N, int64_t ld_x, const int32_t* slot,
                const int32_t* src, int32_t k, int64_t M, void* out, int64_t ld_out, void* stream) {
    if (N > 0 && ((T > 0 && (!x || !slot)) || (M > 0 && (!src || !out)))) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    int rc = check_map(T, N, k, M);
    if (rc != MX_OK) return rc;
    const int64_t esz = elem(dtype);
    if (mxq::dispatch_blocks(T, M, N * esz) * 256 > kMaxThreads) return MX_E_SHAPE;
    const uint64_t xb = matrix_bytes(T, N, ld_x, esz), ob = matrix_bytes(M, N, ld_out, esz);
    if (ld_x < N || ld_out < N || xb == kTooLarge || ob == kTooLarge) return MX_E_STRIDE;
    if (!aligned(x, uintptr_t(esz)) || !aligned(out, uintptr_t(esz)) || !aligned(slot, 4) || !aligned(src, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(out), ob}, {addr(x), xb}, {addr(slot), uint64_t(T) * uint64_t(k) * 4},
                       {addr(src), uint64_t(M) * 4}};
    if (outputs_clash(sp, 1, 4)) return MX_E_OVERLAP;
    if (N == 0 || M == 0) return MX_OK;
    return status(mxq::launch_dispatch(x, dtype, T, N, ld_x, slot, src, k, M, out, ld_out, hip(stream)));
}

int mx_dispatch_i8(const void* x, int32_t dtype, int64_t T, int64_t K, int64_t ld_x, const int32_t* slot,
                   const int32_t* src, int32_t k, int64_t M, int8_t* q, int64_t ld_q, float* s, void* stream) {
    return quantize(x, dtype, T, K, ld_x, slot, src, k, M, q, ld_q, s, true, stream);
}

int i8_quantize_rows(const void* x, int32_t dtype, int64_t T, int64_t K, int64_t ld_x, int8_t* q, int64_t ld_q,
                     float* s, void* stream) {
    return quantize(x, dtype, T, K, ld_x, nullptr, nullptr, 1, T, q, ld_q, s, false, stream);
}

int i8_gemm_nt(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, const float* sB,
               const float* bias, int64_t M, int64_t N, int64_t K, void* C, int64_t ldc, int32_t out_dtype,
               void* stream) {
    return gemm(A, lda, sA, B, ldb, 0, sB, 0, bias, nullptr, 1, false, M, N, K, C, ldc, out_dtype, stream);
}

int64_t i8_linear_workspace(int64_t M, int64_t K) {
    if (M < 0 || K < 0 || M > kMaxRows || K > kMaxCodes) return -1;
    return M * code_pitch(K) + (M * 4 + 15) / 16 * 16;
}

int i8_linear(const void* x, int32_t dtype, int64_t ld_x, const int8_t* B, int64_t ldb, const float* sB,
              const float* bias, int64_t M, int64_t N, int64_t K, void* C, int64_t ldc, int32_t out_dtype,
              void* workspace, int64_t workspace_bytes, void* stream) {
    const bool some = M > 0 && N > 0;
    if (some && ((!x && K > 0) || !workspace)) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    Span sp[7];
    int rc = check_product(code_pitch(K), B, ldb, 0, sB, 0, bias, nullptr, 1, false, M, N, K, C, ldc, out_dtype, sp);
    if (rc != MX_OK) return rc;
    const int64_t need = i8_linear_workspace(M, K);
    if (some && workspace_bytes < need) return MX_E_SHAPE;
    if (mxq::token_blocks(M, M) * 256 > kMaxThreads) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t xb = matrix_bytes(M, K, ld_x, esz);
    if (ld_x < K || xb == kTooLarge) return MX_E_STRIDE;
    if (!aligned(x, uintptr_t(esz)) || !aligned(workspace, 16)) return MX_E_ALIGN;
    sp[4] = sp[0];                                       // C and the workspace first: the outputs
    sp[0] = {addr(workspace), some ? uint64_t(need) : 0};
    sp[5] = sp[1];
    sp[1] = sp[4];
    sp[4] = {addr(x), xb};
    if (outputs_clash(sp, 2, 6)) return MX_E_OVERLAP;
    if (!some) return MX_OK;
    if (mxq::i8_linear_fuses(x, dtype, ld_x, B, ldb, M, N, K))
        return status(mxq::launch_i8_linear_fused(x, dtype, ld_x, B, ldb, sB, bias, C, ldc, M, N, K, out_dtype,
                                                  hip(stream)));
    int8_t* q = static_cast<int8_t*>(workspace);
    const int64_t ld_q = code_pitch(K);
    float* s = reinterpret_cast<float*>(q + M * ld_q);
    hipError_t e = mxq::launch_quantize_rows(x, dtype, M, K, ld_x, nullptr, nullptr, 1, M, q, ld_q, s, hip(stream));
    if (e != hipSuccess) return MX_E_LAUNCH;
    return status(mxq::launch_i8_gemm(q, ld_q, s, B, ldb, 0, sB, 0, bias, C, ldc, M, N, K, nullptr, 0, out_dtype,
                                      hip(stream)));
}

int i8_grouped_gemm_rows(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs,
                         const float* sB, int64_t sb_gs, const int32_t* offs, int32_t G, int64_t M, int64_t N,
                         int64_t K, void* C, int64_t ldc, int32_t out_dtype, void* stream) {
    return gemm(A, lda, sA, B, ldb, b_gs, sB, sb_gs, nullptr, offs, G, true, M, N, K, C, ldc, out_dtype, stream);
}

int mx_combine(const void* rows, int32_t dtype, int64_t M, int64_t N, int64_t ld_r, const int32_t* slot,
               const float* weight, int32_t k, int64_t T, void* y, int64_t ld_y, void* stream) {
    if (N > 0 && T > 0 && ((M > 0 && !rows) || !slot || !y)) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    int rc = check_map(T, N, k, M);
    if (rc != MX_OK) return rc;
    const int64_t esz = elem(dtype);
    if (mxq::combine_blocks(T, N * esz) * 256 > kMaxThreads) return MX_E_SHAPE;
    const uint64_t rb = matrix_bytes(M, N, ld_r, esz), yb = matrix_bytes(T, N, ld_y, esz);
    const uint64_t pk = uint64_t(T) * uint64_t(k) * 4;
    if (ld_r < N || ld_y < N || rb == kTooLarge || yb == kTooLarge) return MX_E_STRIDE;
    if (!aligned(rows, uintptr_t(esz)) || !aligned(y, uintptr_t(esz)) || !aligned(slot, 4) || !aligned(weight, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(y), yb}, {addr(rows), rb}, {addr(slot), pk}, {addr(weight), weight ? pk : 0}};
    if (outputs_clash(sp, 1, 4)) return MX_E_OVERLAP;
    if (N == 0 || T == 0) return MX_OK;
    return status(mxq::launch_combine(rows, dtype, M, N, ld_r, slot, weight, k, T, y, ld_y, hip(stream)));
}

int mx_combine_grad(const void* dy, int32_t dtype, int64_t T, int64_t N, int64_t ld_dy, const void* rows,
                    int64_t ld_r, const int32_t* slot, const float* weight, const int32_t* src, int32_t k, int64_t M,
                    void* drows, int64_t ld_d, float* dweight, void* stream) {
    if (T > 0 && (!slot || (N > 0 && !dy))) return MX_E_NULL;
    if (M > 0 && (!src || (N > 0 && (!drows || (dweight && !rows))))) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    int rc = check_map(T, N, k, M);
    if (rc != MX_OK) return rc;
    if (mxq::token_blocks(T, M) * 256 > kMaxThreads) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t rb = rows ? matrix_bytes(M, N, ld_r, esz) : 0, gb = matrix_bytes(T, N, ld_dy, esz);
    const uint64_t db = matrix_bytes(M, N, ld_d, esz), pk = uint64_t(T) * uint64_t(k) * 4;
    if ((rows && ld_r < N) || ld_dy < N || ld_d < N || rb == kTooLarge || gb == kTooLarge || db == kTooLarge)
        return MX_E_STRIDE;
    if (!aligned(dy, uintptr_t(esz)) || !aligned(rows, uintptr_t(esz)) || !aligned(drows, uintptr_t(esz)) ||
        !aligned(slot, 4) || !aligned(weight, 4) || !aligned(src, 4) || !aligned(dweight, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(drows), db}, {addr(dweight), dweight ? pk : 0}, {addr(dy), gb}, {addr(rows), rb},
                       {addr(slot), pk}, {addr(weight), weight ? pk : 0}, {addr(src), uint64_t(M) * 4}};
    if (outputs_clash(sp, 2, 7)) return MX_E_OVERLAP;
    if (T == 0 && (M == 0 || N == 0)) return MX_OK;
    return status(mxq::launch_combine_grad(dy, dtype, T, N, ld_dy, rows, ld_r, slot, weight, src, k, M, drows, ld_d,
                                           dweight, hip(stream)));
}

}  // extern "C"
