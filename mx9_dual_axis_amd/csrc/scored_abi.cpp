// scored_abi.cpp -- the C ABI declared in include/mxq_scored.h.
//
// As in mxq_abi.cpp: arguments are checked on the host, in the order the
// header lists the errors, before anything is enqueued.
#include "../../include/mxq_scored.h"

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "mxq_host.h"
#include "mxq_kernels.h"

namespace {

bool score_ok(int32_t s) { return s == MX_SCORE_SIGMOID || s == MX_SCORE_SOFTMAX; }

}  // namespace

extern "C" {

int mx_route_scored(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                    const float* bias, int32_t score, int32_t groups, int32_t top_groups, int32_t group_best, int32_t k,
                    int32_t normalize, float scale, int32_t align, int64_t M, int32_t* idx, float* weight, int32_t* slot,
                    int32_t* src, int32_t* counts, int32_t* offs, int32_t* live, float* prob, float* loss, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    if (T > 0 && (!logits || !idx || !weight || !slot)) return MX_E_NULL;
    if (!counts || !offs || !live || !prob || !loss || (M > 0 && !src)) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    if (!score_ok(score)) return MX_E_MODE;
    const int64_t rows = mx_route_rows(T, E, k, align);
    if (rows < 0 || M < rows || M > kMaxRows) return MX_E_SHAPE;
    if (groups < 1 || groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups || group_best < 1 ||
        group_best > 2 || k > top_groups * (E / groups))
        return MX_E_SHAPE;
    const int64_t need = mxq::route_workspace(T, E);
    if (need > 0 && !workspace) return MX_E_NULL;
    if (workspace_bytes < need) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t lb = matrix_bytes(T, E, ld, esz), pk = uint64_t(T) * uint64_t(k) * 4, eb = uint64_t(E) * 4;
    if (ld < E || lb == kTooLarge) return MX_E_STRIDE;
    if (!aligned(logits, uintptr_t(esz)) || !aligned(bias, 4) || !aligned(idx, 4) || !aligned(weight, 4) ||
        !aligned(slot, 4) || !aligned(src, 4) || !aligned(counts, 4) || !aligned(offs, 4) || !aligned(live, 4) ||
        !aligned(prob, 4) || !aligned(loss, 4) || !aligned(workspace, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(idx), pk}, {addr(weight), pk}, {addr(slot), pk}, {addr(src), uint64_t(M) * 4},
                       {addr(counts), eb}, {addr(offs), eb}, {addr(live), 4}, {addr(prob), eb}, {addr(loss), 4},
                       {addr(workspace), uint64_t(need)}, {addr(logits), lb}, {addr(valid), valid ? uint64_t(T) : 0},
                       {addr(bias), bias ? eb : 0}};
    if (outputs_clash(sp, 10, 13)) return MX_E_OVERLAP;
    return status(mxq::launch_route_scored(logits, dtype, T, E, ld, valid, bias, score == MX_SCORE_SOFTMAX, groups,
                                           top_groups, group_best, k, normalize != 0, scale, align, M, idx, weight, slot,
                                           src, counts, offs, live, prob, loss, workspace, hip(stream)));
}

int mx_route_scored_grad(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                         int32_t score, int32_t k, int32_t normalize, float scale, const int32_t* idx,
                         const float* dweight, const int32_t* counts, const int32_t* live, const float* dloss,
                         void* dlogits, int64_t ld_d, void* stream) {
    if (T > 0 && (!logits || !counts || !live || !dlogits || (dweight && !idx))) return MX_E_NULL;
    if (!dtype_ok(dtype)) return MX_E_DTYPE;
    if (!score_ok(score)) return MX_E_MODE;
    if (mx_route_rows(T, E, k, 1) < 0) return MX_E_SHAPE;
    const int64_t esz = elem(dtype);
    const uint64_t lb = matrix_bytes(T, E, ld, esz), db = matrix_bytes(T, E, ld_d, esz);
    const uint64_t pk = dweight ? uint64_t(T) * uint64_t(k) * 4 : 0;
    if (ld < E || ld_d < E || lb == kTooLarge || db == kTooLarge) return MX_E_STRIDE;
    if (!aligned(logits, uintptr_t(esz)) || !aligned(dlogits, uintptr_t(esz)) || !aligned(idx, 4) ||
        !aligned(dweight, 4) || !aligned(counts, 4) || !aligned(live, 4) || !aligned(dloss, 4))
        return MX_E_ALIGN;
    const Span sp[] = {{addr(dlogits), db}, {addr(logits), lb}, {addr(valid), valid ? uint64_t(T) : 0},
                       {addr(idx), pk}, {addr(dweight), pk}, {addr(counts), uint64_t(E) * 4},
                       {addr(live), 4}, {addr(dloss), dloss ? 4u : 0u}};
    if (outputs_clash(sp, 1, 8)) return MX_E_OVERLAP;
    if (T == 0) return MX_OK;
    return status(mxq::launch_route_scored_grad(logits, dtype, T, E, ld, valid, score == MX_SCORE_SOFTMAX, k,
                                                normalize != 0, scale, idx, dweight, counts, live, dloss, dlogits, ld_d,
                                                hip(stream)));
}

int mx_route_bias_step(const float* bias, const int32_t* counts, int32_t E, float rate, float* out, void* stream) {
    if (!bias || !counts || !out) return MX_E_NULL;
    if (E < 1 || E > 1024) return MX_E_SHAPE;
    if (!aligned(bias, 4) || !aligned(counts, 4) || !aligned(out, 4)) return MX_E_ALIGN;
    const uint64_t eb = uint64_t(E) * 4;
    const Span sp[] = {{addr(out), eb}, {addr(counts), eb}, {addr(bias), bias == out ? 0 : eb}};
    if (outputs_clash(sp, 1, 3)) return MX_E_OVERLAP;
    return status(mxq::launch_route_bias_step(bias, counts, E, rate, out, hip(stream)));
}

}  // extern "C"
