// i8_act_launch.h -- the launchers of the 8-bit product with an epilogue, once
// without gates and once with them (two files, which compile side by side).
#include "i8_kernels.h"

namespace mxq {

hipError_t MXQ_ACT_GEMM(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs,
                        const float* sB, int64_t sb_gs, const Epilogue& e, void* C, int64_t ldc, int64_t M, int64_t N,
                        int64_t K, const int32_t* offs, int32_t G, int out_dtype, hipStream_t stream) {
    I8Args p{};
    p.A = A; p.lda = lda; p.sA = sA; p.B = B; p.ldb = ldb; p.b_gs = b_gs; p.sB = sB; p.sb_gs = sb_gs; p.e = e;
    p.C = C; p.ldc = ldc; p.M = M; p.N = N; p.K = K; p.offs = offs; p.G = G;
    using E = Act<MXQ_ACT_GATED>;
    return out_dtype == 0 ? launch<float, E>(p, stream) : launch<__bf16, E>(p, stream);
}

hipError_t MXQ_ACT_LINEAR(const void* x, int dtype, int64_t ld_x, const int8_t* B, int64_t ldb, const float* sB,
                          const Epilogue& e, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K, int out_dtype,
                          hipStream_t stream) {
    I8Args p{};
    p.A = static_cast<const int8_t*>(x); p.lda = ld_x; p.B = B; p.ldb = ldb; p.sB = sB; p.e = e; p.C = C; p.ldc = ldc;
    p.M = M; p.N = N; p.K = K;
    using E = Act<MXQ_ACT_GATED>;
    const bool ring_fits = ring_fuses(x, dtype == 0 ? 4 : 2, ld_x, B, ldb, M, K);
    return dtype == 0 ? fused<float, E>(p, ring_fits, out_dtype, stream) : fused<uint16_t, E>(p, ring_fits, out_dtype, stream);
}

}  // namespace mxq
