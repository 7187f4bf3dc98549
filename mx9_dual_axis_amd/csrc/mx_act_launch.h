// mx_act_launch.h -- the launcher of the MXFP8 contraction with an epilogue,
// once without gates and once with them (two files, which compile side by side).
#include "mx_gemm_kernels.h"

namespace mxq {

hipError_t MXQ_ACT_LAUNCH(const uint8_t* A, int64_t lda, const uint8_t* sA, int64_t sa_rs, int64_t sa_bs, const uint8_t* B,
                          int64_t ldb, int64_t b_gs, const uint8_t* sB, int64_t sb_rs, int64_t sb_bs, int64_t sb_gs,
                          const Epilogue& e, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K, const int32_t* offs,
                          int32_t G, int out_dtype, bool mfma_scales, hipStream_t stream) {
    GemmArgs p{};
    p.A = A; p.lda = lda; p.sA = sA; p.sa_rs = sa_rs; p.sa_bs = sa_bs;
    p.B = B; p.ldb = ldb; p.b_gs = b_gs; p.sB = sB; p.sb_rs = sb_rs; p.sb_bs = sb_bs; p.sb_gs = sb_gs;
    p.C = C; p.ldc = ldc; p.M = M; p.N = N; p.K = K; p.offs = offs; p.G = G; p.e = e;
    if (mfma_scales) {
        // the K/32 scale bytes of each of 64 rows
        p.sa_rs = p.sb_rs = 2 * K;
        p.sa_bs = p.sb_bs = 0;
    }
    return launch_any<Act<MXQ_ACT_GATED>>(p, out_dtype, mfma_scales, stream);
}

}  // namespace mxq
