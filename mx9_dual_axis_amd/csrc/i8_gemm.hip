// i8_gemm.hip -- the product of 8-bit codes with scales and bias alone
// (i8_kernels.h).
#include "i8_kernels.h"

namespace mxq {

// The threads of the largest grid that a product of this shape launches.
uint64_t i8_gemm_threads(int64_t lda, int64_t ldb, int64_t M, int64_t N, int64_t K, bool groups, int32_t G) {
    if (M <= 0 || N <= 0) return 0;
    if (far(lda, ldb)) return choose(M, N, K, groups, G, Rows::kFar).threads;
    const uint64_t a = choose(M, N, K, groups, G, Rows::kBytes).threads, b = choose(M, N, K, groups, G, Rows::kPieces).threads;
    return a > b ? a : b;
}

hipError_t launch_i8_gemm(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs,
                          const float* sB, int64_t sb_gs, const float* bias, void* C, int64_t ldc, int64_t M,
                          int64_t N, int64_t K, const int32_t* offs, int32_t G, int out_dtype, hipStream_t stream) {
    I8Args p{};
    p.A = A; p.lda = lda; p.sA = sA; p.B = B; p.ldb = ldb; p.b_gs = b_gs; p.sB = sB; p.sb_gs = sb_gs; p.bias = bias;
    p.C = C; p.ldc = ldc; p.M = M; p.N = N; p.K = K; p.offs = offs; p.G = G; p.tiles_m = p.tiles_n = 0;
    return out_dtype == 0 ? launch<float, Plain>(p, stream) : launch<__bf16, Plain>(p, stream);
}

bool i8_linear_fuses(const void* x, int dtype, int64_t ld_x, const int8_t* B, int64_t ldb, int64_t M, int64_t N, int64_t K) {
    return ring_fuses(x, dtype == 0 ? 4 : 2, ld_x, B, ldb, M, K) || split_fuses(M, N, K);
}

hipError_t launch_i8_linear_fused(const void* x, int dtype, int64_t ld_x, const int8_t* B, int64_t ldb, const float* sB,
                                  const float* bias, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                  int out_dtype, hipStream_t stream) {
    I8Args p{};
    p.A = static_cast<const int8_t*>(x); p.lda = ld_x; p.sA = nullptr; p.B = B; p.ldb = ldb; p.b_gs = 0; p.sB = sB;
    p.sb_gs = 0; p.bias = bias; p.C = C; p.ldc = ldc; p.M = M; p.N = N; p.K = K; p.offs = nullptr; p.G = 0;
    p.tiles_m = p.tiles_n = 0;
    const bool ring_fits = ring_fuses(x, dtype == 0 ? 4 : 2, ld_x, B, ldb, M, K);
    return dtype == 0 ? fused<float, Plain>(p, ring_fits, out_dtype, stream) : fused<uint16_t, Plain>(p, ring_fits, out_dtype, stream);
}

}  // namespace mxq
