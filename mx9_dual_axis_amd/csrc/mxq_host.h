// Host-side argument checks shared by the C-ABI files.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxq.h"

namespace {

constexpr uint64_t kMaxThreads = 0xFFFFFFFFull - 256;   // grid.x * block.x must fit 32 bits

struct Span {
    uintptr_t p;
    uint64_t n;   // bytes
};

inline bool overlap(const Span& a, const Span& b) {
    return a.n != 0 && b.n != 0 && a.p < b.p + b.n && b.p < a.p + a.n;
}

inline bool any_overlap(const Span* s, int k) {
    for (int i = 0; i < k; ++i)
        for (int j = i + 1; j < k; ++j)
            if (overlap(s[i], s[j])) return true;
    return false;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// No device buffer spans more bytes than a 48-bit virtual address space.
constexpr uint64_t kMaxSpan = uint64_t(1) << 48;
constexpr uint64_t kTooLarge = ~uint64_t(0);

// Bytes spanned by a [rows, cols] matrix with row pitch ld (elements), or
// kTooLarge when that exceeds kMaxSpan (computed without overflow).
inline uint64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t esz) {
    if (rows <= 0 || cols <= 0) return 0;
    const unsigned __int128 b =
        (static_cast<unsigned __int128>(rows - 1) * uint64_t(ld) + uint64_t(cols)) * uint64_t(esz);
    return b > kMaxSpan ? kTooLarge : uint64_t(b);
}

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxCodes = 131071;     // of an 8-bit contraction: 131071 * 128 * 128 < 2^31

inline hipStream_t hip(void* stream) { return static_cast<hipStream_t>(stream); }
inline int status(hipError_t e) { return e == hipSuccess ? MX_OK : MX_E_LAUNCH; }

inline bool dtype_ok(int32_t d) { return d == MX_DTYPE_F32 || d == MX_DTYPE_BF16; }
inline int64_t elem(int32_t d) { return d == MX_DTYPE_F32 ? 4 : 2; }

// The first n_out spans are outputs: disjoint from each other and from the
// inputs that follow; inputs may overlap each other.
inline bool outputs_clash(const Span* s, int n_out, int n) {
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(s[i], s[j])) return true;
    return false;
}

// Bytes spanned by a strided scale view of rows x blocks (non-negative strides).
inline uint64_t scale_span(int64_t rows, int64_t blocks, int64_t rs, int64_t bs) {
    if (rows <= 0 || blocks <= 0) return 0;
    return uint64_t((rows - 1) * rs + (blocks - 1) * bs + 1);
}

constexpr int64_t kMaxGemm = int64_t(1) << 24;

// Checks shared by the contraction calls: operand pitches and alignment,
// scale strides, the output type and pitch.  K is the contraction extent.
inline int check_gemm(const uint8_t* A, int64_t lda, const uint8_t* sA, int64_t sa_rs, int64_t sa_bs,
               const uint8_t* B, int64_t ldb, const uint8_t* sB, int64_t sb_rs, int64_t sb_bs,
               int64_t M, int64_t N, int64_t K, const void* C, int64_t ldc, int32_t out_dtype, bool mfma) {
    const bool empty = M == 0 || N == 0;
    if (!empty && (!A || !sA || !B || !sB || !C)) return MX_E_NULL;
    if (out_dtype != MX_DTYPE_F32 && out_dtype != MX_DTYPE_BF16) return MX_E_DTYPE;
    if (M < 0 || N < 0 || K < 0 || M > kMaxGemm || N > kMaxGemm || K > kMaxGemm ||
        M % 128 != 0 || N % 128 != 0 || K % 128 != 0)
        return MX_E_SHAPE;
    if (lda < K || ldb < K || lda % 16 != 0 || ldb % 16 != 0 || lda > kMaxGemm || ldb > kMaxGemm || ldc < N ||
        ldc > kMaxGemm || sa_rs < 0 || sa_bs < 0 || sb_rs < 0 || sb_bs < 0)
        return MX_E_STRIDE;
    const uintptr_t esz = out_dtype == MX_DTYPE_F32 ? 4 : 2;
    if (!empty && (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, esz))) return MX_E_ALIGN;
    if (!empty && mfma && (!aligned(sA, 16) || !aligned(sB, 16))) return MX_E_ALIGN;
    return MX_OK;
}

// Whether every contraction kernel the call may launch has a grid whose
// thread count fits 32 bits: the general kernel (128 x 128 tiles of 256
// threads), the pipelined kernel (256 x 256 tiles of 512 threads, or for row
// groups 8 XCD shares of at most ceil(M/128/8) + 1 row tiles of 128 x 256),
// times the group count for contraction groups.
inline bool gemm_grid_fits(int64_t M, int64_t N, int32_t G, bool row_groups, bool k_groups) {
    const uint64_t g = k_groups ? uint64_t(G) : 1u;
    const uint64_t general = uint64_t(M / 128) * uint64_t(N / 128) * g * 256u;
    const uint64_t pipe = row_groups ? 8u * (uint64_t(M / 128 + 7) / 8u + 1u) * uint64_t((N + 255) / 256) * 512u
                                     : uint64_t((M + 255) / 256) * uint64_t((N + 255) / 256) * g * 512u;
    return general <= kMaxThreads && pipe <= kMaxThreads;
}

// Bytes of one operand's scales: a strided view, or rows * K/32 in the matrix-core layout.
inline uint64_t scale_bytes(bool mfma, int64_t rows, int64_t K, int64_t rs, int64_t bs) {
    return mfma ? uint64_t(rows) * uint64_t(K / 32) : scale_span(rows, K / 32, rs, bs);
}

}  // namespace
