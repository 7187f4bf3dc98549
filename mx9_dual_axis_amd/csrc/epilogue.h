// epilogue.h -- what a product does with its sums before their only rounding:
//
//   x = sum + bias[n]              (the caller has added the bias)
//   y = act(x) (+ residual), or where gated act(x[n]) x[n + up] (+ residual)
//
// y, and x where it is kept, are rounded once to the output's type.  A gated
// product's tile holds the rows of B of its channels n and, as many rows
// further on, those of n + up: each wave's columns are half the one, half the
// other, so that both factors of a result meet in the wave's own LDS.
//
// The sums wait in LDS in fp32, 16 rows at a time, and each lane takes 16 bytes
// of a result's row: residual, kept values and results move in whole 16-byte
// pieces.  The residual of the 16 rows to come is read while these are
// computed (but for 128 fp32 columns, where that would spill).
//
// What it adds to a product, 8192^3 MXFP8 to bf16 (us, calls with a pause before
// each; without pauses the clock is lower, 452 for the product alone): the
// product alone 405; with this epilogue and no activation 425, SiLU 446, tanh GELU
// 452, GELU 465, its bias 466, a residual 474, the kept sums 484.  The tile's waves
// compute it while the matrix cores wait (a tile's accumulators leave no room for
// a second tile on the CU), so an activation costs its instructions: act.h.  The
// residual and the kept sums cost their 134 MB each.
#pragma once

#include "act.h"
#include "mxq_kernels.h"

namespace mxq {
namespace {

typedef unsigned int ep_u4 __attribute__((ext_vector_type(4)));

// Which epilogue a kernel has.
struct Plain {
    static constexpr bool kOn = false, kGated = false;
};
template <bool kG>
struct Act {
    static constexpr bool kOn = true, kGated = kG;
};

template <typename O> __device__ __forceinline__ O ep_round(float x);
template <> __device__ __forceinline__ float ep_round<float>(float x) { return x; }
template <> __device__ __forceinline__ __bf16 ep_round<__bf16>(float x) { return __bf16(x); }   // nearest-even

// An addition by itself: fused with the product before it where the two meet in
// the code, and rounded twice elsewhere, a row's bits would go by the form that
// its batch takes.
__device__ __forceinline__ float ep_add(float x, float y) {
#pragma clang fp contract(off)
    return x + y;
}

// kCols columns (results) of 16 rows of one wave.
template <typename O, int kCols>
struct EpRows {
    static constexpr int kPer = 16 / int(sizeof(O)), kPieces = kCols / kPer, kAll = 16 * kPieces, kQ = (kAll + 63) / 64;
    static constexpr bool kAhead = kQ <= 4;      // the registers hold the residual of 16 rows more
    static_assert(kCols % kPer == 0, "whole pieces");

    static __device__ __forceinline__ bool whole(const void* p, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % kPer == 0;
    }
    static __device__ __forceinline__ bool place(int q, uint32_t rows, uint32_t cols, uint32_t* row, uint32_t* col) {
        const uint32_t piece = 64u * uint32_t(q) + (threadIdx.x & 63u);
        *row = piece / uint32_t(kPieces);
        *col = piece % uint32_t(kPieces) * uint32_t(kPer);
        return (kAll % 64 == 0 || piece < uint32_t(kAll)) && *row < rows && *col < cols;
    }

    // The residual's pieces (rows and cols: what is left of the result from row0, col0).
    ep_u4 res[kQ];
    __device__ __forceinline__ void read(const Epilogue& e, int64_t row0, int64_t col0, uint32_t rows, uint32_t cols) {
        const O* R = static_cast<const O*>(e.residual);
        const bool w = whole(R, e.ld_res);
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            uint32_t row, col;
            res[q] = ep_u4{0u, 0u, 0u, 0u};
            if (!place(q, rows, cols, &row, &col)) continue;
            const O* from = R + (row0 + row) * e.ld_res + col0 + col;
            if (col + uint32_t(kPer) <= cols) {
                if (w) res[q] = __builtin_nontemporal_load(reinterpret_cast<const ep_u4*>(from));
                else __builtin_memcpy(&res[q], from, 16);
            } else {
                O part[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) part[i] = from[min(uint32_t(i), cols - 1u - col)];
                __builtin_memcpy(&res[q], part, 16);
            }
        }
    }

    static __device__ __forceinline__ void put(O* to, const O (&v)[kPer], bool w, uint32_t left) {
        if (left >= uint32_t(kPer)) {
            ep_u4 x;
            __builtin_memcpy(&x, v, 16);
            if (w) __builtin_nontemporal_store(x, reinterpret_cast<ep_u4*>(to));
            else __builtin_memcpy(to, &x, 16);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (uint32_t(i) < left) to[i] = v[i];
        }
    }

    // The staged rows (fp32, `pitch` bytes apart; gated: the second factors
    // kCols columns on) to C, and to pre.
    template <int kAct, bool kGated>
    __device__ __forceinline__ void write(const Epilogue& e, O* C, int64_t ldc, const uint8_t* staged, int pitch,
                                          int64_t row0, int64_t col0, uint32_t rows, uint32_t cols, bool zero) const {
        O* P = static_cast<O*>(e.pre);
        const bool wc = whole(C, ldc), wp = whole(P, e.ld_pre) && (!kGated || e.up % kPer == 0);
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            uint32_t row, col;
            if (!place(q, rows, cols, &row, &col)) continue;
            const float* x = reinterpret_cast<const float*>(staged + row * pitch) + col;
            const float* u = x + kCols;
            O r[kPer], y[kPer], g[kPer], h[kPer];
            __builtin_memcpy(r, &res[q], 16);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                float v = act_value<kAct>(x[i]);
                if (kGated) v *= u[i];
                if (e.residual) v = ep_add(v, float(r[i]));
                y[i] = ep_round<O>(zero ? 0.f : v);
                g[i] = ep_round<O>(zero ? 0.f : x[i]);
                if (kGated) h[i] = ep_round<O>(zero ? 0.f : u[i]);
            }
            put(C + (row0 + row) * ldc + col0 + col, y, wc, cols - col);
            if (P) {
                O* to = P + (row0 + row) * e.ld_pre + col0 + col;
                put(to, g, wp, cols - col);
                if (kGated) put(to + e.up, h, wp, cols - col);
            }
        }
    }
};

// f(std::integral_constant<int, i>) for a uniform i in [0, N): a choice among
// registers, in a loop that is not unrolled so that what follows it (five
// activations' code) exists once.  The branches end and begin unlike each other:
// alike, they would be merged into one that chooses an address, and the
// registers would move to memory.
template <int I>
__device__ __forceinline__ void branch_mark() {
    if constexpr (I == 0) asm volatile("; rows 0");
    if constexpr (I == 1) asm volatile("; rows 1");
    if constexpr (I == 2) asm volatile("; rows 2");
    if constexpr (I == 3) asm volatile("; rows 3");
}
template <int N, typename F>
__device__ __forceinline__ void each_index(int i, F&& f) {
    static_assert(N <= 4, "a mark for each");
    if constexpr (N > 1) {
        if (i < N - 1) return each_index<N - 1>(i, f);
    }
    branch_mark<N - 1>();
    f(std::integral_constant<int, N - 1>{});
    branch_mark<N - 1>();
}

// One result by itself.
template <typename O, bool kGated>
__device__ __forceinline__ O ep_one(const Epilogue& e, float x, float u, float residual) {
    float v = x;
    act_switch(e.act, [&](auto a) { v = act_value<decltype(a)::value>(x); });
    if (kGated) v *= u;
    if (e.residual) v = ep_add(v, residual);
    return ep_round<O>(v);
}

}  // namespace
}  // namespace mxq
