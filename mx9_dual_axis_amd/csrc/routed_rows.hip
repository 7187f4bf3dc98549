// routed_rows.hip -- token rows to their experts' rows of the padded buffer
// and back: dispatch (copied, or quantized to 8-bit integers), the weighted
// combine and its gradient.
//
//   dispatch      out[slot[t][j]] = x[t]                     rows without a token: 0
//   quantize      a = max(max |x|, 127 2^-126), q = rne(x (127 (1 / a))), s = a / 127
//                 (a row with Inf or NaN: q = 0, s = NaN, so that what is
//                 computed from it is NaN)
//   combine       y[t] = sum_j w[t][j] rows[slot[t][j]]      fp32, j ascending, rounded once
//   its gradient  drows[slot[t][j]] = w[t][j] dy[t], dw[t][j] = <dy[t], rows[slot[t][j]]>
//
// All are bound by HBM: each token row is read once and each expert row
// written (or read) once.  Rows move in 16-byte pieces whatever their
// alignment (the hardware takes unaligned pieces).  A row that is not whole
// pieces ends with a piece that overlaps the one before, whose common part
// is written twice with the same bytes; rows shorter than a piece go by
// element.  A slot outside [0, M) is skipped, so that no access leaves the
// operands whatever the map holds.
#include "mxq_kernels.h"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kPadRows = 16;     // rows of the map that one wave (or block) looks through for padding

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct Piece {
    u32x4 v;
};

__device__ __forceinline__ u32x4 load16(const char* p) {
    Piece q;
    __builtin_memcpy(&q, p, 16);
    return q.v;
}
__device__ __forceinline__ void store16(char* p, u32x4 v) {
    Piece q{v};
    __builtin_memcpy(p, &q, 16);
}

// Elements of a piece as fp32.
template <typename T> struct Elem;
template <> struct Elem<float> {
    static constexpr int kPer = 4;
    static __device__ __forceinline__ void get(u32x4 v, float (&f)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
    }
    static __device__ __forceinline__ u32x4 put(const float (&f)[4]) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
        return v;
    }
    static __device__ __forceinline__ float one(const char* p) { return *reinterpret_cast<const float*>(p); }
    static __device__ __forceinline__ void one(char* p, float f) { *reinterpret_cast<float*>(p) = f; }
};
template <> struct Elem<uint16_t> {
    static constexpr int kPer = 8;
    static __device__ __forceinline__ void get(u32x4 v, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint32_t bits(float f) {
        return __builtin_bit_cast(uint16_t, __bf16(f));                    // nearest-even
    }
    static __device__ __forceinline__ u32x4 put(const float (&f)[8]) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = bits(f[2 * i]) | (bits(f[2 * i + 1]) << 16);
        return v;
    }
    static __device__ __forceinline__ float one(const char* p) {
        return __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16);
    }
    static __device__ __forceinline__ void one(char* p, float f) { *reinterpret_cast<uint16_t*>(p) = uint16_t(bits(f)); }
};

// Zero `bytes` (a multiple of esz) at p with n threads.
__device__ __forceinline__ void zero_row(char* p, int64_t bytes, int esz, uint32_t t, uint32_t n) {
    if (bytes >= 16) {
        const u32x4 z = {0u, 0u, 0u, 0u};
        const int64_t pieces = (bytes + 15) / 16;
        for (int64_t c = t; c < pieces; c += n) store16(p + (16 * c + 16 > bytes ? bytes - 16 : 16 * c), z);
    } else if (int64_t(t) * esz < bytes) {
        for (int b = 0; b < esz; ++b) p[int64_t(t) * esz + b] = 0;
    }
}

constexpr int kMaxPicks = 64;

// Which of the kPadRows rows from r0 belong to no token: one load, one bit each.
__device__ __forceinline__ uint32_t pad_rows(const int32_t* src, int64_t r0, int64_t M) {
    const uint32_t lane = threadIdx.x & 63u;
    bool pad = false;
    if (lane < kPadRows && r0 + lane < M) pad = src[r0 + lane] < 0;
    return uint32_t(__ballot(pad));
}

// ------------------------------------------------------------------ dispatch
struct DispatchArgs {
    const char* x;
    int64_t T, ld_x;             // bytes
    const int32_t *slot, *src;
    int32_t k;
    int64_t M;
    char* out;
    int64_t ld_out, row;         // bytes per row
    int32_t esz;
    int64_t chunks;              // 4 KiB chunks per row
};

constexpr int64_t kChunk = 4096;

// One wave per token and 4 KiB chunk of its row, then one wave per 16 rows of
// the map and chunk for the rows without a token.  [4096, 5120] bf16 to 24576
// rows, 4 picks a token: 49 us, 293.6 MB at 6.0 TB/s.
__global__ __launch_bounds__(kThreads) void dispatch_kernel(DispatchArgs p) {
    const uint32_t lane = threadIdx.x & 63u;
    const int64_t w = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tokens = p.T * p.chunks;
    if (w < tokens) {
        const int64_t t = w / p.chunks, c0 = (w - t * p.chunks) * kChunk;
        const char* x = p.x + t * p.ld_x;
        const int32_t* slot = p.slot + t * p.k;
        if (p.row >= 16) {
            u32x4 v[4];
            int64_t at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t b = c0 + 1024 * i + 16 * int64_t(lane);
                at[i] = b < p.row ? (b + 16 > p.row ? p.row - 16 : b) : -1;
                if (at[i] >= 0) v[i] = load16(x + at[i]);
            }
            for (int32_t j = 0; j < p.k; ++j) {
                const int64_t s = slot[j];
                if (s < 0 || s >= p.M) continue;
                char* o = p.out + s * p.ld_out;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at[i] >= 0) store16(o + at[i], v[i]);
            }
        } else if (int64_t(lane) < p.row) {
            for (int32_t j = 0; j < p.k; ++j) {
                const int64_t s = slot[j];
                if (s >= 0 && s < p.M) p.out[s * p.ld_out + lane] = x[lane];
            }
        }
        return;
    }
    const int64_t u = w - tokens, g = u / p.chunks, c0 = (u - g * p.chunks) * kChunk;
    const int64_t r0 = g * kPadRows;
    if (r0 >= p.M) return;
    uint32_t rows = pad_rows(p.src, r0, p.M);
    const int64_t n = p.row - c0 < kChunk ? p.row - c0 : kChunk;
    // a last chunk shorter than a piece is zeroed with the piece before it
    const int64_t from = n < 16 && c0 > 0 ? c0 - 16 : c0;
    while (rows) {
        const int r = __builtin_ctz(rows);
        rows &= rows - 1;
        zero_row(p.out + (r0 + r) * p.ld_out + from, n + (c0 - from), p.esz, lane, 64);
    }
}

// ----------------------------------------------------- dispatch, quantized
struct QuantArgs {
    const char* x;
    int64_t T, K, ld_x;          // elements, bytes
    const int32_t *slot, *src;   // src null: no map, row t goes to row t
    int32_t k;
    int64_t M;
    int8_t* q;
    int64_t ld_q;
    float* s;
};

// Four codes of four products, packed.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    const int ia = int(rintf(a)), ib = int(rintf(b)), ic = int(rintf(c)), id = int(rintf(d));
    return uint32_t(ia & 255) | (uint32_t(ib & 255) << 8) | (uint32_t(ic & 255) << 16) | (uint32_t(id) << 24);
}

// One block per token: the largest magnitude, then codes.  kHold pieces of
// the row stay in each thread's registers between the two; a longer row's
// rest is read again, from the cache.  [8192, 8192] bf16: 39 us, 201 MB at 5.2
// TB/s; [4096, 5120] bf16 to 24576 rows 31 us, 168 MB at 5.4 TB/s.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantArgs p) {
    constexpr int kPer = Elem<T>::kPer, kHold = 4;
    constexpr float kFloor = 127.f * 0x1p-126f;
    __shared__ uint32_t sh[4];
    __shared__ int32_t rows[kMaxPicks];                                     // where this token's codes go, or -1
    const uint32_t t = threadIdx.x;
    if (int64_t(blockIdx.x) >= p.T) {
        const int64_t r0 = (int64_t(blockIdx.x) - p.T) * kPadRows;
        for (uint32_t pads = pad_rows(p.src, r0, p.M); pads != 0; pads &= pads - 1) {
            const int64_t r = r0 + __builtin_ctz(pads);
            zero_row(reinterpret_cast<char*>(p.q) + r * p.ld_q, p.K, 1, t, kThreads);
            if (t == 0) p.s[r] = kFloor / 127.f;
        }
        return;
    }
    const int64_t tok = blockIdx.x;
    const int32_t n = p.src ? p.k : 1;
    if (t < uint32_t(n)) {
        const int64_t r = p.src ? int64_t(p.slot[tok * n + t]) : tok;
        rows[t] = r >= 0 && r < p.M ? int32_t(r) : -1;
    }
    const char* x = p.x + tok * p.ld_x;
    const int64_t bytes = p.K * int64_t(sizeof(T));
    const bool whole = bytes >= 16;
    const int64_t pieces = whole ? (bytes + 15) / 16 : 0;
    u32x4 hold[kHold];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int64_t c = int64_t(i) * kThreads + t;
        if (c < pieces) {
            hold[i] = load16(x + (16 * c + 16 > bytes ? bytes - 16 : 16 * c));
            float f[kPer];
            Elem<T>::get(hold[i], f);
#pragma unroll
            for (int e = 0; e < kPer; ++e) m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);
        }
    }
    for (int64_t c = int64_t(kHold) * kThreads + t; c < pieces; c += kThreads) {
        float f[kPer];
        Elem<T>::get(load16(x + (16 * c + 16 > bytes ? bytes - 16 : 16 * c)), f);
#pragma unroll
        for (int e = 0; e < kPer; ++e) m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    }
    float lone = 0.f;
    if (!whole && int64_t(t) < p.K) {
        lone = Elem<T>::one(x + int64_t(t) * sizeof(T));
        m = __float_as_uint(lone) & 0x7FFFFFFFu;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), d, 64)));
    if ((t & 63u) == 0) sh[t >> 6] = m;
    __syncthreads();
    m = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
    const bool bad = m >= 0x7F800000u;
    const float a = fmaxf(__uint_as_float(m), kFloor);
    const float inv = bad ? 0.f : 127.f * (1.f / a);                        // as torch forms 127 / a: the same codes
    const float s = bad ? __uint_as_float(0x7FC00000u) : a / 127.f;

    auto put = [&](int64_t c, u32x4 v) {
        float f[kPer];
        Elem<T>::get(v, f);
        uint32_t o[kPer / 4];
#pragma unroll
        for (int e = 0; e < kPer / 4; ++e) {
            o[e] = pack4(f[4 * e] * inv, f[4 * e + 1] * inv, f[4 * e + 2] * inv, f[4 * e + 3] * inv);
            o[e] = bad ? 0u : o[e];
        }
        const int64_t at = c * kPer + kPer > p.K ? p.K - kPer : c * kPer;
        for (int32_t j = 0; j < n; ++j) {
            const int64_t r = rows[j];
            if (r >= 0) __builtin_memcpy(p.q + r * p.ld_q + at, o, kPer);
        }
    };
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const int64_t c = int64_t(i) * kThreads + t;
        if (c < pieces) put(c, hold[i]);
    }
    for (int64_t c = int64_t(kHold) * kThreads + t; c < pieces; c += kThreads)
        put(c, load16(x + (16 * c + 16 > bytes ? bytes - 16 : 16 * c)));
    for (int32_t j = 0; j < n; ++j) {
        const int64_t r = rows[j];
        if (r < 0) continue;
        if (!whole && int64_t(t) < p.K) p.q[r * p.ld_q + t] = bad ? int8_t(0) : int8_t(int(rintf(lone * inv)));
        if (t == 0) p.s[r] = s;
    }
}

// ------------------------------------------------------------------- combine
struct CombineArgs {
    const char* rows;
    int64_t M, N, ld_r;          // bytes
    const int32_t* slot;
    const float* weight;         // null: 1
    int32_t k;
    int64_t T;
    char* y;
    int64_t ld_y;
    int64_t chunks;              // 64-piece chunks per row
};

// One wave per token and 64 pieces of its row.  4096 tokens of 4 rows of 5120
// in bf16: 38 us when called over and over, 210 MB at 5.5 TB/s (48 to 55 us
// among other kernels).  Reading four rows before the first is added gained
// nothing there (38.2 us) and cost half again with one row (19.8 us for 13.8).
template <typename T>
__global__ __launch_bounds__(kThreads) void combine_kernel(CombineArgs p) {
    constexpr int kPer = Elem<T>::kPer;
    const uint32_t lane = threadIdx.x & 63u;
    const int64_t w = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= p.T * p.chunks) return;
    const int64_t t = w / p.chunks, c = (w - t * p.chunks) * 64 + lane;
    const int32_t* slot = p.slot + t * p.k;
    const float* weight = p.weight ? p.weight + t * p.k : nullptr;
    const int64_t bytes = p.N * int64_t(sizeof(T));
    if (bytes >= 16) {
        if (16 * c >= bytes) return;
        const int64_t at = 16 * c + 16 > bytes ? bytes - 16 : 16 * c;
        float acc[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
        for (int32_t j = 0; j < p.k; ++j) {
            const int64_t s = slot[j];
            if (s < 0 || s >= p.M) continue;
            const float wt = weight ? weight[j] : 1.f;
            float f[kPer];
            Elem<T>::get(load16(p.rows + s * p.ld_r + at), f);
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] = __fmaf_rn(wt, f[e], acc[e]);
        }
        store16(p.y + t * p.ld_y + at, Elem<T>::put(acc));
    } else if (c < p.N) {
        const int64_t at = c * int64_t(sizeof(T));
        float acc = 0.f;
        for (int32_t j = 0; j < p.k; ++j) {
            const int64_t s = slot[j];
            if (s < 0 || s >= p.M) continue;
            acc = __fmaf_rn(weight ? weight[j] : 1.f, Elem<T>::one(p.rows + s * p.ld_r + at), acc);
        }
        Elem<T>::one(p.y + t * p.ld_y + at, acc);
    }
}

struct CombineGradArgs {
    const char* dy;
    int64_t T, N, ld_dy;         // bytes
    const char* rows;
    int64_t ld_r;
    const int32_t *slot, *src;
    const float* weight;         // null: 1
    int32_t k;
    int64_t M;
    char* drows;
    int64_t ld_d;
    float* dweight;
};

// One block per token: dy stays in registers over the token's rows.  4096 tokens
// of 4 rows of 5120 in bf16, 24576 rows written: 84 us, 462 MB at 5.5 TB/s.
template <typename T>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(CombineGradArgs p) {
    constexpr int kPer = Elem<T>::kPer, kHold = 4;
    __shared__ float dots[4][kMaxPicks];
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6;
    const int64_t bytes = p.N * int64_t(sizeof(T));
    if (int64_t(blockIdx.x) >= p.T) {
        const int64_t r0 = (int64_t(blockIdx.x) - p.T) * kPadRows;
        for (uint32_t pads = pad_rows(p.src, r0, p.M); pads != 0; pads &= pads - 1)
            zero_row(p.drows + (r0 + __builtin_ctz(pads)) * p.ld_d, bytes, int(sizeof(T)), t, kThreads);
        return;
    }
    const int64_t tok = blockIdx.x;
    const char* dy = p.dy + tok * p.ld_dy;
    for (int32_t j = int32_t(t); j < p.k; j += kThreads) dots[0][j] = dots[1][j] = dots[2][j] = dots[3][j] = 0.f;
    __syncthreads();
    const int64_t pieces = bytes >= 16 ? (bytes + 15) / 16 : 0;
    for (int64_t c0 = 0; c0 < pieces; c0 += kHold * kThreads) {
        float g[kHold][kPer];
        int64_t at[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int64_t c = c0 + int64_t(i) * kThreads + t;
            at[i] = c < pieces ? (16 * c + 16 > bytes ? bytes - 16 : 16 * c) : -1;
            if (at[i] >= 0) Elem<T>::get(load16(dy + at[i]), g[i]);
        }
        for (int32_t j = 0; j < p.k; ++j) {
            const int64_t s = p.slot[tok * p.k + j];
            if (s < 0 || s >= p.M) continue;
            const float w = p.weight ? p.weight[tok * p.k + j] : 1.f;
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                if (at[i] < 0) continue;
                float o[kPer];
                if (p.dweight) {
                    float f[kPer];
                    Elem<T>::get(load16(p.rows + s * p.ld_r + at[i]), f);
                    // the part that the piece before has already: a row's last piece overlaps it
                    const int skip = int((16 * (c0 + int64_t(i) * kThreads + t) - at[i]) / int64_t(sizeof(T)));
#pragma unroll
                    for (int e = 0; e < kPer; ++e) dot = e >= skip ? __fmaf_rn(g[i][e], f[e], dot) : dot;
                }
#pragma unroll
                for (int e = 0; e < kPer; ++e) o[e] = w * g[i][e];
                store16(p.drows + s * p.ld_d + at[i], Elem<T>::put(o));
            }
            if (p.dweight) {
#pragma unroll
                for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, 64);
                if (lane == 0) dots[wave][j] += dot;
            }
        }
    }
    if (pieces == 0 && wave == 0) {
        for (int32_t j = 0; j < p.k; ++j) {
            const int64_t s = p.slot[tok * p.k + j];
            if (s < 0 || s >= p.M) continue;
            const float w = p.weight ? p.weight[tok * p.k + j] : 1.f;
            float dot = 0.f;
            if (int64_t(lane) < p.N) {
                const int64_t at = int64_t(lane) * int64_t(sizeof(T));
                const float g = Elem<T>::one(dy + at);
                if (p.dweight) dot = g * Elem<T>::one(p.rows + s * p.ld_r + at);
                Elem<T>::one(p.drows + s * p.ld_d + at, w * g);
            }
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, 64);
            if (lane == 0) dots[0][j] = dot;
        }
    }
    __syncthreads();
    if (p.dweight)
        for (int32_t j = int32_t(t); j < p.k; j += kThreads)
            p.dweight[tok * p.k + j] = (dots[0][j] + dots[1][j]) + (dots[2][j] + dots[3][j]);
}

int64_t pad_groups(int64_t M) { return (M + kPadRows - 1) / kPadRows; }

}  // namespace

// Grids in blocks; the caller rejects those whose threads would not fit 32 bits.
uint64_t dispatch_blocks(int64_t T, int64_t M, int64_t row_bytes) {
    const uint64_t chunks = uint64_t((row_bytes + kChunk - 1) / kChunk);
    return ((uint64_t(T) + uint64_t(pad_groups(M))) * chunks + 3) / 4;
}
uint64_t combine_blocks(int64_t T, int64_t row_bytes) {
    return (uint64_t(T) * uint64_t((row_bytes + 1023) / 1024) + 3) / 4;
}
uint64_t token_blocks(int64_t T, int64_t M) { return uint64_t(T) + uint64_t(pad_groups(M)); }

hipError_t launch_dispatch(const void* x, int dtype, int64_t T, int64_t N, int64_t ld_x, const int32_t* slot,
                           const int32_t* src, int32_t k, int64_t M, void* out, int64_t ld_out, hipStream_t stream) {
    const int esz = dtype == 0 ? 4 : 2;
    DispatchArgs p;
    p.x = static_cast<const char*>(x); p.T = T; p.ld_x = ld_x * esz; p.slot = slot; p.src = src; p.k = k; p.M = M;
    p.out = static_cast<char*>(out); p.ld_out = ld_out * esz; p.row = N * esz; p.esz = esz;
    p.chunks = (p.row + kChunk - 1) / kChunk;
    hipLaunchKernelGGL(dispatch_kernel, dim3(uint32_t(dispatch_blocks(T, M, p.row))), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_quantize_rows(const void* x, int dtype, int64_t T, int64_t K, int64_t ld_x, const int32_t* slot,
                                const int32_t* src, int32_t k, int64_t M, int8_t* q, int64_t ld_q, float* s,
                                hipStream_t stream) {
    const int esz = dtype == 0 ? 4 : 2;
    QuantArgs p;
    p.x = static_cast<const char*>(x); p.T = T; p.K = K; p.ld_x = ld_x * esz; p.slot = slot; p.src = src; p.k = k;
    p.M = M; p.q = q; p.ld_q = ld_q; p.s = s;
    const dim3 grid(uint32_t(src ? token_blocks(T, M) : uint64_t(T))), block(kThreads);
    if (dtype == 0) hipLaunchKernelGGL(quantize_kernel<float>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(quantize_kernel<uint16_t>, grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_combine(const void* rows, int dtype, int64_t M, int64_t N, int64_t ld_r, const int32_t* slot,
                          const float* weight, int32_t k, int64_t T, void* y, int64_t ld_y, hipStream_t stream) {
    const int esz = dtype == 0 ? 4 : 2;
    CombineArgs p;
    p.rows = static_cast<const char*>(rows); p.M = M; p.N = N; p.ld_r = ld_r * esz; p.slot = slot; p.weight = weight;
    p.k = k; p.T = T; p.y = static_cast<char*>(y); p.ld_y = ld_y * esz;
    p.chunks = (N * esz + 1023) / 1024;
    const dim3 grid(uint32_t(combine_blocks(T, N * esz))), block(kThreads);
    if (dtype == 0) hipLaunchKernelGGL(combine_kernel<float>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(combine_kernel<uint16_t>, grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_combine_grad(const void* dy, int dtype, int64_t T, int64_t N, int64_t ld_dy, const void* rows,
                               int64_t ld_r, const int32_t* slot, const float* weight, const int32_t* src, int32_t k,
                               int64_t M, void* drows, int64_t ld_d, float* dweight, hipStream_t stream) {
    const int esz = dtype == 0 ? 4 : 2;
    CombineGradArgs p;
    p.dy = static_cast<const char*>(dy); p.T = T; p.N = N; p.ld_dy = ld_dy * esz;
    p.rows = static_cast<const char*>(rows); p.ld_r = ld_r * esz; p.slot = slot; p.src = src; p.weight = weight;
    p.k = k; p.M = M; p.drows = static_cast<char*>(drows); p.ld_d = ld_d * esz; p.dweight = dweight;
    const dim3 grid(uint32_t(token_blocks(T, M))), block(kThreads);
    if (dtype == 0) hipLaunchKernelGGL(combine_grad_kernel<float>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(combine_grad_kernel<uint16_t>, grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace mxq
