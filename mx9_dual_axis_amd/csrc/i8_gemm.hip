// i8_gemm.hip -- matrix product in 8-bit integers with a scale for each row
// of A (token) and each row of B (output channel), dense and by expert.
//
//   C[m][n] = (float(sum_k A[m][k] B[n][k]) sA[m]) sB[n] (+ bias[n])
//
// Both operands hold the contraction contiguous.  The sum is exact in 32-bit
// integers for any codes while K <= 131071 (131071 * 128 * 128 < 2^31), so
// neither tiles, nor splits, nor their order change a result; it is rounded
// once to fp32, then by each multiplication, and to the output type.
//
// v_mfma_i32_16x16x64_i8: lane L holds 16 consecutive codes of operand row
// L % 16; both operands are read alike, so the position of those codes in
// the contraction is free as long as A and B agree.  The result
// C[4 (L/16) + v][L % 16] is element v of lane L's four accumulators.
//
// Row groups: rows offs[g-1] <= m < offs[g] take B + g b_gs, sB + g sb_gs;
// rows from offs[G-1] on give 0.  Groups may have any size.  Row tiles are
// numbered group by group (a group's tiles start at its first row), the tail
// as a last group; every wave finds its tile's group by a prefix sum over
// 64 group ends at a time.
#include "mxq_kernels.h"

namespace mxq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

struct I8Args {
    const int8_t* A;
    int64_t lda;
    const float* sA;
    const int8_t* B;
    int64_t ldb, b_gs;
    const float* sB;
    int64_t sb_gs;
    const float* bias;           // null: none
    void* C;
    int64_t ldc;
    int64_t M, N, K;
    const int32_t* offs;         // null: dense
    int32_t G;
    uint32_t tiles_m, tiles_n;
};

__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// The rows [m0, m1) of row tile `tile` of TM rows and its group (G: the
// tail).  The ends are clamped to an ascending sequence in [0, M], so that
// the tiles partition the rows whatever offs holds.  False past the last tile.
struct RowTile {
    int64_t m0, m1;
    int32_t g;
};

template <int TM>
__device__ bool find_tile(const int32_t* offs, int32_t G, int64_t M, uint32_t tile, RowTile* out) {
    if (offs == nullptr) {
        out->m0 = int64_t(tile) * TM;
        out->m1 = M;
        out->g = 0;
        return out->m0 < M;
    }
    const uint32_t lane = threadIdx.x & 63u;
    int32_t end_carry = 0;       // the last group's end
    uint32_t tiles = 0;          // tiles of the groups before
    for (int32_t base = 0; base <= G; base += 64) {
        const int32_t g = base + int32_t(lane);
        int32_t c = 0;
        if (g < G) c = offs[g];
        if (g >= G) c = int32_t(M);                                // the tail ends with the rows
        c = c < 0 ? 0 : (int64_t(c) > M ? int32_t(M) : c);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(c, d, 64);
            if (lane >= uint32_t(d)) c = max(c, o);
        }
        c = max(c, end_carry);
        int32_t start = __shfl_up(c, 1, 64);
        if (lane == 0) start = end_carry;
        const uint32_t own = g <= G ? uint32_t(c - start + TM - 1) / uint32_t(TM) : 0u;
        uint32_t sum = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = uint32_t(__shfl_up(int(sum), d, 64));
            if (lane >= uint32_t(d)) sum += o;
        }
        const uint64_t past = __ballot(tiles + sum > tile);
        if (past != 0) {
            const int w = __builtin_ctzll(past);
            const uint32_t before = tiles + uint32_t(uniform(__shfl(int(sum - own), w, 64)));
            const int32_t s = uniform(__shfl(start, w, 64)), e = uniform(__shfl(c, w, 64));
            out->m0 = int64_t(s) + int64_t(tile - before) * TM;
            out->m1 = e;
            out->g = base + w;
            return true;
        }
        tiles += uint32_t(uniform(__shfl(int(sum), 63, 64)));
        end_carry = uniform(__shfl(c, 63, 64));
    }
    return false;
}

// Row tiles that any offsets can give: every group and the tail may end in a
// tile of its own.
int64_t tile_bound(int64_t M, int64_t TM, bool groups, int32_t G) {
    const int64_t full = M / TM;
    if (!groups) return (M + TM - 1) / TM;
    const int64_t parts = int64_t(G) + 1;
    return full + (parts < M ? parts : M);
}

// 16 codes of a row at k, zeros from K on; the row is any address.
__device__ __forceinline__ v4i load_codes(const int8_t* row, int64_t k, int64_t K) {
    v4i v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (k < K) {
        uint32_t w[4] = {0, 0, 0, 0};
        const int n = int(K - k);
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (i < n) w[i >> 2] |= uint32_t(uint8_t(row[k + i])) << (8 * (i & 3));
        v = v4i{int(w[0]), int(w[1]), int(w[2]), int(w[3])};
    }
    return v;
}

template <typename O> struct Out;
template <> struct Out<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
};
template <> struct Out<__bf16> {
    static __device__ __forceinline__ __bf16 get(float x) { return __bf16(x); }   // nearest-even
};

// ---- any shape, pitch and alignment: 128 x 128 tiles, 128 codes a step ----
//
// 4 waves, each a 64 x 64 quarter (4 x 4 instructions, twice per step).  The
// next step's 16-byte pieces wait in registers while this one's are
// multiplied from LDS, whose rows of 8 pieces are stored under an XOR of the
// piece with the row (mod 8), so that neither side conflicts.
constexpr int kTile = 128;

template <typename O>
__global__ __launch_bounds__(256, 2) void i8_gemm_kernel(I8Args p) {
    __shared__ v4i lds[2][2][kTile * 8];
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6;
    const uint32_t wm = wave >> 1, wn = wave & 1u;
    const uint32_t tm = blockIdx.x / p.tiles_n, tn = blockIdx.x - tm * p.tiles_n;
    RowTile r;
    if (!find_tile<kTile>(p.offs, p.G, p.M, tm, &r)) return;       // uniform
    const int64_t n0 = int64_t(tn) * kTile;
    const bool zero = p.offs != nullptr && r.g >= p.G;
    const int8_t* B = p.B + (zero ? 0 : int64_t(r.g) * p.b_gs);
    const float* sB = p.sB + (zero ? 0 : int64_t(r.g) * p.sb_gs);

    v4i acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4i{0, 0, 0, 0};

    if (!zero) {
        // this thread's pieces: rows r0 + 32 i, piece ch; rows past the end repeat the last
        const uint32_t r0 = t >> 3, ch = t & 7u;
        const int8_t *ga[4], *gb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t ar = r.m0 + r0 + 32 * i, br = n0 + r0 + 32 * i;
            ga[i] = p.A + (ar < r.m1 ? ar : r.m1 - 1) * p.lda;
            gb[i] = B + (br < p.N ? br : p.N - 1) * p.ldb;
        }
        const uint32_t slot = r0 * 8u + (ch ^ (r0 & 7u));
        v4i va[4], vb[4];
        auto load = [&](int64_t k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                va[i] = load_codes(ga[i], k + 16 * ch, p.K);
                vb[i] = load_codes(gb[i], k + 16 * ch, p.K);
            }
        };
        auto store = [&](int b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lds[b][0][slot + 256 * i] = va[i];
                lds[b][1][slot + 256 * i] = vb[i];
            }
        };
        load(0);
        store(0);
        __syncthreads();
        int buf = 0;
        for (int64_t k = 0; k < p.K; k += 128) {
            const bool more = k + 128 < p.K;
            if (more) load(k + 128);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v4i af[4], bf[4];
                const uint32_t piece = 4u * h + (lane >> 4);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t ar = wm * 64 + 16 * s + (lane & 15u), br = wn * 64 + 16 * s + (lane & 15u);
                    af[s] = lds[buf][0][ar * 8u + (piece ^ (ar & 7u))];
                    bf[s] = lds[buf][1][br * 8u + (piece ^ (br & 7u))];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i], bf[j], acc[i][j], 0, 0, 0);
            }
            if (more) store(buf ^ 1);
            __syncthreads();
            buf ^= 1;
        }
    }

    O* C = static_cast<O*>(p.C);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t col = n0 + wn * 64 + 16 * j + (lane & 15u);
        if (col >= p.N) continue;
        const float sb = sB[col], bi = p.bias ? p.bias[col] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t row = r.m0 + wm * 64 + 16 * i + 4 * (lane >> 4) + v;
                if (row >= r.m1) continue;
                float x = float(acc[i][j][v]) * p.sA[row];
                x = p.bias ? __builtin_fmaf(x, sb, bi) : x * sb;
                C[row * p.ldc + col] = Out<O>::get(zero ? 0.f : x);
            }
        }
    }
}

// ---- few tiles: operands streamed from memory into the instructions ----
//
// One workgroup of kW waves computes (16 MS) x (16 NS) of C; its waves split
// the contraction, each reading its own range of both operands straight into
// fragments (no element is used by two waves, so LDS would only add a copy),
// and their integer sums meet in LDS.  A lane's 16 bytes of 16 rows make 64
// contiguous bytes of each row per load.  kU steps of 64 codes are loaded
// before the first is multiplied.  With one to a few tokens this reads the
// weights once at the rate of memory; with more it is used while whole tiles
// would leave most CUs without work.
//
// X != void: A is not codes but the activations themselves (float or bf16
// bits): every workgroup quantizes the few rows into LDS, after its first
// weights are under way, which saves a kernel and its wait.
constexpr int kFuseBytes = 32 * 1024;    // of activations at most

template <typename X> struct Raw;
template <> struct Raw<void> {
    using T = float;
    static constexpr int kPer = 0;
};
template <> struct Raw<float> {
    using T = float;
    static constexpr int kPer = 4;
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int e) { return __uint_as_float(w[e]); }
};
template <> struct Raw<uint16_t> {
    using T = uint16_t;
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(const uint32_t (&w)[4], int e) {
        return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    }
};

template <typename X>
__device__ __forceinline__ void quantize_to_lds(const I8Args& p, uint8_t* codes, uint32_t pitch, float* scales,
                                                uint32_t* maxes, uint32_t t, uint32_t threads) {
    constexpr int kPer = Raw<X>::kPer, kHold = 4;          // kFuseBytes / 16 pieces over 512 threads
    const uint32_t per_row = uint32_t(p.K) / kPer, pieces = per_row * uint32_t(p.M);
    uint32_t w[kHold][4];
    if (t < 16) maxes[t] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const uint32_t c = t + uint32_t(i) * threads;
        if (c < pieces) {
            const uint32_t row = c / per_row;
            __builtin_memcpy(w[i], reinterpret_cast<const char*>(p.A) +
                                       (int64_t(row) * p.lda + int64_t(c - row * per_row) * kPer) * int64_t(sizeof(X)), 16);
        }
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const uint32_t c = t + uint32_t(i) * threads;
        uint32_t m = 0;
        if (c < pieces) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) m = max(m, __float_as_uint(Raw<X>::get(w[i], e)) & 0x7FFFFFFFu);
        }
        if (per_row % 64 == 0) {                           // a wave's pieces are one row's
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), d, 64)));
            if ((t & 63u) == 0 && c < pieces) atomicMax(&maxes[c / per_row], m);
        } else if (c < pieces) {
            atomicMax(&maxes[c / per_row], m);
        }
    }
    __syncthreads();
    if (t < uint32_t(p.M)) {
        const uint32_t m = maxes[t];
        scales[t] = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(m), 127.f * 0x1p-126f) / 127.f;
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        const uint32_t c = t + uint32_t(i) * threads;
        if (c >= pieces) continue;
        const uint32_t row = c / per_row, m = maxes[row];
        const float inv = 127.f / fmaxf(__uint_as_float(m), 127.f * 0x1p-126f);
        uint32_t o[kPer / 4];
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            uint32_t v = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v |= uint32_t(int(rintf(Raw<X>::get(w[i], 4 * q + e) * inv)) & 255) << (8 * e);
            o[q] = m >= 0x7F800000u ? 0u : v;
        }
        uint32_t* at = reinterpret_cast<uint32_t*>(codes + row * pitch + (c - row * per_row) * kPer);
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) at[q] = o[q];
    }
    // zeros up to whole steps
    const uint32_t pad = (64u - uint32_t(p.K) % 64u) % 64u / 16u;
    for (uint32_t c = t; c < pad * uint32_t(p.M); c += threads)
        *reinterpret_cast<uint4*>(codes + (c / pad) * pitch + uint32_t(p.K) + 16u * (c % pad)) = uint4{0, 0, 0, 0};
    __syncthreads();
}

__device__ __forceinline__ v4i load16(const int8_t* p) {
    v4i v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

template <typename O, int MS, int NS, int kW, int kU, typename X>
__global__ __launch_bounds__(64 * kW) void i8_stream_kernel(I8Args p) {
    constexpr bool kFuse = Raw<X>::kPer != 0;
    constexpr int kRegs = MS * NS * 4;
    constexpr int kSums = kW * kRegs * 256, kCodes = kFuse ? kFuseBytes / int(sizeof(typename Raw<X>::T)) + 16 * 80 : 0;
    __shared__ __attribute__((aligned(16))) uint8_t dyn[kSums > kCodes ? kSums : kCodes];   // sums, the codes before them
    __shared__ float scales[16];
    __shared__ uint32_t maxes[16];
    const uint32_t t = threadIdx.x, lane = t & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = uint32_t(uniform(int32_t(t >> 6)));
    const uint32_t tm = p.offs ? blockIdx.x / p.tiles_n : blockIdx.x % p.tiles_m;
    const uint32_t tn = p.offs ? blockIdx.x - tm * p.tiles_n : blockIdx.x / p.tiles_m;
    RowTile r;
    if (!find_tile<16 * MS>(p.offs, p.G, p.M, tm, &r)) return;             // uniform
    const int64_t n0 = int64_t(tn) * (16 * NS);
    const bool zero = p.offs != nullptr && r.g >= p.G;
    const int8_t* B = p.B + (zero ? 0 : int64_t(r.g) * p.b_gs);
    const float* sB = p.sB + (zero ? 0 : int64_t(r.g) * p.sb_gs);

    const int64_t per = (p.K + kW * 128 - 1) / (kW * 128) * 128;
    const int64_t k0 = zero ? p.K : min(int64_t(wave) * per, p.K), k1 = min(k0 + per, p.K);
    const int8_t *pa[MS], *pb[NS];
    const uint32_t pitch = kFuse ? (uint32_t(p.K) + 63u) / 64u * 64u + 16u : 0u;
#pragma unroll
    for (int i = 0; i < MS; ++i) {
        const int64_t row = r.m0 + 16 * i + l16;
        if constexpr (!kFuse) pa[i] = p.A + (row < r.m1 ? row : r.m1 - 1) * p.lda + 16 * g;
        else pa[i] = reinterpret_cast<const int8_t*>(dyn) + uint32_t(row < p.M ? row : p.M - 1) * pitch + 16 * g;
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int64_t row = n0 + 16 * j + l16;
        pb[j] = B + (row < p.N ? row : p.N - 1) * p.ldb + 16 * g;
    }
    v4i acc[MS][NS];
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) acc[i][j] = v4i{0, 0, 0, 0};

    v4i b[kU][NS];
    int64_t k = k0;
    const bool first = k + 64 * kU <= k1;
    auto load_b = [&]() {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int j = 0; j < NS; ++j) b[u][j] = load16(pb[j] + k + 64 * u);
    };
    if constexpr (kFuse) {
        if (first) load_b();
        quantize_to_lds<typename Raw<X>::T>(p, dyn, pitch, scales, maxes, t, 64 * kW);
    }
    for (; k + 64 * kU <= k1; k += 64 * kU) {
        if (!kFuse || k != k0) load_b();
        v4i a[kU][MS];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < MS; ++i) a[u][i] = load16(pa[i] + k + 64 * u);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < MS; ++i)
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][i], b[u][j], acc[i][j], 0, 0, 0);
    }
    for (; k < k1; k += 64) {
        v4i a[MS], c[NS];
#pragma unroll
        for (int i = 0; i < MS; ++i) a[i] = kFuse ? load16(pa[i] + k) : load_codes(pa[i] - 16 * g, k + 16 * g, p.K);
#pragma unroll
        for (int j = 0; j < NS; ++j) c[j] = load_codes(pb[j] - 16 * g, k + 16 * g, p.K);
#pragma unroll
        for (int i = 0; i < MS; ++i)
#pragma unroll
            for (int j = 0; j < NS; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], c[j], acc[i][j], 0, 0, 0);
    }

    // ---- the waves' sums ----
    if (kFuse) __syncthreads();                                            // the codes are read
    int* red = reinterpret_cast<int*>(dyn);
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[(wave * kRegs + (i * NS + j) * 4 + v) * 64 + lane] = acc[i][j][v];
    __syncthreads();
    O* C = static_cast<O*>(p.C);
    for (uint32_t q = wave; q < uint32_t(kRegs); q += kW) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) sum += red[(w * kRegs + q) * 64 + lane];
        const uint32_t i = q / (4 * NS), j = q / 4 % NS, v = q & 3u;
        const int64_t row = r.m0 + 16 * i + 4 * g + v, col = n0 + 16 * j + l16;
        if (row >= r.m1 || col >= p.N) continue;
        const float sa = kFuse ? scales[row] : p.sA[row];
        float x = float(sum) * sa;
        x = p.bias ? __builtin_fmaf(x, sB[col], p.bias[col]) : x * sB[col];
        C[row * p.ldc + col] = Out<O>::get(zero ? 0.f : x);
    }
}

// ---- many tiles, aligned operands: pipelined through LDS ----
//
// WM x WN waves, each (16 MS) x (16 NS) of the tile.  A stage holds 128 codes
// of every row of both operands; buffer loads put 16-byte pieces from memory
// straight into LDS (no registers stage them), the swizzle applied to the
// address they read, and run kStages - 1 steps ahead.  Loads complete in
// order, so a step waits only until the later steps' loads are the ones
// outstanding; wait and barrier are one asm block, because the compiler's
// barrier would wait for every load.  Within a step a wave keeps all its A
// fragments and reads B one column ahead of the instructions.
//
// Rows past the tile's last repeat it.  In the last step, pieces past the
// end of the contraction (K is whole pieces) load that step's first piece
// again; A's are then cleared in LDS, and any integer times 0 is 0.
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4i pipe_rsrc(const int8_t* base, uint64_t bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    return v4i{uniform(int32_t(uint32_t(b))), uniform(int32_t(uint32_t(b >> 32))), uniform(int32_t(uint32_t(bytes))),
               0x00020000};
}
// 16 bytes per lane from voff + soff of the buffer to LDS at lds + 16 lane.
__device__ __forceinline__ void pipe_load16(v4i r, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(r), "s"(soff), "{m0}"(lds)
                 : "memory");
}
// The same, hinting that the line is not read again from this L2.
__device__ __forceinline__ void pipe_load16_nt(v4i r, uint32_t lds, uint32_t voff, uint32_t soff) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds" ::"v"(voff), "s"(r), "s"(soff), "{m0}"(lds)
                 : "memory");
}
// At most kLeft loads of this wave outstanding, its LDS accesses done, then
// the workgroup's barrier.
template <int kLeft>
__device__ __forceinline__ void pipe_sync() {
    static_assert(kLeft >= 0 && kLeft < 64, "vmcnt immediate");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
}

template <int MS, int NS, int WM, int WN>
struct Pipe {
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int kTM = 16 * MS * WM, kTN = 16 * NS * WN;
    static constexpr int kLA = kTM / 8 / kWaves, kLB = kTN / 8 / kWaves;    // loads per wave and step
    static constexpr uint32_t kB = uint32_t(kTM) * 128, kStage = kB + uint32_t(kTN) * 128;
    static constexpr int kStages = (152 * 1024) / kStage >= 3 ? 3 : 2;
    static constexpr uint32_t kScales = kStages * kStage;                   // sA, sB, bias of the tile
    static constexpr uint32_t kLds = kScales + uint32_t(kTM + 2 * kTN) * 4;
    static constexpr int kLoads = kLA + kLB;
    static_assert(kLA * kWaves * 8 == kTM && kLB * kWaves * 8 == kTN && kLds <= 160 * 1024, "tile");
    static_assert(kThreads >= kTM && kThreads >= kTN, "scales: one per thread");
};

__device__ __forceinline__ v8i fragment(const v4i* tile, uint32_t row, uint32_t lane) {
    const uint32_t g = lane >> 4, sw = lane & 7u;                           // row % 8 == lane % 8
    const v4i lo = tile[row * 8u + (g ^ sw)], hi = tile[row * 8u + ((4u + g) ^ sw)];
    return v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}
__device__ __forceinline__ v4i lo4(const v8i& v) { return v4i{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ v4i hi4(const v8i& v) { return v4i{v[4], v[5], v[6], v[7]}; }

// Row tiles of the groups, and all of them with the tail's.
template <int TM>
__device__ void count_tiles(const int32_t* offs, int32_t G, int64_t M, uint32_t* covered, uint32_t* all) {
    const uint32_t lane = threadIdx.x & 63u;
    int32_t end_carry = 0;
    uint32_t tiles = 0;
    for (int32_t base = 0; base < G; base += 64) {
        const int32_t g = base + int32_t(lane);
        int32_t c = g < G ? offs[g] : 0;
        c = c < 0 ? 0 : (int64_t(c) > M ? int32_t(M) : c);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(c, d, 64);
            if (lane >= uint32_t(d)) c = max(c, o);
        }
        c = max(c, end_carry);
        int32_t start = __shfl_up(c, 1, 64);
        if (lane == 0) start = end_carry;
        uint32_t own = uint32_t(c - start + TM - 1) / uint32_t(TM);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) own += uint32_t(__shfl_xor(int(own), d, 64));
        tiles += uint32_t(uniform(int32_t(own)));
        end_carry = uniform(__shfl(c, 63, 64));
    }
    *covered = tiles;
    *all = tiles + uint32_t((M - end_carry + TM - 1) / TM);
}

// The tile of this workgroup.  Workgroups are dealt to the 8 XCDs in turn, each
// with its own L2.  Row groups: XCD x takes a contiguous eighth of the covered
// row tiles, all column tiles of a row tile in a row, then its eighth of the
// tail.
template <int TM>
__device__ bool place_tile(const I8Args& p, RowTile* r, uint32_t* tn) {
    if (p.offs == nullptr) {
        r->m0 = int64_t(blockIdx.x % p.tiles_m) * TM;
        r->m1 = p.M;
        r->g = 0;
        *tn = blockIdx.x / p.tiles_m;
        return true;
    }
    const uint32_t xcd = blockIdx.x & 7u, j = blockIdx.x >> 3, lr = j / p.tiles_n;
    *tn = j - lr * p.tiles_n;
    uint32_t cov, all;
    count_tiles<TM>(p.offs, p.G, p.M, &cov, &all);
    const uint32_t tail = all - cov;
    const uint32_t c0 = uint32_t(uint64_t(cov) * xcd / 8u), c1 = uint32_t(uint64_t(cov) * (xcd + 1u) / 8u);
    const uint32_t t0 = cov + uint32_t(uint64_t(tail) * xcd / 8u), t1 = cov + uint32_t(uint64_t(tail) * (xcd + 1u) / 8u);
    uint32_t tm;
    if (lr < c1 - c0) tm = c0 + lr;
    else if (lr < (c1 - c0) + (t1 - t0)) tm = t0 + (lr - (c1 - c0));
    else return false;
    return find_tile<TM>(p.offs, p.G, p.M, tm, r);
}

// The tile's scales and bias into LDS.
template <typename P>
__device__ __forceinline__ void load_scales(const I8Args& p, uint8_t* lds, const float* sB, const RowTile& r, int64_t n0,
                                            uint32_t rows, uint32_t cols) {
    const uint32_t t = threadIdx.x;
    float* sc = reinterpret_cast<float*>(lds + P::kScales);
    if (t < uint32_t(P::kTM)) sc[t] = p.sA[r.m0 + min(t, rows - 1u)];
    if (t < uint32_t(P::kTN)) {
        sc[P::kTM + t] = sB[min(t, cols - 1u)];
        sc[P::kTM + P::kTN + t] = p.bias ? p.bias[n0 + min(t, cols - 1u)] : 0.f;
    }
}

// A wave's staged rows (kCols columns at a pitch in bytes) to C: 16-byte
// non-temporal stores where C allows them.
template <typename O, int kCols, int kRows>
__device__ __forceinline__ void store_rows(const I8Args& p, const uint8_t* ep, int pitch, int64_t row0, int64_t col0,
                                           uint32_t rows, uint32_t cols) {
    constexpr int kPer = 16 / int(sizeof(O)), kPieces = kCols / kPer;
    const uint32_t lane = threadIdx.x & 63u;
    O* C = static_cast<O*>(p.C);
    const bool whole = reinterpret_cast<uintptr_t>(C) % 16 == 0 && (p.ldc * int64_t(sizeof(O))) % 16 == 0;
#pragma unroll
    for (int q = 0; q < kRows * kPieces / 64; ++q) {
        const uint32_t piece = 64u * q + lane, row = piece / kPieces, col = piece % kPieces * kPer;
        const uint8_t* from = ep + row * pitch + col * sizeof(O);
        if (row >= rows || col >= cols) continue;
        O* to = C + (row0 + row) * p.ldc + col0 + col;
        if (whole && col + kPer <= cols) {
            const uint4 val = *reinterpret_cast<const uint4*>(from);
            const u32x4 vv = {val.x, val.y, val.z, val.w};
            __builtin_nontemporal_store(vv, reinterpret_cast<u32x4*>(to));
        } else {
#pragma unroll 1
            for (uint32_t e = 0; e < kPer && col + e < cols; ++e) to[e] = reinterpret_cast<const O*>(from)[e];
        }
    }
}

// Results of a workgroup's tile, through LDS (whose stages are free now), 16
// rows of the wave tile at a time.
template <typename O, int MS, int NS, typename P>
__device__ __forceinline__ void store_tile(const I8Args& p, const v4i (&acc)[MS][NS], uint8_t* lds, const RowTile& r,
                                           int64_t n0, uint32_t rows, uint32_t cols, uint32_t wave, uint32_t wm,
                                           uint32_t wn, bool zero) {
    constexpr int kPitch = 16 * NS * int(sizeof(O)) + 16;
    static_assert(P::kWaves * 16 * kPitch <= int(P::kScales), "result staging");
    const uint32_t lane = threadIdx.x & 63u, c0 = wn * 16u * NS;
    const float* sc = reinterpret_cast<const float*>(lds + P::kScales);
    uint8_t* ep = lds + wave * (16 * kPitch);
    float sb[NS], bi[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        sb[j] = sc[P::kTM + c0 + 16u * j + (lane & 15u)];
        bi[j] = sc[P::kTM + P::kTN + c0 + 16u * j + (lane & 15u)];
    }
#pragma unroll
    for (int i = 0; i < MS; ++i) {
        const uint32_t r0 = wm * 16u * MS + 16u * i;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t row = 4u * (lane >> 4) + v;
            const float sa = sc[r0 + row];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                float x = float(acc[i][j][v]) * sa;
                x = p.bias ? __builtin_fmaf(x, sb[j], bi[j]) : x * sb[j];
                reinterpret_cast<O*>(ep + row * kPitch)[16 * j + (lane & 15u)] = Out<O>::get(zero ? 0.f : x);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);                                 // lgkmcnt(0)
        __builtin_amdgcn_wave_barrier();
        store_rows<O, 16 * NS, 16>(p, ep, kPitch, r.m0 + r0, n0 + c0, rows - min(rows, r0), cols - min(cols, c0));
        __builtin_amdgcn_s_waitcnt(0xC07F);                                 // reads done before the next rows' writes
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename O, int MS, int NS, int WM, int WN, bool kStreamB>
__global__ __launch_bounds__(64 * WM * WN, WM * WN >= 8 ? 2 : 1) void i8_pipe_kernel(I8Args p) {
    using P = Pipe<MS, NS, WM, WN>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[P::kLds];

    const uint32_t t = threadIdx.x, lane = t & 63u;
    const uint32_t wave = uint32_t(uniform(int32_t(t >> 6)));
    const uint32_t wm = wave / WN, wn = wave % WN;

    RowTile r;
    uint32_t tn;
    if (!place_tile<P::kTM>(p, &r, &tn)) return;                            // uniform
    const bool zero = p.offs != nullptr && r.g >= p.G;
    const int64_t n0 = int64_t(tn) * P::kTN;
    const uint32_t rows = uint32_t(min(int64_t(P::kTM), r.m1 - r.m0)), cols = uint32_t(min(int64_t(P::kTN), p.N - n0));
    const int8_t* B = p.B + (zero ? 0 : int64_t(r.g) * p.b_gs) + n0 * p.ldb;
    const float* sB = p.sB + (zero ? 0 : int64_t(r.g) * p.sb_gs) + n0;
    const uint32_t K = uint32_t(p.K), n = zero ? 0u : (K + 127u) / 128u;

    // load plan: load j of an operand fills rows 8 j .. 8 j + 7 of its tile
    const uint32_t lda = uint32_t(p.lda), ldb = uint32_t(p.ldb);
    const uint32_t lr = lane >> 3, lc = 16u * ((lane & 7u) ^ lr);
    const v4i ra = pipe_rsrc(p.A + r.m0 * p.lda, uint64_t(rows - 1u) * lda + K);
    const v4i rb = pipe_rsrc(B, uint64_t(cols - 1u) * ldb + K);
    uint32_t va[P::kLA], vb[P::kLB];
#pragma unroll
    for (int q = 0; q < P::kLA; ++q) va[q] = min(8u * (uint32_t(P::kLA) * wave + q) + lr, rows - 1u) * lda + lc;
#pragma unroll
    for (int q = 0; q < P::kLB; ++q) vb[q] = min(8u * (uint32_t(P::kLB) * wave + q) + lr, cols - 1u) * ldb + lc;
    const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(lds));
    const uint32_t cut = K % 128u != 0 && lc >= K % 128u ? lc : 0u;          // the last step's pieces past K read piece 0
    auto issue = [&](uint32_t step, uint32_t stage) {
        const uint32_t k = step * 128u, st = lds0 + stage * P::kStage, back = step + 1u == n ? cut : 0u;
#pragma unroll
        for (int q = 0; q < P::kLA; ++q) pipe_load16(ra, st + 1024u * (uint32_t(P::kLA) * wave + q), va[q] - back, k);
#pragma unroll
        for (int q = 0; q < P::kLB; ++q) {
            const uint32_t at = st + P::kB + 1024u * (uint32_t(P::kLB) * wave + q);
            if constexpr (kStreamB) pipe_load16_nt(rb, at, vb[q] - back, k);
            else pipe_load16(rb, at, vb[q] - back, k);
        }
    };

    v4i acc[MS][NS];
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) acc[i][j] = v4i{0, 0, 0, 0};

#pragma unroll
    for (uint32_t s = 0; s + 1 < uint32_t(P::kStages); ++s)
        if (s < n) issue(s, s);
    load_scales<P>(p, lds, sB, r, n0, rows, cols);                          // while the first stage is on its way
    uint32_t stage = 0;
    for (uint32_t s = 0; s < n; ++s) {
        if constexpr (P::kStages == 3) {
            if (s + 1 < n) pipe_sync<P::kLoads>();
            else pipe_sync<0>();
        } else {
            pipe_sync<0>();
        }
        if (s + P::kStages - 1 < n) {
            const uint32_t free = stage == 0 ? uint32_t(P::kStages - 1) : stage - 1u;
            issue(s + P::kStages - 1, free);
        }
        uint8_t* st = lds + stage * P::kStage;
        if (s + 1 == n && K % 128u != 0) {
            const uint32_t c0 = K % 128u / 16u, left = 8u - c0;              // K is whole pieces
            for (uint32_t c = t; c < left * uint32_t(P::kTM); c += uint32_t(P::kThreads)) {
                const uint32_t row = c / left, piece = c0 + c % left;
                reinterpret_cast<v4i*>(st)[row * 8u + (piece ^ (row & 7u))] = v4i{0, 0, 0, 0};
            }
            pipe_sync<0>();
        }
        const v4i* ta = reinterpret_cast<const v4i*>(st);
        const v4i* tb = reinterpret_cast<const v4i*>(st + P::kB);
        v8i a[MS];
#pragma unroll
        for (int i = 0; i < MS; ++i) a[i] = fragment(ta, wm * 16u * MS + 16u * i + (lane & 15u), lane);
        v8i b = fragment(tb, wn * 16u * NS + (lane & 15u), lane);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            v8i nb = b;
            if (j + 1 < NS) nb = fragment(tb, wn * 16u * NS + 16u * (j + 1) + (lane & 15u), lane);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < MS; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(lo4(a[i]), lo4(b), acc[i][j], 0, 0, 0);
#pragma unroll
            for (int i = 0; i < MS; ++i)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(hi4(a[i]), hi4(b), acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            b = nb;
        }
        stage = stage + 1u == uint32_t(P::kStages) ? 0u : stage + 1u;
    }
    __syncthreads();

    store_tile<O, MS, NS, P>(p, acc, lds, r, n0, rows, cols, wave, wm, wn, zero);
}

// Workgroups of a pipelined product.
template <int MS, int NS, int WM, int WN>
uint64_t pipe_blocks(int64_t M, int64_t N, bool groups, int32_t G, int64_t* tiles_m, int64_t* tiles_n) {
    using P = Pipe<MS, NS, WM, WN>;
    *tiles_m = tile_bound(M, P::kTM, groups, G);
    *tiles_n = (N + P::kTN - 1) / P::kTN;
    // an XCD's share: at most a ceiling of the covered tiles and one of the tail's
    return groups ? uint64_t(8 * ((*tiles_m + 7) / 8 + 1)) * uint64_t(*tiles_n) : uint64_t(*tiles_m) * uint64_t(*tiles_n);
}

template <typename O, int MS, int NS, int WM, int WN, bool kStreamB>
hipError_t launch_pipe(I8Args& p, hipStream_t stream) {
    int64_t tm, tn;
    const uint64_t blocks = pipe_blocks<MS, NS, WM, WN>(p.M, p.N, p.offs != nullptr, p.G, &tm, &tn);
    p.tiles_m = uint32_t(tm);
    p.tiles_n = uint32_t(tn);
    hipLaunchKernelGGL((i8_pipe_kernel<O, MS, NS, WM, WN, kStreamB>), dim3(uint32_t(blocks)), dim3(64 * WM * WN), 0,
                       stream, p);
    return hipGetLastError();
}

template <typename O, int MS, int NS, int kW, int kU, typename X>
hipError_t launch_stream(I8Args& p, hipStream_t stream) {
    p.tiles_m = uint32_t(tile_bound(p.M, 16 * MS, p.offs != nullptr, p.G));
    p.tiles_n = uint32_t((p.N + 16 * NS - 1) / (16 * NS));
    hipLaunchKernelGGL((i8_stream_kernel<O, MS, NS, kW, kU, X>), dim3(p.tiles_m * p.tiles_n), dim3(64 * kW), 0, stream, p);
    return hipGetLastError();
}

template <typename O>
hipError_t launch_tiles(I8Args& p, hipStream_t stream) {
    p.tiles_m = uint32_t(tile_bound(p.M, kTile, p.offs != nullptr, p.G));
    p.tiles_n = uint32_t((p.N + kTile - 1) / kTile);
    hipLaunchKernelGGL(i8_gemm_kernel<O>, dim3(p.tiles_m * p.tiles_n), dim3(256), 0, stream, p);
    return hipGetLastError();
}

// Which kernel.
enum class Kind { kStream, kTiles, kPipe };
struct Form {
    Kind kind;
    int ms, ns;                  // kStream: 16-row sub-tiles; kPipe: ms 64-row units (1, 2 or 4) by 256 columns
    uint64_t threads;            // of the grid
};

// pipe: the operands are whole aligned 16-byte pieces.
//
// Row groups, by the mean rows of a group (64 experts of [2048, 5120], group
// sizes spread by e^0.6; us for tiles of 64, 128 and 256 rows, and streamed):
//   rows    4: 108.0  117.6           145.5       rows  48: 141.8  147.3  156.3  266.1
//   rows   16: 107.6  113.9           186.6       rows 128: 234.1  173.5  201.1
//   rows   24: 134.7  113.1  159.4    204.1       rows 192:        229.1  214.0
//   rows   32: 135.3  115.0  153.9    217.3       rows 384:        394.6  320.1
// (the 671 MB of weights alone take 108 us at 6.2 TB/s).  Groups of unaligned
// operands are streamed while they are small.
Form choose(int64_t M, int64_t N, bool groups, int32_t G, bool pipe) {
    auto stream = [&](int ms, int ns, int waves) {
        return Form{Kind::kStream, ms, ns,
                    uint64_t(tile_bound(M, 16 * ms, groups, G)) * uint64_t((N + 16 * ns - 1) / (16 * ns)) * 64u * uint64_t(waves)};
    };
    auto piped = [&](int units) {
        int64_t tm, tn;
        const uint64_t blocks = units == 1   ? pipe_blocks<2, 4, 2, 4>(M, N, groups, G, &tm, &tn)
                                : units == 2 ? pipe_blocks<4, 4, 2, 4>(M, N, groups, G, &tm, &tn)
                                             : pipe_blocks<4, 8, 4, 2>(M, N, groups, G, &tm, &tn);
        return Form{Kind::kPipe, units, 0, blocks * 512};
    };
    const Form tiles{Kind::kTiles, 0, 0, uint64_t(tile_bound(M, kTile, groups, G)) * uint64_t((N + kTile - 1) / kTile) * 256};
    if (groups) {
        const int64_t rows = (M + G - 1) / G;
        if (pipe) return piped(rows <= 16 ? 1 : rows <= 160 ? 2 : 4);
        if (rows <= 8) return stream(1, 2, 8);
        if (rows <= 20) return stream(2, 2, 8);
        if (rows <= 48) return stream(4, 2, 8);
        return tiles;
    }
    if (M <= 16) return N >= 16384 ? stream(1, 2, 8) : stream(1, 1, 8);
    if (((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile) >= 192) return pipe ? piped(4) : tiles;
    return ((M + 63) / 64) * ((N + 63) / 64) >= 192 ? stream(4, 4, 4) : stream(2, 2, 8);
}

bool pipe_fits(const I8Args& p) {
    const auto aligned = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    return aligned(p.A) && aligned(p.B) && p.lda % 16 == 0 && p.ldb % 16 == 0 && p.b_gs % 16 == 0 && p.K % 16 == 0 &&
           p.K > 0 && p.lda < (1 << 23) && p.ldb < (1 << 23);
}

template <typename O>
hipError_t launch(I8Args& p, hipStream_t stream) {
    const Form f = choose(p.M, p.N, p.offs != nullptr, p.G, pipe_fits(p));
    if (f.kind == Kind::kPipe) {
        // experts' weights pass through each L2 about once (measured: 113 us with
        // the hint, 126 without, at 24 rows a group); dense tiles meet in the L2
        // (428 us without, 470 with it, for 8192 cubed)
        if (f.ms == 1) return launch_pipe<O, 2, 4, 2, 4, true>(p, stream);
        if (f.ms == 2) return launch_pipe<O, 4, 4, 2, 4, true>(p, stream);
        return p.offs ? launch_pipe<O, 4, 8, 4, 2, true>(p, stream) : launch_pipe<O, 4, 8, 4, 2, false>(p, stream);
    }
    if (f.kind == Kind::kTiles) return launch_tiles<O>(p, stream);
    switch (f.ms * 8 + f.ns) {
        case 8 + 1: return launch_stream<O, 1, 1, 8, 8, void>(p, stream);
        case 8 + 2: return launch_stream<O, 1, 2, 8, 4, void>(p, stream);
        case 16 + 2: return launch_stream<O, 2, 2, 8, 4, void>(p, stream);
        case 32 + 2: return launch_stream<O, 4, 2, 8, 2, void>(p, stream);
        default: return launch_stream<O, 4, 4, 4, 2, void>(p, stream);
    }
}

}  // namespace

// The threads of the largest grid that a product of this shape launches.
uint64_t i8_gemm_threads(int64_t M, int64_t N, bool groups, int32_t G) {
    if (M <= 0 || N <= 0) return 0;
    const uint64_t a = choose(M, N, groups, G, false).threads, b = choose(M, N, groups, G, true).threads;
    return a > b ? a : b;
}

hipError_t launch_i8_gemm(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs,
                          const float* sB, int64_t sb_gs, const float* bias, void* C, int64_t ldc, int64_t M,
                          int64_t N, int64_t K, const int32_t* offs, int32_t G, int out_dtype, hipStream_t stream) {
    I8Args p;
    p.A = A; p.lda = lda; p.sA = sA; p.B = B; p.ldb = ldb; p.b_gs = b_gs; p.sB = sB; p.sb_gs = sb_gs; p.bias = bias;
    p.C = C; p.ldc = ldc; p.M = M; p.N = N; p.K = K; p.offs = offs; p.G = G; p.tiles_m = p.tiles_n = 0;
    return out_dtype == 0 ? launch<float>(p, stream) : launch<__bf16>(p, stream);
}

bool i8_linear_fuses(int64_t M, int64_t K, int dtype) {
    return M <= 16 && K > 0 && K % 16 == 0 && M * K * (dtype == 0 ? 4 : 2) <= kFuseBytes;
}

hipError_t launch_i8_linear_fused(const void* x, int dtype, int64_t ld_x, const int8_t* B, int64_t ldb, const float* sB,
                                  const float* bias, void* C, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                  int out_dtype, hipStream_t stream) {
    I8Args p;
    p.A = static_cast<const int8_t*>(x); p.lda = ld_x; p.sA = nullptr; p.B = B; p.ldb = ldb; p.b_gs = 0; p.sB = sB;
    p.sb_gs = 0; p.bias = bias; p.C = C; p.ldc = ldc; p.M = M; p.N = N; p.K = K; p.offs = nullptr; p.G = 0;
    p.tiles_m = p.tiles_n = 0;
    if (dtype == 0)
        return out_dtype == 0 ? launch_stream<float, 1, 1, 8, 8, float>(p, stream)
                              : launch_stream<__bf16, 1, 1, 8, 8, float>(p, stream);
    return out_dtype == 0 ? launch_stream<float, 1, 1, 8, 8, uint16_t>(p, stream)
                          : launch_stream<__bf16, 1, 1, 8, 8, uint16_t>(p, stream);
}

}  // namespace mxq
