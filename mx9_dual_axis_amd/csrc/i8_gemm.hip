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

// Which kernel: a streamed one of (16 MS) x (16 NS) tiles, or whole tiles.
struct Form {
    int ms, ns, threads;         // ms == 0: 128 x 128 tiles
};

Form choose(int64_t M, int64_t N, bool groups, int32_t G) {
    if (groups) {
        const int64_t rows = (M + G - 1) / G;
        if (rows <= 8) return {1, 2, 512};
        if (rows <= 20) return {2, 2, 512};
        if (rows <= 48) return {4, 2, 512};
        return {0, 0, 256};
    }
    if (M <= 16) return N >= 16384 ? Form{1, 2, 512} : Form{1, 1, 512};
    const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
    if (tiles >= 192) return {0, 0, 256};
    return ((M + 63) / 64) * ((N + 63) / 64) >= 192 ? Form{4, 4, 256} : Form{2, 2, 512};
}

template <typename O>
hipError_t launch(I8Args& p, hipStream_t stream) {
    const Form f = choose(p.M, p.N, p.offs != nullptr, p.G);
    switch (f.ms * 8 + f.ns) {
        case 8 + 1: return launch_stream<O, 1, 1, 8, 8, void>(p, stream);
        case 8 + 2: return launch_stream<O, 1, 2, 8, 4, void>(p, stream);
        case 16 + 2: return launch_stream<O, 2, 2, 8, 4, void>(p, stream);
        case 32 + 2: return launch_stream<O, 4, 2, 8, 2, void>(p, stream);
        case 32 + 4: return launch_stream<O, 4, 4, 4, 2, void>(p, stream);
        default: return launch_tiles<O>(p, stream);
    }
}

}  // namespace

// The threads of the grid that a product launches.
uint64_t i8_gemm_threads(int64_t M, int64_t N, bool groups, int32_t G) {
    if (M <= 0 || N <= 0) return 0;
    const Form f = choose(M, N, groups, G);
    const int64_t tm = f.ms ? 16 * f.ms : kTile, tn = f.ms ? 16 * f.ns : kTile;
    return uint64_t(tile_bound(M, tm, groups, G)) * uint64_t((N + tn - 1) / tn) * uint64_t(f.threads);
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
