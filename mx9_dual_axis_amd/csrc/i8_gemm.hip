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

}  // namespace

uint64_t i8_gemm_blocks(int64_t M, int64_t N, bool groups, int32_t G) {
    return uint64_t(tile_bound(M, kTile, groups, G)) * uint64_t((N + kTile - 1) / kTile);
}

hipError_t launch_i8_gemm(const int8_t* A, int64_t lda, const float* sA, const int8_t* B, int64_t ldb, int64_t b_gs,
                          const float* sB, int64_t sb_gs, const float* bias, void* C, int64_t ldc, int64_t M,
                          int64_t N, int64_t K, const int32_t* offs, int32_t G, int out_dtype, hipStream_t stream) {
    I8Args p;
    p.A = A; p.lda = lda; p.sA = sA; p.B = B; p.ldb = ldb; p.b_gs = b_gs; p.sB = sB; p.sb_gs = sb_gs; p.bias = bias;
    p.C = C; p.ldc = ldc; p.M = M; p.N = N; p.K = K; p.offs = offs; p.G = G;
    p.tiles_m = uint32_t(tile_bound(M, kTile, offs != nullptr, G));
    p.tiles_n = uint32_t((N + kTile - 1) / kTile);
    const dim3 grid(p.tiles_m * p.tiles_n), block(256);
    if (out_dtype == 0) hipLaunchKernelGGL(i8_gemm_kernel<float>, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(i8_gemm_kernel<__bf16>, grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace mxq
