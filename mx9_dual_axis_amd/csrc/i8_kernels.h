// i8_kernels.h -- matrix product in 8-bit integers with a scale for each row
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
//
// Forms, from few rows to many (choose() in i8_forms.h has the rules and both sides of each):
//   ring   up to 16 rows: bound by the weights' one way from HBM; each wave
//          streams its share through LDS for itself.  One token through [14336,
//          4096]: 12.1 us, its quantization within, 58.7 MB at 4.9 TB/s.
//   pipe   operands in whole 16-byte pieces: tiles of 64 x 64 to 256 x 256,
//          loads straight to LDS.  8192 cubed: 430 to 525 us (2.1 to 2.6 PFLOP/s;
//          the clock falls as the matrix cores fill), 64 experts of [2048, 5120]
//          with 2 rows each 87 us (the weights' 580 MB), with 256 245 us.
//   split  rows that start at any byte, few tiles: the waves of a workgroup
//          split the contraction.  77 x 1000 x 1111: 4.8 us in a graph, 6.8
//          with fp32 activations that it quantizes itself.
//   staged rows that start at any byte, many tiles: as pipe, through registers.
//          512 x 8191 x 4095: 36 us.
#pragma once

#include "epilogue.h"
#include "i8_forms.h"
#include "mxq_kernels.h"

#include <type_traits>

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
    Epilogue e;                  // of the kernels that have one; N counts results then
};

// A row group's bias (the tail's is never added).
template <typename E>
__device__ __forceinline__ const float* bias_of(const I8Args& p, int64_t g, bool zero) {
    if constexpr (!E::kOn) return p.bias;
    else return p.e.bias == nullptr ? nullptr : p.e.bias + (zero ? 0 : g * p.e.bias_gs);
}

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

// 16 codes at any address (the hardware takes it whole; aligning it by hand
// from whole dwords took up to twice the time of a product).
__device__ __forceinline__ v4i load16(const int8_t* p) {
    v4i v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// 16 codes of a row at k, zeros from `end` on, where the row is K long (end <=
// K): near the row's end its last 16 codes are read and shifted.
__device__ __forceinline__ v4i load_codes(const int8_t* row, int64_t k, int64_t end, int64_t K) {
    if (K < 16) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll 1
        for (int i = 0; k + i < end; ++i) w[i >> 2] |= uint32_t(uint8_t(row[k + i])) << (8 * (i & 3));
        return v4i{int(w[0]), int(w[1]), int(w[2]), int(w[3])};
    }
    const int64_t at = k + 16 <= K ? k : K - 16;
    const v4i v = load16(row + at);
    uint64_t lo = uint32_t(v[0]) | (uint64_t(uint32_t(v[1])) << 32), hi = uint32_t(v[2]) | (uint64_t(uint32_t(v[3])) << 32);
    const int skip = int(k - at < 16 ? k - at : 16) * 8;                    // bits before k
    if (skip >= 64) {
        lo = skip < 128 ? hi >> (skip - 64) : 0;
        hi = 0;
    } else if (skip > 0) {
        lo = (lo >> skip) | (hi << (64 - skip));
        hi >>= skip;
    }
    const bool none = k >= end;                                             // `end` is K or whole pieces away
    return none ? v4i{0, 0, 0, 0} : v4i{int(uint32_t(lo)), int(uint32_t(lo >> 32)), int(uint32_t(hi)), int(uint32_t(hi >> 32))};
}

template <typename O> struct Out;
template <> struct Out<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
};
template <> struct Out<__bf16> {
    static __device__ __forceinline__ __bf16 get(float x) { return __bf16(x); }   // nearest-even
};

// ---- few tiles, any alignment: every wave for itself ----
//
// One workgroup of kW waves computes 16 x (16 NS) of C.  Wave w takes the
// steps (128 codes) w, w + kW, ... of the contraction: it loads eight lanes to
// a row, 16 bytes each, lays the pieces out in its own part of LDS (next
// step's loads under way), and multiplies; the waves' integer sums meet at the
// end.  (Loading fragments straight into registers, sixteen rows at a time,
// touched four times as many cache lines per load: 77 x 1000 x 1111 took 8.8
// us, 5.2 so.)

// What a wave multiplies its share of a workgroup's sums by: accumulators
// wave, wave + kW, ... of the 16 x (16 NS) tile.  Read before the contraction,
// whose loads hide theirs.
template <typename O, int NS, int kW, typename E>
struct Share {
    static constexpr int kRegs = (E::kGated ? NS / 2 : NS) * 4, kN = (kRegs + kW - 1) / kW;   // results
    float sa[kN], sb[kN], bias[kN];
    float sb_up[E::kGated ? kN : 1], bias_up[E::kGated ? kN : 1], res[E::kOn ? kN : 1];

    static __device__ __forceinline__ void place(uint32_t q, const RowTile& r, int64_t n0, int64_t* row, int64_t* col) {
        const uint32_t lane = threadIdx.x & 63u;
        *row = r.m0 + 4 * (lane >> 4) + (q & 3u);
        *col = n0 + 16 * (q >> 2) + (lane & 15u);
    }
    __device__ __forceinline__ void load(const I8Args& p, const RowTile& r, int64_t n0, uint32_t wave, const float* sA,
                                         const float* sB, const float* add) {
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            int64_t row, col;
            place(wave + kW * x, r, n0, &row, &col);
            row = row < r.m1 ? row : r.m1 - 1;
            col = col < p.N ? col : p.N - 1;
            sa[x] = sA ? sA[row] : 0.f;
            sb[x] = sB[col];
            bias[x] = add ? add[col] : 0.f;
            if constexpr (E::kGated) {
                sb_up[x] = sB[p.e.up + col];
                bias_up[x] = add ? add[p.e.up + col] : 0.f;
            }
            if constexpr (E::kOn) res[x] = p.e.residual ? float(static_cast<const O*>(p.e.residual)[row * p.e.ld_res + col]) : 0.f;
        }
    }
};

// The sums of a workgroup's waves, which split the contraction, meet in LDS
// and become C's tile.  sA: in LDS, or null where the share has them.
template <typename O, int NS, int kW, typename E>
__device__ __forceinline__ void store_sums(const I8Args& p, const v4i (&acc)[NS], int* sums, const RowTile& r, int64_t n0,
                                           uint32_t wave, const Share<O, NS, kW, E>& share, const float* sA, bool add, bool zero) {
    using S = Share<O, NS, kW, E>;
    constexpr int kAll = NS * 4;
    const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) sums[(wave * kAll + j * 4 + v) * 64 + lane] = acc[j][v];
    __syncthreads();
    O* C = static_cast<O*>(p.C);
#pragma unroll
    for (int x = 0; x < S::kN; ++x) {
        const uint32_t q = wave + kW * x;
        if (q >= uint32_t(S::kRegs)) break;                                 // uniform
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) sum += sums[(w * kAll + q) * 64 + lane];
        int64_t row, col;
        S::place(q, r, n0, &row, &col);
        if (row >= r.m1 || col >= p.N) continue;
        const float sa = sA ? sA[row - r.m0] : share.sa[x];
        float y = float(sum) * sa;
        y = add ? __builtin_fmaf(y, share.sb[x], share.bias[x]) : y * share.sb[x];
        if constexpr (E::kOn) {
            float u = 0.f;
            if constexpr (E::kGated) {
                int other = 0;
#pragma unroll
                for (int w = 0; w < kW; ++w) other += sums[(w * kAll + S::kRegs + q) * 64 + lane];
                u = float(other) * sa;
                u = add ? __builtin_fmaf(u, share.sb_up[x], share.bias_up[x]) : u * share.sb_up[x];
            }
            const O z = ep_one<O, E::kGated>(p.e, y, u, share.res[x]);
            C[row * p.ldc + col] = zero ? Out<O>::get(0.f) : z;
        } else {
            C[row * p.ldc + col] = Out<O>::get(zero ? 0.f : y);
        }
    }
}

// Row of B that a workgroup of few tiles keeps as row 8 q + lr of its own 16 NS:
// channels from n0 on, those past the last repeating it; gated, half of them
// gates and half what these multiply.
template <typename E, int NS>
__device__ __forceinline__ int64_t b_row(const I8Args& p, int64_t n0, int q, uint32_t lr) {
    const bool up = E::kGated && q >= NS;
    const int64_t col = n0 + 8 * (up ? q - NS : q) + lr;
    return (up ? p.e.up : 0) + (col < p.N ? col : p.N - 1);
}

template <typename O, int NS, int kW, typename E>
__global__ __launch_bounds__(64 * kW) void i8_split_kernel(I8Args p) {
    static_assert(!E::kGated || NS % 2 == 0, "both factors' channels");
    constexpr int kRows = 16 * (1 + NS), kLA = 2, kL = 2 * (1 + NS);
    static_assert(kRows * 8 * 4 >= NS * 4 * 64, "the sums take a wave's part of LDS");
    __shared__ v4i lds[kW * kRows * 8];
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = uint32_t(uniform(int32_t(threadIdx.x >> 6)));
    const uint32_t tm = p.offs ? blockIdx.x / p.tiles_n : blockIdx.x % p.tiles_m;
    const uint32_t tn = p.offs ? blockIdx.x - tm * p.tiles_n : blockIdx.x / p.tiles_m;
    RowTile r;
    if (!find_tile<16>(p.offs, p.G, p.M, tm, &r)) return;                  // uniform
    const int64_t n0 = int64_t(tn) * (16 * (E::kGated ? NS / 2 : NS));
    const bool zero = p.offs != nullptr && r.g >= p.G;
    const int8_t* B = p.B + (zero ? 0 : int64_t(r.g) * p.b_gs);
    const float* sB = p.sB + (zero ? 0 : int64_t(r.g) * p.sb_gs);
    const float* add = bias_of<E>(p, r.g, zero);
    Share<O, NS, kW, E> share;
    share.load(p, r, n0, wave, p.sA, sB, add);

    // load q brings rows 8 q .. 8 q + 7 of A's tile, then of B's; rows past the end repeat the last
    const uint32_t lr = lane >> 3, piece = lane & 7u;
    const int8_t* from[kL];
#pragma unroll
    for (int q = 0; q < kL; ++q) {
        const int64_t ar = r.m0 + 8 * q + lr;
        from[q] = q < kLA ? p.A + (ar < r.m1 ? ar : r.m1 - 1) * p.lda : B + b_row<E, NS>(p, n0, q - kLA, lr) * p.ldb;
    }
    v4i* part = lds + wave * (kRows * 8);
    const uint32_t at = lr * 8u + (piece ^ lr);
    v4i v[kL];
    auto load = [&](int64_t k) {
        if (k + 128 <= p.K) {                                              // uniform
#pragma unroll
            for (int q = 0; q < kL; ++q) v[q] = load16(from[q] + k + 16 * piece);
        } else {
#pragma unroll
            for (int q = 0; q < kL; ++q) v[q] = load_codes(from[q], k + 16 * piece, p.K, p.K);
        }
    };
    v4i acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = v4i{0, 0, 0, 0};
    int64_t k = zero ? p.K : 128 * int64_t(wave);
    if (k < p.K) load(k);
    for (; k < p.K; k += 128 * kW) {
#pragma unroll
        for (int q = 0; q < kL; ++q) part[64 * q + at] = v[q];
        if (k + 128 * kW < p.K) load(k + 128 * kW);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t c = (4u * h + g) ^ (l16 & 7u);
            const v4i a = part[l16 * 8u + c];
            v4i b[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) b[j] = part[(16u * (1 + j) + l16) * 8u + c];
#pragma unroll
            for (int j = 0; j < NS; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b[j], acc[j], 0, 0, 0);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();                                                       // every part is read
    store_sums<O, NS, kW, E>(p, acc, reinterpret_cast<int*>(lds), r, n0, wave, share, nullptr, add != nullptr, zero);
}

// ---- many tiles, aligned operands: pipelined through LDS ----
//
// WM x WN waves, each MS x NS fragments of 16 x 16.  A wave's row fragments lie
// 16 WM apart, so that every wave has its part of a tile of few rows, and
// groups multiply only the fragments that hold rows (64 experts of [2048, 5120],
// mean rows 64 and 128: 151 and 164 us so, 169 and 171 with whole tiles).  A
// stage holds 128 codes of every row of an operand; buffer loads put 16-byte
// pieces from memory straight into LDS (no registers stage them), the swizzle
// applied to the address they read, and run SA - 1 (A) and SB - 1 (B) steps
// ahead.  Experts' B comes from HBM, A mostly from L2, so there B runs further
// ahead (mean rows 384 and 512: 2 and 3 stages 317 and 411 us, 2 and 2 325 and
// 433); dense operands, both from L2, gain nothing by it.  Loads complete in
// order, so a step waits only until what was issued after its own is what is
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

template <int MS, int NS, int WM, int WN, int SA, int SB>
struct Pipe {
    static constexpr int kWM = WM, kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int kTM = 16 * MS * WM, kTN = 16 * NS * WN;
    static constexpr int kLA = kTM / 8 / kWaves, kLB = kTN / 8 / kWaves;    // loads per wave and step
    static constexpr uint32_t kStageA = uint32_t(kTM) * 128, kStageB = uint32_t(kTN) * 128;
    static constexpr uint32_t kB = SA * kStageA, kLds = kB + SB * kStageB;  // B's stages follow A's
    static constexpr uint32_t kScales = kLds - uint32_t(kTM + 2 * kTN) * 4; // sA, sB, bias of the tile, once the stages are free
    // loads that may be outstanding while a step's own have arrived
    static constexpr int kLater = (SA - 2) * (kLA + kLB) + (SB > SA ? kLB : 0);
    static_assert(kLA * kWaves * 8 == kTM && kLB * kWaves * 8 == kTN && kLds <= 160 * 1024, "tile");
    static_assert(kThreads >= kTM && kThreads >= kTN && SA >= 2 && SB >= SA && kLater < 64, "scales: one per thread; vmcnt");
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
// with its own L2.  Dense: the tiles are numbered in bands of 8 row tiles,
// column by column, and XCD x takes a contiguous eighth: a column's B is read
// into one L2 (two at a seam), for all its row tiles at once.  (Dealt out
// tile by tile every B was read into several L2s: [8192, 8192] by 128, 512 and
// 1024 rows took 39.1, 74.0 and 80.1 us instead of 25.5, 42.4 and 66.8.)  Row
// groups: XCD x takes a contiguous eighth of the covered row tiles, all column
// tiles of a row tile in a row, then its eighth of the tail.
constexpr uint32_t kBand = 8;

template <int TM>
__device__ bool place_tile(const I8Args& p, RowTile* r, uint32_t* tn) {
    const uint32_t xcd = blockIdx.x & 7u, j = blockIdx.x >> 3;
    if (p.offs == nullptr) {
        const uint32_t tiles = p.tiles_m * p.tiles_n;
        const uint32_t lo = uint32_t(uint64_t(tiles) * xcd / 8u), hi = uint32_t(uint64_t(tiles) * (xcd + 1u) / 8u);
        if (lo + j >= hi) return false;
        const uint32_t band = (lo + j) / (kBand * p.tiles_n), in = lo + j - band * kBand * p.tiles_n;
        const uint32_t height = min(kBand, p.tiles_m - band * kBand);
        *tn = in / height;
        r->m0 = int64_t(band * kBand + in - *tn * height) * TM;
        r->m1 = p.M;
        r->g = 0;
        return true;
    }
    const uint32_t lr = j / p.tiles_n;
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

// Tiles of MS x NS fragments a wave with an epilogue that pairs channels: of a
// wave's 16 NS rows of B the second half are what the first half's results
// multiply.  The channel, from the tile's first, of its row b of B.
template <int NS>
__device__ __forceinline__ uint32_t pair_channel(uint32_t b, bool* up) {
    const uint32_t in = b % (16u * NS);
    *up = in >= 8u * NS;
    return b / (16u * NS) * (8u * NS) + in % (8u * NS);
}

// The tile's scales and bias: read by one thread each while the first steps are
// on their way, put into LDS when the stages are free.
template <typename P, int NS, typename E>
struct Scales {
    float a = 0.f, b = 0.f, bias = 0.f;
    __device__ __forceinline__ void read(const I8Args& p, const float* sB, const float* add, const RowTile& r, int64_t n0,
                                         uint32_t rows, uint32_t cols) {
        const uint32_t t = threadIdx.x;
        if (t < uint32_t(P::kTM)) a = p.sA[r.m0 + min(t, rows - 1u)];
        if (t < uint32_t(P::kTN)) {
            int64_t c = min(t, cols - 1u);
            if constexpr (E::kGated) {
                bool up;
                c = min(pair_channel<NS>(t, &up), cols - 1u);
                if (up) c += p.e.up;
            }
            b = sB[c];
            if (add) bias = add[n0 + c];
        }
    }
    __device__ __forceinline__ void write(uint8_t* lds) const {
        const uint32_t t = threadIdx.x;
        float* sc = reinterpret_cast<float*>(lds + P::kScales);
        if (t < uint32_t(P::kTM)) sc[t] = a;
        if (t < uint32_t(P::kTN)) {
            sc[P::kTM + t] = b;
            sc[P::kTM + P::kTN + t] = bias;
        }
    }
};

// A wave's staged rows (kCols columns at a pitch in bytes) to C in 16-byte
// pieces: non-temporal where C has them whole, else through the L2, where
// neighbours meet (4000 x 5001 x 333: 35 us so, 61 by element).
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
        if (col + kPer <= cols) {
            const uint4 val = *reinterpret_cast<const uint4*>(from);
            const u32x4 vv = {val.x, val.y, val.z, val.w};
            if (whole) __builtin_nontemporal_store(vv, reinterpret_cast<u32x4*>(to));
            else __builtin_memcpy(to, &vv, 16);
        } else {
#pragma unroll 1
            for (uint32_t e = 0; e < kPer && col + e < cols; ++e) to[e] = reinterpret_cast<const O*>(from)[e];
        }
    }
}

// Results of a workgroup's tile, through LDS (whose stages are free now), 16
// rows of the wave tile at a time.
template <typename O, int MS, int NS, typename P, typename E>
__device__ __forceinline__ void store_tile_act(const I8Args& p, const v4i (&acc)[MS][NS], uint8_t* lds, const RowTile& r,
                                               int64_t n0, uint32_t rows, uint32_t cols, uint32_t wave, uint32_t wm,
                                               uint32_t wn, bool add, bool zero) {
    constexpr int kPitch = 16 * NS * 4 + 16, kCols = E::kGated ? 8 * NS : 16 * NS;
    static_assert(P::kWaves * 16 * kPitch <= int(P::kScales), "result staging");
    using R = EpRows<O, kCols>;
    const uint32_t lane = threadIdx.x & 63u, c0 = wn * 16u * NS, o0 = wn * uint32_t(kCols);
    const float* sc = reinterpret_cast<const float*>(lds + P::kScales);
    uint8_t* ep = lds + wave * (16 * kPitch);
    float sb[NS], bi[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        sb[j] = sc[P::kTM + c0 + 16u * j + (lane & 15u)];
        bi[j] = sc[P::kTM + P::kTN + c0 + 16u * j + (lane & 15u)];
    }
    const uint32_t left = cols - min(cols, o0);
    auto first = [&](int i) { return 16u * (uint32_t(P::kWM) * uint32_t(i) + wm); };
    R now;
    if (R::kAhead && p.e.residual) now.read(p.e, r.m0 + first(0), n0 + o0, rows - min(rows, first(0)), left);
#pragma unroll 1
    for (int i = 0; i < MS; ++i) {
        const uint32_t r0 = first(i);
        R next;
        if (!R::kAhead && p.e.residual) now.read(p.e, r.m0 + r0, n0 + o0, rows - min(rows, r0), left);
        if (R::kAhead && i + 1 < MS && p.e.residual)
            next.read(p.e, r.m0 + first(i + 1), n0 + o0, rows - min(rows, first(i + 1)), left);
        each_index<MS>(i, [&](auto at) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const uint32_t row = 4u * (lane >> 4) + v;
                const float sa = sc[r0 + row];
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    const float x = float(acc[decltype(at)::value][j][v]) * sa;
                    reinterpret_cast<float*>(ep + row * kPitch)[16 * j + (lane & 15u)] =
                        add ? __builtin_fmaf(x, sb[j], bi[j]) : x * sb[j];
                }
            }
        });
        __builtin_amdgcn_s_waitcnt(0xC07F);                                 // lgkmcnt(0)
        __builtin_amdgcn_wave_barrier();
        act_switch(p.e.act, [&](auto a) {
            now.template write<decltype(a)::value, E::kGated>(p.e, static_cast<O*>(p.C), p.ldc, ep, kPitch, r.m0 + r0, n0 + o0,
                                                              rows - min(rows, r0), left, zero);
        });
        __builtin_amdgcn_s_waitcnt(0xC07F);                                 // reads done before the next rows' writes
        __builtin_amdgcn_wave_barrier();
        if (R::kAhead) now = next;
    }
}

template <typename O, int MS, int NS, typename P, typename E>
__device__ __forceinline__ void store_tile(const I8Args& p, const v4i (&acc)[MS][NS], uint8_t* lds, const RowTile& r,
                                           int64_t n0, uint32_t rows, uint32_t cols, uint32_t wave, uint32_t wm,
                                           uint32_t wn, bool add, bool zero) {
    if constexpr (E::kOn) return store_tile_act<O, MS, NS, P, E>(p, acc, lds, r, n0, rows, cols, wave, wm, wn, add, zero);
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
        const uint32_t r0 = 16u * (uint32_t(P::kWM) * i + wm);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint32_t row = 4u * (lane >> 4) + v;
            const float sa = sc[r0 + row];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                float x = float(acc[i][j][v]) * sa;
                x = add ? __builtin_fmaf(x, sb[j], bi[j]) : x * sb[j];
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

// One step of a wave: its first I row fragments by all its columns.
template <int I, int MS, int NS, int WM>
__device__ __forceinline__ void multiply(const v4i* ta, const v4i* tb, v4i (&acc)[MS][NS], uint32_t wm, uint32_t wn,
                                         uint32_t lane) {
    v8i a[I];
#pragma unroll
    for (int i = 0; i < I; ++i) a[i] = fragment(ta, 16u * (uint32_t(WM) * i + wm) + (lane & 15u), lane);
    v8i b = fragment(tb, wn * 16u * NS + (lane & 15u), lane);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        v8i nb = b;
        if (j + 1 < NS) nb = fragment(tb, wn * 16u * NS + 16u * (j + 1) + (lane & 15u), lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < I; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(lo4(a[i]), lo4(b), acc[i][j], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < I; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(hi4(a[i]), hi4(b), acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        b = nb;
    }
}

// f(n) for a uniform n in [1, MS].
template <int MS, typename F>
__device__ __forceinline__ void each_count(uint32_t n, F&& f) {
    if constexpr (MS > 1) {
        if (n < uint32_t(MS)) return each_count<MS - 1>(n, f);
    }
    f(std::integral_constant<int, MS>{});
}

template <typename O, int MS, int NS, int WM, int WN, int SA, int SB, bool kGroups, typename E>
__global__ __launch_bounds__(64 * WM * WN, 2) void i8_pipe_kernel(I8Args p) {
    using P = Pipe<MS, NS, WM, WN, SA, SB>;
    constexpr int kOut = E::kGated ? P::kTN / 2 : P::kTN;                   // results of a tile's row
    static_assert(!E::kGated || WM >= 2, "a wave loads rows of one half");
    __shared__ __attribute__((aligned(16))) uint8_t lds[P::kLds];

    const uint32_t t = threadIdx.x, lane = t & 63u;
    const uint32_t wave = uint32_t(uniform(int32_t(t >> 6)));
    const uint32_t wm = wave / WN, wn = wave % WN;

    RowTile r;
    uint32_t tn;
    if (!place_tile<P::kTM>(p, &r, &tn)) return;                            // uniform
    const bool zero = p.offs != nullptr && r.g >= p.G;
    const int64_t n0 = int64_t(tn) * kOut;
    const uint32_t rows = uint32_t(min(int64_t(P::kTM), r.m1 - r.m0)), cols = uint32_t(min(int64_t(kOut), p.N - n0));
    // this wave's part of B's tile begins at its row 8 kLB wave
    bool up = false;
    const uint32_t b0 = E::kGated ? pair_channel<NS>(8u * uint32_t(P::kLB) * wave, &up) : 8u * uint32_t(P::kLB) * wave;
    const int8_t* B = p.B + (zero ? 0 : int64_t(r.g) * p.b_gs) + (n0 + (E::kGated && up ? p.e.up : 0)) * p.ldb;
    const float* sB = p.sB + (zero ? 0 : int64_t(r.g) * p.sb_gs) + n0;
    const float* add = bias_of<E>(p, r.g, zero);
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
    for (int q = 0; q < P::kLB; ++q) vb[q] = min(b0 + 8u * q + lr, cols - 1u) * ldb + lc;
    const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(lds));
    const uint32_t cut = K % 128u != 0 && lc >= K % 128u ? lc : 0u;          // the last step's pieces past K read piece 0
    auto issue_a = [&](uint32_t step, uint32_t slot) {
        const uint32_t k = step * 128u, back = step + 1u == n ? cut : 0u;
#pragma unroll
        for (int q = 0; q < P::kLA; ++q)
            pipe_load16(ra, lds0 + slot * P::kStageA + 1024u * (uint32_t(P::kLA) * wave + q), va[q] - back, k);
    };
    auto issue_b = [&](uint32_t step, uint32_t slot) {
        const uint32_t k = step * 128u, back = step + 1u == n ? cut : 0u;
#pragma unroll
        for (int q = 0; q < P::kLB; ++q) {
            const uint32_t at = lds0 + P::kB + slot * P::kStageB + 1024u * (uint32_t(P::kLB) * wave + q);
            if constexpr (kGroups) pipe_load16_nt(rb, at, vb[q] - back, k);
            else pipe_load16(rb, at, vb[q] - back, k);
        }
    };

    v4i acc[MS][NS];
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) acc[i][j] = v4i{0, 0, 0, 0};

#pragma unroll
    for (uint32_t s = 0; s + 1 < uint32_t(SB); ++s) {                       // as the steps before the first would
        if (s + SA >= uint32_t(SB) && s + SA - SB < n) issue_a(s + SA - SB, s + SA - SB);
        if (s < n) issue_b(s, s);
    }
    Scales<P, NS, E> scales;
    scales.read(p, sB, add, r, n0, rows, cols);
    // The contraction for the first I row fragments of every wave.
    auto contract = [&](auto fragments) {
        constexpr int I = decltype(fragments)::value;
        uint32_t slot_a = 0, slot_b = 0;
        for (uint32_t s = 0; s < n; ++s) {
            // step s has arrived, and of what was issued later the most there can be
            // is under way (near the end, where fewer are, all are waited for)
            if (P::kLater > 0 && s + SB - 2 < n) pipe_sync<P::kLater>();
            else pipe_sync<0>();
            if (s + SA - 1 < n) issue_a(s + SA - 1, slot_a == 0 ? uint32_t(SA - 1) : slot_a - 1u);
            if (s + SB - 1 < n) issue_b(s + SB - 1, slot_b == 0 ? uint32_t(SB - 1) : slot_b - 1u);
            uint8_t* st = lds + slot_a * P::kStageA;
            if (s + 1 == n && K % 128u != 0) {
                const uint32_t c0 = K % 128u / 16u, left = 8u - c0;              // K is whole pieces
                for (uint32_t c = t; c < left * uint32_t(P::kTM); c += uint32_t(P::kThreads)) {
                    const uint32_t row = c / left, piece = c0 + c % left;
                    reinterpret_cast<v4i*>(st)[row * 8u + (piece ^ (row & 7u))] = v4i{0, 0, 0, 0};
                }
                pipe_sync<0>();
            }
            const v4i* ta = reinterpret_cast<const v4i*>(st);
            const v4i* tb = reinterpret_cast<const v4i*>(lds + P::kB + slot_b * P::kStageB);
            multiply<I, MS, NS, WM>(ta, tb, acc, wm, wn, lane);
            slot_a = slot_a + 1u == uint32_t(SA) ? 0u : slot_a + 1u;
            slot_b = slot_b + 1u == uint32_t(SB) ? 0u : slot_b + 1u;
        }
    };
    if constexpr (kGroups) {
        const uint32_t need = (rows + 16u * WM - 1u) / (16u * WM);          // uniform
        each_count<MS>(need, contract);
    } else {
        contract(std::integral_constant<int, MS>{});
    }
    __syncthreads();
    scales.write(lds);
    __syncthreads();

    store_tile<O, MS, NS, P, E>(p, acc, lds, r, n0, rows, cols, wave, wm, wn, add != nullptr, zero);
}

// ---- many tiles, rows that start at any byte: pipelined through registers ----
//
// The tiles, LDS layout and steps of the form above, but a thread's pieces come
// by ordinary loads (which take any address), wait in registers through the
// step before theirs, and are written to the slot that the step before that one
// has left.  Near a row's end the row's last piece is shifted, zeros behind it.
// The loads' rate bounds it (about a clock a lane where they straddle dwords),
// not their latency: two or four steps under way in registers instead of one
// took 19.4 and 19.7 us for 20.1 (128 x 8191 x 4095, 64 x 64 tiles), 46.5 and 48.9
// for 44.5 (512 rows, 128 x 64; two and three).
template <typename O, int MS, int NS, int WM, int WN, typename E>
__global__ __launch_bounds__(64 * WM * WN, 2) void i8_staged_kernel(I8Args p) {
    using P = Pipe<MS, NS, WM, WN, 2, 2>;
    constexpr int kOut = E::kGated ? P::kTN / 2 : P::kTN;                   // results of a tile's row
    static_assert(!E::kGated || WM >= 2, "a wave loads rows of one half");
    __shared__ __attribute__((aligned(16))) uint8_t lds[P::kLds];

    const uint32_t t = threadIdx.x, lane = t & 63u;
    const uint32_t wave = uint32_t(uniform(int32_t(t >> 6)));
    const uint32_t wm = wave / WN, wn = wave % WN;

    RowTile r;
    uint32_t tn;
    if (!place_tile<P::kTM>(p, &r, &tn)) return;                            // uniform
    const bool zero = p.offs != nullptr && r.g >= p.G;
    const int64_t n0 = int64_t(tn) * kOut;
    const uint32_t rows = uint32_t(min(int64_t(P::kTM), r.m1 - r.m0)), cols = uint32_t(min(int64_t(kOut), p.N - n0));
    const int8_t* A = p.A + r.m0 * p.lda;
    // this wave's part of B's tile begins at its row 8 kLB wave
    bool up = false;
    const uint32_t b0 = E::kGated ? pair_channel<NS>(8u * uint32_t(P::kLB) * wave, &up) : 8u * uint32_t(P::kLB) * wave;
    const int8_t* B = p.B + (zero ? 0 : int64_t(r.g) * p.b_gs) + (n0 + (E::kGated && up ? p.e.up : 0)) * p.ldb;
    const float* sB = p.sB + (zero ? 0 : int64_t(r.g) * p.sb_gs) + n0;
    const float* add = bias_of<E>(p, r.g, zero);
    const uint32_t K = uint32_t(p.K), n = zero ? 0u : (K + 127u) / 128u;

    const uint32_t lda = uint32_t(p.lda), ldb = uint32_t(p.ldb);
    const uint32_t lr = lane >> 3, lc = 16u * ((lane & 7u) ^ lr);
    uint32_t va[P::kLA], vb[P::kLB];                                        // of the tile: below 2^31
#pragma unroll
    for (int q = 0; q < P::kLA; ++q) va[q] = min(8u * (uint32_t(P::kLA) * wave + q) + lr, rows - 1u) * lda + lc;
#pragma unroll
    for (int q = 0; q < P::kLB; ++q) vb[q] = min(b0 + 8u * q + lr, cols - 1u) * ldb + lc;
    v4i ha[P::kLA], hb[P::kLB];
    auto load = [&](uint32_t step) {
        const uint32_t k = step * 128u;
        if (k + 128u <= K) {                                                // uniform
            const int8_t *a = A + k, *b = B + k;
#pragma unroll
            for (int q = 0; q < P::kLA; ++q) ha[q] = load16(a + va[q]);
#pragma unroll
            for (int q = 0; q < P::kLB; ++q) hb[q] = load16(b + vb[q]);
        } else {
#pragma unroll
            for (int q = 0; q < P::kLA; ++q) ha[q] = load_codes(A + (va[q] - lc), k + lc, K, K);
#pragma unroll
            for (int q = 0; q < P::kLB; ++q) hb[q] = load_codes(B + (vb[q] - lc), k + lc, K, K);
        }
    };
    auto put = [&](uint32_t slot) {
        v4i* a = reinterpret_cast<v4i*>(lds + slot * P::kStageA) + lane;
        v4i* b = reinterpret_cast<v4i*>(lds + P::kB + slot * P::kStageB) + lane;
#pragma unroll
        for (int q = 0; q < P::kLA; ++q) a[64u * (uint32_t(P::kLA) * wave + q)] = ha[q];
#pragma unroll
        for (int q = 0; q < P::kLB; ++q) b[64u * (uint32_t(P::kLB) * wave + q)] = hb[q];
    };

    v4i acc[MS][NS];
#pragma unroll
    for (int i = 0; i < MS; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) acc[i][j] = v4i{0, 0, 0, 0};

    Scales<P, NS, E> scales;
    if (n > 0) load(0);
    scales.read(p, sB, add, r, n0, rows, cols);
    if (n > 0) put(0);
    if (n > 1) load(1);
    auto contract = [&](auto fragments) {
        constexpr int I = decltype(fragments)::value;
        for (uint32_t s = 0; s < n; ++s) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // step s is in LDS; loads stay under way
            if (s + 1 < n) put((s + 1) & 1u);
            if (s + 2 < n) load(s + 2);
            multiply<I, MS, NS, WM>(reinterpret_cast<const v4i*>(lds + (s & 1u) * P::kStageA),
                                    reinterpret_cast<const v4i*>(lds + P::kB + (s & 1u) * P::kStageB), acc, wm, wn, lane);
        }
    };
    each_count<MS>((rows + 16u * WM - 1u) / (16u * WM), contract);          // uniform
    __syncthreads();
    scales.write(lds);
    __syncthreads();

    store_tile<O, MS, NS, P, E>(p, acc, lds, r, n0, rows, cols, wave, wm, wn, add != nullptr, zero);
}

// ---- up to 16 rows, aligned operands: a ring of LDS slots for each wave ----
//
// One workgroup of kW waves computes 16 x (16 NS) of C.  Wave w takes the steps
// (128 codes) w, w + kW, ... of the contraction for itself: its loads go
// straight into its own ring of kS slots, eight whole 128-byte lines of the
// operands at a time, and it waits for nothing but them, so up to kS steps of
// every wave are under way at any moment and there is no barrier before the
// sums meet.  (Fragments loaded into registers touch sixteen 64-byte pieces per
// quarter wave instead, four times the cache lookups: one row through [8192, 8192]
// takes 13.1 us here and 15.1 us so, 16 rows 13.7 and 20.8.)
//
// X != void: A is not codes but the activations themselves (float or bf16
// bits): every workgroup quantizes the few rows into LDS, with its first
// weights under way, which saves a kernel and its wait.

template <typename X> struct Raw;
template <> struct Raw<void> {
    using T = float;
    static constexpr int kPer = 0;
};
template <> struct Raw<float> {
    using T = float;
    static constexpr int kPer = 4;
    static __device__ __forceinline__ float get(const v4i& w, int e) { return __int_as_float(w[e]); }
    static __device__ __forceinline__ float one(float x) { return x; }
};
template <> struct Raw<uint16_t> {
    using T = uint16_t;
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(const v4i& w, int e) {
        return __uint_as_float(e & 1 ? uint32_t(w[e >> 1]) & 0xFFFF0000u : uint32_t(w[e >> 1]) << 16);
    }
    static __device__ __forceinline__ float one(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
};

// A barrier that leaves loads on their way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ uint32_t row_max(uint32_t x) {                    // over 16 lanes, by DPP rotations
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x128, 0xF, 0xF, false)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x124, 0xF, 0xF, false)));
    x = max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x122, 0xF, 0xF, false)));
    return max(x, uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x121, 0xF, 0xF, false)));
}

// Rows of activations to codes (rows `pitch` bytes apart, zeros up to whole
// 128-code steps) and scales in LDS.  The activations go to LDS themselves
// first (`raw`), every thread's pieces to where it reads them, and `then` puts
// the weights on their way right behind them; `arrived` waits for the former.
template <typename X, int kThr, typename F, typename W>
__device__ __forceinline__ void quantize_to_lds(const I8Args& p, uint8_t* raw, uint8_t* codes, uint32_t pitch,
                                                float* scales, uint32_t* maxes, F&& then, W&& arrived) {
    constexpr int kPer = Raw<X>::kPer, kHold = kFuseBytes / 16 / kThr;
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = uint32_t(uniform(int32_t(t >> 6)));
    const uint32_t per_row = uint32_t(p.K) / kPer, pieces = per_row * uint32_t(p.M), M = uint32_t(p.M);
    const v4i rx = pipe_rsrc(p.A, uint64_t((p.M - 1) * p.lda + p.K) * sizeof(X));
    const uint32_t base = uint32_t(reinterpret_cast<uintptr_t>(raw)) + 1024u * wave;
    uint32_t row[kHold], piece[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        if (uint32_t(i * kThr) >= pieces) break;                            // uniform
        const uint32_t c = min(t + uint32_t(i * kThr), pieces - 1u);        // past the last: that one again
        row[i] = c / per_row;
        piece[i] = c - row[i] * per_row;
        pipe_load16(rx, base + uint32_t(i * kThr) * 16u, (row[i] * uint32_t(p.lda) + piece[i] * kPer) * sizeof(X), 0u);
    }
    then();
    if (t < M) maxes[t] = 0;
    lds_barrier();
    arrived();
    v4i w[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        if (uint32_t(i * kThr) >= pieces) break;
        w[i] = *reinterpret_cast<const v4i*>(raw + uint32_t(i * kThr) * 16u + 1024u * wave + 16u * lane);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) m = max(m, __float_as_uint(Raw<X>::get(w[i], e)) & 0x7FFFFFFFu);
        if (per_row % 16u == 0) {                                           // 16 lanes hold one row's pieces
            m = row_max(m);
            if ((lane & 15u) == 0) atomicMax(&maxes[row[i]], m);
        } else {
            atomicMax(&maxes[row[i]], m);
        }
    }
    lds_barrier();
    if (t < M) {
        const uint32_t m = maxes[t];
        scales[t] = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(m), 127.f * 0x1p-126f) / 127.f;
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        if (uint32_t(i * kThr) >= pieces) break;
        const uint32_t m = maxes[row[i]];
        const float inv = 127.f * (1.f / fmaxf(__uint_as_float(m), 127.f * 0x1p-126f));
        uint32_t* at = reinterpret_cast<uint32_t*>(codes + row[i] * pitch + piece[i] * kPer);
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            uint32_t v = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v |= uint32_t(int(rintf(Raw<X>::get(w[i], 4 * q + e) * inv)) & 255) << (8 * e);
            at[q] = m >= 0x7F800000u ? 0u : v;
        }
    }
    const uint32_t pad = (128u - uint32_t(p.K) % 128u) % 128u / 16u;
    for (uint32_t c = t; c < pad * M; c += kThr)
        *reinterpret_cast<v4i*>(codes + (c / pad) * pitch + uint32_t(p.K) + 16u * (c % pad)) = v4i{0, 0, 0, 0};
    lds_barrier();
}

template <typename O, int NS, int kW, int kS, typename X, typename E>
__global__ __launch_bounds__(64 * kW) void i8_ring_kernel(I8Args p) {
    static_assert(!E::kGated || NS % 2 == 0, "both factors' channels");
    constexpr int kOut = 16 * (E::kGated ? NS / 2 : NS);                    // results of a row
    constexpr bool kFuse = Raw<X>::kPer != 0;
    constexpr int kLA = kFuse ? 0 : 2, kLB = 2 * NS, kLoads = kLA + kLB;
    constexpr uint32_t kSlot = uint32_t(kLoads) * 1024u, kRing = kW * kS * kSlot;
    // codes: rows of a multiple of 128, 16 more against bank conflicts
    constexpr uint32_t kCodes = kFuse ? kFuseBytes / uint32_t(sizeof(typename Raw<X>::T)) + 16 * 128 : 0u;
    constexpr uint32_t kRaw = kFuse ? kFuseBytes : 0u;
    static_assert(kRing + kCodes + kRaw <= 160 * 1024 - 256 && kRing >= kW * NS * 1024u && kS * kLoads < 64, "LDS, vmcnt");
    __shared__ __attribute__((aligned(16))) uint8_t lds[kRing + kCodes + kRaw];
    __shared__ float scales[kFuse ? 16 : 1];
    __shared__ uint32_t maxes[kFuse ? 16 : 1];
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = uint32_t(uniform(int32_t(threadIdx.x >> 6)));
    const int64_t n0 = int64_t(blockIdx.x) * kOut;
    const RowTile r{0, p.M, 0};
    const uint32_t K = uint32_t(p.K), steps = (K + 127u) / 128u;
    const uint32_t mine = steps > wave ? (steps - wave + kW - 1u) / kW : 0u;
    const uint32_t rows = uint32_t(p.M), cols = uint32_t(min(int64_t(kOut), p.N - n0));
    const uint32_t lda = uint32_t(p.lda), ldb = uint32_t(p.ldb);
    const uint32_t lr = lane >> 3, lc = 16u * ((lane & 7u) ^ lr);
    const v4i ra = pipe_rsrc(p.A, kFuse ? 0 : uint64_t(rows - 1u) * lda + K);
    const v4i rb = pipe_rsrc(p.B + n0 * p.ldb, uint64_t(cols - 1u) * ldb + K);
    const v4i ru = pipe_rsrc(p.B + (n0 + (E::kGated ? p.e.up : 0)) * p.ldb, uint64_t(cols - 1u) * ldb + K);
    uint32_t va[2], vb[kLB];
#pragma unroll
    for (int q = 0; q < 2; ++q) va[q] = min(8u * q + lr, rows - 1u) * lda + lc;
#pragma unroll
    for (int q = 0; q < kLB; ++q) vb[q] = min(8u * (E::kGated ? q % NS : q) + lr, cols - 1u) * ldb + lc;
    const uint32_t cut = K % 128u != 0 && lc >= K % 128u ? lc : 0u;          // the last step's pieces past K read piece 0
    const uint32_t ring = uint32_t(reinterpret_cast<uintptr_t>(lds)) + wave * (kS * kSlot);
    auto issue = [&](uint32_t i, uint32_t slot) {
        const uint32_t step = wave + kW * i, back = step + 1u == steps ? cut : 0u, at = ring + slot * kSlot;
#pragma unroll
        for (int q = 0; q < kLB; ++q) pipe_load16_nt(E::kGated && q >= NS ? ru : rb, at + 1024u * q, vb[q] - back, step * 128u);
#pragma unroll
        for (int q = 0; q < kLA; ++q) pipe_load16(ra, at + 1024u * (kLB + q), va[q] - back, step * 128u);
    };
    auto fill = [&]() {
#pragma unroll
        for (uint32_t i = 0; i < uint32_t(kS); ++i)
            if (i < mine) issue(i, i);
    };
    const float* add = bias_of<E>(p, 0, false);
    Share<O, NS, kW, E> share;
    share.load(p, r, n0, wave, kFuse ? nullptr : p.sA, p.sB, add);
    const uint32_t pitch = (K + 127u) / 128u * 128u + 16u;
    uint8_t* codes = lds + kRing;
    if constexpr (kFuse) {
        quantize_to_lds<X, 64 * kW>(p, codes + kCodes, codes, pitch, scales, maxes, fill, [&]() {
            if (mine >= uint32_t(kS)) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kS * kLoads) : "memory");
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        });
    } else {
        fill();
    }

    v4i acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = v4i{0, 0, 0, 0};
    uint32_t slot = 0;
    for (uint32_t i = 0; i < mine; ++i) {
        // step i has arrived; near the end, where fewer are under way, all are waited for
        if (i + kS <= mine) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kS - 1) * kLoads) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint32_t step = wave + kW * i;
        const uint8_t* at = lds + wave * (kS * kSlot) + slot * kSlot;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t piece = 4u * h + g;
            v4i a;
            if constexpr (kFuse) {
                a = *reinterpret_cast<const v4i*>(codes + min(l16, rows - 1u) * pitch + step * 128u + 16u * piece);
            } else {
                a = reinterpret_cast<const v4i*>(at + 1024u * kLB)[l16 * 8u + (piece ^ (l16 & 7u))];
                // codes past K: cleared, and any integer times 0 is 0
                if (step + 1u == steps && step * 128u + 16u * piece >= K) a = v4i{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const v4i b = reinterpret_cast<const v4i*>(at)[(16u * j + l16) * 8u + (piece ^ (l16 & 7u))];
                acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc[j], 0, 0, 0);
            }
        }
        if (i + kS < mine) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");               // the slot is read
            issue(i + kS, slot);
        }
        slot = slot + 1u == uint32_t(kS) ? 0u : slot + 1u;
    }
    __syncthreads();                                                         // every ring is read
    store_sums<O, NS, kW, E>(p, acc, reinterpret_cast<int*>(lds), r, n0, wave, share, kFuse ? scales : nullptr, add != nullptr,
                             false);
}

// ---- few tiles, activations quantized on the way ----
//
// The split form with float or bf16 activations (at any element) as its left
// operand: a wave holds its two steps of 16 rows in registers, the waves'
// largest magnitudes meet in LDS, and each quantizes what it holds.  A column
// tile quantizes the rows anew; while that is little, it costs no more than a
// kernel before the product, and a call saves a launch (fp32, us in a graph and
// as a call, two kernels and this one: 77 x 1000 x 1111, 160 workgroups, 7.9,
// 10.9 and 6.8, 8.7; 64 x 2047 x 2047, 256, 8.9, 11.5 and 9.1, 9.0; 300 x 600 x
// 600, 361, 7.6, 11.5 and 6.8, 8.8; 128 x 1500 x 1023, 376, 7.9, 11.4 and 9.3,
// 9.2; 250 x 770 x 2047, 400, 13.9, 14.0 and 14.3, 14.0).  16 columns a
// workgroup instead of 32: 8.1, 12.1, 8.8, 11.6 and 20.6 in a graph.

template <typename O, typename X, typename E>
__global__ __launch_bounds__(512) void i8_split_fused_kernel(I8Args p) {
    constexpr int NS = 2, kW = 8, kRows = 16 * (1 + NS), kPer = Raw<X>::kPer;
    __shared__ v4i lds[kW * kRows * 8];
    __shared__ uint32_t maxes[kW][16];
    __shared__ float scales[16];
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u, g = lane >> 4;
    const uint32_t wave = uint32_t(uniform(int32_t(threadIdx.x >> 6)));
    const uint32_t tm = blockIdx.x % p.tiles_m, tn = blockIdx.x / p.tiles_m;
    const RowTile r{int64_t(tm) * 16, p.M, 0};
    const int64_t n0 = int64_t(tn) * (16 * (E::kGated ? NS / 2 : NS));
    const uint32_t K = uint32_t(p.K), lr = lane >> 3, piece = lane & 7u;
    const uint32_t k0 = 128u * wave;
    const X* rowx[2];
    const int8_t* rowb[2 * NS];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        rowx[q] = reinterpret_cast<const X*>(p.A) + min(r.m0 + 8 * q + int64_t(lr), p.M - 1) * p.lda;
#pragma unroll
    for (int q = 0; q < 2 * NS; ++q) rowb[q] = p.B + b_row<E, NS>(p, n0, q, lr) * p.ldb;

    // x[h][q]: 16 of row 8 q + lr from 128 (wave + 8 h) + 16 piece, zeros past K
    float x[2][2][16];
    auto read_x = [&](uint32_t h) {
        const uint32_t from = k0 + 1024u * h, k = from + 16u * piece;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (from + 128u <= K) {                                         // uniform
                v4i w[16 / kPer];
#pragma unroll
                for (int c = 0; c < 16 / kPer; ++c) w[c] = load16(reinterpret_cast<const int8_t*>(rowx[q] + k + c * kPer));
#pragma unroll
                for (int e = 0; e < 16; ++e) x[h][q][e] = Raw<X>::get(w[e / kPer], e % kPer);
            } else {
                X w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = rowx[q][min(k + e, K - 1u)];
#pragma unroll
                for (int e = 0; e < 16; ++e) x[h][q][e] = k + e < K ? Raw<X>::one(w[e]) : 0.f;
            }
        }
    };
    v4i b[2][2 * NS];
    auto read_b = [&](uint32_t h) {
        const uint32_t from = k0 + 1024u * h;
#pragma unroll
        for (int q = 0; q < 2 * NS; ++q)
            b[h][q] = from + 128u <= K ? load16(rowb[q] + from + 16u * piece) : load_codes(rowb[q], from + 16u * piece, K, K);
    };
    const bool first = k0 < K, second = k0 + 1024u < K;                     // uniform
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 16; ++e) x[h][q][e] = 0.f;
    if (first) read_x(0);
    if (second) read_x(1);
    if (first) read_b(0);
    if (second) read_b(1);
    const float* add = bias_of<E>(p, 0, false);
    Share<O, NS, kW, E> share;
    share.load(p, r, n0, wave, nullptr, p.sB, add);

#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t m = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(x[h][q][e]) & 0x7FFFFFFFu);
        m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0xB1, 0xF, 0xF, false)));    // quad_perm: lane ^ 1
        m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x4E, 0xF, 0xF, false)));    // quad_perm: lane ^ 2
        m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x141, 0xF, 0xF, false)));   // row_half_mirror
        if (piece == 0) maxes[wave][8 * q + lr] = m;
    }
    lds_barrier();
    v4i a[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) m = max(m, maxes[w][8 * q + lr]);
        const float top = fmaxf(__uint_as_float(m), 127.f * 0x1p-126f);
        const float inv = 127.f * (1.f / top);
        const bool bad = m >= 0x7F800000u;
        if (wave == 0 && piece == 0) scales[8 * q + lr] = bad ? __uint_as_float(0x7FC00000u) : top / 127.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t v = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) v |= uint32_t(int(rintf(x[h][q][4 * c + e] * inv)) & 255) << (8 * e);
                a[h][q][c] = bad ? 0 : int(v);
            }
    }

    v4i* part = lds + wave * (kRows * 8);
    const uint32_t at = lr * 8u + (piece ^ lr);
    v4i acc[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) acc[j] = v4i{0, 0, 0, 0};
    auto step = [&](int h) {
#pragma unroll
        for (int q = 0; q < 2; ++q) part[64 * q + at] = a[h][q];
#pragma unroll
        for (int q = 0; q < 2 * NS; ++q) part[64 * (2 + q) + at] = b[h][q];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t c = (4u * i + g) ^ (l16 & 7u);
            const v4i u = part[l16 * 8u + c];
#pragma unroll
            for (int j = 0; j < NS; ++j)
                acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(u, part[(16u * (1 + j) + l16) * 8u + c], acc[j], 0, 0, 0);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    if (first) step(0);
    if (second) step(1);
    __syncthreads();                                                       // every part is read
    store_sums<O, NS, kW, E>(p, acc, reinterpret_cast<int*>(lds), r, n0, wave, share, scales, add != nullptr, false);
}

template <typename O, typename X, typename E>
hipError_t launch_split_fused(I8Args& p, hipStream_t stream) {
    constexpr int kOut = E::kGated ? 16 : 32;
    p.tiles_m = uint32_t((p.M + 15) / 16);
    p.tiles_n = uint32_t((p.N + kOut - 1) / kOut);
    hipLaunchKernelGGL((i8_split_fused_kernel<O, X, E>), dim3(p.tiles_m * p.tiles_n), dim3(512), 0, stream, p);
    return hipGetLastError();
}

template <typename O, int NS, int kW, int kS, typename X, typename E>
hipError_t launch_ring(I8Args& p, hipStream_t stream) {
    constexpr int kOut = 16 * (E::kGated ? NS / 2 : NS);
    hipLaunchKernelGGL((i8_ring_kernel<O, NS, kW, kS, X, E>), dim3(uint32_t((p.N + kOut - 1) / kOut)), dim3(64 * kW), 0,
                       stream, p);
    return hipGetLastError();
}

template <typename O, int MS, int NS, int WM, int WN, int SA, int SB, bool kGroups, typename E>
hipError_t launch_pipe(I8Args& p, hipStream_t stream) {
    using P = Pipe<MS, NS, WM, WN, SA, SB>;
    constexpr int kOut = E::kGated ? P::kTN / 2 : P::kTN;
    const int64_t tm = tile_bound(p.M, P::kTM, p.offs != nullptr, p.G);
    p.tiles_m = uint32_t(tm);
    p.tiles_n = uint32_t((p.N + kOut - 1) / kOut);
    const uint32_t blocks = p.offs ? uint32_t(group_tiles(tm)) * p.tiles_n : (uint32_t(tm) * p.tiles_n + 7u) / 8u * 8u;
    hipLaunchKernelGGL((i8_pipe_kernel<O, MS, NS, WM, WN, SA, SB, kGroups, E>), dim3(blocks), dim3(64 * WM * WN), 0,
                       stream, p);
    return hipGetLastError();
}

template <typename O, int MS, int NS, int WM, int WN, typename E>
hipError_t launch_staged(I8Args& p, hipStream_t stream) {
    using P = Pipe<MS, NS, WM, WN, 2, 2>;
    constexpr int kOut = E::kGated ? P::kTN / 2 : P::kTN;
    const int64_t tm = tile_bound(p.M, P::kTM, p.offs != nullptr, p.G);
    p.tiles_m = uint32_t(tm);
    p.tiles_n = uint32_t((p.N + kOut - 1) / kOut);
    const uint32_t blocks = p.offs ? uint32_t(group_tiles(tm)) * p.tiles_n : (uint32_t(tm) * p.tiles_n + 7u) / 8u * 8u;
    hipLaunchKernelGGL((i8_staged_kernel<O, MS, NS, WM, WN, E>), dim3(blocks), dim3(64 * WM * WN), 0, stream, p);
    return hipGetLastError();
}

template <typename O, int NS, int kW, typename E>
hipError_t launch_split(I8Args& p, hipStream_t stream) {
    constexpr int kOut = 16 * (E::kGated ? NS / 2 : NS);
    p.tiles_m = uint32_t(tile_bound(p.M, 16, p.offs != nullptr, p.G));
    p.tiles_n = uint32_t((p.N + kOut - 1) / kOut);
    const dim3 grid(p.tiles_m * p.tiles_n), block(64 * kW);
    hipLaunchKernelGGL((i8_split_kernel<O, NS, kW, E>), grid, block, 0, stream, p);
    return hipGetLastError();
}

// Rows of B: a gated product has two to a result.
template <typename E>
int64_t channels(const I8Args& p) {
    return E::kGated ? 2 * p.N : p.N;
}

template <typename O, typename X, typename E>
hipError_t ring(I8Args& p, hipStream_t stream) {
    const int columns = ring_columns(channels<E>(p));
    if constexpr (E::kGated) {
        return columns <= 2 ? launch_ring<O, 2, 4, 3, X, E>(p, stream) : launch_ring<O, 4, 4, 2, X, E>(p, stream);
    } else {
        switch (columns) {
            case 1: return launch_ring<O, 1, 8, 2, X, E>(p, stream);
            case 2: return launch_ring<O, 2, 4, 3, X, E>(p, stream);
            default: return launch_ring<O, 4, 4, 2, X, E>(p, stream);
        }
    }
}

bool pipe_fits(const I8Args& p) {
    const auto aligned = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
    return aligned(p.A) && aligned(p.B) && p.lda % 16 == 0 && p.ldb % 16 == 0 && p.b_gs % 16 == 0 && p.K % 16 == 0 &&
           p.K > 0;
}

template <typename O, typename E>
hipError_t launch(I8Args& p, hipStream_t stream) {
    const Rows rows = far(p.lda, p.ldb) ? Rows::kFar : pipe_fits(p) ? Rows::kPieces : Rows::kBytes;
    const Form f = choose(p.M, channels<E>(p), p.K, p.offs != nullptr, p.G, rows);
    if (f.kind == Kind::kRing) return ring<O, void, E>(p, stream);
    if (f.kind == Kind::kPipe) {
        // experts' weights pass through each L2 about once (measured: 113 us with
        // the hint, 126 without, at 24 rows a group); dense tiles meet in the L2
        // (428 us without, 470 with it, for 8192 cubed)
        if (p.offs) {
            if (f.ms == 1) return launch_pipe<O, 2, 4, 2, 4, 3, 3, true, E>(p, stream);
            if (f.ms == 2) return launch_pipe<O, 4, 4, 2, 4, 2, 4, true, E>(p, stream);
            return launch_pipe<O, 4, 8, 4, 2, 2, 3, true, E>(p, stream);
        }
        if (f.ms == 4) return launch_pipe<O, 4, 8, 4, 2, 2, 2, false, E>(p, stream);
        if (f.ms == 1) return launch_pipe<O, 1, 2, 4, 2, 4, 4, false, E>(p, stream);
        if (f.ns == 4) return launch_pipe<O, 4, 4, 2, 4, 3, 3, false, E>(p, stream);
        if (f.ns == 2) return launch_pipe<O, 2, 4, 4, 2, 4, 4, false, E>(p, stream);
        return launch_pipe<O, 2, 2, 4, 2, 6, 6, false, E>(p, stream);
    }
    if (f.kind == Kind::kStaged) {
        if (f.ms == 1) return launch_staged<O, 1, 2, 4, 2, E>(p, stream);
        if (f.ns == 1) return launch_staged<O, 2, 2, 4, 2, E>(p, stream);
        if (f.ns == 2) return launch_staged<O, 2, 4, 4, 2, E>(p, stream);
        return launch_staged<O, 4, 4, 2, 4, E>(p, stream);
    }
    if constexpr (!E::kGated) {
        if (f.ns == 1) return launch_split<O, 1, 8, E>(p, stream);
    }
    return launch_split<O, 2, 8, E>(p, stream);
}

template <typename X, typename E>
hipError_t fused(I8Args& p, bool ring_fits, int out_dtype, hipStream_t stream) {
    if (ring_fits) return out_dtype == 0 ? ring<float, X, E>(p, stream) : ring<__bf16, X, E>(p, stream);
    return out_dtype == 0 ? launch_split_fused<float, X, E>(p, stream) : launch_split_fused<__bf16, X, E>(p, stream);
}

}  // namespace
}  // namespace mxq
