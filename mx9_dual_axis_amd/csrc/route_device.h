// route_device.h -- what the routing kernels share: scores in registers, 16 lanes
// to a token, keys and their sorting, softmax statistics, prefixes of groups.
#pragma once

#include "mxq_kernels.h"

#include <utility>

namespace mxq {

struct RouteArgs {
    const void* logits;
    int64_t ld;
    const uint8_t* valid;
    int64_t T, M;
    int32_t E, k, align;
    bool normalize;
    int32_t *idx, *slot, *src, *counts, *offs, *live;
    float *weight, *prob, *loss;
    int32_t passes;              // of 64 tokens per block
    int32_t blocks;
    float* ws_prob;              // [blocks][E]
    int32_t* ws_base;            // [blocks][E]: picks of the blocks before (three kernels only)
    int32_t* ws_live;            // [blocks]
    uint16_t* ws_counts;         // [blocks][E]
};

// Blocks of 64-token passes, and what follows the first kernel where there is
// more than one block: totals and prefixes, picks to their rows (route.hip).
// route_begin fills passes, blocks and the workspace's parts.
void route_begin(RouteArgs& p, void* workspace);
hipError_t route_rest(const RouteArgs& p, hipStream_t stream);

namespace {

constexpr int kTok = 64;         // tokens per pass of a block: one 64-bit mask per expert
constexpr int kMaxK = 16;

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), kCtrl, 0xF, 0xF, false));
}
template <int kCtrl>
__device__ __forceinline__ float dpp(float x) {
    return __uint_as_float(dpp<kCtrl>(__float_as_uint(x)));
}
__device__ __forceinline__ uint32_t key_max(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t key_min(uint32_t a, uint32_t b) { return a < b ? a : b; }
// A choice between two values (a conditional between two array elements would
// choose an address, and the array would leave the registers).
template <typename T>
__device__ __forceinline__ T choose(bool c, T a, T b) {
    return c ? a : b;
}

// All-reduce over the 16 lanes of a DPP row (rotations by 8, 4, 2, 1).
__device__ __forceinline__ uint32_t row_top(uint32_t x) {
    x = key_max(x, dpp<0x128>(x));
    x = key_max(x, dpp<0x124>(x));
    x = key_max(x, dpp<0x122>(x));
    return key_max(x, dpp<0x121>(x));
}
__device__ __forceinline__ float row_sum(float x) {
    x += dpp<0x128>(x);
    x += dpp<0x124>(x);
    x += dpp<0x122>(x);
    return x + dpp<0x121>(x);
}
__device__ __forceinline__ uint32_t row_least(uint32_t x) {
    x = key_min(x, dpp<0x128>(x));
    x = key_min(x, dpp<0x124>(x));
    x = key_min(x, dpp<0x122>(x));
    return key_min(x, dpp<0x121>(x));
}
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, dpp<0x128>(x));
    x = fmaxf(x, dpp<0x124>(x));
    x = fmaxf(x, dpp<0x122>(x));
    return fmaxf(x, dpp<0x121>(x));
}

// Scores in memory.  A lane's V scores are V / kC pieces of kC; score v of
// lane l is expert (v / kC) 16 kC + l kC + v % kC.
template <typename L, int V>
struct Scores {
    static constexpr int kC = V < 16 / int(sizeof(L)) ? V : 16 / int(sizeof(L));
    static __device__ __forceinline__ int32_t expert(uint32_t l16, int v) {
        return (v / kC) * (16 * kC) + int32_t(l16) * kC + v % kC;
    }
};
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
template <typename L> __device__ __forceinline__ L narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float x) { return __builtin_bit_cast(uint16_t, __bf16(x)); }

// This lane's scores of one row (-inf past E): in pieces when every lane has
// them whole, else by element, where those past the end read the last one and
// are then replaced.  Either way no load waits for another.
template <typename L, int V, bool kWhole>
__device__ __forceinline__ void fetch_row(const L* row, uint32_t l16, int32_t E, L (&w)[V]) {
    using S = Scores<L, V>;
    if constexpr (kWhole) {
#pragma unroll
        for (int q = 0; q < V / S::kC; ++q)
            __builtin_memcpy(w + q * S::kC, row + S::expert(l16, q * S::kC), S::kC * sizeof(L));
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = row[min(S::expert(l16, v), E - 1)];
    }
}
template <typename L, int V, bool kWhole>
__device__ __forceinline__ void widen_row(const L (&w)[V], uint32_t l16, int32_t E, float (&z)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = kWhole || Scores<L, V>::expert(l16, v) < E ? widen(w[v]) : -INFINITY;
}
// At once (one branch for both halves: with two of them the gradient of 131072
// tokens of 256 fp32 scores took 75 us instead of 57).
template <typename L, int V>
__device__ __forceinline__ void load_row(const L* row, uint32_t l16, int32_t E, float (&z)[V]) {
    L w[V];
    if (E == 16 * V) {                                                      // uniform
        fetch_row<L, V, true>(row, l16, E, w);
        widen_row<L, V, true>(w, l16, E, z);
    } else {
        fetch_row<L, V, false>(row, l16, E, w);
        widen_row<L, V, false>(w, l16, E, z);
    }
}

// Keys: kBits leading bits of the score, ordered, over the inverted expert.
template <typename L> struct Key {
    static constexpr uint32_t kLow = sizeof(L) == 2 ? 0xFFFFu : 0x3FFu;     // the expert's bits
    static constexpr bool kExact = sizeof(L) == 2;
    static __device__ __forceinline__ uint32_t make(float z, int32_t e) {
        const uint32_t b = __float_as_uint(z + 0.f);                        // -0 is +0
        const uint32_t o = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
        return (o & ~kLow) + (kLow - uint32_t(e));
    }
    static __device__ __forceinline__ bool some(uint32_t k) { return k >= 0x00800000u; }   // above -inf
    static __device__ __forceinline__ uint32_t expert(uint32_t k) { return kLow - (k & kLow); }
    static __device__ __forceinline__ float score(uint32_t k) {             // where the key is exact
        const uint32_t o = k & ~kLow;
        return __uint_as_float((o ^ (o & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu)) & ~kLow);
    }
    static __device__ __forceinline__ bool tied(uint32_t a, uint32_t b) { return (a ^ b) <= kLow; }
};

__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
    const uint32_t hi = key_max(a, b);
    b = key_min(a, b);
    a = hi;
}
// Batcher's odd-even merge sort, descending, N a power of two.  The pairs are
// a compile-time list, so that the keys stay in registers.
template <int N>
struct Network {
    int lo[N * 5], hi[N * 5], n;
    constexpr Network() : lo{}, hi{}, n(0) {
        for (int p = 1; p < N; p *= 2)
            for (int q = p; q >= 1; q /= 2)
                for (int j = q % p; j + q < N; j += 2 * q)
                    for (int i = 0; i < q; ++i)
                        if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                            lo[n] = i + j;
                            hi[n++] = i + j + q;
                        }
    }
};
template <int N, int... I>
__device__ __forceinline__ void sort_pairs(uint32_t (&a)[N], std::integer_sequence<int, I...>) {
    constexpr Network<N> net{};
    (exchange(a[net.lo[I]], a[net.hi[I]]), ...);
}
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&a)[N]) {
    constexpr Network<N> net{};
    sort_pairs(a, std::make_integer_sequence<int, net.n>{});
}
// a: the best N of a and b, both descending (the larger of opposite ends is
// bitonic, then log2 N half cleaners).
template <int N>
__device__ __forceinline__ void keep_best(uint32_t (&a)[N], const uint32_t (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = key_max(a[i], b[N - 1 - i]);
#pragma unroll
    for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & d) == 0) exchange(a[i], a[i + d]);
}

// Softmax statistics of a token, given its largest finite score.  p becomes
// exp(z - top); a NaN or +inf among the scores makes the sum NaN or +inf.
struct Row {
    float top, inv;
    bool live, bad;
};
template <int V>
__device__ __forceinline__ Row softmax_row(const float (&z)[V], float top, bool some, float (&p)[V]) {
    Row r;
    r.top = some ? top : 0.f;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = __expf(z[v] - r.top);
        s += p[v];
    }
    s = row_sum(s);
    r.bad = !(s < INFINITY);
    r.live = some || r.bad;
    r.inv = r.bad ? __uint_as_float(0x7FC00000u) : (some ? 1.f / s : 0.f);
    return r;
}

// x of this lane's row plus that of the rows 16 and 32 lanes away, in every
// lane (the swaps put the low and the high half of a pair into one register
// each).
__device__ __forceinline__ float rows_sum(float x) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ float wave_sum(float x) { return rows_sum(row_sum(x)); }

// Inclusive prefix sums over the wave: shifts within the rows of 16, then the
// rows' last lanes handed to the rows after them.
__device__ __forceinline__ int32_t wave_prefix(int32_t x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);         // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);         // row_bcast:15, to rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);         // row_bcast:31, to rows 2 and 3
    return x;
}

// Group starts from counts, by one wave; returns the last group's end.
struct Groups {
    const int32_t* counts;       // LDS
    const float* prob;           // or null
    int32_t* starts;             // LDS
    int32_t* offs;               // or null
    float dot;                   // this lane's part of sum counts * prob
};
__device__ __forceinline__ int32_t scan_groups(int32_t E, int32_t align, Groups& g) {
    const uint32_t lane = threadIdx.x & 63u;
    int32_t carry = 0;
    for (int32_t b = 0; b < E; b += 64) {
        const int32_t e = b + int32_t(lane);
        const int32_t c = e < E ? g.counts[e] : 0;
        const int32_t pad = int32_t(uint32_t(c + align - 1) / uint32_t(align)) * align;
        const int32_t x = wave_prefix(pad);
        if (e < E) {
            g.starts[e] = carry + x - pad;
            if (g.offs) g.offs[e] = carry + x;
            if (g.prob) g.dot += float(c) * g.prob[e];
        }
        carry += __builtin_amdgcn_readlane(x, 63);
    }
    return carry;
}

// After a pass's picks are in LDS: what the block's experts have so far grows by
// theirs; beyond one block, experts and ranks within the block go to memory.
template <int kThr>
__device__ __forceinline__ void note_picks(const RouteArgs& p, int64_t first, const uint16_t* pick, const unsigned long long* mask,
                                           int32_t* sh_count, bool alone) {
    const uint32_t t = threadIdx.x;
    if (!alone) {
        // ranks within the block until the last kernel
        const int64_t left = p.T - first;
        const uint32_t picks = uint32_t(left < kTok ? left : kTok) * uint32_t(p.k);
        for (uint32_t i = t; i < picks; i += kThr) {
            const uint32_t tok = i / uint32_t(p.k), e = pick[i];
            p.idx[first * p.k + i] = e == 0xFFFFu ? -1 : int32_t(e);
            p.slot[first * p.k + i] = e == 0xFFFFu ? -1 : sh_count[e] + __popcll(mask[e] & ((1ull << tok) - 1ull));
        }
        __syncthreads();
    }
    for (uint32_t e = t; e < uint32_t(p.E); e += kThr) sh_count[e] += __popcll(mask[e]);
}

// The block's sums of probabilities (acc, by lane) and its counts: the results
// where it is the only block, else its part of the workspace.
template <int V, int kThr, typename L>
__device__ __forceinline__ void finish_block(const RouteArgs& p, float (&acc)[V], float (*red)[16 * V], const unsigned long long* mask,
                                             const uint16_t* pick, const int32_t* sh_count, int32_t* sh_start,
                                             const int32_t* live, bool alone) {
    using S = Scores<L, V>;
    const uint32_t t = threadIdx.x, l16 = t & 15u, wave = t >> 6;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        acc[v] = rows_sum(acc[v]);
        if ((t & 63u) < 16u) red[wave][S::expert(l16, v)] = acc[v];
    }
    __syncthreads();
    const float n = float(max(live[0], 1));
    for (uint32_t e = t; e < uint32_t(p.E); e += kThr) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kThr / 64; ++w) s += red[w][e];
        const int32_t c = sh_count[e];
        if (alone) {
            p.counts[e] = c;
            red[0][e] = s / n;
            p.prob[e] = s / n;
        } else {
            p.ws_counts[int64_t(blockIdx.x) * p.E + e] = uint16_t(c);
            p.ws_prob[int64_t(blockIdx.x) * p.E + e] = s;
        }
    }
    if (!alone) {
        if (t == 0) p.ws_live[blockIdx.x] = live[0];
        return;
    }
    __syncthreads();
    if (wave == 0) {
        Groups g{sh_count, red[0], sh_start, p.offs, 0.f};
        scan_groups(p.E, p.align, g);
        const float dot = wave_sum(g.dot);
        if (t == 0) {
            p.live[0] = live[0];
            p.loss[0] = float(p.E) * dot / (float(p.k) * n);
        }
    }
    __syncthreads();
    const uint32_t picks = uint32_t(p.T) * uint32_t(p.k);
    for (uint32_t i = t; i < picks; i += kThr) {
        const uint32_t tok = i / uint32_t(p.k), e = pick[i];
        int32_t s = -1;
        if (e != 0xFFFFu) {
            s = sh_start[e] + __popcll(mask[e] & ((1ull << tok) - 1ull));
            p.src[s] = int32_t(i);
        }
        p.idx[i] = e == 0xFFFFu ? -1 : int32_t(e);
        p.slot[i] = s;
    }
}

}  // namespace
}  // namespace mxq
