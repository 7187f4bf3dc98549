// route.hip -- expert routing of a batch of tokens, and the gradient of its
// weights and balance loss.
//
//   live token   valid[t] and some logit above -inf
//   p[t][e]      softmax of the logits of a live token, else 0
//   picks        the k largest logits above -inf, equal ones lowest expert
//                first; weight = p of the pick, or that over the picks' sum
//   counts[e]    picks of e; group e of the padded buffer holds them in token
//                order and ends at offs[e], a multiple of align
//   prob[e]      mean of p[t][e] over the live tokens
//   loss         E sum_e counts[e] / (k live) prob[e]
//
// Lanes: 16 lanes of a wave hold one token's scores, V = 2^n >= E/16 each (four
// tokens per wave); reductions over a token stay inside a 16-lane row, where
// DPP rotations need no LDS.  A lane's scores come in 16-byte pieces that
// alternate between the lanes, so a load covers contiguous memory.
//
// Selection: each score becomes a 32-bit key, its leading bits in an order
// of unsigned integers over the inverted expert, so keys are unique and equal
// scores go to the lowest expert.  A lane sorts its keys once (merge networks
// keep its best 8 or 16), then each pick is a maximum over the row's heads and
// the winner drops its head: a round costs 4 DPP steps and a few moves,
// however many experts there are.  A bf16 score fits its key whole.  Of an
// fp32 score 22 bits do; the picks are then checked by their scores, and where
// those are out of order, or the last pick's 22 bits equal those of the score
// after it (or a lane has given away all the keys it kept), the four tokens of the wave are selected again by exact
// comparisons (about one wave in seven for scores spread like a normal
// distribution over 256 experts).  Measured for 131072 tokens of 256 fp32
// scores: exact maxima over all scores for each pick 86.6 us, sorted 64-bit
// keys (double) 88 us, this selection 56 us.
//
// Order: a block takes 64 tokens at a time, so the tokens that picked an
// expert are one 64-bit mask in LDS, and a pick's rank is a population count
// below its token's bit.  Ranks, counts and every floating sum are therefore
// in a fixed order: the same inputs give the same bits.  Up to 64 tokens one
// block does everything.  Beyond, each block leaves its counts, and a second
// kernel adds those of the blocks before and places the picks; when that is
// much to read for every block, a kernel between them forms the prefixes.
#include "mxq_kernels.h"

#include <utility>

namespace mxq {
namespace {

constexpr int kTok = 64;         // tokens per pass of a block: one 64-bit mask per expert
constexpr int kMaxK = 16;

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

// Rows of the padded buffer that no pick owns: the end of each group (a wave
// for each expert in turn) and what follows the last group.
__device__ __forceinline__ void clear_pads(const RouteArgs& p, const int32_t* counts, const int32_t* starts,
                                           int32_t total, uint32_t block, uint32_t blocks, uint32_t threads) {
    const uint32_t lane = threadIdx.x & 63u, waves = threads / 64u;
    const int32_t w = __builtin_amdgcn_readfirstlane(int32_t(block * waves + (threadIdx.x >> 6)));
    for (int32_t e = w; e < p.E; e += int32_t(blocks * waves)) {
        const int32_t end = e + 1 < p.E ? starts[e + 1] : total;
        for (int32_t r = starts[e] + counts[e] + int32_t(lane); r < end; r += 64) p.src[r] = -1;
    }
    for (int64_t r = total + int64_t(block) * threads + threadIdx.x; r < p.M; r += int64_t(blocks) * threads)
        p.src[r] = -1;
}

// kThr threads: kThr / 16 tokens at once.  kKeep: the sorted keys a lane
// keeps, enough for k (or all V).
template <typename L, int V, int kKeep, int kThr>
__global__ __launch_bounds__(kThr) void route_kernel(RouteArgs p) {
    using KT = Key<L>;
    using S = Scores<L, V>;
    __shared__ unsigned long long mask[16 * V];
    __shared__ float red[kThr / 64][16 * V];
    // the scores, for the picks to read theirs (a row's own wave alone uses it)
    __shared__ __attribute__((aligned(16))) float stash[KT::kExact ? 1 : kThr / 16][KT::kExact ? 1 : 16 * V];
    __shared__ uint16_t pick[kTok * kMaxK];
    __shared__ int32_t sh_count[16 * V], sh_start[16 * V];
    __shared__ int32_t sh_live;

    const uint32_t t = threadIdx.x, l16 = t & 15u, grp = t >> 4, wave = t >> 6;
    const bool alone = gridDim.x == 1;
    for (uint32_t e = t; e < 16u * V; e += kThr) sh_count[e] = 0;
    if (t == 0) sh_live = 0;
    if (alone)                                                              // the picks' rows are written over this
        for (int64_t r = t; r < p.M; r += kThr) p.src[r] = -1;

    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    const L* logits = static_cast<const L*>(p.logits);
    // Scores are read a round ahead where the registers allow it at four waves a
    // SIMD and a block has several rounds (the three kernels, without and with it: 131072 tokens of 256 fp32
    // scores 72.6 and 71.5 us, of 64 bf16 scores 37.1 and 35.8, 65536 of 160
    // 39.3 and 36.7).
    constexpr bool kAhead = V <= 16 && kThr == 256;
    L ahead[kAhead ? V : 1];
    uint8_t take_ahead = 1;
    if constexpr (kAhead) {
        const int64_t row = int64_t(blockIdx.x) * p.passes * kTok + grp;
        const int64_t at = row < p.T ? row : p.T - 1;
        if (p.T > 0) {
            take_ahead = p.valid ? p.valid[at] : uint8_t(1);
            if (p.E == 16 * V) fetch_row<L, V, true>(logits + at * p.ld, l16, p.E, ahead);
            else fetch_row<L, V, false>(logits + at * p.ld, l16, p.E, ahead);
        }
    }
    for (int32_t pass = 0; pass < p.passes; ++pass) {
        const int64_t first = (int64_t(blockIdx.x) * p.passes + pass) * kTok;
        if (first >= p.T && first > 0) break;                               // uniform
        for (uint32_t e = t; e < 16u * V; e += kThr) mask[e] = 0;
        __syncthreads();
        for (uint32_t sub = 0; sub < kTok; sub += kThr / 16) {
            const uint32_t tok = sub + grp;
            // What follows from the lane alone is formed anew for each token:
            // kept over the loop it would take half the registers.
            uint32_t l16 = t & 15u;
            asm volatile("" : "+v"(l16));
            const int64_t row = first + tok;
            if (first + sub >= p.T) break;                                  // uniform
            // a row past the end reads the last one; its scores do not count
            const int64_t at = row < p.T ? row : p.T - 1;
            float z[V], q[V];
            uint8_t take;
            if constexpr (kAhead) {
                if (p.E == 16 * V) widen_row<L, V, true>(ahead, l16, p.E, z);  // uniform
                else widen_row<L, V, false>(ahead, l16, p.E, z);
                take = take_ahead;
                // the next tokens' scores, while these are sorted
                if (sub + kThr / 16 < uint32_t(kTok) || pass + 1 < p.passes) {
                    const int64_t next = row + kThr / 16 < p.T ? row + kThr / 16 : p.T - 1;
                    take_ahead = p.valid ? p.valid[next] : uint8_t(1);
                    if (p.E == 16 * V) fetch_row<L, V, true>(logits + next * p.ld, l16, p.E, ahead);
                    else fetch_row<L, V, false>(logits + next * p.ld, l16, p.E, ahead);
                }
            } else {
                take = p.valid ? p.valid[at] : uint8_t(1);
                load_row<L, V>(logits + at * p.ld, l16, p.E, z);
            }
            const bool in = (row < p.T) & (take != 0);
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = choose(in, z[v], -INFINITY);
            if constexpr (!KT::kExact) {
#pragma unroll
                for (int v = 0; v < V; ++v) stash[grp][S::expert(l16, v)] = z[v];
            }
            float high = z[0];
#pragma unroll
            for (int v = 1; v < V; ++v) high = fmaxf(high, z[v]);
            high = row_max(high);
            const bool some = high > -INFINITY;
            const Row r = softmax_row<V>(z, high, some, q);
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = __fmaf_rn(q[v], r.inv, acc[v]);
            if (l16 == 0 && r.live) atomicAdd(&sh_live, 1);
            __builtin_amdgcn_sched_barrier(0);                              // the probabilities are dead from here

            uint32_t best[kKeep];
#pragma unroll
            for (int v = 0; v < kKeep; ++v) best[v] = KT::make(z[v], S::expert(l16, v));
            sort_desc(best);
#pragma unroll
            for (int b = kKeep; b < V; b += kKeep) {
                uint32_t more[kKeep];
#pragma unroll
                for (int v = 0; v < kKeep; ++v) more[v] = KT::make(z[b + v], S::expert(l16, b + v));
                sort_desc(more);
                keep_best(best, more);
            }
            uint32_t mine = 0, last = 0;
#pragma unroll 1
            for (int j = 0; j < p.k; ++j) {
                last = row_top(best[0]);
                mine = l16 == uint32_t(j) ? last : mine;
                const bool win = best[0] == last;
#pragma unroll
                for (int i = 0; i + 1 < kKeep; ++i) best[i] = choose(win, best[i + 1], best[i]);
                best[kKeep - 1] = choose(win, 0u, best[kKeep - 1]);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            // this lane's pick: its expert and score
            bool ok = KT::some(mine);
            uint32_t expert = ok ? KT::expert(mine) : 0u;
            float score = KT::score(mine);
            if constexpr (!KT::kExact) {
                score = ok ? stash[grp][expert] : -INFINITY;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const float after = dpp<0x101>(score);                      // the next lane's (row_shl:1)
                const uint32_t next = row_top(best[0]);
                // a lane that won kKeep rounds has no key left (0 is none's) and may have
                // dropped the score after the last pick
                const bool wrong = (l16 + 1u < uint32_t(p.k) && score < after) || (KT::some(next) && KT::tied(last, next)) ||
                                   (V > kKeep && best[0] == 0u);
                if (__ballot(wrong) != 0) {                                 // uniform: the wave's four tokens
                    // the best score that comes after the last pick, k times
                    ok = false;
                    float top = INFINITY;
                    uint32_t least = 0;
#pragma unroll 1
                    for (int j = 0; j < p.k; ++j) {
                        float m = -INFINITY;
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const bool left = (z[v] < top) | ((z[v] == top) & (uint32_t(S::expert(l16, v)) > least));
                            m = fmaxf(m, choose(left, z[v], -INFINITY));
                        }
                        m = row_max(m);
                        uint32_t e = 0xFFFFFFFFu;
#pragma unroll
                        for (int v = V - 1; v >= 0; --v) {
                            const uint32_t x = uint32_t(S::expert(l16, v));
                            e = choose((z[v] == m) & ((m < top) | (x > least)), x, e);
                        }
                        e = row_least(e);
                        top = m;
                        least = e;
                        if (l16 == uint32_t(j) && m > -INFINITY) {
                            ok = true;
                            expert = e;
                            score = m;
                        }
                    }
                }
            }
            ok = ok && !r.bad;
            float w = r.bad ? r.inv : (ok ? __expf(score - r.top) * r.inv : 0.f);
            if (p.normalize) {
                const float sum = row_sum(l16 < uint32_t(p.k) ? w : 0.f);
                if (r.live) w /= sum;
            }
            if (l16 < uint32_t(p.k) && row < p.T) {
                const uint32_t e = ok ? expert : 0xFFFFu;
                pick[tok * uint32_t(p.k) + l16] = uint16_t(e);
                if (ok) atomicOr(&mask[e], 1ull << tok);
                p.weight[row * p.k + l16] = w;
            }
        }
        __syncthreads();
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

    // ---- the block's sums ----
#pragma unroll
    for (int v = 0; v < V; ++v) {
        acc[v] = rows_sum(acc[v]);
        if ((t & 63u) < 16u) red[wave][S::expert(l16, v)] = acc[v];
    }
    __syncthreads();
    const float n = float(max(sh_live, 1));
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
        if (t == 0) p.ws_live[blockIdx.x] = sh_live;
        return;
    }
    __syncthreads();
    if (wave == 0) {
        Groups g{sh_count, red[0], sh_start, p.offs, 0.f};
        scan_groups(p.E, p.align, g);
        const float dot = wave_sum(g.dot);
        if (t == 0) {
            p.live[0] = sh_live;
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

// The sums over all blocks of 16 experts: totals, prefixes, mean probability.
// One workgroup for 16 experts, 64 segments of the blocks each.
__global__ __launch_bounds__(1024) void route_scan_kernel(RouteArgs p) {
    __shared__ int32_t sc[64][17];
    __shared__ float sp[64][17];
    __shared__ int32_t sl[16];
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6;
    int32_t n = 0;
    for (int32_t b = int32_t(t); b < p.blocks; b += 1024) n += p.ws_live[b];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d, 64);
    if (lane == 0) sl[wave] = n;

    const uint32_t seg = t >> 4, col = t & 15u;
    const int32_t e = int32_t(blockIdx.x) * 16 + int32_t(col);
    const int32_t per = (p.blocks + 63) / 64;
    const int32_t b0 = min(int32_t(seg) * per, p.blocks), b1 = min(b0 + per, p.blocks);
    int32_t c = 0;
    float s = 0.f;
    if (e < p.E) {
#pragma unroll 8
        for (int32_t b = b0; b < b1; ++b) {
            c += p.ws_counts[int64_t(b) * p.E + e];
            s += p.ws_prob[int64_t(b) * p.E + e];
        }
    }
    sc[seg][col] = c;
    sp[seg][col] = s;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) n += sl[w];
    {
        // wave w: the segments of column w
        const int32_t own = sc[lane][wave];
        const int32_t x = wave_prefix(own);
        const float tot = wave_sum(sp[lane][wave]);
        const int32_t we = int32_t(blockIdx.x) * 16 + int32_t(wave);
        if (lane == 63u && we < p.E) {
            p.counts[we] = x;
            p.prob[we] = tot / float(max(n, 1));
        }
        __syncthreads();
        sc[lane][wave] = x - own;
    }
    __syncthreads();
    if (e < p.E) {
        int32_t run = sc[seg][col];
#pragma unroll 8
        for (int32_t b = b0; b < b1; ++b) {
            p.ws_base[int64_t(b) * p.E + e] = run;
            run += p.ws_counts[int64_t(b) * p.E + e];
        }
    }
    if (blockIdx.x == 0 && t == 0) p.live[0] = n;
}


// Places the picks of one block of the first kernel per workgroup.  kSum: the
// workgroup adds the counts of the blocks before its own itself, and the first
// one (which places nothing) the totals.
template <bool kSum, int kPlaceThr>
__global__ __launch_bounds__(kPlaceThr) void route_place_kernel(RouteArgs p) {
    constexpr int kHold = 4;     // picks per thread that are read before the sums are waited for
    __shared__ int32_t sh_count[1024], sh_start[1024];
    __shared__ int32_t sh_before[kSum ? 1024 : 1];
    __shared__ float sh_prob[kSum ? 1024 : 1];   // segments x experts, then the experts' means
    __shared__ int32_t sh_total, sh_live;
    const uint32_t t = threadIdx.x;
    const bool first = blockIdx.x == 0;
    const int32_t block = kSum ? int32_t(blockIdx.x) - 1 : int32_t(blockIdx.x);
    const int64_t from = int64_t(block) * p.passes * kTok, left = p.T - from, most = int64_t(p.passes) * kTok;
    const uint32_t picks = block < 0 ? 0u : uint32_t(most < left ? most : left) * uint32_t(p.k);
    int32_t he[kHold], hs[kHold];
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const uint32_t i = t + uint32_t(h) * kPlaceThr;
        he[h] = i < picks ? p.idx[from * p.k + i] : -1;
        hs[h] = i < picks ? p.slot[from * p.k + i] : -1;
    }
    if constexpr (kSum) {
        for (int32_t e = int32_t(t); e < p.E; e += kPlaceThr) {
            sh_count[e] = 0;
            sh_before[e] = 0;
        }
        if (t == 0) sh_live = 0;
        __syncthreads();
        if (first) {
            int32_t n = 0;
            for (int32_t b = int32_t(t); b < p.blocks; b += kPlaceThr) n += p.ws_live[b];
            if (n) atomicAdd(&sh_live, n);
        }
        // a thread adds a segment of the blocks for one expert (integer sums
        // have no order; the probabilities' segments are added in turn below)
        const int32_t segs = max(1, kPlaceThr / p.E), per = (p.blocks + segs - 1) / segs;
        for (int32_t i = int32_t(t); i < p.E * segs; i += kPlaceThr) {
            const int32_t e = i % p.E, s = i / p.E;
            if (first) {
                float sum = 0.f;
#pragma unroll 16
                for (int32_t b = s * per; b < min((s + 1) * per, p.blocks); ++b) sum += p.ws_prob[int64_t(b) * p.E + e];
                sh_prob[i] = sum;
            }
            const int32_t b0 = s * per, b1 = min(b0 + per, p.blocks);
            int32_t c = 0, before = 0;
#pragma unroll 16
            for (int32_t b = b0; b < b1; ++b) {
                const int32_t x = p.ws_counts[int64_t(b) * p.E + e];
                c += x;
                before += b < block ? x : 0;
            }
            if (c) atomicAdd(&sh_count[e], c);
            if (before) atomicAdd(&sh_before[e], before);
        }
        __syncthreads();
        if (first) {
            const float n = float(max(sh_live, 1));
            for (int32_t e = int32_t(t); e < p.E; e += kPlaceThr) {
                float sum = 0.f;
                for (int32_t s = 0; s < segs; ++s) sum += sh_prob[s * p.E + e];
                sh_prob[e] = sum / n;
                p.prob[e] = sum / n;
                p.counts[e] = sh_count[e];
            }
            if (t == 0) p.live[0] = sh_live;
            __syncthreads();
        }
    } else {
        for (int32_t e = int32_t(t); e < p.E; e += kPlaceThr) sh_count[e] = p.counts[e];
        if (t == 0) sh_live = p.live[0];
        __syncthreads();
    }
    if (t < 64) {
        Groups g{sh_count, first ? (kSum ? sh_prob : p.prob) : nullptr, sh_start, first ? p.offs : nullptr, 0.f};
        const int32_t total = scan_groups(p.E, p.align, g);
        const float dot = wave_sum(g.dot);
        if (t == 0) {
            sh_total = total;
            if (first) p.loss[0] = float(p.E) * dot / (float(p.k) * float(max(sh_live, 1)));
        }
    }
    __syncthreads();
    auto place = [&](uint32_t i, int32_t e, int32_t rank) {
        if (e < 0) return;
        const int64_t at = from * p.k + i;
        const int32_t s = sh_start[e] + (kSum ? sh_before[e] : p.ws_base[int64_t(block) * p.E + e]) + rank;
        p.slot[at] = s;
        p.src[s] = int32_t(at);
    };
#pragma unroll
    for (int h = 0; h < kHold; ++h) place(t + uint32_t(h) * kPlaceThr, he[h], hs[h]);
    for (uint32_t i = t + kHold * kPlaceThr; i < picks; i += kPlaceThr) place(i, p.idx[from * p.k + i], p.slot[from * p.k + i]);
    clear_pads(p, sh_count, sh_start, sh_total, blockIdx.x, gridDim.x, kPlaceThr);
}

// ---- gradient ----
//
//   a[e] = dloss E counts[e] / (k live^2)          (balance loss, by p)
//   not normalized: a[t][idx_j] += dweight_j,      dlogits = p (a - sum_e p a)
//   normalized:     dlogits = p (a - sum_e p a), + w_j (dweight_j - sum w dweight) at idx_j
//
// One pass: the row is in registers between the softmax and the result.
struct RouteGradArgs {
    const void* logits;
    int64_t ld;
    const uint8_t* valid;
    int64_t T;
    int32_t E, k;
    bool normalize;
    const int32_t *idx, *counts, *live;
    const float *weight, *dweight, *dloss;
    void* dlogits;
    int64_t ld_d;
};

constexpr int kGradThr = 256;

// The gradient reads logits and writes dlogits once: HBM bounds it, at the
// latency of a row's loads.  A row's memory is therefore read a round ahead
// (up to 256 experts, where the registers allow four waves a SIMD), and the
// loss's part of each expert stays in LDS, not in registers.  131072 tokens of
// 256 fp32 scores take 51 us (a copy kernel moves as many bytes in 54; 58
// without either measure), of 256 bf16 scores 42 (27; 59), 65536 of 384 bf16
// scores 40 (20; 90).
template <typename L, int V>
__global__ __launch_bounds__(kGradThr) void route_grad_kernel(RouteGradArgs p) {
    using S = Scores<L, V>;
    constexpr int kC = S::kC;
    __shared__ __attribute__((aligned(16))) float up[kGradThr / 16][16 * V];   // each row's own wave alone uses it
    __shared__ __attribute__((aligned(16))) float share[16 * V];           // the loss's part of each expert
    const uint32_t t = threadIdx.x, l16 = t & 15u, grp = t >> 4;
    const bool whole = p.E == 16 * V, picks = p.dweight != nullptr && l16 < uint32_t(p.k);
    // what a row takes from memory, read a round ahead
    L ahead[V];
    uint8_t take = 1;
    int32_t e_ahead = -1;
    float c_ahead = 0.f, w_ahead = 0.f;
    auto fetch = [&](int64_t at, uint32_t l16) {
        if (p.valid) take = p.valid[at];
        if (whole) fetch_row<L, V, true>(static_cast<const L*>(p.logits) + at * p.ld, l16, p.E, ahead);
        else fetch_row<L, V, false>(static_cast<const L*>(p.logits) + at * p.ld, l16, p.E, ahead);
        if (picks) {
            e_ahead = p.idx[at * p.k + l16];
            c_ahead = p.dweight[at * p.k + l16];
            w_ahead = p.weight[at * p.k + l16];
        }
    };
    int64_t row = int64_t(blockIdx.x) * (kGradThr / 16) + grp;
    const int64_t step = int64_t(gridDim.x) * (kGradThr / 16);
    constexpr bool kAhead = V <= 16;
    if (kAhead) fetch(row < p.T ? row : p.T - 1, l16);
    const float n = float(max(p.live[0], 1));
    const float unit = p.dloss ? p.dloss[0] * float(p.E) / (float(p.k) * n * n) : 0.f;
    for (uint32_t e = t; e < 16u * V; e += kGradThr) share[e] = int32_t(e) < p.E ? unit * float(p.counts[e]) : 0.f;
    __syncthreads();
    for (; row < p.T; row += step) {
        uint32_t l16 = t & 15u;                                             // formed anew, as in routing
        asm volatile("" : "+v"(l16));
        if (!kAhead) fetch(row, l16);
        float z[V], q[V];
        const bool in = take != 0;
        if (whole) widen_row<L, V, true>(ahead, l16, p.E, z);
        else widen_row<L, V, false>(ahead, l16, p.E, z);
        int32_t e = e_ahead;
        float c = c_ahead, w = w_ahead;
        if (uint32_t(e) >= uint32_t(p.E)) {
            e = -1;
            c = w = 0.f;
        }
        if (kAhead && row + step < p.T) fetch(row + step, l16);
        // the picks' direct part, scattered over the row through LDS
        float d[V];
        if (p.dweight != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) up[grp][S::expert(l16, v)] = 0.f;
            if (p.normalize) c = w * (c - row_sum(w * c));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (e >= 0) up[grp][e] = c;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = up[grp][S::expert(l16, v)];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = 0.f;
        }
        float m = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = choose(in, z[v], -INFINITY);
            m = fmaxf(m, z[v]);
        }
        m = row_max(m);
        const Row r = softmax_row<V>(z, m, m > -INFINITY, q);
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            q[v] *= r.inv;
            const float a = share[S::expert(l16, v)];
            s += q[v] * (p.normalize ? a : a + d[v]);
        }
        s = row_sum(s);
        L* out = static_cast<L*>(p.dlogits) + row * p.ld_d;
#pragma unroll
        for (int b = 0; b < V / kC; ++b) {
            const int32_t e0 = S::expert(l16, b * kC);
            L o[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const int v = b * kC + i;
                const float a = share[e0 + i];
                const float g = p.normalize ? q[v] * (a - s) + d[v] : q[v] * (a + d[v] - s);
                o[i] = narrow<L>(r.live ? g : 0.f);
            }
            if (e0 + kC <= p.E) {
                __builtin_memcpy(out + e0, o, kC * sizeof(L));
            } else {
#pragma unroll
                for (int i = 0; i < kC; ++i)
                    if (e0 + i < p.E) out[e0 + i] = o[i];
            }
        }
    }
}

template <typename L, int V, int kKeep>
hipError_t run_first(const RouteArgs& p, hipStream_t stream) {
    const dim3 grid(uint32_t(p.blocks));
    if (p.T <= 4) {
        hipLaunchKernelGGL((route_kernel<L, V, kKeep, 64>), grid, dim3(64), 0, stream, p);
        return hipGetLastError();
    }
    // Few blocks of many threads hide more of their loads: up to 512 blocks of up
    // to 128 experts, up to a block a CU beyond (256, 512 and 1024 threads, the
    // three kernels: 16384 x 256 fp32 29.6, 24.8 and 24.4 us, 4096 x 256 26.2, 21.3
    // and 20.4, 8192 x 512 40.5, 32.4 and 40.7; but 32768 x 256 34.5, 37.4 and 36.7,
    // and 131072 x 256 71.5, 97.3 and 96.5).
    constexpr int kMany = V <= 16 ? 1024 : 512;
    if constexpr (V <= 32) {
        if (V <= 8 ? p.passes == 1 : p.blocks <= 256) {
            hipLaunchKernelGGL((route_kernel<L, V, kKeep, kMany>), grid, dim3(kMany), 0, stream, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((route_kernel<L, V, kKeep, 256>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

template <typename L>
hipError_t route_first(const RouteArgs& p, hipStream_t stream) {
    if (p.E <= 16) return run_first<L, 1, 1>(p, stream);
    if (p.E <= 32) return run_first<L, 2, 2>(p, stream);
    if (p.E <= 64) return run_first<L, 4, 4>(p, stream);
    if (p.E <= 128) return run_first<L, 8, 8>(p, stream);
    if (p.E <= 256) return p.k <= 8 ? run_first<L, 16, 8>(p, stream) : run_first<L, 16, 16>(p, stream);
    if (p.E <= 512) return p.k <= 8 ? run_first<L, 32, 8>(p, stream) : run_first<L, 32, 16>(p, stream);
    return p.k <= 8 ? run_first<L, 64, 8>(p, stream) : run_first<L, 64, 16>(p, stream);
}

template <typename L>
hipError_t route_grad(const RouteGradArgs& p, hipStream_t stream) {
    const int64_t blocks = (p.T + 15) / 16;
    // 1024, 2048 and 4096 blocks: 128.9, 126.4 and 127.7 us for routing and
    // gradient of 131072 tokens of 256 fp32 scores
    const dim3 grid(static_cast<uint32_t>(blocks < 2048 ? blocks : 2048)), block(kGradThr);
    if (p.E <= 16) hipLaunchKernelGGL((route_grad_kernel<L, 1>), grid, block, 0, stream, p);
    else if (p.E <= 32) hipLaunchKernelGGL((route_grad_kernel<L, 2>), grid, block, 0, stream, p);
    else if (p.E <= 64) hipLaunchKernelGGL((route_grad_kernel<L, 4>), grid, block, 0, stream, p);
    else if (p.E <= 128) hipLaunchKernelGGL((route_grad_kernel<L, 8>), grid, block, 0, stream, p);
    else if (p.E <= 256) hipLaunchKernelGGL((route_grad_kernel<L, 16>), grid, block, 0, stream, p);
    else if (p.E <= 512) hipLaunchKernelGGL((route_grad_kernel<L, 32>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_grad_kernel<L, 64>), grid, block, 0, stream, p);
    return hipGetLastError();
}

// 64 tokens per block while that is at most 512 blocks; then 128, which halves
// what the later kernels read (131072 tokens of 256 experts, the three
// kernels: 64 a block 82 us, 128 75 us, 256 91 us, whose first kernel has too
// few waves); 4096 where the grid's threads would not fit 32 bits.
int32_t route_passes(int64_t T) { return T <= 512 * kTok ? 1 : (T <= (int64_t(1) << 24) ? 2 : 64); }
int64_t route_blocks(int64_t T) {
    const int64_t per = int64_t(route_passes(T)) * kTok;
    return T <= per ? 1 : (T + per - 1) / per;
}

// Up to this many counts every workgroup of the last kernel adds them itself.
constexpr int64_t kSumCounts = 32768;

}  // namespace

int64_t route_workspace(int64_t T, int32_t E) {
    const int64_t b = route_blocks(T);
    return b <= 1 ? 0 : b * (10 * int64_t(E) + 4);
}

hipError_t launch_route(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                        int32_t k, bool normalize, int32_t align, int64_t M, int32_t* idx, float* weight,
                        int32_t* slot, int32_t* src, int32_t* counts, int32_t* offs, int32_t* live, float* prob,
                        float* loss, void* workspace, hipStream_t stream) {
    RouteArgs p;
    p.logits = logits; p.ld = ld; p.valid = valid; p.T = T; p.M = M; p.E = E; p.k = k; p.align = align;
    p.normalize = normalize; p.idx = idx; p.slot = slot; p.src = src; p.counts = counts; p.offs = offs;
    p.live = live; p.weight = weight; p.prob = prob; p.loss = loss;
    p.passes = route_passes(T);
    p.blocks = int32_t(route_blocks(T));
    const int64_t cells = int64_t(p.blocks) * E;
    p.ws_prob = static_cast<float*>(workspace);
    p.ws_base = reinterpret_cast<int32_t*>(p.ws_prob + cells);
    p.ws_live = p.ws_base + cells;
    p.ws_counts = reinterpret_cast<uint16_t*>(p.ws_live + p.blocks);
    hipError_t e = dtype == 0 ? route_first<float>(p, stream) : route_first<uint16_t>(p, stream);
    if (e != hipSuccess || p.blocks == 1) return e;
    if (cells <= kSumCounts) {
        hipLaunchKernelGGL((route_place_kernel<true, 1024>), dim3(uint32_t(p.blocks) + 1u), dim3(1024), 0, stream, p);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(route_scan_kernel, dim3((uint32_t(E) + 15u) / 16u), dim3(1024), 0, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((route_place_kernel<false, 512>), dim3(uint32_t(p.blocks)), dim3(512), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_route_grad(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                             int32_t k, bool normalize, const int32_t* idx, const float* weight, const float* dweight,
                             const int32_t* counts, const int32_t* live, const float* dloss, void* dlogits,
                             int64_t ld_d, hipStream_t stream) {
    RouteGradArgs p;
    p.logits = logits; p.ld = ld; p.valid = valid; p.T = T; p.E = E; p.k = k; p.normalize = normalize;
    p.idx = idx; p.weight = weight; p.dweight = dweight; p.counts = counts; p.live = live; p.dloss = dloss;
    p.dlogits = dlogits; p.ld_d = ld_d;
    return dtype == 0 ? route_grad<float>(p, stream) : route_grad<uint16_t>(p, stream);
}

}  // namespace mxq
