// route_scored.hip -- expert routing by sigmoid or softmax scores with a
// balancing bias and groups of experts, and the gradient of its weights and
// balance loss; the bias's step.
//
//   s[e]      1 / (1 + e^-z), or the softmax of the token's logits
//   u[e]      s[e] + bias[e]: what picks go by.  Without a bias the logits
//             themselves, which have the scores' order
//   worth[g]  sum of the best (1 or 2) u (s without a bias) of the experts of
//             group g that the token may use
//   picks     out of the top groups by worth (equal ones lowest first) the k
//             experts of largest u (equal ones lowest first)
//   weight    scale s[pick], or scale s[pick] / (sum over the picks + 1e-20)
//   share[e]  s[e] / (sum over the experts + 1e-20) of sigmoid scores, s[e] of
//             softmax ones; prob and loss are of the shares as route.hip's
//
// Blocks, lanes, ranks, counts and what follows the first kernel are those of
// route.hip.
//
// Selection is exact though scores are fp32: u is compared as the binary64
// value of the formula.  A lane's keys are u on a grid of 2^22 steps between
// the token's least and largest u (an fp32 u has no more digits there), over
// the inverted expert; they are sorted and merged as in route.hip.  Then every
// decision that the rounding of u, of the keys or of a worth could have turned
// is looked for: a pick and its successor closer than that, an expert left out
// that comes as close to the last pick, the last group that stays as close to
// the first that does not.  Experts with the same logit and the same bias are
// truly equal and in order by their keys.  Where one is found the experts that
// come close enough to be picks (mostly one or two more than k) are ranked by
// their binary64 values, a lane to each or two; where it is groups that are
// close, or more than 32 experts, or the u span too little or too much for a
// grid, the four tokens of the wave are decided again in binary64 from the
// logits in LDS, pick by pick.
//
// 131072 x 256 fp32 by sigmoid scores, a bias and 8 groups: 128 us, without groups
// 102 (the first kernel 119).  A round of four tokens is 1420 vector instructions,
// which fill 49% of the first kernel's cycles.  The rest is mostly its end: tokens
// are decided again after the pass, so that what they need takes no registers from
// the others (within it the call took 301 us), and though they are few, about one
// in 1500 here, a block waits some 10 us for one; by fp32 values alone the call
// takes 97 us.  Scores formed in fewer operations (within 1.25 |z| 2^-24 of
// themselves; prob and loss are sums of them in fp32): 122 us.
#include "act.h"
#include "route_device.h"

namespace mxq {
namespace {

struct ScoredArgs {
    const float* bias;           // null: none
    int32_t softmax, groups, top, best, size;   // size: experts of a group
    uint32_t inverse;            // ceil(2^20 / size): e / size = e inverse >> 20 for e < 1024
    float scale;
};

constexpr float kEps = 1e-20f;
constexpr int kMaxGroups = 32;

__device__ __forceinline__ float row_min(float x) {
    x = fminf(x, dpp<0x128>(x));
    x = fminf(x, dpp<0x124>(x));
    x = fminf(x, dpp<0x122>(x));
    return fminf(x, dpp<0x121>(x));
}
__device__ __forceinline__ uint32_t row_or(uint32_t x) {
    x |= dpp<0x128>(x);
    x |= dpp<0x124>(x);
    x |= dpp<0x122>(x);
    return x | dpp<0x121>(x);
}
__device__ __forceinline__ int32_t row_count(int32_t x) {
    x += int32_t(dpp<0x128>(uint32_t(x)));
    x += int32_t(dpp<0x124>(uint32_t(x)));
    x += int32_t(dpp<0x122>(uint32_t(x)));
    return x + int32_t(dpp<0x121>(uint32_t(x)));
}
__device__ __forceinline__ void row_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// What was derived from x (comparisons, addresses) is formed anew from here on:
// kept, it would take registers that a third or fourth wave could use.
template <int N>
__device__ __forceinline__ void forget(float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
    __builtin_amdgcn_sched_barrier(0);
}

// A token's scores: of a logit z.  Sigmoid: top and inv are not used.
struct Score {
    bool softmax;
    float top, inv;
    __device__ __forceinline__ float of(float z) const {
        float q;
        return softmax ? __expf(z - top) * inv : act_logistic(z, &q);
    }
};

// e^x in binary64, within a few ulp: 2^n e^r, |r| <= ln 2 / 2, by 14 terms of the
// series (r^14 / 14! < 2^-54).  A function of its own: inlined six times its
// constants take the registers of a wave, and the code, which most blocks fetch
// once, is longer (16384 x 256, 8 groups: 40.1 us instead of 37.9).
__device__ __attribute__((noinline)) double exact_exp(double x) {
    constexpr double kFactorial[14] = {1, 1, 2, 6, 24, 120, 720, 5040, 40320, 362880, 3628800, 39916800, 479001600, 6227020800.};
    x = fmax(fmin(x, 1000.0), -1000.0);
    const double n = rint(x * 1.4426950408889634);
    const double r = fma(-n, 2.3190468138462996e-17, fma(-n, 0.6931471805599453, x));    // ln 2 in two parts
    double s = 1.0 / 87178291200.;
#pragma unroll
    for (int i = 13; i >= 0; --i) s = fma(s, r, 1.0 / kFactorial[i]);
    return ldexp(s, int(n));
}

// A token decided in binary64, out of its logits in LDS.
struct Exact {
    const float *z, *bias;       // LDS
    const ScoredArgs& a;
    int32_t E;
    double top, sum;

    // the softmax's sum, by the row's 16 lanes
    __device__ double all(uint32_t l16, int32_t row0) const;
    __device__ double score(double x) const { return a.softmax ? exact_exp(x - top) / sum : 1.0 / (1.0 + exact_exp(-x)); }
    __device__ bool can(int32_t e) const { return z[e] > -INFINITY && (a.bias == nullptr || fabsf(bias[e]) < INFINITY); }
    // what groups are weighed by
    __device__ double worth_of(int32_t e) const {
        const double s = score(double(z[e]));
        return a.bias == nullptr ? s : s + double(bias[e]);
    }
    // what picks go by
    __device__ double value(int32_t e) const { return a.bias == nullptr ? double(z[e]) : worth_of(e); }
};

__device__ __forceinline__ double row_shift(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = uint32_t(__shfl(int(uint32_t(b)), lane, 64)), hi = uint32_t(__shfl(int(uint32_t(b >> 32)), lane, 64));
    return __builtin_bit_cast(double, lo | (uint64_t(hi) << 32));
}

__device__ double Exact::all(uint32_t l16, int32_t row0) const {
    double s = 0.0;
#pragma unroll 1
    for (int32_t e = int32_t(l16); e < E; e += 16) s += exact_exp(double(z[e]) - top);
#pragma unroll 1
    for (int d = 8; d >= 1; d >>= 1) s += row_shift(s, row0 + int(l16 ^ uint32_t(d)));
    return s;
}

__device__ __forceinline__ int32_t uniform_lane(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// The groups of the largest worths; a lane has those of groups l16 and l16 + 16.
__device__ __forceinline__ uint32_t best_groups(const ScoredArgs& a, double worth0, double worth1) {
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u;
    const int32_t row0 = int32_t(lane & 48u);
    int32_t ahead0 = 0, ahead1 = 0;
#pragma unroll 1
    for (int32_t h = 0; h < a.groups; ++h) {
        const double w = row_shift(h < 16 ? worth0 : worth1, row0 + (h & 15));
        ahead0 += w > worth0 || (w == worth0 && h < int32_t(l16));
        ahead1 += w > worth1 || (w == worth1 && h < int32_t(l16) + 16);
    }
    return row_or((int32_t(l16) < a.groups && ahead0 < a.top ? 1u << l16 : 0u) |
                  (int32_t(l16) + 16 < a.groups && ahead1 < a.top ? 1u << (l16 + 16u) : 0u));
}

// All four tokens of the wave again.  Returns this lane's pick (-1: none).
__device__ int32_t pick_exactly(const ScoredArgs& a, int32_t E, int32_t k, const float* z, const float* bias, float top) {
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u;
    const int32_t row0 = int32_t(lane & 48u);
    Exact x{z, bias, a, E, double(top), 1.0};
    if (a.softmax) x.sum = x.all(l16, row0);
    uint32_t stays = 0xFFFFFFFFu;
    if (a.top < a.groups) {                                                 // uniform
        double worth[2];                                                    // of groups l16 and l16 + 16
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            const int32_t g = int32_t(l16) + 16 * i;
            double first = -INFINITY, second = -INFINITY;
            if (g < a.groups) {
#pragma unroll 1
                for (int32_t e = g * a.size; e < (g + 1) * a.size; ++e) {
                    if (!x.can(e)) continue;
                    const double w = x.worth_of(e);
                    second = fmax(second, fmin(first, w));
                    first = fmax(first, w);
                }
            }
            const double w = a.best == 2 && second > -INFINITY ? first + second : first;
            if (i == 0) worth[0] = w;
            else worth[1] = w;
        }
        stays = best_groups(a, worth[0], worth[1]);
    }
    int32_t mine = -1;
    double last = INFINITY;
    int32_t least = -1;
    bool more = true;
#pragma unroll 1
    for (int32_t j = 0; j < k; ++j) {
        // the best expert after the last pick
        double best = -INFINITY;
        int32_t at = 0x7FFFFFFF;
#pragma unroll 1
        for (int32_t e = int32_t(l16); e < E; e += 16) {
            if (!x.can(e) || ((stays >> (uint32_t(e) * a.inverse >> 20)) & 1u) == 0) continue;
            const double u = x.value(e);
            if ((j == 0 || u < last || (u == last && e > least)) && u > best) {
                best = u;
                at = e;
            }
        }
#pragma unroll 1
        for (int d = 8; d >= 1; d >>= 1) {
            const int from = row0 + int(l16 ^ uint32_t(d));
            const double o = row_shift(best, from);
            const int32_t oe = __shfl(at, from, 64);
            if (o > best || (o == best && oe < at)) {
                best = o;
                at = oe;
            }
        }
        more = more && at != 0x7FFFFFFF;
        if (more && int32_t(l16) == j) mine = at;
        last = best;
        least = at;
    }
    return mine;
}

// The candidates of each of the wave's tokens, `total` experts in `list` (at
// most 32), by their binary64 values.  Returns this lane's pick (-1: none).
__device__ int32_t rank_exactly(const ScoredArgs& a, int32_t E, int32_t k, const float* z, const float* bias, float top,
                                uint16_t* list, int32_t total) {
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u;
    const int32_t row0 = int32_t(lane & 48u);
    Exact x{z, bias, a, E, double(top), 1.0};
    if (a.softmax && a.bias != nullptr) x.sum = x.all(l16, row0);
    int32_t e0 = 0x7FFFFFFF, e1 = 0x7FFFFFFF;
    double u0 = -INFINITY, u1 = -INFINITY;
    if (int32_t(l16) < total) {
        e0 = list[l16];
        u0 = x.value(e0);
    }
    if (int32_t(l16) + 16 < total) {
        e1 = list[l16 + 16u];
        u1 = x.value(e1);
    }
    int32_t most = total;                                                   // of the four tokens
    most = max(most, __shfl_xor(most, 16, 64));
    most = uniform_lane(max(most, __shfl_xor(most, 32, 64)));
    int32_t r0 = 0, r1 = 0;
#pragma unroll 1
    for (int32_t j = 0; j < most; ++j) {
        const int from = row0 + (j & 15);
        const double u = row_shift(j < 16 ? u0 : u1, from);
        const int32_t e = __shfl(j < 16 ? e0 : e1, from, 64);
        r0 += u > u0 || (u == u0 && e < e0);
        r1 += u > u1 || (u == u1 && e < e1);
    }
    row_fence();                                                            // the list is read
    if (int32_t(l16) < total && r0 < k) list[r0] = uint16_t(e0);
    if (int32_t(l16) + 16 < total && r1 < k) list[r1] = uint16_t(e1);
    row_fence();
    return int32_t(l16) < min(k, total) ? int32_t(list[l16]) : -1;
}

// How close to a worth w without a bias another tells nothing: scores are within
// 2^-16 of their own size (a softmax one |d| <= 87 below the largest; a sigmoid
// one within 2^-21), and below 2^-126 they may be 0: two to each worth, 2^-124.
__device__ __forceinline__ float close_worths(float w) { return 0x1p-15f * w + 0x1p-123f; }

// What is kept of a token that is decided again.
struct Again {
    float least;                 // experts of smaller u in those groups cannot be picks
    uint32_t stays;              // groups
    float top, inv;              // of its scores
    float near;                  // how close two u tell nothing
    int32_t doubt;               // 0; 1 the groups are in doubt; 2 everything is
};

// A token's picks, one to a lane, and their weights.
__device__ __forceinline__ void write_picks(const RouteArgs& p, const ScoredArgs& a, const Score& sc, int64_t row, uint32_t tok,
                                            uint32_t l16, bool ok, uint32_t expert, float z, bool bad, float nan, uint16_t* pick,
                                            unsigned long long* mask) {
    float w = bad ? nan : (ok ? sc.of(z) : 0.f);
    if (p.normalize) {
        const float all = row_sum(l16 < uint32_t(p.k) ? w : 0.f);
        w = w / (all + kEps);
    }
    w *= a.scale;
    if (l16 < uint32_t(p.k) && row < p.T) {
        const uint32_t e = ok ? expert : 0xFFFFu;
        pick[tok * uint32_t(p.k) + l16] = uint16_t(e);
        if (ok) atomicOr(&mask[e], 1ull << tok);
        p.weight[row * p.k + l16] = w;
    }
}

// The groups that stay by their binary64 worths: of each group the experts whose
// fp32 values come close to the best two (or one), four at most (else *many),
// are weighed in binary64.
__device__ __forceinline__ uint32_t groups_exactly(const RouteArgs& p, const ScoredArgs& a, const Score& sc, const Again& r,
                                                   const float* z, const float* bias, bool* many) {
    const uint32_t lane = threadIdx.x & 63u, l16 = lane & 15u;
    const int32_t row0 = int32_t(lane & 48u);
    Exact x{z, bias, a, p.E, double(r.top), 1.0};
    if (a.softmax) x.sum = x.all(l16, row0);
    double worth0 = -INFINITY, worth1 = -INFINITY;                          // of groups l16 and l16 + 16
    bool over = false;
#pragma unroll 1
    for (int32_t i = 0; i < 2; ++i) {
        const int32_t g = int32_t(l16) + 16 * i, e0 = g * a.size, e1 = g < a.groups ? e0 + a.size : e0;
        float one = -INFINITY, two = -INFINITY;
#pragma unroll 1
        for (int32_t e = e0; e < e1; ++e) {
            const float w = x.can(e) ? sc.of(z[e]) + (a.bias ? bias[e] : 0.f) : -INFINITY;
            two = __builtin_amdgcn_fmed3f(one, two, w);
            one = fmaxf(one, w);
        }
        const float low = a.best == 2 && two > -INFINITY ? two : one;
        const float from = low - (a.bias ? r.near : close_worths(low));
        int32_t n = 0, c0 = 0, c1 = 0, c2 = 0, c3 = 0;
#pragma unroll 1
        for (int32_t e = e0; e < e1; ++e) {
            if (!x.can(e) || !(sc.of(z[e]) + (a.bias ? bias[e] : 0.f) >= from)) continue;
            c3 = n == 3 ? e : c3;
            c2 = n == 2 ? e : c2;
            c1 = n == 1 ? e : c1;
            c0 = n == 0 ? e : c0;
            ++n;
        }
        over |= n > 4;
        double first = -INFINITY, second = -INFINITY;
#pragma unroll 1
        for (int32_t q = 0; q < 4; ++q) {
            if (q >= n) continue;
            const double w = x.worth_of(q == 0 ? c0 : q == 1 ? c1 : q == 2 ? c2 : c3);
            second = fmax(second, fmin(first, w));
            first = fmax(first, w);
        }
        const double w = a.best == 2 && second > -INFINITY ? first + second : first;
        worth0 = i == 0 ? w : worth0;
        worth1 = i == 1 ? w : worth1;
    }
    *many = row_or(over) != 0;
    return best_groups(a, worth0, worth1);
}

// One token (where `on`) by its 16 lanes, in binary64.
template <typename L, int V>
__device__ __forceinline__ void decide_again(const RouteArgs& p, const ScoredArgs& a, const L* logits, const Again& r, float* z,
                                             const float* bias, uint16_t* list, int64_t row, uint32_t tok, bool on,
                                             uint16_t* pick, unsigned long long* mask) {
    const uint32_t t = threadIdx.x, l16 = t & 15u;
    const Score sc{a.softmax != 0, r.top, r.inv};
    row_fence();
#pragma unroll 4
    for (int32_t e = int32_t(l16); e < p.E; e += 16) z[e] = widen(logits[e]);
    row_fence();
    const auto can = [&](int32_t e) { return z[e] > -INFINITY && fabsf(bias[e]) < INFINITY; };
    const auto u_of = [&](int32_t e) { return a.bias == nullptr ? z[e] : sc.of(z[e]) + bias[e]; };
    uint32_t stays = r.stays;
    float least = r.least;
    bool all = r.doubt == 2;
    if (__ballot(on && r.doubt == 1) != 0) {
        bool many = false;
        const uint32_t exact = groups_exactly(p, a, sc, r, z, bias, &many);
        if (r.doubt == 1) {
            all |= many;
            if (exact != stays) {
                // other groups: their k-th largest u, by fp32 values in order
                stays = exact;
                const auto in = [&](int32_t e) { return can(e) && ((stays >> (uint32_t(e) * a.inverse >> 20)) & 1u) != 0; };
                float last = INFINITY;
                int32_t at = -1;
#pragma unroll 1
                for (int32_t j = 0; j < p.k; ++j) {
                    float m = -INFINITY;
                    int32_t me = 0x7FFFFFFF;
#pragma unroll 1
                    for (int32_t e = int32_t(l16); e < p.E; e += 16) {
                        const float u = u_of(e);
                        if (in(e) && (u < last || (u == last && e > at)) && u > m) {
                            m = u;
                            me = e;
                        }
                    }
                    last = row_max(m);
                    at = int32_t(row_least(m == last ? uint32_t(me) : 0x7FFFFFFFu));
                }
                // (r.near knows the best u of these groups, not the k-th, whose
                // rounding is 2^-24 of its own size, as the next one's)
                least = last > -INFINITY ? last - r.near - (a.bias ? 0x1p-22f * fabsf(last) : 0.f) : -INFINITY;
            }
        }
    }
    // the experts that may be picks, in a list
    int32_t total = 0;
#pragma unroll 1
    for (int32_t e0 = 0; e0 < p.E; e0 += 16) {
        const int32_t e = e0 + int32_t(l16);
        const bool in = e < p.E && can(e) && ((stays >> (uint32_t(e) * a.inverse >> 20)) & 1u) != 0 && u_of(e) >= least;
        const uint32_t lanes = uint32_t(__ballot(in) >> (t & 48u)) & 0xFFFFu;
        if (in) {
            const int32_t to = total + __popc(lanes & ((1u << l16) - 1u));
            if (to < 32) list[to] = uint16_t(e);
        }
        total += __popc(lanes);
    }
    row_fence();
    int32_t e;
    if (__ballot(on && (all || total > 32)) != 0) e = pick_exactly(a, p.E, p.k, z, bias, r.top);
    else e = rank_exactly(a, p.E, p.k, z, bias, r.top, list, min(total, 32));
    const uint32_t expert = e >= 0 ? uint32_t(e) : 0u;
    if (on) write_picks(p, a, sc, row, tok, l16, e >= 0, expert, z[expert], false, 0.f, pick, mask);
    row_fence();
}

template <typename L, int V, int kKeep, int kThr>
__global__ __launch_bounds__(kThr, kThr == 256 && V == 16 ? 4 : 1) void route_scored_kernel(RouteArgs p, ScoredArgs a) {
    using S = Scores<L, V>;
    __shared__ unsigned long long mask[16 * V];
    __shared__ float red[kThr / 64][16 * V];
    // worths' scores, then the logits, for a row's own wave
    __shared__ __attribute__((aligned(16))) float stash[kThr / 16][16 * V];
    __shared__ __attribute__((aligned(16))) float bias[16 * V];
    __shared__ float worths[kThr / 16][kMaxGroups];
    __shared__ uint16_t lists[kThr / 16][32];
    __shared__ Again redo[kTok];
    __shared__ unsigned long long again;                                    // tokens of the pass to decide again
    __shared__ uint16_t pick[kTok * kMaxK];
    __shared__ int32_t sh_count[16 * V], sh_start[16 * V];
    __shared__ int32_t sh_live;

    const uint32_t t = threadIdx.x, grp = t >> 4, wave = t >> 6;
    const bool alone = gridDim.x == 1, biased = a.bias != nullptr, grouped = a.top < a.groups;
    for (uint32_t e = t; e < 16u * V; e += kThr) {
        sh_count[e] = 0;
        bias[e] = biased && int32_t(e) < p.E ? a.bias[e] : 0.f;
    }
    if (t == 0) {
        sh_live = 0;
        again = 0;
    }
    if (alone)                                                              // the picks' rows are written over this
        for (int64_t r = t; r < p.M; r += kThr) p.src[r] = -1;

    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    const L* logits = static_cast<const L*>(p.logits);
    // A group's experts are scanned by 2^part lanes, in pieces of four where they
    // have such, beginning where the lanes of a wave meet few of each other's banks.
    const int32_t part = a.groups <= 2 ? 3 : a.groups <= 4 ? 2 : a.groups <= 8 ? 1 : 0;
    const int32_t own = (a.size + (1 << part) - 1) >> part;
    const bool pieces = a.size % (4 << part) == 0;
    const int32_t start = pieces ? int32_t(((t & 15u) >> 2) + (grp & 3u)) % (own >> 2) : 0;
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
            float z[V], u[V];
            const uint8_t take = p.valid ? p.valid[at] : uint8_t(1);
            load_row<L, V>(logits + at * p.ld, l16, p.E, z);
            const bool in = (row < p.T) & (take != 0);
            float high = -INFINITY;
            bool nan = false;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                z[v] = choose(in, z[v], -INFINITY);
                nan |= !(z[v] < INFINITY);                                  // NaN or +inf
                high = fmaxf(high, z[v]);
            }
            high = row_max(high);
            const bool bad = row_or(nan) != 0, some = high > -INFINITY || bad;
            Score sc{a.softmax != 0, some && !bad ? high : 0.f, 0.f};
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float q;
                u[v] = sc.softmax ? __expf(z[v] - sc.top) : act_logistic(z[v], &q);
                sum += u[v];
            }
            sum = row_sum(sum);
            const float inv = bad ? __uint_as_float(0x7FC00000u) : !some ? 0.f : sc.softmax ? 1.f / sum : 1.f / (sum + kEps);
            sc.inv = sc.softmax ? inv : 1.f;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = __fmaf_rn(u[v], inv, acc[v]);
            if (l16 == 0 && some) atomicAdd(&sh_live, 1);
            // How far a score may be from its binary64 value.  Sigmoid: e^-|z| within
            // 1.6 2^-23 of itself, which moves s by a quarter of that at most, the sum and
            // the reciprocal 1.5 2^-23: 2^-22 in all.  Softmax: p |d| 2^-23 <= 2^-24, and
            // 2^-24 p for each of V + 4 additions and the mean |d| <= ln E of the sum.
            const float off = sc.softmax ? 0x1p-24f * (1.f + float(V + 24) * inv) : 0x1p-22f;
            // what groups are weighed by: u with a bias, else s
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float b = bias[S::expert(l16, v)];
                u[v] = u[v] * sc.inv + b;
                u[v] = choose((z[v] > -INFINITY) & (fabsf(b) < INFINITY), u[v], -INFINITY);
            }
            forget(u);
            bool unsure = false;
            uint32_t staying = 0xFFFFFFFFu;
            float largest = 0.f;                                            // of the best u, those of groups that go among them
            if (grouped) {                                                  // uniform
#pragma unroll
                for (int v = 0; v < V; ++v) stash[grp][S::expert(l16, v)] = u[v];
                row_fence();
                float mag = 0.f, inside = INFINITY, outside = -INFINITY;    // least worth that stays, largest that does not
                uint32_t stays = 0;
                const int32_t in_group = int32_t(l16) & ((1 << part) - 1);
                auto weigh = [&](int32_t g) {
                    float one = -INFINITY, two = -INFINITY;
                    auto take_one = [&](float x) {
                        two = __builtin_amdgcn_fmed3f(one, two, x);         // two <= one: the second of the three
                        one = fmaxf(one, x);
                    };
                    if (g < a.groups) {
                        const float* from = &stash[grp][g * a.size + in_group * own];
                        if (pieces) {
                            const int32_t n = own >> 2;
                            int32_t j = start;
#pragma unroll 4
                            for (int32_t i = 0; i < n; ++i) {
                                const float4 x = *reinterpret_cast<const float4*>(from + 4 * j);
                                take_one(x.x);
                                take_one(x.y);
                                take_one(x.z);
                                take_one(x.w);
                                j = j + 1 == n ? 0 : j + 1;
                            }
                        } else {
                            const int32_t n = min(own, a.size - in_group * own);
#pragma unroll 4
                            for (int32_t i = 0; i < n; ++i) take_one(from[i]);
                        }
                    }
                    auto merge = [&](float o1, float o2) {
                        two = fmaxf(fminf(one, o1), fmaxf(two, o2));
                        one = fmaxf(one, o1);
                    };
                    if (part >= 1) merge(dpp<0xB1>(one), dpp<0xB1>(two));   // lane ^ 1
                    if (part >= 2) merge(dpp<0x4E>(one), dpp<0x4E>(two));   // lane ^ 2
                    if (part >= 3) merge(dpp<0x141>(one), dpp<0x141>(two)); // the other four of eight
                    const bool both = a.best == 2 && two > -INFINITY;
                    if (one > -INFINITY) mag = fmaxf(mag, fabsf(one) + (both ? fabsf(two) : 0.f));
                    return both ? one + two : one;
                };
                auto settle = [&](int32_t g, float w, int32_t ahead) {
                    if (ahead < a.top) {
                        stays |= 1u << g;
                        inside = fminf(inside, w);
                    } else {
                        outside = fmaxf(outside, w);
                    }
                };
                if (a.groups <= 16) {                                       // every lane's group against the others', by rotations
                    const int32_t g = int32_t(l16) >> part;
                    const float w = weigh(g);
                    int32_t ahead = 0;
                    auto against = [&](float x, uint32_t r) { ahead += (x > w) | ((x == w) & (l16 >= r)); };
                    against(dpp<0x128>(w), 8u);                             // from lane l16 - 8, or l16 + 8 of a lower one
                    if (part < 3) {
                        against(dpp<0x124>(w), 4u);
                        against(dpp<0x12C>(w), 12u);
                    }
                    if (part < 2) {
                        against(dpp<0x122>(w), 2u);
                        against(dpp<0x126>(w), 6u);
                        against(dpp<0x12A>(w), 10u);
                        against(dpp<0x12E>(w), 14u);
                    }
                    if (part < 1) {
                        against(dpp<0x121>(w), 1u);
                        against(dpp<0x123>(w), 3u);
                        against(dpp<0x125>(w), 5u);
                        against(dpp<0x127>(w), 7u);
                        against(dpp<0x129>(w), 9u);
                        against(dpp<0x12B>(w), 11u);
                        against(dpp<0x12D>(w), 13u);
                        against(dpp<0x12F>(w), 15u);
                    }
                    if (g < a.groups) settle(g, w, ahead);
                } else {
                    float w[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        w[i] = weigh(int32_t(l16) + 16 * i);
                        worths[grp][l16 + 16u * i] = w[i];
                    }
                    row_fence();
                    int32_t ahead[2] = {0, 0};
#pragma unroll 4
                    for (int32_t h = 0; h < a.groups; ++h) {
                        const float x = worths[grp][h];
                        ahead[0] += (x > w[0]) | ((x == w[0]) & (h < int32_t(l16)));
                        ahead[1] += (x > w[1]) | ((x == w[1]) & (h < int32_t(l16) + 16));
                    }
                    settle(int32_t(l16), w[0], ahead[0]);
                    if (int32_t(l16) + 16 < a.groups) settle(int32_t(l16) + 16, w[1], ahead[1]);
                }
                staying = stays = row_or(stays);
                inside = row_min(inside);
                outside = row_max(outside);
                mag = row_max(mag);
                largest = mag;
                // two scores to a worth, two worths to a comparison
                const float near = biased ? 4.f * off + 0x1p-21f * mag : close_worths(inside);
                unsure = outside > -INFINITY && !(inside - outside > near);
                auto kept = [&](int v) { return ((stays >> (uint32_t(S::expert(l16, v)) * a.inverse >> 20)) & 1u) != 0; };
                if (a.size % S::kC == 0) {                                  // a lane's pieces lie in one group each
#pragma unroll
                    for (int q = 0; q < V / S::kC; ++q) {
                        const bool in_one = kept(q * S::kC);
#pragma unroll
                        for (int i = 0; i < S::kC; ++i) u[q * S::kC + i] = choose(in_one, u[q * S::kC + i], -INFINITY);
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) u[v] = choose(kept(v), u[v], -INFINITY);
                }
                row_fence();
            }
#pragma unroll
            for (int v = 0; v < V; ++v) stash[grp][S::expert(l16, v)] = z[v];
            forget(u);
            // what picks go by, and its keys
            float low = INFINITY, up = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!biased) u[v] = choose(u[v] > -INFINITY, z[v], -INFINITY);
                up = fmaxf(up, u[v]);
                low = fminf(low, choose(u[v] > -INFINITY, u[v], INFINITY));
            }
            up = row_max(up);
            low = row_min(low);
            const float range = up - low;                                   // -inf where there is nothing
            // no grid where a step of it, or its inverse, would leave fp32: everything is
            // decided again
            const bool gridless = range >= 1e30f || (up > low && range < 0x1p-100f);
            const float grid = up > low && !gridless ? 4194240.f / range : 0.f;
            forget(u);
            // steps from 1 on; 0 of an expert that is none (no key below 1024 counts)
            auto key = [&](int v) {
                const uint32_t n = uint32_t(fmaxf(__builtin_fmaf(u[v] - low, grid, 1.f), 0.f));
                return (n << 10) + (1023u - uint32_t(S::expert(l16, v)));
            };
            uint32_t best[kKeep];
#pragma unroll
            for (int v = 0; v < kKeep; ++v) best[v] = key(v);
            sort_desc(best);
#pragma unroll
            for (int b = kKeep; b < V; b += kKeep) {
                uint32_t more[kKeep];
#pragma unroll
                for (int v = 0; v < kKeep; ++v) more[v] = key(b + v);
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
            row_fence();
            forget(u);
            forget(z);
            asm volatile("" : "+v"(l16));
            bool ok = mine >= 1024u;
            uint32_t expert = ok ? 1023u - (mine & 1023u) : 0u;
            float zp = ok ? stash[grp][expert] : 0.f;
            const float bp = ok ? bias[expert] : 0.f;
            const float x = ok ? (biased ? sc.of(zp) + bp : zp) : -INFINITY;
            // two u's with a bias: their scores, and 2^-24 of each sum; two steps of the grid
            const float near = biased ? 2.f * off + 0x1p-23f * fmaxf(fabsf(up), fabsf(low)) : 0.f, step = range * 0x1.1p-21f;
            // picks out of order, or too close to tell; the next lane's (row_shl:1)
            const float xn = dpp<0x101>(x), zn = dpp<0x101>(zp), bn = dpp<0x101>(bp);
            const bool okn = dpp<0x101>(uint32_t(ok)) != 0;
            bool close_picks = l16 + 1u < uint32_t(p.k) && ok && okn && !(zp == zn && bp == bn) &&
                               (biased ? x - xn <= near + step : x < xn);
            // experts that come close to the last pick, but for it and its equals
            const int32_t from = int32_t((t & 48u) + uint32_t(p.k) - 1u);
            const float xl = __shfl(x, from, 64), zl = __shfl(zp, from, 64), bl = __shfl(bp, from, 64);
            // (counted with the picks first: those that come close are mostly k)
            const bool full = last >= 1024u;
            const float reach = biased ? xl - near : xl;
            int32_t close = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) close += u[v] >= reach ? 1 : 0;
            close = full ? row_count(close) - p.k : 0;
            if (__ballot(close != 0) != 0) {                                // uniform: its equals apart
                int32_t apart = 0;
                forget(u);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool same = (z[v] == zl) & (!biased || bias[S::expert(l16, v)] == bl);
                    apart += (u[v] >= reach && !same) ? 1 : 0;
                }
                apart -= (l16 < uint32_t(p.k) && !(zp == zl && bp == bl)) ? 1 : 0;
                apart = row_count(apart);
                if (close != 0) close = apart;
            }
            close_picks = (row_or(close_picks) | uint32_t(close)) != 0;
            if ((close_picks || unsure || gridless) && !bad) {
                // decided again after the pass
                if (l16 == 0) {
                    atomicOr(&again, 1ull << tok);
                    Again& r = redo[tok];
                    r.least = full ? xl - near - step : -INFINITY;
                    r.near = near + 0x1p-23f * largest;
                    r.doubt = gridless ? 2 : unsure ? 1 : 0;
                    r.stays = staying;
                    r.top = sc.top;
                    r.inv = sc.inv;
                }
            } else {
                write_picks(p, a, sc, row, tok, l16, ok && !bad, expert, zp, bad, inv, pick, mask);
            }
            row_fence();                                                    // the stash is read
        }
        __syncthreads();
        const unsigned long long left = again;
        if (left != 0) {                                                    // uniform
            int32_t skip = int32_t(grp);
            const int32_t todo = __popcll(left);
            // all four rows of a wave go round together
            for (int32_t n = 0; n < todo; n += kThr / 16, skip += kThr / 16) {
                if (n + int32_t(wave) * 4 >= todo) break;                   // uniform for the wave
                const bool on = skip < todo;
                unsigned long long bits = left;
                for (int32_t i = on ? skip : todo - 1; i > 0; --i) bits &= bits - 1ull;
                const uint32_t tok = uint32_t(__builtin_ctzll(bits));
                const int64_t row = first + tok;
                __builtin_amdgcn_s_setprio(3);                              // the block waits for this wave
                decide_again<L, V>(p, a, logits + row * p.ld, redo[tok], stash[grp], bias, lists[grp], row, tok, on, pick, mask);
            }
            __builtin_amdgcn_s_setprio(0);
            __syncthreads();
            if (t == 0) again = 0;
        }
        note_picks<kThr>(p, first, pick, mask, sh_count, alone);
    }
    finish_block<V, kThr, L>(p, acc, red, mask, pick, sh_count, sh_start, &sh_live, alone);
}

// ---- gradient ----
//
//   a[e] = dloss E counts[e] / (k live^2)                 (balance loss, by share)
//   d_j  = scale dweight_j, normalized: (d_j - sum_i d_i w_i) / S,
//          w_j = s_j / S, S = sum of the picks' s + 1e-20
//   sigmoid: ds[e] = m (a[e] - m sum a s), m = 1 / (sum s + 1e-20), + d_j at idx_j;
//            dlogits = ds s (1 - s)
//   softmax: dlogits = s (a - sum a s) - s sum_j d_j s_j, + d_j s_j at idx_j
//
// One pass, as route.hip's gradient: a row is in registers between its scores
// and the result.  131072 x 256 fp32: 62 us, 4.5 TB/s; the vector instructions
// fill 64% of the cycles.
struct ScoredGradArgs {
    const void* logits;
    int64_t ld;
    const uint8_t* valid;
    int64_t T;
    int32_t E, k, softmax;
    bool normalize;
    float scale;
    const int32_t *idx, *counts, *live;
    const float *dweight, *dloss;
    void* dlogits;
    int64_t ld_d;
};

constexpr int kGradThr = 256;

template <typename L, int V>
__global__ __launch_bounds__(kGradThr) void route_scored_grad_kernel(ScoredGradArgs p) {
    using S = Scores<L, V>;
    constexpr int kC = S::kC;
    __shared__ __attribute__((aligned(16))) float part[kGradThr / 16][16 * V];   // each row's own wave alone uses it
    __shared__ __attribute__((aligned(16))) float share[16 * V];           // the loss's part of each expert
    const uint32_t t = threadIdx.x, l16 = t & 15u, grp = t >> 4;
    const bool whole = p.E == 16 * V, picks = p.dweight != nullptr && l16 < uint32_t(p.k);
    // what a row takes from memory, read a round ahead
    L ahead[V];
    uint8_t take = 1;
    int32_t e_ahead = -1;
    float d_ahead = 0.f;
    auto fetch = [&](int64_t at, uint32_t l16) {
        if (p.valid) take = p.valid[at];
        if (whole) fetch_row<L, V, true>(static_cast<const L*>(p.logits) + at * p.ld, l16, p.E, ahead);
        else fetch_row<L, V, false>(static_cast<const L*>(p.logits) + at * p.ld, l16, p.E, ahead);
        if (picks) {
            e_ahead = p.idx[at * p.k + l16];
            d_ahead = p.dweight[at * p.k + l16];
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
        float z[V], s[V];
        const bool in = take != 0;
        if (whole) widen_row<L, V, true>(ahead, l16, p.E, z);
        else widen_row<L, V, false>(ahead, l16, p.E, z);
        int32_t e = uint32_t(e_ahead) < uint32_t(p.E) ? e_ahead : -1;
        float d = e >= 0 ? d_ahead * p.scale : 0.f;
        if (kAhead && row + step < p.T) fetch(row + step, l16);
        float high = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = choose(in, z[v], -INFINITY);
            nan |= !(z[v] < INFINITY);
            high = fmaxf(high, z[v]);
        }
        high = row_max(high);
        const bool bad = row_or(nan) != 0, live = high > -INFINITY || bad;
        const float top = live && !bad ? high : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float q;
            s[v] = p.softmax ? __expf(z[v] - top) : act_logistic(z[v], &q);
            if (!p.softmax) z[v] = q;                                       // 1 - s
            sum += s[v];
        }
        sum = row_sum(sum);
        const float m = bad ? __uint_as_float(0x7FC00000u) : !live ? 0.f : p.softmax ? 1.f / sum : 1.f / (sum + kEps);
        if (p.softmax) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] *= m;
        }
        // the picks' part, gathered from and scattered over the row through LDS
        float all = 0.f;                                                    // softmax: sum_j d_j s_j (normalized: mean 1e-20 / S)
        if (p.dweight != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) part[grp][S::expert(l16, v)] = s[v];
            row_fence();
            const float sj = e >= 0 ? part[grp][e] : 0.f;
            row_fence();
#pragma unroll
            for (int v = 0; v < V; ++v) part[grp][S::expert(l16, v)] = 0.f;
            if (p.normalize) {
                // by the weights themselves: the only pick's is 1 and its part 0
                const float q = row_sum(sj) + kEps, w = sj / q, mean = row_sum(d * w);
                d = p.softmax ? w * (d - mean) : (d - mean) / q;
                all = mean * (kEps / q);
            } else if (p.softmax) {
                d *= sj;
                all = row_sum(d);
            }
            row_fence();
            if (e >= 0) part[grp][e] = d;
            row_fence();
        }
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) dot += share[S::expert(l16, v)] * s[v];
        dot = row_sum(dot);
        const float both = dot + all;
        L* out = static_cast<L*>(p.dlogits) + row * p.ld_d;
#pragma unroll
        for (int b = 0; b < V / kC; ++b) {
            const int32_t e0 = S::expert(l16, b * kC);
            L o[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const int v = b * kC + i;
                const float a = share[e0 + i], c = p.dweight != nullptr ? part[grp][e0 + i] : 0.f;
                float g;
                if (p.softmax) g = s[v] * (a - both) + c;
                else g = (m * (a - m * dot) + c) * (s[v] * z[v]);
                g = bad ? m : g;
                o[i] = narrow<L>(live ? g : 0.f);
            }
            if (e0 + kC <= p.E) {
                __builtin_memcpy(out + e0, o, kC * sizeof(L));
            } else {
#pragma unroll
                for (int i = 0; i < kC; ++i)
                    if (e0 + i < p.E) out[e0 + i] = o[i];
            }
        }
        row_fence();                                                        // the row's part is read
    }
}

// ---- the bias's step ----
//
//   out[e] = bias[e] + rate sign(sum of counts - E counts[e])
//
// in exact integers: towards the experts that have fewer picks than the mean.
__global__ __launch_bounds__(1024) void bias_step_kernel(const float* bias, const int32_t* counts, int32_t E, float rate,
                                                         float* out) {
    __shared__ long long total;
    const int32_t e = int32_t(threadIdx.x);
    if (e == 0) total = 0;
    __syncthreads();
    const long long c = e < E ? counts[e] : 0;
    if (e < E) atomicAdd(reinterpret_cast<unsigned long long*>(&total), static_cast<unsigned long long>(c));
    __syncthreads();
    if (e >= E) return;
    const long long d = total - c * E;
    const float b = bias[e];
    out[e] = d > 0 ? b + rate : d < 0 ? b - rate : b;
}

template <typename L, int V, int kKeep>
hipError_t run_scored(const RouteArgs& p, const ScoredArgs& a, hipStream_t stream) {
    const dim3 grid(uint32_t(p.blocks));
    if (p.T <= 4) {
        hipLaunchKernelGGL((route_scored_kernel<L, V, kKeep, 64>), grid, dim3(64), 0, stream, p, a);
        return hipGetLastError();
    }
    // few blocks: all 64 tokens of a pass at once
    constexpr int kMany = V <= 16 ? 1024 : 512;
    if constexpr (V <= 32) {
        if (p.blocks <= 256) {
            hipLaunchKernelGGL((route_scored_kernel<L, V, kKeep, kMany>), grid, dim3(kMany), 0, stream, p, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((route_scored_kernel<L, V, kKeep, 256>), grid, dim3(256), 0, stream, p, a);
    return hipGetLastError();
}

template <typename L>
hipError_t scored_first(const RouteArgs& p, const ScoredArgs& a, hipStream_t stream) {
    if (p.E <= 16) return run_scored<L, 1, 1>(p, a, stream);
    if (p.E <= 32) return run_scored<L, 2, 2>(p, a, stream);
    if (p.E <= 64) return run_scored<L, 4, 4>(p, a, stream);
    if (p.E <= 128) return run_scored<L, 8, 8>(p, a, stream);
    if (p.E <= 256) return p.k <= 8 ? run_scored<L, 16, 8>(p, a, stream) : run_scored<L, 16, 16>(p, a, stream);
    if (p.E <= 512) return p.k <= 8 ? run_scored<L, 32, 8>(p, a, stream) : run_scored<L, 32, 16>(p, a, stream);
    return p.k <= 8 ? run_scored<L, 64, 8>(p, a, stream) : run_scored<L, 64, 16>(p, a, stream);
}

template <typename L>
hipError_t scored_grad(const ScoredGradArgs& p, hipStream_t stream) {
    const int64_t blocks = (p.T + 15) / 16;
    const dim3 grid(static_cast<uint32_t>(blocks < 2048 ? blocks : 2048)), block(kGradThr);
    if (p.E <= 16) hipLaunchKernelGGL((route_scored_grad_kernel<L, 1>), grid, block, 0, stream, p);
    else if (p.E <= 32) hipLaunchKernelGGL((route_scored_grad_kernel<L, 2>), grid, block, 0, stream, p);
    else if (p.E <= 64) hipLaunchKernelGGL((route_scored_grad_kernel<L, 4>), grid, block, 0, stream, p);
    else if (p.E <= 128) hipLaunchKernelGGL((route_scored_grad_kernel<L, 8>), grid, block, 0, stream, p);
    else if (p.E <= 256) hipLaunchKernelGGL((route_scored_grad_kernel<L, 16>), grid, block, 0, stream, p);
    else if (p.E <= 512) hipLaunchKernelGGL((route_scored_grad_kernel<L, 32>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_scored_grad_kernel<L, 64>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_scored(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                               const float* bias, bool softmax, int32_t groups, int32_t top, int32_t best, int32_t k,
                               bool normalize, float scale, int32_t align, int64_t M, int32_t* idx, float* weight,
                               int32_t* slot, int32_t* src, int32_t* counts, int32_t* offs, int32_t* live, float* prob,
                               float* loss, void* workspace, hipStream_t stream) {
    RouteArgs p;
    p.logits = logits; p.ld = ld; p.valid = valid; p.T = T; p.M = M; p.E = E; p.k = k; p.align = align;
    p.normalize = normalize; p.idx = idx; p.slot = slot; p.src = src; p.counts = counts; p.offs = offs;
    p.live = live; p.weight = weight; p.prob = prob; p.loss = loss;
    route_begin(p, workspace);
    const int32_t size = E / groups;
    const ScoredArgs a{bias, softmax ? 1 : 0, groups, top, best, size, uint32_t(((1 << 20) + size - 1) / size), scale};
    const hipError_t e = dtype == 0 ? scored_first<float>(p, a, stream) : scored_first<uint16_t>(p, a, stream);
    return e != hipSuccess ? e : route_rest(p, stream);
}

hipError_t launch_route_scored_grad(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                                    bool softmax, int32_t k, bool normalize, float scale, const int32_t* idx,
                                    const float* dweight, const int32_t* counts, const int32_t* live, const float* dloss,
                                    void* dlogits, int64_t ld_d, hipStream_t stream) {
    ScoredGradArgs p;
    p.logits = logits; p.ld = ld; p.valid = valid; p.T = T; p.E = E; p.k = k; p.softmax = softmax ? 1 : 0;
    p.normalize = normalize; p.scale = scale; p.idx = idx; p.counts = counts; p.live = live; p.dweight = dweight;
    p.dloss = dloss; p.dlogits = dlogits; p.ld_d = ld_d;
    return dtype == 0 ? scored_grad<float>(p, stream) : scored_grad<uint16_t>(p, stream);
}

hipError_t launch_route_bias_step(const float* bias, const int32_t* counts, int32_t E, float rate, float* out,
                                  hipStream_t stream) {
    hipLaunchKernelGGL(bias_step_kernel, dim3(1), dim3(1024), 0, stream, bias, counts, E, rate, out);
    return hipGetLastError();
}

}  // namespace mxq
