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
// Lanes: 16 lanes of a wave hold one token's scores, V = 2^n >= E/16
// consecutive experts each (four tokens per wave).  Reductions over a token
// stay inside a 16-lane row, where DPP rotations need no LDS, and the lowest
// expert among equal scores is the lowest lane's first one.
//
// Order: a block takes 64 tokens, so the tokens that picked an expert are one
// 64-bit mask in LDS; a pick's rank within the block is a population count
// below its token's bit.  Ranks, counts and every floating sum are therefore
// in a fixed order: the same inputs give the same bits.  Up to 64 tokens one
// block does everything; beyond, a second kernel turns the blocks' counts
// into exclusive prefixes and a third places the picks.
#include "mxq_kernels.h"

namespace mxq {
namespace {

constexpr int kTok = 64;         // tokens per block: one 64-bit mask per expert
constexpr int kThreads = 256;
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
    int32_t* ws_counts;          // [blocks][E], then exclusive prefixes over the blocks
    float* ws_prob;              // [blocks][E]
    int32_t* ws_live;            // [blocks]
    int32_t blocks;
};

template <int kCtrl>
__device__ __forceinline__ float dpp_f(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), kCtrl, 0xF, 0xF, false));
}
// All-reduce over the 16 lanes of a DPP row (rotations by 8, 4, 2, 1).
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, dpp_f<0x128>(x));
    x = fmaxf(x, dpp_f<0x124>(x));
    x = fmaxf(x, dpp_f<0x122>(x));
    return fmaxf(x, dpp_f<0x121>(x));
}
__device__ __forceinline__ float row_sum(float x) {
    x += dpp_f<0x128>(x);
    x += dpp_f<0x124>(x);
    x += dpp_f<0x122>(x);
    return x + dpp_f<0x121>(x);
}
__device__ __forceinline__ uint32_t row_ballot(bool b) {
    return uint32_t(__ballot(b) >> (threadIdx.x & 48u)) & 0xFFFFu;
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ void store_logit(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_logit(uint16_t* p, float x) {
    const __bf16 b = __bf16(x);
    *p = __builtin_bit_cast(uint16_t, b);
}

// This lane's V scores of token `row` (-inf past E and for rows that do not
// take part).
template <typename L, int V>
__device__ __forceinline__ void load_row(const L* base, int64_t ld, int64_t row, bool in, uint32_t l16, int32_t E,
                                         float (&z)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int32_t e = int32_t(l16) * V + v;
        z[v] = in && e < E ? load_logit(base + row * ld + e) : -INFINITY;
    }
}

// Softmax statistics of a token.  bad: a NaN or +inf among the scores.
struct Row {
    float top, inv;
    bool live, bad;
};

template <int V>
__device__ __forceinline__ Row softmax_row(const float (&z)[V], float (&p)[V]) {
    Row r;
    bool bad = false;
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bad = bad || !(z[v] < INFINITY);
        m = fmaxf(m, z[v]);
    }
    r.bad = row_ballot(bad) != 0;
    r.top = row_max(m);
    r.live = r.bad || r.top > -INFINITY;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = r.live ? __expf(z[v] - r.top) : 0.f;
        s += p[v];
    }
    s = row_sum(s);
    r.inv = r.bad ? __int_as_float(0x7FC00000) : (r.live ? 1.f / s : 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] *= r.inv;
    return r;
}

// Group starts from counts (LDS), by one wave: starts[e] = the padded sizes
// of the groups before e; the caller's lambda gets (e, count, start, end).
template <typename F>
__device__ __forceinline__ int32_t scan_groups(int32_t E, int32_t align, F&& each) {
    const uint32_t lane = threadIdx.x & 63u;
    int32_t carry = 0;
    for (int32_t b = 0; b < E; b += 64) {
        const int32_t e = b + int32_t(lane);
        const int32_t c = e < E ? each.count(e) : 0;
        const int32_t pad = (c + align - 1) / align * align;
        int32_t x = pad;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(x, d, 64);
            if (lane >= uint32_t(d)) x += o;
        }
        if (e < E) each.put(e, c, carry + x - pad, carry + x);
        carry += __shfl(x, 63, 64);
    }
    return carry;
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
    return x;
}

// What the last stage keeps in LDS per expert.
struct Groups {
    const int32_t* counts;       // LDS or global
    const float* prob;
    int32_t* starts;             // LDS
    int32_t* offs;               // global, or null
    float dot;                   // this lane's sum of counts * prob
    __device__ int32_t count(int32_t e) const { return counts[e]; }
    __device__ void put(int32_t e, int32_t c, int32_t start, int32_t end) {
        starts[e] = start;
        if (offs) offs[e] = end;
        if (prob) dot += float(c) * prob[e];
    }
};

// Rows of the padded buffer that no pick owns: the end of each group (this
// block's share of the experts) and what follows the last group.
__device__ __forceinline__ void clear_pads(const RouteArgs& p, const int32_t* counts, const int32_t* starts,
                                           int32_t total, uint32_t block, uint32_t blocks) {
    for (int32_t e = int32_t(block); e < p.E; e += int32_t(blocks)) {
        const int32_t c = counts[e];
        const int32_t end = starts[e] + (c + p.align - 1) / p.align * p.align;
        for (int32_t r = starts[e] + c + int32_t(threadIdx.x); r < end; r += kThreads) p.src[r] = -1;
    }
    for (int64_t r = total + int64_t(block) * kThreads + threadIdx.x; r < p.M; r += int64_t(blocks) * kThreads)
        p.src[r] = -1;
}

template <typename L, int V>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs p) {
    __shared__ unsigned long long mask[16 * V];
    __shared__ float red[4][16 * V];
    __shared__ uint16_t pick[kTok * kMaxK];
    __shared__ int32_t sh_count[16 * V], sh_start[16 * V];
    __shared__ int32_t sh_live, sh_total;

    const uint32_t t = threadIdx.x, l16 = t & 15u, grp = t >> 4, wave = t >> 6;
    const int64_t first = int64_t(blockIdx.x) * kTok;
    for (uint32_t e = t; e < 16u * V; e += kThreads) mask[e] = 0;
    if (t == 0) sh_live = 0;
    __syncthreads();

    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    for (uint32_t pass = 0; pass < kTok / 16; ++pass) {
        const uint32_t tok = pass * 16 + grp;
        const int64_t row = first + tok;
        if (first + pass * 16 >= p.T) break;                      // uniform
        const bool in = row < p.T && (p.valid == nullptr || p.valid[row] != 0);
        float z[V], q[V];
        load_row<L, V>(static_cast<const L*>(p.logits), p.ld, row, in, l16, p.E, z);
        const Row r = softmax_row<V>(z, q);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            acc[v] += q[v];
            if (r.bad) z[v] = -INFINITY;                          // a bad row picks nothing
        }
        if (l16 == 0 && r.live) atomicAdd(&sh_live, 1);

        float sum = 0.f, mine = 0.f;
        for (int j = 0; j < p.k; ++j) {
            float best = z[0];
#pragma unroll
            for (int v = 1; v < V; ++v) best = fmaxf(best, z[v]);
            const float top = row_max(best);
            const bool ok = top > -INFINITY;
            const uint32_t who = row_ballot(ok && best == top);
            const bool win = ok && l16 == uint32_t(__builtin_ctz(who | 0x10000u));
            int at = 0;
#pragma unroll
            for (int v = V - 1; v >= 0; --v) at = z[v] == top ? v : at;
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = win && v == at ? -INFINITY : z[v];
            if (win) {
                const uint32_t e = l16 * V + uint32_t(at);
                pick[tok * p.k + j] = uint16_t(e);
                atomicOr(&mask[e], 1ull << tok);
            } else if (!ok && l16 == 0) {
                pick[tok * p.k + j] = 0xFFFFu;
            }
            const float w = r.bad ? r.inv : (ok ? __expf(top - r.top) * r.inv : 0.f);
            sum += w;
            mine = l16 == uint32_t(j) ? w : mine;
        }
        if (row < p.T && l16 < uint32_t(p.k))
            p.weight[row * p.k + l16] = p.normalize && r.live ? mine / sum : mine;
    }

    // ---- the block's sums ----
#pragma unroll
    for (int v = 0; v < V; ++v) {
        acc[v] += __shfl_xor(acc[v], 16, 64);
        acc[v] += __shfl_xor(acc[v], 32, 64);
        if ((t & 63u) < 16u) red[wave][l16 * V + v] = acc[v];
    }
    __syncthreads();
    const bool alone = gridDim.x == 1;
    const float n = float(max(sh_live, 1));
    for (uint32_t e = t; e < uint32_t(p.E); e += kThreads) {
        const float s = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
        const int32_t c = __popcll(mask[e]);
        if (alone) {
            sh_count[e] = c;
            p.counts[e] = c;
            red[0][e] = s / n;
            p.prob[e] = s / n;
        } else {
            p.ws_counts[int64_t(blockIdx.x) * p.E + e] = c;
            p.ws_prob[int64_t(blockIdx.x) * p.E + e] = s;
        }
    }
    if (!alone && t == 0) p.ws_live[blockIdx.x] = sh_live;
    if (alone) {
        __syncthreads();
        if (wave == 0) {
            Groups g{sh_count, red[0], sh_start, p.offs, 0.f};
            const int32_t total = scan_groups(p.E, p.align, g);
            const float dot = wave_sum(g.dot);
            if (t == 0) {
                sh_total = total;
                p.live[0] = sh_live;
                p.loss[0] = float(p.E) * dot / (float(p.k) * n);
            }
        }
        __syncthreads();
        clear_pads(p, sh_count, sh_start, sh_total, 0, 1);
    }
    const int64_t left = p.T - first;
    const uint32_t picks = uint32_t(left < kTok ? (left < 0 ? 0 : left) : kTok) * uint32_t(p.k);
    for (uint32_t i = t; i < picks; i += kThreads) {
        const uint32_t tok = i / uint32_t(p.k), e = pick[i];
        const int64_t at = first * p.k + i;
        int32_t rank = -1;
        if (e != 0xFFFFu) {
            rank = __popcll(mask[e] & ((1ull << tok) - 1ull));
            if (alone) {
                rank += sh_start[e];
                p.src[rank] = int32_t(at);
            }
        }
        p.idx[at] = e == 0xFFFFu ? -1 : int32_t(e);
        p.slot[at] = rank;                                        // the rank in the block until the last kernel
    }
}

// Exclusive prefixes of the blocks' counts (in place), and the totals: one
// block for 16 experts, 64 segments of the blocks each.
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
        int32_t x = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(x, d, 64);
            if (lane >= uint32_t(d)) x += o;
        }
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
        for (int32_t b = b0; b < b1; ++b) {
            int32_t* at = p.ws_counts + int64_t(b) * p.E + e;
            const int32_t own = *at;
            *at = run;
            run += own;
        }
    }
    if (blockIdx.x == 0 && t == 0) p.live[0] = n;
}

constexpr int kPlaceTok = 256;   // tokens per block of the last kernel

__global__ __launch_bounds__(kThreads) void route_place_kernel(RouteArgs p) {
    __shared__ int32_t sh_count[1024], sh_start[1024];
    __shared__ int32_t sh_total;
    const uint32_t t = threadIdx.x;
    for (int32_t e = int32_t(t); e < p.E; e += kThreads) sh_count[e] = p.counts[e];
    __syncthreads();
    if (t < 64) {
        const bool out = blockIdx.x == 0;
        Groups g{sh_count, out ? p.prob : nullptr, sh_start, out ? p.offs : nullptr, 0.f};
        const int32_t total = scan_groups(p.E, p.align, g);
        const float dot = wave_sum(g.dot);
        if (t == 0) {
            sh_total = total;
            if (out) p.loss[0] = float(p.E) * dot / (float(p.k) * float(max(p.live[0], 1)));
        }
    }
    __syncthreads();
    clear_pads(p, sh_count, sh_start, sh_total, blockIdx.x, gridDim.x);
    const int64_t first = int64_t(blockIdx.x) * kPlaceTok;
    const int64_t left = p.T - first;
    const uint32_t picks = uint32_t(left < kPlaceTok ? left : kPlaceTok) * uint32_t(p.k);
    for (uint32_t i = t; i < picks; i += kThreads) {
        const int64_t at = first * p.k + i;
        const int32_t e = p.idx[at];
        if (e >= 0) {
            const int64_t blk = (first + i / uint32_t(p.k)) / kTok;
            const int32_t s = sh_start[e] + p.ws_counts[blk * p.E + e] + p.slot[at];
            p.slot[at] = s;
            p.src[s] = int32_t(at);
        }
    }
}

// ---- gradient ----
//
//   a[e] = dloss E counts[e] / (k live^2)          (balance loss, by p)
//   not normalized: a[t][idx_j] += dweight_j,      dlogits = p (a - sum_e p a)
//   normalized:     dlogits = p (a - sum_e p a), + w_j (dweight_j - sum w dweight) at idx_j
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

template <typename L, int V>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradArgs p) {
    __shared__ float up[16][16 * V + 1];
    const uint32_t t = threadIdx.x, l16 = t & 15u, grp = t >> 4;
    const float n = float(max(p.live[0], 1));
    const float unit = p.dloss ? p.dloss[0] * float(p.E) / (float(p.k) * n * n) : 0.f;
    float a[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int32_t e = int32_t(l16) * V + v;
        a[v] = e < p.E ? unit * float(p.counts[e]) : 0.f;
    }
    for (int64_t first = int64_t(blockIdx.x) * 16; first < p.T; first += int64_t(gridDim.x) * 16) {
        const int64_t row = first + grp;
        const bool in = row < p.T && (p.valid == nullptr || p.valid[row] != 0);
        float z[V], q[V];
        load_row<L, V>(static_cast<const L*>(p.logits), p.ld, row, in, l16, p.E, z);
        const Row r = softmax_row<V>(z, q);
        // the picks' direct part, scattered over the row through LDS
#pragma unroll
        for (int v = 0; v < V; ++v) up[grp][l16 * V + v] = 0.f;
        __syncthreads();
        if (p.dweight != nullptr) {
            int32_t e = -1;
            float c = 0.f, w = 0.f;
            if (row < p.T && l16 < uint32_t(p.k)) {
                e = p.idx[row * p.k + l16];
                if (uint32_t(e) < uint32_t(p.E)) {
                    c = p.dweight[row * p.k + l16];
                    w = p.weight[row * p.k + l16];
                } else {
                    e = -1;
                }
            }
            if (p.normalize) c = w * (c - row_sum(w * c));
            if (e >= 0) up[grp][e] = c;
        }
        __syncthreads();
        float s = 0.f, d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            d[v] = up[grp][l16 * V + v];
            s += q[v] * (p.normalize ? a[v] : a[v] + d[v]);
        }
        s = row_sum(s);
        __syncthreads();
        if (row < p.T) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int32_t e = int32_t(l16) * V + v;
                const float g = p.normalize ? q[v] * (a[v] - s) + d[v] : q[v] * (a[v] + d[v] - s);
                if (e < p.E) store_logit(static_cast<L*>(p.dlogits) + row * p.ld_d + e, r.live ? g : 0.f);
            }
        }
    }
}

template <typename L>
hipError_t route_first(const RouteArgs& p, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(p.blocks)), block(kThreads);
    if (p.E <= 16) hipLaunchKernelGGL((route_kernel<L, 1>), grid, block, 0, stream, p);
    else if (p.E <= 32) hipLaunchKernelGGL((route_kernel<L, 2>), grid, block, 0, stream, p);
    else if (p.E <= 64) hipLaunchKernelGGL((route_kernel<L, 4>), grid, block, 0, stream, p);
    else if (p.E <= 128) hipLaunchKernelGGL((route_kernel<L, 8>), grid, block, 0, stream, p);
    else if (p.E <= 256) hipLaunchKernelGGL((route_kernel<L, 16>), grid, block, 0, stream, p);
    else if (p.E <= 512) hipLaunchKernelGGL((route_kernel<L, 32>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_kernel<L, 64>), grid, block, 0, stream, p);
    return hipGetLastError();
}

template <typename L>
hipError_t route_grad(const RouteGradArgs& p, hipStream_t stream) {
    const int64_t blocks = (p.T + 15) / 16;
    const dim3 grid(static_cast<uint32_t>(blocks < 4096 ? blocks : 4096)), block(kThreads);
    if (p.E <= 16) hipLaunchKernelGGL((route_grad_kernel<L, 1>), grid, block, 0, stream, p);
    else if (p.E <= 32) hipLaunchKernelGGL((route_grad_kernel<L, 2>), grid, block, 0, stream, p);
    else if (p.E <= 64) hipLaunchKernelGGL((route_grad_kernel<L, 4>), grid, block, 0, stream, p);
    else if (p.E <= 128) hipLaunchKernelGGL((route_grad_kernel<L, 8>), grid, block, 0, stream, p);
    else if (p.E <= 256) hipLaunchKernelGGL((route_grad_kernel<L, 16>), grid, block, 0, stream, p);
    else if (p.E <= 512) hipLaunchKernelGGL((route_grad_kernel<L, 32>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_grad_kernel<L, 64>), grid, block, 0, stream, p);
    return hipGetLastError();
}

int64_t route_blocks(int64_t T) { return T <= kTok ? 1 : (T + kTok - 1) / kTok; }

}  // namespace

int64_t route_workspace(int64_t T, int32_t E) {
    const int64_t b = route_blocks(T);
    return b <= 1 ? 0 : b * (8 * int64_t(E) + 4);
}

hipError_t launch_route(const void* logits, int dtype, int64_t T, int32_t E, int64_t ld, const uint8_t* valid,
                        int32_t k, bool normalize, int32_t align, int64_t M, int32_t* idx, float* weight,
                        int32_t* slot, int32_t* src, int32_t* counts, int32_t* offs, int32_t* live, float* prob,
                        float* loss, void* workspace, hipStream_t stream) {
    RouteArgs p;
    p.logits = logits; p.ld = ld; p.valid = valid; p.T = T; p.M = M; p.E = E; p.k = k; p.align = align;
    p.normalize = normalize; p.idx = idx; p.slot = slot; p.src = src; p.counts = counts; p.offs = offs;
    p.live = live; p.weight = weight; p.prob = prob; p.loss = loss;
    p.blocks = int32_t(route_blocks(T));
    p.ws_counts = static_cast<int32_t*>(workspace);
    p.ws_prob = reinterpret_cast<float*>(p.ws_counts + int64_t(p.blocks) * E);
    p.ws_live = reinterpret_cast<int32_t*>(p.ws_prob + int64_t(p.blocks) * E);
    hipError_t e = dtype == 0 ? route_first<float>(p, stream) : route_first<uint16_t>(p, stream);
    if (e != hipSuccess || p.blocks == 1) return e;
    hipLaunchKernelGGL(route_scan_kernel, dim3((uint32_t(E) + 15u) / 16u), dim3(1024), 0, stream, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(route_place_kernel, dim3(uint32_t((T + kPlaceTok - 1) / kPlaceTok)), dim3(kThreads), 0, stream, p);
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
