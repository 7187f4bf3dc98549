// act_grad.hip -- the gradient of a product's epilogue.
//
//   dpre = dy act'(pre), or gated  dpre[n] = dy act'(pre[n]) pre[n + N],
//                                  dpre[n + N] = dy act(pre[n])
//   dbias[n] = sum over rows of dpre[n], before it is rounded; of each group's
//              rows by itself where there are groups
//
// Rows behind the last group give 0 and are not read.
//
// One pass over dy and pre, which bounds it (HBM).  A workgroup takes a few
// rows of one group (row tiles are numbered group by group, as the products
// number theirs) by 32 pieces of 16 bytes: lane c of 32 holds the columns of
// piece c, eight rows at a time, two of them in flight to a thread (four: no
// faster, and half the waves fit), and adds its columns' sums in registers.
// They meet in LDS, and each row tile leaves its sums; a second kernel adds
// those of a group's tiles in their order, so the same inputs give the same
// bits.  dy and pre are read for the last time, so they are loaded past the
// caches: after other work, 16384 x 8192 bf16 GELU took 168 us so and 198 with
// plain loads, and the read of dpre that follows is as fast or faster.  Its
// tiles since (below): 142 us, 5.7 TB/s.  By group nothing overlaps the search
// for a tile's group: gated SiLU over 64 groups of 20608 rows in 24576 x 2048
// takes 98 us (455 MB, 4.7 TB/s) after other work and 81 where its inputs are in
// the last cache; the bias 11 more.
#include "act.h"
#include "mxq_kernels.h"

namespace mxq {
namespace {

typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef u4 u4_at2 __attribute__((aligned(2)));

struct GradArgs {
    const void *dy, *pre;
    int64_t ld_dy, ld_pre;
    void* dpre;
    int64_t ld_d;
    int64_t M, N;
    const int32_t* offs;         // null: one group of all rows
    int32_t G, act;
    int32_t shift;               // a row tile has 2^shift rows
    float* sums;                 // [row tile][W]; null: no bias
    float* dbias;                // [G][W]
};

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <> struct Elem<__bf16> {
    static __device__ __forceinline__ float get(__bf16 x) { return float(x); }
    static __device__ __forceinline__ __bf16 put(float x) { return __bf16(x); }   // nearest-even
};

__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Calls f(group, first row, end, tiles before it) for 64 groups at a time, one
// to a lane, the tail (group G) last; ends are clamped to an ascending
// sequence in [0, M].  f returns true to stop.
template <typename F>
__device__ __forceinline__ void each_group(const GradArgs& p, F&& f) {
    const uint32_t lane = threadIdx.x & 63u;
    int32_t end = 0;
    int64_t tiles = 0;
    for (int32_t base = 0; base <= p.G; base += 64) {
        const int32_t g = base + int32_t(lane);
        int32_t c = g < p.G ? p.offs[g] : int32_t(p.M);
        c = c < 0 ? 0 : (int64_t(c) > p.M ? int32_t(p.M) : c);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(c, d, 64);
            if (lane >= uint32_t(d)) c = max(c, o);
        }
        c = max(c, end);
        int32_t start = __shfl_up(c, 1, 64);
        if (lane == 0) start = end;
        const int32_t own = g <= p.G ? int32_t((int64_t(c) - start + (int64_t(1) << p.shift) - 1) >> p.shift) : 0;
        int32_t sum = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(sum, d, 64);
            if (lane >= uint32_t(d)) sum += o;
        }
        if (f(g, start, c, tiles + sum - own, own)) return;
        tiles += uniform(__shfl(sum, 63, 64));
        end = uniform(__shfl(c, 63, 64));
    }
}

constexpr int kCol = 32, kRow = 8, kThr = kCol * kRow, kDeep = 2;

template <typename T, bool kGated, int kAct>
__device__ __forceinline__ void grad_rows(const GradArgs& p, int64_t m0, int64_t m1, bool zero, int64_t tile, float* lds) {
    constexpr int kPer = 16 / int(sizeof(T)), kParts = kGated ? 2 : 1;
    const uint32_t t = threadIdx.x, c = t & 31u, r = t >> 5;
    const int64_t col = (int64_t(blockIdx.y) * kCol + c) * kPer;
    const bool all = col + kPer <= p.N;
    const T *dy = static_cast<const T*>(p.dy) + col, *pre = static_cast<const T*>(p.pre) + col;
    T* out = static_cast<T*>(p.dpre) + col;
    float sum[kParts][kPer];
#pragma unroll
    for (int h = 0; h < kParts; ++h)
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[h][i] = 0.f;
    auto one = [&](float g, float x, float u, int i, float& a, float& b) {
        float value;
        a = g * act_slope<kAct>(x, &value);
        if constexpr (kGated) {
            a *= u;
            b = g * value;
            sum[1][i] += b;
        }
        sum[0][i] += a;
    };
    struct Row {
        u4 d, x, u;
    };
    auto piece = [](const T* from) { return __builtin_nontemporal_load(reinterpret_cast<const u4_at2*>(from)); };
    auto fetch = [&](Row& w, int64_t m) {
        w.d = piece(dy + m * p.ld_dy);
        w.x = piece(pre + m * p.ld_pre);
        if constexpr (kGated) w.u = piece(pre + m * p.ld_pre + p.N);
    };
    auto finish = [&](const Row& w, int64_t m) {
        T d[kPer], x[kPer], u[kPer], o[kPer], ou[kPer];
        __builtin_memcpy(d, &w.d, 16);
        __builtin_memcpy(x, &w.x, 16);
        if constexpr (kGated) __builtin_memcpy(u, &w.u, 16);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float a, b = 0.f;
            one(Elem<T>::get(d[i]), Elem<T>::get(x[i]), kGated ? Elem<T>::get(u[i]) : 0.f, i, a, b);
            o[i] = Elem<T>::put(a);
            if constexpr (kGated) ou[i] = Elem<T>::put(b);
        }
        __builtin_memcpy(out + m * p.ld_d, o, 16);
        if constexpr (kGated) __builtin_memcpy(out + m * p.ld_d + p.N, ou, 16);
    };
    int64_t m = m0 + r;
    if (zero) {
        const u4 o = {};
        for (; m < m1; m += kRow) {
            if (all) {
                __builtin_memcpy(out + m * p.ld_d, &o, 16);
                if constexpr (kGated) __builtin_memcpy(out + m * p.ld_d + p.N, &o, 16);
                continue;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (col + i >= p.N) continue;
                out[m * p.ld_d + i] = Elem<T>::put(0.f);
                if constexpr (kGated) out[m * p.ld_d + p.N + i] = Elem<T>::put(0.f);
            }
        }
    } else if (all) {
        // kDeep rows of the thread are read before the first is worked on
        for (; m + (kDeep - 1) * kRow < m1; m += kDeep * kRow) {
            Row w[kDeep];
#pragma unroll
            for (int i = 0; i < kDeep; ++i) fetch(w[i], m + i * kRow);
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                finish(w[i], m + i * kRow);
            }
        }
        for (; m < m1; m += kRow) {
            Row w;
            fetch(w, m);
            finish(w, m);
        }
    } else {
        // the last piece of a row that ends inside it
        for (; m < m1; m += kRow) {
            T d[kPer], x[kPer], u[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (col + i >= p.N) continue;
                d[i] = dy[m * p.ld_dy + i];
                x[i] = pre[m * p.ld_pre + i];
                if constexpr (kGated) u[i] = pre[m * p.ld_pre + p.N + i];
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (col + i >= p.N) continue;
                float a, b = 0.f;
                one(Elem<T>::get(d[i]), Elem<T>::get(x[i]), kGated ? Elem<T>::get(u[i]) : 0.f, i, a, b);
                out[m * p.ld_d + i] = Elem<T>::put(a);
                if constexpr (kGated) out[m * p.ld_d + p.N + i] = Elem<T>::put(b);
            }
        }
    }
    if (p.sums == nullptr || zero) return;                                  // uniform
    const int64_t W = p.N * kParts;
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
        if (h > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) lds[(r * kPer + i) * kCol + c] = sum[h][i];
        __syncthreads();
        // column i of piece c: kCol kPer of them
        for (uint32_t q = t; q < uint32_t(kCol * kPer); q += kThr) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kRow; ++w) s += lds[w * (kPer * kCol) + q];
            const int64_t n = (int64_t(blockIdx.y) * kCol + (q & 31u)) * kPer + (q >> 5);
            if (n < p.N) p.sums[tile * W + h * p.N + n] = s;
        }
    }
}

template <typename T, bool kGated>
__global__ __launch_bounds__(kThr) void act_grad_kernel(GradArgs p) {
    __shared__ float lds[kRow * kCol * (16 / int(sizeof(T)))];
    const int64_t tile = blockIdx.x;
    int64_t m0 = tile << p.shift, m1 = min(m0 + (int64_t(1) << p.shift), p.M);
    bool zero = false;
    if (p.offs != nullptr) {
        bool found = false;
        each_group(p, [&](int32_t g, int32_t start, int32_t end, int64_t before, int32_t own) {
            const uint64_t at = __ballot(own > 0 && before <= tile && tile < before + own);
            if (at == 0) return false;
            const int w = __builtin_ctzll(at);
            const int64_t s = uniform(__shfl(start, w, 64)), e = uniform(__shfl(end, w, 64));
            const int32_t skip = int32_t(tile) - uniform(__shfl(int32_t(before), w, 64));
            m0 = s + (int64_t(skip) << p.shift);
            m1 = min(m0 + (int64_t(1) << p.shift), e);
            zero = uniform(__shfl(g, w, 64)) >= p.G;
            found = true;
            return true;
        });
        if (!found) return;                                                 // uniform
    }
    act_switch(p.act, [&](auto a) { grad_rows<T, kGated, decltype(a)::value>(p, m0, m1, zero, tile, lds); });
}

// The sums of one group's row tiles for 64 channels: kSeg segments of the tiles
// in turn, eight loads in flight, then the segments.  16 segments where groups
// have many tiles, else four and smaller workgroups.
template <int kSeg>
__global__ __launch_bounds__(64 * kSeg) void bias_sum_kernel(GradArgs p, int64_t W) {
    __shared__ float lds[kSeg][64];
    const uint32_t t = threadIdx.x, c = t & 63u, seg = t >> 6;
    const int32_t g = int32_t(blockIdx.y);
    int64_t first = 0, tiles = (p.M + (int64_t(1) << p.shift) - 1) >> p.shift;
    if (p.offs != nullptr) {
        each_group(p, [&](int32_t at, int32_t, int32_t, int64_t before, int32_t own) {
            const uint64_t mine = __ballot(at == g);
            if (mine == 0) return false;
            const int w = __builtin_ctzll(mine);
            first = uniform(__shfl(int32_t(before), w, 64));
            tiles = uniform(__shfl(own, w, 64));
            return true;
        });
    }
    const int64_t n = int64_t(blockIdx.x) * 64 + c, per = (tiles + kSeg - 1) / kSeg;
    const int64_t b0 = min(int64_t(seg) * per, tiles), b1 = min(b0 + per, tiles);
    const float* from = p.sums + first * W + min(n, W - 1);
    float s = 0.f;
    for (int64_t b = b0; b < b1; b += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = from[min(b + i, b1 - 1) * W];
#pragma unroll
        for (int i = 0; i < 8; ++i) s += b + i < b1 ? v[i] : 0.f;
    }
    lds[seg][c] = s;
    __syncthreads();
    if (seg != 0 || n >= W) return;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kSeg; ++w) s += lds[w][c];
    p.dbias[int64_t(g) * W + n] = s;
}

// Rows of a tile: at least 16 and at most 256, while there are 4096 workgroups
// (16 to a CU: 16384 x 8192 bf16 took 161 us with half of them, 141 so; twice as
// many cost 20480 x 2048 gated in 64 groups 8 us in the sums of the bias) or
// 1024 row tiles (a bias adds one number of each).
int grad_shift(int64_t M, int64_t N, int esz) {
    const int64_t slabs = (N * esz + 16 * kCol - 1) / (16 * kCol);
    int s = 8;
    for (; s > 4; --s) {
        const int64_t tiles = (M + (int64_t(1) << s) - 1) >> s;
        if (tiles * slabs >= 4096 || tiles >= 1024) break;
    }
    return s;
}
int64_t grad_tiles(int64_t M, int32_t G, bool groups, int shift) {
    const int64_t full = (M + (int64_t(1) << shift) - 1) >> shift;
    return groups ? full + (int64_t(G) + 1 < M ? int64_t(G) + 1 : M) : full;
}

}  // namespace

int64_t act_grad_workspace(int64_t M, int64_t N, int dtype, bool gated, bool groups, int32_t G) {
    return M <= 0 ? 0 : grad_tiles(M, G, groups, grad_shift(M, N, dtype == 0 ? 4 : 2)) * N * (gated ? 2 : 1) * 4;
}

uint64_t act_grad_threads(int64_t M, int64_t N, int dtype, bool groups, int32_t G) {
    return uint64_t(grad_tiles(M, G, groups, grad_shift(M, N, dtype == 0 ? 4 : 2))) * kThr;
}

hipError_t launch_act_grad(const void* dy, int64_t ld_dy, const void* pre, int64_t ld_pre, int dtype, int64_t M, int64_t N,
                           int act, bool gated, const int32_t* offs, int32_t G, void* dpre, int64_t ld_d, float* dbias,
                           float* workspace, hipStream_t stream) {
    GradArgs p;
    p.dy = dy; p.pre = pre; p.ld_dy = ld_dy; p.ld_pre = ld_pre; p.dpre = dpre; p.ld_d = ld_d; p.M = M; p.N = N;
    p.offs = offs; p.G = offs ? G : 1; p.act = act; p.sums = dbias ? workspace : nullptr; p.dbias = dbias;
    const int esz = dtype == 0 ? 4 : 2;
    p.shift = grad_shift(M, N, esz);
    const int64_t W = N * (gated ? 2 : 1);
    if (M > 0) {
        const dim3 grid(uint32_t(grad_tiles(M, p.G, offs != nullptr, p.shift)), uint32_t((N * esz + 16 * kCol - 1) / (16 * kCol)));
        if (dtype == 0) {
            if (gated) hipLaunchKernelGGL((act_grad_kernel<float, true>), grid, dim3(kThr), 0, stream, p);
            else hipLaunchKernelGGL((act_grad_kernel<float, false>), grid, dim3(kThr), 0, stream, p);
        } else {
            if (gated) hipLaunchKernelGGL((act_grad_kernel<__bf16, true>), grid, dim3(kThr), 0, stream, p);
            else hipLaunchKernelGGL((act_grad_kernel<__bf16, false>), grid, dim3(kThr), 0, stream, p);
        }
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dbias) {
        const dim3 grid(uint32_t((W + 63) / 64), uint32_t(p.G));
        if ((M >> p.shift) / p.G < 32)
            hipLaunchKernelGGL((bias_sum_kernel<4>), grid, dim3(256), 0, stream, p, W);
        else
            hipLaunchKernelGGL((bias_sum_kernel<16>), grid, dim3(1024), 0, stream, p, W);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace mxq
