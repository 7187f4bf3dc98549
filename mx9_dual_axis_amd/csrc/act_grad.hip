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
// piece c, eight rows at a time, and adds its columns' sums in registers.  They
// meet in LDS, and each row tile leaves its sums; a second kernel adds those
// of a group's tiles in their order, so the same inputs give the same bits.
// Row tiles are as tall as still gives every CU a few workgroups.
#include "act.h"
#include "mxq_kernels.h"

namespace mxq {
namespace {

typedef unsigned int u4 __attribute__((ext_vector_type(4)));

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

constexpr int kCol = 32, kRow = 8, kThr = kCol * kRow;

template <typename T, bool kGated, int kAct>
__device__ __forceinline__ void grad_rows(const GradArgs& p, int64_t m0, int64_t m1, bool zero, int64_t tile, float* lds) {
    constexpr int kPer = 16 / int(sizeof(T)), kParts = kGated ? 2 : 1;
    const uint32_t t = threadIdx.x, c = t & 31u, r = t >> 5;
    const int64_t col = (int64_t(blockIdx.y) * kCol + c) * kPer;
    const bool some = col < p.N, all = col + kPer <= p.N;
    const T *dy = static_cast<const T*>(p.dy) + col, *pre = static_cast<const T*>(p.pre) + col;
    T* out = static_cast<T*>(p.dpre) + col;
    float sum[kParts][kPer];
#pragma unroll
    for (int h = 0; h < kParts; ++h)
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[h][i] = 0.f;
    auto load = [&](const T* from, T (&v)[kPer]) {
        if (all) {
            __builtin_memcpy(v, from, 16);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[i] = from[min(int64_t(i), p.N - 1 - col)];
        }
    };
    auto store = [&](T* to, const T (&v)[kPer]) {
        if (all) {
            u4 x;
            __builtin_memcpy(&x, v, 16);
            __builtin_memcpy(to, &x, 16);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (col + i < p.N) to[i] = v[i];
        }
    };
    if (some) {
        for (int64_t m = m0 + r; m < m1; m += kRow) {
            T d[kPer], x[kPer], u[kPer], o[kPer], ou[kPer];
            if (!zero) {
                load(dy + m * p.ld_dy, d);
                load(pre + m * p.ld_pre, x);
                if (kGated) load(pre + m * p.ld_pre + p.N, u);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (zero) {
                    o[i] = ou[i] = Elem<T>::put(0.f);
                    continue;
                }
                float value;
                const float slope = act_slope<kAct>(Elem<T>::get(x[i]), &value), g = Elem<T>::get(d[i]);
                float a = g * slope;
                if (kGated) {
                    a *= Elem<T>::get(u[i]);
                    const float b = g * value;
                    sum[kParts - 1][i] += b;
                    ou[i] = Elem<T>::put(b);
                }
                sum[0][i] += a;
                o[i] = Elem<T>::put(a);
            }
            store(out + m * p.ld_d, o);
            if (kGated) store(out + m * p.ld_d + p.N, ou);
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

// The sums of one group's row tiles, for 64 channels: 16 segments of the tiles
// in turn, then the segments.
__global__ __launch_bounds__(1024) void bias_sum_kernel(GradArgs p, int64_t W) {
    __shared__ float lds[16][64];
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
    const int64_t n = int64_t(blockIdx.x) * 64 + c, per = (tiles + 15) / 16;
    const int64_t b0 = min(int64_t(seg) * per, tiles), b1 = min(b0 + per, tiles);
    float s = 0.f;
    if (n < W) {
#pragma unroll 8
        for (int64_t b = b0; b < b1; ++b) s += p.sums[(first + b) * W + n];
    }
    lds[seg][c] = s;
    __syncthreads();
    if (seg == 0 && n < W) {
        s = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) s += lds[w][c];
        p.dbias[int64_t(g) * W + n] = s;
    }
}

// Rows of a tile: at least 16 and at most 256, while there are 1024 workgroups
// (four to a CU).
int grad_shift(int64_t M, int64_t N, int esz) {
    const int64_t slabs = (N * esz + 16 * kCol - 1) / (16 * kCol);
    int s = 8;
    while (s > 4 && ((M + (int64_t(1) << s) - 1) >> s) * slabs < 1024) --s;
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
        hipLaunchKernelGGL(bias_sum_kernel, dim3(uint32_t((W + 63) / 64), uint32_t(p.G)), dim3(1024), 0, stream, p, W);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace mxq
