// act.h -- activations of a product's epilogue and their slopes, in fp32.
//
//   relu       max(x, 0)
//   silu       x p(x),             p(x) = 1 / (1 + e^-x)
//   gelu       x Phi(x),           Phi the normal distribution's integral
//   gelu_tanh  x p(t),             t = 2 sqrt(2 / pi) (x + 0.044715 x^3)
//
// e^x carries the rounding of its argument's product with log2 e, Phi is formed
// from erfc (1 + erf loses its leading bits below 0), and 1 - p(x) is p(-x), so
// that tails keep their digits.  Largest errors measured over 2^20 points of each
// of eleven ranges in [-80, 80], relative to the value: silu 2^-21.7, gelu
// 2^-20.9; gelu_tanh 2^-21.5 for |x| <= 1 and 3.4 |t| 2^-24 beyond, since t is
// rounded on the way (2^-18.6 at x = -5, 2^-16.3 at -10).  Slopes p + x p' have
// the same errors, relative to |p| + |x p'|.  e^x ends at 2^-126: values below
// 2^-118 may be 0.  A NaN gives NaN.
//
// One formula whatever the results are rounded to: a bf16 result is the fp32 one,
// rounded.  (Formed in fewer operations for bf16, within 2^-16 of the value,
// 8192^3 took 513 us instead of 524 in MXFP8 with GELU, bias, residual and kept
// sums, and 509 instead of 518 in int8 with tanh GELU; shorter products the same
// within 0.3 us.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace mxq {

// Which activation: MX_ACT_* of the header.
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

namespace {

// e^x for x in [-250, 250]: 2^(h + l), h + l = x log2 e, 2^l = 1 + l ln 2.
__device__ __forceinline__ float act_exp(float x) {
    const float h = x * 1.44269502f;
    const float l = __builtin_fmaf(x, 1.44269502f, -h) + x * 1.92596303e-8f;
    const float e = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(e, l * 0.693147182f, e);
}
__device__ __forceinline__ float act_clamp(float x, float m) { return __builtin_amdgcn_fmed3f(x, -m, m); }
// p(x) = 1 / (1 + e^-x) and p(-x), from e^-|x| (which ends at 2^-126).
__device__ __forceinline__ float act_logistic(float x, float* other) {
    const float z = act_exp(-__builtin_fabsf(act_clamp(x, 250.f)));
    const float p = __builtin_amdgcn_rcpf(1.f + z), q = z * p;
    *other = x < 0.f ? p : q;
    return x < 0.f ? q : p;
}

// erfc(|x| / sqrt 2) / 2 = e^(-x^2 / 2) R(1 / (1 + 0.38 |x| / sqrt 2)): R fitted to
// erfcx / 2 for |x| <= 20 (weighted least squares, weights moved until the
// relative error was level: 2.6e-8), the square's rounding carried along.
__device__ __forceinline__ float act_half_erfc(float x, float* density) {
    const float a = act_clamp(x, 20.f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(a), 0.38f * 0.707106769f, 1.f));
    const float q = a * a, lo = __builtin_fmaf(a, a, -q);
    const float e = act_exp(-0.5f * q);
    const float g = __builtin_fmaf(e, -0.5f * lo, e);
    float r = 0.5f * 0.0582896769f;
    r = __builtin_fmaf(r, t, 0.5f * -0.259262949f);
    r = __builtin_fmaf(r, t, 0.5f * 0.358198434f);
    r = __builtin_fmaf(r, t, 0.5f * -0.155643195f);
    r = __builtin_fmaf(r, t, 0.5f * 0.226468056f);
    r = __builtin_fmaf(r, t, 0.5f * 0.139968276f);
    r = __builtin_fmaf(r, t, 0.5f * 0.203619704f);
    r = __builtin_fmaf(r, t, 0.5f * 0.213952541f);
    r = __builtin_fmaf(r, t, 0.5f * 0.214409426f);
    *density = g;                                                           // e^(-x^2 / 2)
    return r * t * g;
}

__device__ __forceinline__ float act_tanh_arg(float x) {
    return 1.59576912f * __builtin_fmaf(0.044715f * x * x, x, x);
}

template <int kAct>
__device__ __forceinline__ float act_value(float x) {
    if constexpr (kAct == kActRelu) return x < 0.f ? 0.f : x;
    float q;
    if constexpr (kAct == kActSilu) return x * act_logistic(x, &q);
    if constexpr (kAct == kActGelu) {
        float d;
        const float r = act_half_erfc(x, &d);
        return x * (x < 0.f ? r : 1.f - r);
    }
    if constexpr (kAct == kActGeluTanh) return x * act_logistic(act_tanh_arg(x), &q);
    return x;
}

// The activation and its slope at x (the slope's limits at the infinities).
template <int kAct>
__device__ __forceinline__ float act_slope(float x, float* value) {
    const float f = x != x ? x : act_clamp(x, 3e4f);                        // what the slope multiplies
    if constexpr (kAct == kActRelu) {
        *value = x < 0.f ? 0.f : x;
        return x > 0.f ? 1.f : x <= 0.f ? 0.f : x;
    }
    if constexpr (kAct == kActSilu) {
        float q;
        const float p = act_logistic(x, &q);
        *value = x * p;
        return p * __builtin_fmaf(f, q, 1.f);
    }
    if constexpr (kAct == kActGelu) {
        float d;
        const float r = act_half_erfc(x, &d), phi = x < 0.f ? r : 1.f - r;
        *value = x * phi;
        return __builtin_fmaf(f * d, 0.398942280f, phi);
    }
    if constexpr (kAct == kActGeluTanh) {
        float q;
        const float p = act_logistic(act_tanh_arg(x), &q);
        *value = x * p;
        return p * __builtin_fmaf(f * q, 1.59576912f * __builtin_fmaf(3.f * 0.044715f * f, f, 1.f), 1.f);
    }
    *value = x;
    return 1.f;
}

// f(std::integral_constant<int, act>) for a uniform act.
template <typename F>
__device__ __forceinline__ void act_switch(int act, F&& f) {
    switch (act) {
        case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
        case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
        default: f(std::integral_constant<int, kActNone>{}); break;
    }
}

}  // namespace
}  // namespace mxq
