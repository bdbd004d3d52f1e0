// Activations of the gated feed-forward block and their derivatives, in
// float.  Written so that both tails keep their accuracy relative to the value
// down to the smallest floats: the logistic function with its complement, each
// from the exponential that is small on its side, for silu, sigmoid and
// tanh-gelu (0.5 (1 + tanh v) = 1 / (1 + exp(-2v))), and erfc for gelu (0.5 (1 +
// erf(g / sqrt 2)) = 0.5 erfc(-g / sqrt 2)).  None of these cancels or overflows
// before its value does.  What is left is the rounding of the exponent: a
// relative 2^-24 times its size.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

namespace sgemm {

// sgemm_act_t
enum Act { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3, ACT_SIGMOID = 4 };

// exp(x) for x <= 0: x / ln 2 in its nearest integer and a rest of at most a
// half, from ln 2's inverse in two floats (Cody and Waite's reduction).  Off by
// two units in the last place at most, the instruction's one and the rest's
// rounding; expf's cases for large x are not needed here.
__device__ __forceinline__ float exp_neg(float x) {
    const float c = x < -110.0f ? -110.0f : x;  // 0 from -104 on; NaN stays NaN
    const float n = rintf(c * 1.44269504f);
    const float f = fmaf(c, 1.92596303e-8f, fmaf(c, 1.44269504f, -n));
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), int(n));
}
// 1 / d for d in 1 .. 2: one Newton step on the instruction's estimate, off by a
// little over half a unit.  A quotient n (1 / d) rounds once more.
__device__ __forceinline__ float rcp_1to2(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return fmaf(fmaf(-d, r, 1.0f), r, r);
}

// 1 / (1 + exp(-v)) and its complement 1 / (1 + exp(v)).
struct Logistic {
    float s, r;
};
__device__ __forceinline__ Logistic logistic2(float v) {
    const float e = exp_neg(-fabsf(v)), q = rcp_1to2(1.0f + e);
    return v < 0.0f ? Logistic{e * q, q} : Logistic{q, e * q};
}
// n / (1 + exp(-v)), the numerator selected (4096 x 8192 x 4096 with G and U kept
// 3850 us; with expf and the compiler's division 3905; of these with exp(-v)
// whatever its sign, which overflows below -88.7, 3896).
__device__ __forceinline__ float logistic_of(float n, float v) {
    const float e = exp_neg(-fabsf(v));
    return (v < 0.0f ? n * e : n) * rcp_1to2(1.0f + e);
}

// 2 c (g + 0.044715 g^3), c = sqrt(2 / pi): twice the argument of tanh.
__device__ __forceinline__ float gelu_tanh_arg2(float g) {
    return 1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f);
}

__device__ __forceinline__ float act_value(int act, float g) {
    switch (act) {
        case ACT_SILU: return logistic_of(g, g);
        case ACT_GELU: return 0.5f * g * erfcf(-0.70710678118654752f * g);
        case ACT_GELU_TANH: return logistic_of(g, gelu_tanh_arg2(g));
        case ACT_RELU: return g <= 0.0f ? 0.0f : g;  // NaN stays NaN
        default: return logistic_of(1.0f, g);
    }
}

// N activations with one branch on which.
template <int N>
__device__ __forceinline__ void act_values(int act, const float (&g)[N], float (&a)[N]) {
    auto all = [&](auto which) {
#pragma unroll
        for (int i = 0; i < N; i++) a[i] = act_value(decltype(which)::value, g[i]);
    };
    switch (act) {
        case ACT_SILU: return all(std::integral_constant<int, ACT_SILU>{});
        case ACT_GELU: return all(std::integral_constant<int, ACT_GELU>{});
        case ACT_GELU_TANH: return all(std::integral_constant<int, ACT_GELU_TANH>{});
        case ACT_RELU: return all(std::integral_constant<int, ACT_RELU>{});
        default: return all(std::integral_constant<int, ACT_SIGMOID>{});
    }
}

// act(g) and act'(g).  relu'(0) = 0.
__device__ __forceinline__ void act_grad(int act, float g, float* a, float* da) {
    switch (act) {
        case ACT_SILU: {
            const Logistic l = logistic2(g);
            *a = g * l.s;
            *da = l.s * fmaf(g, l.r, 1.0f);
            return;
        }
        case ACT_GELU: {
            const float c = 0.5f * erfcf(-0.70710678118654752f * g);
            *a = g * c;
            *da = fmaf(g * 0.39894228040143268f, expf(-0.5f * g * g), c);
            return;
        }
        case ACT_GELU_TANH: {
            const Logistic l = logistic2(gelu_tanh_arg2(g));
            *a = g * l.s;
            // da = s + g s (1 - s) v', v' = 2 c (1 + 0.134145 g^2).  s (1 - s) is
            // exp(-|v|) or less, 0 in float from |g| = 11 on (v = 112): formed
            // first, and with g cut there in the other factors, the product is 0
            // and not 0 times an overflow.
            const float t = l.s * l.r, gc = fminf(fmaxf(g, -12.0f), 12.0f);
            *da = fmaf(gc * t, 1.5957691216057308f * fmaf(0.134145f * gc, gc, 1.0f), l.s);
            return;
        }
        case ACT_RELU:
            *a = g <= 0.0f ? 0.0f : g;
            *da = g > 0.0f ? 1.0f : 0.0f;
            return;
        default: {
            const Logistic l = logistic2(g);
            *a = l.s;
            *da = l.s * l.r;
            return;
        }
    }
}

}  // namespace sgemm
