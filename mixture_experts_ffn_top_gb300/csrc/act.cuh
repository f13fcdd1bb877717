// act.cuh -- activations of the 16-bit products' epilogues, in fp32, two values at a time.  Near 0 they are off by a few
// 2^-21 of the result.  Far on the negative side the exponent's own roundings count: with e^-s, s up to 87 off by some
// 2^-24 of itself, SiLU stays within 2^-16 of its value and GELU, whose s is a square, within 2^-18 above -4 and within
// 2^-15 below.  Results below 2^-126 may be 0.
#pragma once

#include "pair.cuh"

namespace moe {

__device__ __forceinline__ float act_exp2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float act_rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float act_relu(float v) {  // a NaN stays
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}

// v / (1 + e^-v), the denominator scaled by 2^-8: the reciprocal is flushed to 0 below 2^-126, where the result can still be
// 88 times as large, a normal bf16 number (the product behind it is not flushed).
__device__ __forceinline__ float act_silu(float v) {
    return v * (act_rcp(act_exp2(fmaf(v, -1.44269504f, -8.0f)) + 0.00390625f) * 0.00390625f);
}

// v Phi(v) = max(v, 0) - |v| Q(|v|), Phi the normal distribution, Q = 1 - Phi = erfc(z) / 2 with z = |v| / sqrt(2).
// With t = 1 / (1 + 0.35 z), erfc(z) e^(z^2) = t p(t), p a polynomial fitted to it over all z >= 0 (weighted least
// squares, 8.3e-7 relative; halved here).  No cancellation on the negative side, where 1 + erf would have lost the
// digits.  An infinity meets Q = 0 as 1e5.
__device__ __forceinline__ void act_gelu(float &a, float &b) {
    const float x = fabsf(a), y = fabsf(b);
    const F2 t = pair_of(act_rcp(fmaf(x, 0.24748737f, 1.0f)), act_rcp(fmaf(y, 0.24748737f, 1.0f)));
    auto c = [](float v) { return pair_of(v, v); };
    F2 p = c(-0.0425522731f);
    p = fma(p, t, c(0.100603354f));
    p = fma(p, t, c(-0.00727276437f));
    p = fma(p, t, c(0.0814700965f));
    p = fma(p, t, c(0.0773370025f));
    p = fma(p, t, c(0.09295445f));
    p = fma(p, t, c(0.09872658f));
    p = fma(p, t, c(0.0987331425f));
    const F2 z = pair_of(x * 0.84932180f, y * 0.84932180f);  // z^2 log2(e) = (|v| sqrt(log2(e) / 2))^2
    const float2 s = values_of(mul(z, z));
    const float2 q = values_of(mul(mul(t, p), pair_of(act_exp2(-s.x), act_exp2(-s.y))));
    a = fmaf(-fminf(x, 1e5f), q.x, act_relu(a));
    b = fmaf(-fminf(y, 1e5f), q.y, act_relu(b));
}

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    switch (act) {
        case MOE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_relu(v[i]);
            break;
        case MOE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_silu(v[i]);
            break;
        case MOE_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float none = 0.0f;
                act_gelu(v[i], i + 1 < N ? v[i + 1] : none);
            }
            break;
        default: break;
    }
}

}  // namespace moe
