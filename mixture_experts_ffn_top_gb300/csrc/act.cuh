// act.cuh -- activations of the 16-bit products' epilogues, in fp32, a few 2^-21 of the result.
#pragma once

#include "moe_internal.cuh"

namespace moe {

__device__ __forceinline__ float act_relu(float v) { return v < 0.0f ? 0.0f : v; }  // a NaN stays

// v / (1 + e^-v); for v below -88 the exponential is infinite and the result -0, as the definition rounds
__device__ __forceinline__ float act_silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

// v Phi(v), Phi the normal distribution: with z = |v| / sqrt(2) and t = 1 / (1 + 0.35 z),
// erfc(z) e^(z^2) = t p(t), p a polynomial fitted to it over all z >= 0 (weighted least squares, 8.3e-7 relative).
// No cancellation on the negative side, where 1 + erf would have lost the digits.
__device__ __forceinline__ float act_gelu(float v) {
    const float z = fabsf(v) * 0.70710678f;
    const float t = __fdividef(1.0f, fmaf(z, 0.35f, 1.0f));
    float p = -0.0851045461f;
    p = fmaf(p, t, 0.201206708f);
    p = fmaf(p, t, -0.0145455287f);
    p = fmaf(p, t, 0.162940193f);
    p = fmaf(p, t, 0.154674005f);
    p = fmaf(p, t, 0.1859089f);
    p = fmaf(p, t, 0.19745316f);
    p = fmaf(p, t, 0.197466285f);
    const float q = 0.5f * t * p * __expf(-z * z);
    return v * (v < 0.0f ? q : 1.0f - q);
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
            for (int i = 0; i < N; ++i) v[i] = act_gelu(v[i]);
            break;
        default: break;
    }
}

}  // namespace moe
