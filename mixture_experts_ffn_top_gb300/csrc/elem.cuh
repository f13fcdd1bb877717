// elem.cuh -- element types of the token and 4-bit operators (fp32, fp16, bf16): conversion to and
// from fp32 and accesses of V consecutive elements.  Device code only.
#pragma once

#include <cuda_bf16.h>

#include "moe_internal.cuh"

namespace moe {

__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ float elem_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T elem_of(float v);
template <>
__device__ __forceinline__ float elem_of<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half elem_of<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 elem_of<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements as one access of V * sizeof(T) bytes (2, 4, 8 or 16, so aligned).
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

inline size_t dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

}  // namespace moe
