// elem.cuh -- element types of the token and 4-bit operators (fp32, fp16, bf16): accesses of V
// consecutive elements, kept packed in registers, and their conversion from and to fp32.
#pragma once

#include <cuda_bf16.h>
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {

template <typename T>
__device__ __forceinline__ T elem_of(float v);
template <>
__device__ __forceinline__ float elem_of<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half elem_of<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 elem_of<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements in the bits of one access of V * sizeof(T) bytes (2, 4, 8 or 16, so aligned).
template <typename T, int V>
struct Pack {
    static constexpr int BYTES = sizeof(T) * V;
    using Word = std::conditional_t<BYTES == 2, uint16_t, uint32_t>;
    using Access = std::conditional_t<BYTES == 16, uint4, std::conditional_t<BYTES == 8, uint2, Word>>;
    static constexpr int WORDS = BYTES < 4 ? 1 : BYTES / 4;
    union {
        Access a;
        Word w[WORDS];
    };

    __device__ __forceinline__ float get(int i) const {
        if constexpr (std::is_same_v<T, float>) {
            return __uint_as_float(w[i]);
        } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            if (V == 1) return __uint_as_float((uint32_t)w[0] << 16);
            return __uint_as_float((i & 1) ? (uint32_t)w[i / 2] & 0xffff0000u : (uint32_t)w[i / 2] << 16);
        } else {
            if (V == 1) return __half2float(__ushort_as_half((unsigned short)w[0]));
            return __half2float(__ushort_as_half((unsigned short)((uint32_t)w[i / 2] >> (16 * (i & 1)))));
        }
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {  // one rounding each
        if constexpr (std::is_same_v<T, float>) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
        } else if constexpr (V == 1) {
            const T v = elem_of<T>(f[0]);
            w[0] = *reinterpret_cast<const uint16_t *>(&v);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                if constexpr (std::is_same_v<T, __half>) {
                    const __half2 v = __floats2half2_rn(f[i], f[i + 1]);
                    w[i / 2] = *reinterpret_cast<const uint32_t *>(&v);
                } else {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(f[i], f[i + 1]);
                    w[i / 2] = *reinterpret_cast<const uint32_t *>(&v);
                }
            }
        }
    }
    __device__ __forceinline__ void load(const T *p) { a = *reinterpret_cast<const Access *>(p); }
    __device__ __forceinline__ void load_once(const T *p) { a = __ldcs(reinterpret_cast<const Access *>(p)); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Access *>(p) = a; }
};

inline size_t dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

}  // namespace moe
