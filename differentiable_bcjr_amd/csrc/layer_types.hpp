// layer_types.hpp -- the element types of the layer's matrices: conversions and eight-element loads.
#pragma once
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mfma_tile.hpp"

namespace bcjr {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__hip_bfloat16 x) {
    return __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, x) << 16);
}
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ _Float16 from_f32<_Float16>(float x) { return (_Float16)x; }
template <>
__device__ __forceinline__ __hip_bfloat16 from_f32<__hip_bfloat16>(float x) { return __float2bfloat16(x); }

// 8 elements from p on, the first `count` of them present (the rest 0).  `wide`: all 8 are, on a 16-byte boundary.
template <class T>
__device__ __forceinline__ void load8(const T* p, int count, bool wide, float (&v)[8]) {
    if (wide) {
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 8; j += kPer) {
            const v4i w = *(const v4i*)(p + j);
            T e[kPer];
            __builtin_memcpy(e, &w, 16);
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[j + i] = to_f32(e[i]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < count ? to_f32(p[j]) : 0.0f;
    }
}

}  // namespace bcjr
