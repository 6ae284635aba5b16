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

typedef v4i v4i_any __attribute__((aligned(2)));   // 16 bytes on the boundary of any element

// Eight neighbouring elements as they lie in memory.
template <class T>
struct Eight {
    static constexpr int kWords = sizeof(T) / 2;   // of 16 bytes
    v4i w[kWords];

    __device__ __forceinline__ float at(int j) const {
        constexpr int kPer = 16 / sizeof(T);
        T e[kPer];
        __builtin_memcpy(e, &w[j / kPer], 16);
        return to_f32(e[j % kPer]);
    }
    // All eight from p on.
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = *((const v4i_any*)p + i);
    }
    // From p on, the first `count` of them present, the rest 0 (count below 1: none is read).  All eight take 16-byte
    // loads on any boundary of an element: the hardware takes them unaligned.
    __device__ __forceinline__ void load(const T* p, int64_t count) {
        if (count >= 8) {
            load(p);
        } else {
            T e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[j] = T{};
                if (j < count) e[j] = p[j];
            }
            __builtin_memcpy(w, e, sizeof(e));
        }
    }
};

// The largest of the 16 lanes of a row of lanes, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#define BCJR_ROTATE(n) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xf, 0xf, false))
    BCJR_ROTATE(1);
    BCJR_ROTATE(2);
    BCJR_ROTATE(4);
    BCJR_ROTATE(8);
#undef BCJR_ROTATE
    return v;
}

}  // namespace bcjr
