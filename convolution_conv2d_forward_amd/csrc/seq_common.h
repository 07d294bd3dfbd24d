// Device helpers of the attention-layer kernels (linear, qk_rope, attention).
#pragma once

#include "attention_internal.h"
#include "device_common.h"

namespace conv2d {

typedef __bf16 bf16;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return (float)v; }

// One rounding to nearest even for bf16.
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
    return (T)v;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    typedef f32x4 v4;
    static constexpr int chunk = 4;   // elements of 16 bytes
};
template <>
struct Vec<bf16> {
    typedef bf16x4 v4;
    static constexpr int chunk = 8;
};

__device__ __forceinline__ f32x4 to_f32(f32x4 v) { return v; }
__device__ __forceinline__ f32x4 to_f32(bf16x4 v) { return __builtin_convertvector(v, f32x4); }

template <typename T>
__device__ __forceinline__ typename Vec<T>::v4 from_f32(f32x4 v) {
    return __builtin_convertvector(v, typename Vec<T>::v4);
}

}  // namespace conv2d
