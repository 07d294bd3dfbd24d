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

// Eight elements at a 16-byte boundary.
template <typename T>
__device__ __forceinline__ f32x8 load8(const T* p) {
    typedef T V __attribute__((ext_vector_type(8)));
    return __builtin_convertvector(*(const V*)p, f32x8);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, f32x8 v) {
    typedef T V __attribute__((ext_vector_type(8)));
    *(V*)p = __builtin_convertvector(v, V);
}

// A pointer that is the same in all lanes, in scalar registers.
template <typename P>
__device__ __forceinline__ P* uniform(P* p) {
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (P*)(uintptr_t)(hi << 32 | lo);
}

// 16 bytes per lane from base + off (bytes) straight to LDS: lane l writes
// lds + 16 l (lds wave-uniform).  Inline assembly, so that the compiler does
// not order later LDS reads of the other stage behind it; the kernels' own
// waits order the copies.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_to_lds(const void* base, uint32_t off, const u32x4* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    const uint32_t m = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(m)
                 : "memory", "m0");
#endif
}
// The same for 4 bytes per lane: lane l writes lds + 4 l bytes.
__device__ __forceinline__ void copy4_to_lds(const void* base, uint32_t off, const u32x4* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    const uint32_t m = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(m)
                 : "memory", "m0");
#endif
}
#pragma clang diagnostic pop

// Waits until at most N of this thread's vector memory operations are left.
template <int N>
__device__ __forceinline__ void wait_vmem() {
    static_assert(N < 64, "counter");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

}  // namespace conv2d
