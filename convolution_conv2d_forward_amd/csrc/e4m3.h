// 8-bit numbers of a paged cache and their scales: a row of a head shares the
// power of two 2^(s - 127) of its scale byte s.
//
// The power is the least one that brings the row's largest finite element to
// 448, the largest code, or below: a power of two costs at most one of the
// format's 18 binades and makes every dequantised element exact in bf16 and
// fp32, so that quantising is the only rounding.  Exponents from -117 on keep
// the smallest code, 2^-9, times the scale a normal number, those up to 119 the
// largest finite.
#pragma once

#include "seq_common.h"

namespace conv2d {

constexpr int kLeastExponent = -117, kMostExponent = 119;

// Scale byte of a row whose largest finite magnitude is `top`: with top =
// m 2^E, 1/2 <= m < 1, and 448 = 7/8 * 2^9 the exponent is E - 9, one more
// where m is above 7/8.
__device__ __forceinline__ uint32_t scale_of(float top) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, top);
    const int e = (int)(bits >> 23) - 126 - 9 + ((bits & 0x7fffffu) > 0x600000u);
    return (uint32_t)(min(max(e, kLeastExponent), kMostExponent) + 127);
}
// 2^(s - 127), and 2^(127 - s) for the bytes that scale_of gives.
__device__ __forceinline__ float scale_value(uint32_t s) { return __builtin_bit_cast(float, s << 23); }
__device__ __forceinline__ float scale_inverse(uint32_t s) { return __builtin_bit_cast(float, (254u - s) << 23); }

__device__ __forceinline__ float finite_size(float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.0f; }

// Two codes, rounded to nearest even.  Infinities become NaN; what the largest
// exponent leaves above 448 becomes 448.
__device__ __forceinline__ uint32_t encode2(float a, float b, float inverse, uint32_t old, bool high) {
    a = fabsf(a) < INFINITY ? __builtin_amdgcn_fmed3f(a * inverse, -448.0f, 448.0f) : NAN;
    b = fabsf(b) < INFINITY ? __builtin_amdgcn_fmed3f(b * inverse, -448.0f, 448.0f) : NAN;
    return high ? (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, true)
                : (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, false);
}
__device__ __forceinline__ uint32_t encode4(f32x4 v, float inverse) {
    return encode2(v[2], v[3], inverse, encode2(v[0], v[1], inverse, 0, false), true);
}

// Codes times their scale: four to fp32, eight to bf16, 16 bytes either way.
template <typename T>
struct Codes;
template <>
struct Codes<float> {
    typedef uint32_t type;   // of 16 bytes of T
};
template <>
struct Codes<bf16> {
    typedef u32x2 type;
};
__device__ __forceinline__ u32x4 decode(uint32_t c, float scale, float) {
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, true);
    return __builtin_bit_cast(u32x4, f32x4{lo[0], lo[1], hi[0], hi[1]});
}
__device__ __forceinline__ u32x4 decode(u32x2 c, float scale, bf16) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], scale, false));
        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], scale, true));
    }
    return r;
}
// One code.
__device__ __forceinline__ float decode1(uint32_t c, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, false)[0];
}

}  // namespace conv2d
