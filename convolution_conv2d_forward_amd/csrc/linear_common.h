// Matrix-core steps for both types, and what the kernels of linear_forward
// share.
#pragma once

#include <type_traits>

#include "seq_common.h"

namespace conv2d {

// One 16x16 product step over 64 bytes of each row.  Lane l holds 16 bytes of
// row (l & 15) of each operand, the chunk l >> 4 of the four; the fp32 steps
// use element j of every lane's chunk in step j, which permutes the order of
// the sum alike for both operands.  Result: lane l holds rows 4 (l >> 4) + i
// of A against row (l & 15) of B.
template <typename T>
__device__ __forceinline__ f32x4 mfma_step(u32x4 a, u32x4 b, f32x4 c);

template <>
__device__ __forceinline__ f32x4 mfma_step<bf16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

template <>
__device__ __forceinline__ f32x4 mfma_step<float>(u32x4 a, u32x4 b, f32x4 c) {
    const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[j], fb[j], c, 0, 0, 0);
    return c;
}

// One 32x32 product step over 32 bytes of each row: lane l holds 16 bytes of
// row (l & 31) of each operand, chunk l >> 5 of the two.  Result: lane l holds
// rows 8 (i / 4) + 4 (l >> 5) + i % 4 of A against row (l & 31) of B.
template <typename T>
__device__ __forceinline__ f32x16 mfma32_step(u32x4 a, u32x4 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mfma32_step<bf16>(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
template <>
__device__ __forceinline__ f32x16 mfma32_step<float>(u32x4 a, u32x4 b, f32x16 c) {
    const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[j], fb[j], c, 0, 0, 0);
    return c;
}

// Kinds of activation that kernels are compiled for: one kernel for all would
// hold every activation's code once for each block of outputs, some 300 KB,
// and wait for its instructions.
enum { kActNone, kActPiecewise, kActSilu, kActGelu, kActGeluTanh };

// exp for results of type T.  The hardware's takes x log2(e) rounded, which is
// off by some 2^-24 x: bf16 does not show that, for fp32 what the rounding left,
// `low`, goes onto the result.  (expf has the same correction, which this
// library's -ffp-contract=fast undoes: it fuses a product into a difference
// that relies on the product's rounding.)
template <typename T>
__device__ __forceinline__ float act_exp(float x) {
    const float t = x * kLog2e, r = __builtin_amdgcn_exp2f(t);
    if (sizeof(T) == 2) return r;
    const float low = __builtin_fmaf(x, 1.92596299112661746887e-8f, __builtin_fmaf(x, kLog2e, -t));
    return fabsf(t) < 128.0f ? __builtin_fmaf(r, low * 0.69314718055994530942f, r) : r;
}

// x (1 + erf(x / sqrt 2)) / 2 as x erfc(-x / sqrt 2) / 2.  With z = |x| / sqrt 2
// and t = 1 / (1 + 0.3 z), erfc(z) exp(z^2) is t times a polynomial of t fitted
// to 2e-8 relative for z up to 9.5, where fp32's smallest number lies; 5e-7 as
// evaluated here.  (4096x1024->4096 bf16 47 us, with erfcf 59.)
template <typename T>
__device__ __forceinline__ float gelu_erf(float x) {
    const float c[9] = {0.169189617f, 0.170691982f, 0.148482114f, 0.214437470f, -0.0936339349f,
                        0.546398759f, -0.511229634f, 0.485097945f, -0.129434377f};
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3f * 0.70710678118654752440f * fabsf(x));
    float p = c[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) p = __builtin_fmaf(p, t, c[i]);
    const float q = p * t * act_exp<T>(-0.5f * x * x);
    return 0.5f * x * (x > 0.0f ? 2.0f - q : q);
}

// The activation of N values.  v (1 + tanh u) / 2 is v / (1 + exp(-2u)), and
// v (1 + erf z) / 2 is v erfc(-z) / 2: nothing cancels in them, so the tails
// keep their relative accuracy and +inf stays.
template <typename T, int KIND, int N>
__device__ __forceinline__ void linear_act(const LinearArgs& a, float* v) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x = v[i];
        if constexpr (KIND == kActPiecewise) {
            if (a.act == CONV_ACT_CLIP)
                v[i] = fminf(fmaxf(x, a.act_a), a.act_b);
            else   // RELU (act_a = 0) and LEAKY_RELU; NaN stays
                v[i] = x > 0.0f ? x : a.act_a == 0.0f ? (x != x ? x : 0.0f) : a.act_a * x;
        } else if constexpr (KIND == kActSilu) {
            v[i] = x / (1.0f + act_exp<T>(-x));
        } else if constexpr (KIND == kActGelu) {
            v[i] = gelu_erf<T>(x);
        } else if constexpr (KIND == kActGeluTanh) {
            const float u = 0.79788456080286535588f * (x + 0.044715f * x * x * x);
            v[i] = x / (1.0f + act_exp<T>(-2.0f * u));
        }
    }
}

// Calls f with the kind of a's activation as a compile-time constant.
template <typename F>
hipError_t with_act(const LinearArgs& a, F f) {
    switch (a.act) {
    case CONV_ACT_NONE: return f(std::integral_constant<int, kActNone>{});
    case LINEAR_ACT_SILU: return f(std::integral_constant<int, kActSilu>{});
    case LINEAR_ACT_GELU: return f(std::integral_constant<int, kActGelu>{});
    case LINEAR_ACT_GELU_TANH: return f(std::integral_constant<int, kActGeluTanh>{});
    default: return f(std::integral_constant<int, kActPiecewise>{});
    }
}

// 16 bytes from p on at any alignment of the element, of which `left` elements
// belong to the row: zero past them.
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* p, int left) {
    constexpr int C = Vec<T>::chunk;
    u32x4 r;
    if (left >= C) {
        __builtin_memcpy(&r, p, 16);
        return r;
    }
    T e[C];
#pragma unroll
    for (int i = 0; i < C; ++i) e[i] = i < left ? p[i] : (T)0.0f;
    __builtin_memcpy(&r, e, 16);
    return r;
}

// The same for bf16 put together from the five words that a chunk between
// 4-byte boundaries touches, which hold an element before p and one past p + 7:
// not for chunks at a row's `end`.  Where few waves wait for few chunks that is
// faster than a load of 16 bytes at such an address (24x4097x1126: 17.1 us
// against 27.0), where many are loaded slower (4001x1003x4003: 132 against 71).
__device__ __forceinline__ u32x4 load_words(const bf16* p, bool end, int left) {
    typedef u32x4 __attribute__((aligned(4))) words;
    if (end) return load_chunk<bf16>(p, left);
    const uint32_t odd = (uint32_t)(uintptr_t)p & 2;
    const uint32_t* q = (const uint32_t*)((uintptr_t)p - odd);
    const u32x4 d = *(const words*)q;
    const uint32_t d4 = q[odd ? 4 : 3];
    u32x4 r;
    r[0] = __builtin_amdgcn_alignbit(d[1], d[0], odd * 8);
    r[1] = __builtin_amdgcn_alignbit(d[2], d[1], odd * 8);
    r[2] = __builtin_amdgcn_alignbit(d[3], d[2], odd * 8);
    r[3] = __builtin_amdgcn_alignbit(d4, d[3], odd * 8);
    return r;
}
__device__ __forceinline__ u32x4 load_words(const float* p, bool, int left) { return load_chunk<float>(p, left); }

// Kernels of a call: few rows of x, or few tiles of a long k (linear_rows.hip),
// or tiles of as many rows of x and w (linear_tile.h), 128 with two workgroups
// on a CU or with one and a deeper pipeline.
enum linear_tile_t { LINEAR_ROWS, LINEAR_TILE_64, LINEAR_TILE_128, LINEAR_TILE_128_DEEP, LINEAR_TILE_256 };

// linear_rows: a workgroup's rows of x are 16 MT, k is dealt among its waves.
// As many workgroups as fit one each on the CUs, then as many rows as there
// are, up to 64 (32 through registers): 46x5824x192 fp32 takes 12.0 us with MT
// 1 and 34.2 with 4, 64x4096x4096 43.5 and 27.1.
struct RowsShape {
    int mt, waves;
};
inline RowsShape rows_shape(bool f32, const LinearArgs& a) {
    const int64_t cus = device_cu_count(), m = a.m, n = (a.n + 15) / 16;
    if (m <= 16 || (m + 15) / 16 * n <= cus * 3 / 4) return {1, 8};
    if (!a.vec) return {2, 8};
    if ((m + 31) / 32 * n <= cus) return {2, f32 ? 8 : 4};
    return {a.m <= 32 ? 2 : 4, 4};
}

// Any number of rows of x.
hipError_t launch_linear_rows(int32_t dtype, const LinearArgs& a, hipStream_t s);

template <typename T>
hipError_t launch_linear_tile(const LinearArgs& a, linear_tile_t tile, hipStream_t s);
template <>
hipError_t launch_linear_tile<float>(const LinearArgs& a, linear_tile_t tile, hipStream_t s);
template <>
hipError_t launch_linear_tile<bf16>(const LinearArgs& a, linear_tile_t tile, hipStream_t s);

}  // namespace conv2d
