// Shared by the kernels of linear_forward: matrix-core steps for both types,
// and the epilogue.
#pragma once

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

// erf(x) to fp32: the library's.  tanh(u) through 1 - 2 / (exp(2u) + 1) keeps
// its absolute error near 2^-24, which is what (1 + tanh) is added to.
__device__ __forceinline__ float linear_act(int act, float pa, float pb, float v) {
    switch (act) {
    case CONV_ACT_RELU:
        return v > 0.0f ? v : v != v ? v : 0.0f;
    case CONV_ACT_LEAKY_RELU:
        return v >= 0.0f ? v : pa * v;
    case CONV_ACT_CLIP:
        return fminf(fmaxf(v, pa), pb);
    case LINEAR_ACT_SILU:
        return v / (1.0f + __expf(-v));
    case LINEAR_ACT_GELU:
        return 0.5f * v * (1.0f + erff(v * 0.70710678118654752440f));
    case LINEAR_ACT_GELU_TANH: {
        const float u = 0.79788456080286535588f * (v + 0.044715f * v * v * v);
        return v - v / (1.0f + __expf(2.0f * u));
    }
    default:
        return v;
    }
}

// Four outputs of row m, columns n .. n + 3 (those below a.n).
template <typename T>
__device__ __forceinline__ void linear_store(const LinearArgs& a, int m, int n, f32x4 v) {
    typedef typename Vec<T>::v4 V;
    if (m >= a.m || n >= a.n) return;
    T* y = (T*)a.y + (int64_t)m * a.ys + n;
    const T* r = a.residual ? (const T*)a.residual + (int64_t)m * a.rs + n : nullptr;
    if (a.vec_out) {
        f32x4 b{0, 0, 0, 0}, res{0, 0, 0, 0};
        if (a.bias) b = *(const f32x4*)(a.bias + n);
        if (r) res = to_f32(*(const V*)r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = linear_act(a.act, a.act_a, a.act_b, v[i] + b[i]) + res[i];
        *(V*)y = from_f32<T>(v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= a.n) break;
        const float b = a.bias ? a.bias[n + i] : 0.0f;
        const float res = r ? to_f32(r[i]) : 0.0f;
        y[i] = from_f32<T>(linear_act(a.act, a.act_a, a.act_b, v[i] + b) + res);
    }
}

}  // namespace conv2d
