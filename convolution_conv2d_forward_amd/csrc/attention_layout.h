// Tiles of keys and values in LDS, as attention_tile and paged_tile read them.
#pragma once

#include "seq_common.h"

namespace conv2d {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) float lds_f32;

// An LDS address as a pointer.
template <typename P>
__device__ __forceinline__ P* lds_ptr(uint32_t at) {
    return (P*)(uintptr_t)at;
}

// The other half-wave's value and one's own, in both halves alike.
__device__ __forceinline__ void both_halves(float x, float& a, float& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                    false, false);
    a = __builtin_bit_cast(float, (uint32_t)r[0]);
    b = __builtin_bit_cast(float, (uint32_t)r[1]);
}

template <typename T, int DP, int KW>
struct TileAttn {
    static constexpr bool HALF = sizeof(T) == 2;
    static constexpr int C = Vec<T>::chunk, BK = HALF || KW == 2 ? 64 : 32;   // keys a tile
    static constexpr int TK = BK / 32 / KW, RG = 4 / KW;   // a wave's 32-key products of a tile; 32-row groups
    static constexpr int NC = DP / C, CPR = NC <= 4 ? 4 : NC <= 8 ? 8 : NC <= 16 ? 16 : NC <= 32 ? 32 : 64;   // of a row
    static constexpr int STAGE = 2 * BK * CPR, CP = BK * CPR / 256;   // chunks of K and V; copies of a thread for each
    static constexpr int KS = NC / 2, DT = DP / 32;
    // Stages (copies run S - 1 tiles ahead) and workgroups on a CU: what
    // registers and 160 KB of LDS allow.
    static constexpr int KB = STAGE / 64, S = KB <= 8 ? 4 : KB <= 16 ? 3 : 2;
    static constexpr int OCC = KB <= 8 ? 4 : KB <= 16 ? 3 : KB <= 32 ? 2 : 1;

    // Chunk c of row r is stored at c ^ swizzle(r): the 64 banks are filled
    // once by 16 rows at one chunk, by 4 rows from a multiple of 4 at 4 chunks
    // (the transposing loads, bf16), and by rows r and r + 4 at 8 chunks (fp32).
    static __device__ __forceinline__ constexpr int swizzle(int r) {
        if (CPR == 4) return (r >> 2) & 3;
        if (CPR == 8) return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
        if (HALF) return (r & 3) << 2 | ((r >> 2) & 3);
        return ((r >> 2) & 1) << 3 | ((r >> 3) & 1) << 2 | (r & 3);
    }
    // Where this lane reads a stage, in bytes from its start: K's rows lane % 32
    // in product step 0 (step i: ^ 32 i; 32 rows on: + 512 CPR), V^T as vt()
    // takes it.  swizzle() is a permutation of bits of the row, so a step that
    // sets other bits of the row or the chunk is an exclusive or.
    static __device__ __forceinline__ uint32_t k_at(int lane) {
        const int n = lane & 31;
        return (n * CPR + ((lane >> 5) ^ swizzle(n))) * 16;
    }
    static __device__ __forceinline__ uint32_t v_at(int lane) {
        if (HALF) {
            const int j = lane & 15, r = 4 * (lane >> 5) + (j >> 2), c = 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
            return (BK * CPR + r * CPR + (c ^ swizzle(r))) * 16 + (j & 1) * 8;
        }
        const int r = 4 * (lane >> 5), c = (lane & 31) >> 2;
        return (BK * CPR + r * CPR + (c ^ swizzle(r))) * 16 + (lane & 3) * 4;
    }
    // bf16: 32 rows of V^T, d0 on, against 16 keys from `key` on, in the
    // scores' order: keys 8 i + 4 (lane / 32) + 0..3 for i = 0, then 1.
    static __device__ __forceinline__ bf16x8 vt(uint32_t at, int key, int d0) {
        s16x4 h[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                lds_ptr<lds_s16x4>((at ^ ((swizzle(8 * i) ^ (d0 / C)) * 16)) + (key + 8 * i) * CPR * 16));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // fp32: 32 rows of V^T, d0 on, at the keys of score register i.
    static __device__ __forceinline__ float vt1(uint32_t at, int i, int d0) {
        const int r = 8 * (i >> 2) + (i & 3);
        return *lds_ptr<const lds_f32>((at ^ ((swizzle(r) ^ (d0 / C)) * 16)) + r * CPR * 16);
    }
};

}  // namespace conv2d
