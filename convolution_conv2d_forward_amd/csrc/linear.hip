// y = act(x w^T + bias) + residual: dispatch, and the kernel for any size,
// stride and alignment.
#include "linear_common.h"

namespace conv2d {

namespace {

// 16 bytes of a row from element k on, zero from a.k on.  vec: the chunk is
// aligned, and wholly inside or outside.
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* row, int k, int kend, bool vec) {
    constexpr int C = Vec<T>::chunk;
    u32x4 r{0, 0, 0, 0};
    if (vec) {
        if (k < kend) r = *(const u32x4*)(row + k);
        return r;
    }
    T e[C];
#pragma unroll
    for (int i = 0; i < C; ++i) e[i] = k + i < kend ? row[k + i] : (T)0.0f;
    __builtin_memcpy(&r, e, 16);
    return r;
}

// 64 rows of x by 64 rows of w per workgroup of four waves, each wave a 32x32
// quarter; 128 bytes of every row a step through one LDS buffer, the next
// step's chunks in registers meanwhile.  16-byte chunks are stored at
// chunk ^ (row & 7), so the 16 rows that a wave reads at once lie in
// different banks.
template <typename T>
__global__ __launch_bounds__(256) void linear_any(LinearArgs a, uint32_t tiles_n) {
    constexpr int C = Vec<T>::chunk, BK = 8 * C;
    __shared__ __align__(16) u32x4 lds[2][64 * 8];
    const uint32_t b = xcd_remap(blockIdx.x, gridDim.x);
    const int m0 = (int)(b / tiles_n) * 64, n0 = (int)(b % tiles_n) * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    // Thread's chunks: rows tid/8 and tid/8 + 32 of each tile, chunk tid % 8.
    const int lr = tid >> 3, lc = tid & 7;
    const T* xr[2];
    const T* wr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int m = m0 + lr + 32 * i, n = n0 + lr + 32 * i;
        m = m < a.m ? m : a.m - 1;   // rows past the end repeat the last one; their results are not stored
        n = n < a.n ? n : a.n - 1;
        xr[i] = (const T*)a.x + (int64_t)m * a.xs;
        wr[i] = (const T*)a.w + (int64_t)n * a.k;
    }
    u32x4 rx[2], rw[2];
    const auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rx[i] = load_chunk(xr[i], k0 + lc * C, a.k, a.vec);
            rw[i] = load_chunk(wr[i], k0 + lc * C, a.k, a.vec);
        }
    };
    f32x4 acc[2][2] = {};
    fetch(0);
    for (int k0 = 0; k0 < a.k; k0 += BK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = lr + 32 * i, at = row * 8 + (lc ^ (row & 7));
            lds[0][at] = rx[i];
            lds[1][at] = rw[i];
        }
        __syncthreads();
        if (k0 + BK < a.k) fetch(k0 + BK);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int c = ks * 4 + (lane >> 4), r = lane & 15;
            u32x4 fw[2], fx[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int rw_ = wn + 16 * i + r, rx_ = wm + 16 * i + r;
                fw[i] = lds[1][rw_ * 8 + (c ^ (rw_ & 7))];
                fx[i] = lds[0][rx_ * 8 + (c ^ (rx_ & 7))];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma_step<T>(fw[i], fx[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            linear_store<T>(a, m0 + wm + 16 * j + (lane & 15), n0 + wn + 16 * i + 4 * (lane >> 4), acc[i][j]);
}

template <typename T>
hipError_t run_any(const LinearArgs& a, hipStream_t s) {
    const int64_t tm = ((int64_t)a.m + 63) / 64, tn = ((int64_t)a.n + 63) / 64;
    if (tm * tn > 0x7fffffff) return hipErrorInvalidValue;
    linear_any<T><<<dim3((uint32_t)(tm * tn)), dim3(256), 0, s>>>(a, (uint32_t)tn);
    return hipGetLastError();
}

}  // namespace

const char* linear_kernel_name(int32_t dtype, const LinearArgs& a) {
    return dtype == CONV_DTYPE_F32 ? "linear_any_f32" : "linear_any_bf16";
}

hipError_t launch_linear(int32_t dtype, const LinearArgs& a, hipStream_t s) {
    return dtype == CONV_DTYPE_F32 ? run_any<float>(a, s) : run_any<bf16>(a, s);
}

}  // namespace conv2d
