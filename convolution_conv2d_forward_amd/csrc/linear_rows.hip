// y = act(x w^T + bias) + residual for few rows of x, bound by the bytes of w, and
// for few tiles of a long k, bound by the latency of its units.
#include "linear_common.h"

namespace conv2d {

namespace {

// The activation, its kind at run time: for the few outputs of a thread here.
template <typename T, int N>
__device__ __forceinline__ void linear_act_any(const LinearArgs& a, float* v) {
    switch (a.act) {
    case CONV_ACT_NONE: break;
    case LINEAR_ACT_SILU: linear_act<T, kActSilu, N>(a, v); break;
    case LINEAR_ACT_GELU: linear_act<T, kActGelu, N>(a, v); break;
    case LINEAR_ACT_GELU_TANH: linear_act<T, kActGeluTanh, N>(a, v); break;
    default: linear_act<T, kActPiecewise, N>(a, v);
    }
}

// The waves' sums meet in LDS, and 16 NT x 16 MT outputs from row m0 and
// column n0 on are formed and stored.
template <typename T, int MT, int NT, int NW>
__device__ __forceinline__ void rows_store(const LinearArgs& a, const f32x4 (&acc)[NT][MT], f32x4* red, int m0, int n0,
                                           int wave, int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) red[(wave * NT * MT + i * MT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int t = wave; t < NT * MT; t += NW) {
        const int m = m0 + 16 * (t % MT) + r, n = n0 + 16 * (t / MT) + 4 * g;
        if (m >= a.m || n >= a.n) continue;
        T* y = (T*)a.y + m * a.ys + n;
        const T* res = a.residual ? (const T*)a.residual + m * a.rs + n : nullptr;
        f32x4 v = red[t * 64 + lane];
#pragma unroll
        for (int i = 1; i < NW; ++i) v += red[(i * NT * MT + t) * 64 + lane];
        if (a.vec_out) {
            if (a.bias) v += *(const f32x4*)(a.bias + n);
            linear_act_any<T, 4>(a, (float*)&v);
            if (res) v += to_f32(*(const typename Vec<T>::v4*)res);
            *(typename Vec<T>::v4*)y = from_f32<T>(v);
            continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (a.bias && n + i < a.n) v[i] += a.bias[n + i];
        linear_act_any<T, 4>(a, (float*)&v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.n) y[i] = from_f32<T>(v[i] + (res ? to_f32(res[i]) : 0.0f));
    }
}

// 16 NT rows of w against 16 MT rows of x per workgroup.  Its NW
// waves deal the 128-byte units of the rows among themselves; every lane reads
// its chunks of w and x straight into the operands of the matrix cores, U
// units in flight at a time.
template <typename T, int MT, int NT, int NW, int U>
__global__ __launch_bounds__(64 * NW) void linear_rows(LinearArgs a, int blocks_m) {
    constexpr int C = Vec<T>::chunk, UNIT = 8 * C;
    __shared__ __align__(16) f32x4 red[NW * NT * MT * 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.x % blocks_m * 16 * MT, n0 = blockIdx.x / blocks_m * 16 * NT, r = lane & 15, g = lane >> 4;
    // Rows past the end repeat the last one; their results are not stored.
    const T *w[NT], *x[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) w[i] = (const T*)a.w + (int64_t)min(n0 + 16 * i + r, a.n - 1) * a.k + g * C;
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = (const T*)a.x + (int64_t)min(m0 + 16 * j + r, a.m - 1) * a.xs + g * C;
    f32x4 acc[NT][MT] = {};
    for (int k0 = wave * UNIT; k0 < a.k; k0 += NW * U * UNIT) {
        u32x4 fw[U][2][NT], fx[U][2][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = k0 + u * NW * UNIT + h * 4 * C, left = a.k - k - g * C;   // elements from this lane's first
                // Of the wave's chunks of this step, one starts or ends its row, or lies past it.
                const bool end = k == 0 || k + 4 * C >= a.k;
#pragma unroll
                for (int i = 0; i < NT; ++i) fw[u][h][i] = load_words(w[i] + k, end, left);
#pragma unroll
                for (int j = 0; j < MT; ++j) fx[u][h][j] = load_words(x[j] + k, end, left);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < MT; ++j) acc[i][j] = mfma_step<T>(fw[u][h][i], fx[u][h][j], acc[i][j]);
    }
    rows_store<T, MT, NT, NW>(a, acc, red, m0, n0, wave, lane);
}

// The same through LDS: every wave has a ring of S stages of its own, each one
// unit of all rows, and copies S - 1 units ahead of its products, in pieces of
// W bytes; the copies move whole 128-byte lines, where the operands' layout
// makes register loads take 64 bytes of 16 rows at a time.
template <typename T, int MT, int NT, int NW, int S, int W>
__global__ __launch_bounds__(64 * NW) void linear_rows_ring(LinearArgs a, int blocks_m) {
    constexpr int C = Vec<T>::chunk, UNIT = 8 * C, ROWS = 16 * (NT + MT), PPC = 16 / W, LD = ROWS / 8 * PPC;
    constexpr int RING = NW * S * ROWS * 8, RED = NW * NT * MT * 64;
    __shared__ __align__(16) u32x4 lds[RING > RED ? RING : RED];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = blockIdx.x % blocks_m * 16 * MT, n0 = blockIdx.x / blocks_m * 16 * NT, r = lane & 15, g = lane >> 4;
    u32x4* ring = lds + wave * S * ROWS * 8;
    // Copy i of this lane: piece lane % PPC of the stage's chunk at
    // i * 64 / PPC + lane / PPC; rows of w come first, then x's.  Chunk c of
    // row i is stored at c ^ (i / 2 % 8).
    const auto row_of = [&](int i) { return (i * (64 / PPC) + lane / PPC) / 8; };
    const auto elem_of = [&](int i) {
        return ((lane / PPC % 8) ^ ((row_of(i) >> 1) & 7)) * C + lane % PPC * (W / (int)sizeof(T));
    };
    uint32_t off[LD];
#pragma unroll
    for (int i = 0; i < LD; ++i) {
        const int row = row_of(i);
        const int64_t el = i < 2 * NT * PPC ? (int64_t)(min(n0 + row, a.n - 1) - n0) * a.k
                                            : min(row - 16 * NT, a.m - 1 - m0) * a.xs;
        off[i] = (uint32_t)((el + elem_of(i)) * (int)sizeof(T));
    }
    const T *wb = (const T*)a.w + (int64_t)n0 * a.k, *xb = (const T*)a.x + (int64_t)m0 * a.xs;
    // A piece past k is copied from the unit's start, and zeros are written over it.
    const auto copy = [&](int k0, int stage) {
        if (k0 >= a.k) return;
        const T *wk = uniform(wb + k0), *xk = uniform(xb + k0);
        const u32x4* dst = ring + stage * ROWS * 8;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const T* base = i < 2 * NT * PPC ? wk : xk;
            const uint32_t at = off[i] - (k0 + elem_of(i) < a.k ? 0 : elem_of(i) * (int)sizeof(T));
            if constexpr (W == 16)
                copy16_to_lds(base, at, dst + i * 64);
            else
                copy4_to_lds(base, at, dst + i * 16);
        }
    };
    f32x4 acc[NT][MT] = {};
#pragma unroll
    for (int j = 0; j < S - 1; ++j) copy((wave + j * NW) * UNIT, j);
    int stage = 0;
    for (int k0 = wave * UNIT; k0 < a.k; k0 += NW * UNIT) {
        copy(k0 + (S - 1) * NW * UNIT, stage == 0 ? S - 1 : stage - 1);
        if (k0 + (S - 1) * NW * UNIT < a.k)
            wait_vmem<(S - 1) * LD>();
        else
            wait_vmem<0>();
        u32x4* st = ring + stage * ROWS * 8;
        if (k0 + UNIT > a.k) {
#pragma unroll
            for (int i = 0; i < LD; ++i) {
                if (k0 + elem_of(i) < a.k) continue;
                if constexpr (W == 16)
                    st[i * 64 + lane] = u32x4{0, 0, 0, 0};
                else
                    ((uint32_t*)(st + i * 16))[lane] = 0;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        u32x4 fw[2][NT], fx[2][MT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = (4 * h + g) ^ ((r >> 1) & 7);
#pragma unroll
            for (int i = 0; i < NT; ++i) fw[h][i] = st[(16 * i + r) * 8 + c];
#pragma unroll
            for (int j = 0; j < MT; ++j) fx[h][j] = st[(16 * (NT + j) + r) * 8 + c];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[i][j] = mfma_step<T>(fw[h][i], fx[h][j], acc[i][j]);
        // The stage's reads have returned before it is copied to again.
        __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    __syncthreads();
    rows_store<T, MT, NT, NW>(a, acc, (f32x4*)lds, m0, n0, wave, lane);
}

template <int MT, int NT>
dim3 grid_of(const LinearArgs& a, int& blocks_m) {
    blocks_m = (int)(((int64_t)a.m + 16 * MT - 1) / (16 * MT));
    return dim3((uint32_t)((int64_t)blocks_m * ((a.n + 16 * NT - 1) / (16 * NT))));
}

template <typename T, int MT, int NT, int NW, int S, int W>
hipError_t run_ring(const LinearArgs& a, hipStream_t s) {
    int blocks_m;
    const dim3 grid = grid_of<MT, NT>(a, blocks_m);
    linear_rows_ring<T, MT, NT, NW, S, W><<<grid, dim3(64 * NW), 0, s>>>(a, blocks_m);
    return hipGetLastError();
}

template <typename T, int W>
hipError_t run_ring(const LinearArgs& a, hipStream_t s) {
    // Stages: the fastest of 2 to 8; 16 waves and 32 or 64 rows of w a
    // workgroup were slower or equal at 1 to 128 rows.
    const RowsShape sh = rows_shape(sizeof(T) == 4, a);
    if (sh.mt == 1) return run_ring<T, 1, 1, 8, 2, W>(a, s);
    if (sh.mt == 4) return run_ring<T, 4, 1, 4, 2, W>(a, s);
    if constexpr (sizeof(T) == 4)
        if (sh.waves == 8) return run_ring<T, 2, 1, 8, 2, W>(a, s);
    return run_ring<T, 2, 1, 4, W == 16 ? 3 : 2, W>(a, s);
}

template <typename T>
hipError_t run(const LinearArgs& a, hipStream_t s) {
    if (a.vec == 16) return run_ring<T, 16>(a, s);
    if (a.vec == 4) return run_ring<T, 4>(a, s);
    int blocks_m;
    if (rows_shape(sizeof(T) == 4, a).mt == 1) {
        const dim3 grid = grid_of<1, 1>(a, blocks_m);
        linear_rows<T, 1, 1, 8, 4><<<grid, dim3(512), 0, s>>>(a, blocks_m);
    } else {
        const dim3 grid = grid_of<2, 1>(a, blocks_m);
        linear_rows<T, 2, 1, 8, 2><<<grid, dim3(512), 0, s>>>(a, blocks_m);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_rows(int32_t dtype, const LinearArgs& a, hipStream_t s) {
    return dtype == CONV_DTYPE_F32 ? run<float>(a, s) : run<bf16>(a, s);
}

}  // namespace conv2d
