// y = act(x w^T + bias) + residual as LDS-tiled matrix products, for any size,
// stride and alignment.  Compiled once for each type (linear_f32.hip,
// linear_bf16.hip).
#pragma once

#include "linear_common.h"

namespace conv2d {

namespace {

// Shape of a tile: BM rows of x by BN rows of w, WM * WN waves, CPR chunks of
// 16 bytes of every row a step, S stages of LDS.
template <typename T, int BM_, int BN_, int WM_, int WN_, int CPR_, int S_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, CPR = CPR_, S = S_;
    static constexpr int C = Vec<T>::chunk, BK = CPR * C, NT = 64 * WM * WN;
    static constexpr int RM = BM / WM, RN = BN / WN, MI = RM / 32, NI = RN / 32;   // of a wave; in 32x32 products
    static constexpr int LD = (BM + BN) * CPR / NT, LDX = BM * CPR / NT;   // chunks a thread moves a step; those of x
    static constexpr int STAGE = (BM + BN) * CPR;                          // chunks
    static constexpr int LDS = S * STAGE + WM * WN * 256;                  // chunks: the stages, 4 KB of outputs a wave
    static_assert(BM * CPR % NT == 0 && BN * CPR % NT == 0 && LDS * 16 <= 160 * 1024, "tile shape");
    // Chunk c of row r is stored at c ^ swizzle(r): 16 rows that a wave reads
    // at once then fill the 64 banks once.
    static __device__ __forceinline__ int swizzle(int r) { return CPR == 8 ? (r >> 1) & 7 : (r >> 2) & 3; }
};

// First rows of x and w of tile t.  Tiles go in groups of 8 tile rows, so that
// the workgroups that run at once on an XCD share their rows of x and w in
// its L2.
template <class C>
__device__ __forceinline__ void tile_origin(int t, int tiles_m, int tiles_n, int& m0, int& n0) {
    const int b = (int)xcd_remap(t, tiles_m * tiles_n), per = 8 * tiles_n, grp = b / per, rem = b - grp * per;
    const int gm = min(8, tiles_m - grp * 8);
    m0 = (grp * 8 + rem % gm) * C::BM;
    n0 = rem / gm * C::BN;
}

// Operands of product step s (of CPR / 2) from a stage.
template <class C>
struct Frags {
    u32x4 x[C::MI], w[C::NI];
    __device__ __forceinline__ void load(const u32x4* stage, int wm, int wn, int s, int lane) {
        const int r = lane & 31, c = (2 * s + (lane >> 5)) ^ C::swizzle(r);
#pragma unroll
        for (int i = 0; i < C::NI; ++i) w[i] = stage[(C::BM + wn + 32 * i + r) * C::CPR + c];
#pragma unroll
        for (int i = 0; i < C::MI; ++i) x[i] = stage[(wm + 32 * i + r) * C::CPR + c];
    }
};

// Up to 8 elements from p on, of which `left` are there (at any alignment).
template <typename V, typename E>
__device__ __forceinline__ void load_some(V* v, const E* p, int left) {
    if (left >= 8) {
        __builtin_memcpy(v, p, 8 * sizeof(E));
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < left) (*v)[e] = p[e];
}

// Outputs pass through 4 KB of LDS of the wave's own, 32x32 at a time, so that
// global memory is read and written along rows; the residuals of a column of
// blocks are in flight before the first is used.
template <typename T, class C, int ACT>
__device__ __forceinline__ void tile_store(const LinearArgs& a, const f32x16 (&acc)[C::NI][C::MI], u32x4* os, int m,
                                           int n, int lane) {
    const auto at = [](int r, int c) { return r * 8 + (c ^ ((r >> 1) & 7)); };   // chunk c of the block's row r
    const auto put = [&](const f32x16& v) {
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4 w{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            os[at(lane & 31, 2 * q + (lane >> 5))] = __builtin_bit_cast(u32x4, w);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    // A lane takes 8 columns of rows lane / 4 and lane / 4 + 16, at any
    // alignment; chunks that the row's end cuts go element by element.
    typedef T V __attribute__((ext_vector_type(8)));
    const int r0 = lane >> 2, c0 = lane & 3;
#pragma unroll
    for (int i = 0; i < C::NI; ++i) {
        const int nn = n + 32 * i + 8 * c0, left = a.n - nn;
        V res[C::MI][2] = {};
        if (a.residual)
#pragma unroll
            for (int j = 0; j < C::MI; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int mm = m + 32 * j + r0 + 16 * h;
                    if (mm < a.m) load_some(&res[j][h], (const T*)a.residual + mm * a.rs + nn, left);
                }
        f32x8 b{};
        if (a.bias) load_some(&b, a.bias + nn, left);
#pragma unroll
        for (int j = 0; j < C::MI; ++j) {
            put(acc[i][j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
                __builtin_memcpy(v, &os[at(r0 + 16 * h, 2 * c0)], 16);
                __builtin_memcpy(v + 4, &os[at(r0 + 16 * h, 2 * c0 + 1)], 16);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += b[e];
                linear_act<T, ACT, 8>(a, v);
                const f32x8 r = __builtin_convertvector(res[j][h], f32x8);
                f32x8 o;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = v[e] + r[e];
                const int mm = m + 32 * j + r0 + 16 * h;
                V w = __builtin_convertvector(o, V);
                // Formed by all lanes: a residual left unused in a branch
                // not taken would make the product loop wait for memory.
                asm volatile("" : "+v"(w));
                T* y = (T*)a.y + mm * a.ys + nn;
                if (mm < a.m && left >= 8) {
                    __builtin_memcpy(y, &w, sizeof(w));
                } else if (mm < a.m) {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (e < left) y[e] = w[e];
                }
            }
        }
    }
}

// Chunks are copied straight to a ring of S LDS stages, S - 1 steps ahead of
// their use (a copy takes some 1600 cycles to land, more under load), in
// pieces of W bytes: rows start at W-byte boundaries, and k fills whole
// pieces.  A workgroup takes one tile after the other, and the copies of the
// next tile's first steps run through the outputs of the last one.  The
// operands of product step s + 1 are read while step s multiplies, over the
// border of two stages too: the barrier that frees a stage stands before the
// stage's last products, whose operands are in registers by then, so the
// matrix cores have work while the waves meet.
template <typename T, class C, int ACT, int W>
__global__ __launch_bounds__(C::NT, 2) void linear_tile(LinearArgs a, int tiles_m, int tiles_n) {
    constexpr int S = C::S, BK = C::BK, NT = C::NT, CPR = C::CPR, STEPS = CPR / 2;
    constexpr int PPC = 16 / W, LD = C::LD * PPC, LDX = C::LDX * PPC;   // pieces a chunk; pieces a thread copies a step
    constexpr int AHEAD = LD * (S - 2);                                 // copies that may be in flight past the next step's
    __shared__ __align__(16) u32x4 lds[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN * C::RM, wn = wave % C::WN * C::RN;
    const int tiles = tiles_m * tiles_n;
    // Copy i of this thread: piece tid % PPC of the stage's chunk at
    // i * NT / PPC + tid / PPC, which holds a chunk of this row of the tile.
    const auto row_of = [&](int i) { return (i * (NT / PPC) + tid / PPC) / CPR; };
    const auto elem_of = [&](int i) {
        return ((tid / PPC % CPR) ^ C::swizzle(row_of(i))) * C::C + tid % PPC * (W / (int)sizeof(T));
    };
    // Where the copies are: tile, first element of the step, rows.
    int copy_tile = blockIdx.x, copy_k = 0;
    const T *xb, *wb;
    uint32_t off[LD];
    const auto aim = [&] {
        int m0, n0;
        tile_origin<C>(copy_tile, tiles_m, tiles_n, m0, n0);
        xb = (const T*)a.x + (int64_t)m0 * a.xs;
        wb = (const T*)a.w + (int64_t)n0 * a.k;
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            // Rows past the end repeat the last one; their results are not stored.
            const int r = row_of(i);
            const int64_t el = i < LDX ? min(r, a.m - 1 - m0) * a.xs : (int64_t)min(r - C::BM, a.n - 1 - n0) * a.k;
            off[i] = (uint32_t)((el + elem_of(i)) * (int)sizeof(T));
        }
    };
    // The next step's copies.  In the last step of a row a thread whose piece
    // lies past k copies the step's first piece instead, and writes zeros over
    // it once it has landed.
    const auto copy = [&](int stage) {
        if (copy_tile >= tiles) return;
        u32x4* dst = lds + stage * C::STAGE;
        const T *xk = uniform(xb + copy_k), *wk = uniform(wb + copy_k);
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const T* base = i < LDX ? xk : wk;
            const uint32_t at = off[i] - (copy_k + elem_of(i) < a.k ? 0 : elem_of(i) * (int)sizeof(T));
            if constexpr (W == 16)
                copy16_to_lds(base, at, dst + i * NT + wave * 64);
            else
                copy4_to_lds(base, at, dst + i * (NT / PPC) + wave * 16);
        }
        copy_k += BK;
        if (copy_k >= a.k) {
            copy_k = 0;
            copy_tile += gridDim.x;
            if (copy_tile < tiles) aim();
        }
    };
    // Before a stage's operands are read: this thread's copies of the step
    // from k0 have landed (later ones may be in flight), then all threads'.
    const auto meet = [&](int k0, int stage) {
        if (AHEAD && copy_tile < tiles)
            wait_vmem<AHEAD>();
        else
            wait_vmem<0>();
        if (k0 + BK > a.k) {
#pragma unroll
            for (int i = 0; i < LD; ++i) {
                if (k0 + elem_of(i) < a.k) continue;
                if constexpr (W == 16)
                    lds[stage * C::STAGE + i * NT + tid] = u32x4{0, 0, 0, 0};
                else
                    ((uint32_t*)(lds + stage * C::STAGE + i * (NT / PPC)))[tid] = 0;
            }
        }
        __syncthreads();
    };
    aim();
#pragma unroll
    for (int j = 0; j < S - 1; ++j) copy(j);
    meet(0, 0);
    copy(S - 1);
    int stage = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        // Read again at a tile's start, so that these registers are free while
        // the outputs are formed.
        Frags<C> f[2];
        f[0].load(lds + stage * C::STAGE, wm, wn, 0, lane);
        f32x16 acc[C::NI][C::MI] = {};
        for (int k0 = 0; k0 < a.k; k0 += BK) {
            const int next = stage == S - 1 ? 0 : stage + 1;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s + 1 < STEPS) {
                    f[(s + 1) & 1].load(lds + stage * C::STAGE, wm, wn, s + 1, lane);
                } else {
                    // After a tile's last step this reads what is not used.
                    meet(k0 + BK < a.k ? k0 + BK : 0, next);
                    f[0].load(lds + next * C::STAGE, wm, wn, 0, lane);
                    copy(stage);
                }
                __builtin_amdgcn_sched_barrier(0);   // the reads of the next operands stay ahead of these products
#pragma unroll
                for (int i = 0; i < C::NI; ++i)
#pragma unroll
                    for (int j = 0; j < C::MI; ++j)
                        acc[i][j] = mfma32_step<T>(f[s & 1].w[i], f[s & 1].x[j], acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
            stage = next;
        }
        int m0, n0;
        tile_origin<C>(t, tiles_m, tiles_n, m0, n0);
        tile_store<T, C, ACT>(a, acc, lds + S * C::STAGE + wave * 256, m0 + wm, n0 + wn, lane);
    }
}

// Any alignment of the element and any k: the chunks pass through registers,
// one step ahead.
template <typename T, class C, int ACT>
__global__ __launch_bounds__(C::NT, 2) void linear_staged(LinearArgs a, int tiles_m, int tiles_n) {
    constexpr int LD = C::LD, BK = C::BK, NT = C::NT, CPR = C::CPR;
    __shared__ __align__(16) u32x4 lds[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN * C::RM, wn = wave % C::WN * C::RN;
    int m0, n0;
    tile_origin<C>(blockIdx.x, tiles_m, tiles_n, m0, n0);
    const int lr = tid / CPR, lc = (tid % CPR) ^ C::swizzle(lr);
    const T* row[LD];
#pragma unroll
    for (int i = 0; i < LD; ++i) {
        const int r = lr + (i < C::LDX ? i : i - C::LDX) * (NT / CPR);
        row[i] = i < C::LDX ? (const T*)a.x + min(m0 + r, a.m - 1) * a.xs
                            : (const T*)a.w + (int64_t)min(n0 + r, a.n - 1) * a.k;
    }
    u32x4 reg[LD];
#pragma unroll
    for (int i = 0; i < LD; ++i) reg[i] = load_chunk<T>(row[i] + lc * C::C, a.k - lc * C::C);
    f32x16 acc[C::NI][C::MI] = {};
    int stage = 0;
    for (int k0 = 0; k0 < a.k; k0 += BK) {
        u32x4* st = lds + stage * C::STAGE;
#pragma unroll
        for (int i = 0; i < LD; ++i) st[i * NT + tid] = reg[i];
        __syncthreads();
        if (k0 + BK < a.k)
#pragma unroll
            for (int i = 0; i < LD; ++i) reg[i] = load_chunk<T>(row[i] + k0 + BK + lc * C::C, a.k - (k0 + BK + lc * C::C));
#pragma unroll
        for (int s = 0; s < CPR / 2; ++s) {
            Frags<C> f;
            f.load(st, wm, wn, s, lane);
#pragma unroll
            for (int i = 0; i < C::NI; ++i)
#pragma unroll
                for (int j = 0; j < C::MI; ++j) acc[i][j] = mfma32_step<T>(f.w[i], f.x[j], acc[i][j]);
        }
        stage ^= 1;
    }
    tile_store<T, C, ACT>(a, acc, lds + 2 * C::STAGE + wave * 256, m0 + wm, n0 + wn, lane);
}

// W: bytes of a copy, 0: through registers.
template <typename T, int W, int BM, int BN, int WM, int WN, int CPR, int S>
hipError_t run(const LinearArgs& a, hipStream_t s) {
    typedef Tile<T, BM, BN, WM, WN, CPR, S> C;
    const int64_t tm = ((int64_t)a.m + BM - 1) / BM, tn = ((int64_t)a.n + BN - 1) / BN;
    return with_act(a, [&](auto act) {
        if constexpr (W > 0) {
            const int64_t fit = (int64_t)device_cu_count() * (160 * 1024 / (C::LDS * 16)) & ~7;   // workgroups at once
            linear_tile<T, C, act(), W>
                <<<dim3((uint32_t)(tm * tn < fit ? tm * tn : fit)), dim3(C::NT), 0, s>>>(a, (int)tm, (int)tn);
        } else {
            linear_staged<T, C, act()><<<dim3((uint32_t)(tm * tn)), dim3(C::NT), 0, s>>>(a, (int)tm, (int)tn);
        }
        return hipGetLastError();
    });
}

template <typename T, int W>
hipError_t run(const LinearArgs& a, linear_tile_t tile, hipStream_t s) {
    if constexpr (sizeof(T) == 2 && W == 16)
        if (tile == LINEAR_TILE_256) return run<T, W, 256, 256, 2, 4, 8, 2>(a, s);
    if (tile == LINEAR_TILE_64) return run<T, W, 64, 64, 2, 2, 8, 4>(a, s);
    // Pieces of 4 bytes always take the deep pipeline: four waves would have 32
    // copies a step each to address (1571x770x2309 fp32: 502 us against 67).
    if constexpr (W == 16)
        if (tile == LINEAR_TILE_128) return run<T, W, 128, 128, 2, 2, 8, 2>(a, s);
    return run<T, W, 128, 128, 2, 4, 8, 4>(a, s);
}

template <typename T>
hipError_t run(const LinearArgs& a, linear_tile_t tile, hipStream_t s) {
    if (a.vec == 16) return run<T, 16>(a, tile, s);
    if (a.vec == 4) return run<T, 4>(a, tile, s);
    return tile == LINEAR_TILE_64 ? run<T, 0, 64, 64, 2, 2, 8, 2>(a, s) : run<T, 0, 128, 128, 2, 2, 8, 2>(a, s);
}

}  // namespace

template <>
hipError_t launch_linear_tile<LINEAR_T>(const LinearArgs& a, linear_tile_t tile, hipStream_t s) {
    return run<LINEAR_T>(a, tile, s);
}

}  // namespace conv2d
