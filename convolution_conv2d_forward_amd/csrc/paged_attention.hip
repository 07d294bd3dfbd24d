// Dispatch of paged_attention_forward, and the join of divided results.
#include <numeric>

#include "linear_common.h"
#include "paged_common.h"

namespace conv2d {

namespace {

// Where row r of a (tile, head)'s outputs go; false where there is nothing to
// join: one result was written whole, or there is no such row.
template <typename T>
__device__ __forceinline__ bool out_row(const PagedArgs& a, const PagedRecord& rec, int h, int r, T*& out) {
    if (rec.n == 0 || r >= rec.rows) return false;
    const int token = token_of(a, r + rec.skip), hq = h * a.group + r + rec.skip - token * a.group;
    out = (T*)a.out + (int64_t)(rec.first + token) * a.o_s + (int64_t)hq * a.d;
    return true;
}

// The row of the workspace that holds the i-th result's row r of a head.
template <int R>
__device__ __forceinline__ int64_t result_row(const PagedArgs& a, const PagedRecord& rec, int sub, int i, int r) {
    return ((int64_t)(i == 0 ? rec.slot0 : rec.slot1 + rec.step * i) * a.group_heads + sub) * R + r;
}

// Few results: as many threads as a row is wide add up its outputs, 256 / W rows
// a workgroup.
template <typename T, int R, int DP>
__device__ __forceinline__ void join_few(const PagedArgs& a, uint32_t b) {
    constexpr int W = DP / 4, ROWS = 256 / W;
    const int e = ((int)threadIdx.x % W) * 4;
    const PagedWs w = paged_ws<R>(a);
    const int unit = (int)(b / (R / ROWS)), r = (int)(b % (R / ROWS)) * ROWS + (int)threadIdx.x / W;
    const int sub = unit % a.group_heads;
    const PagedRecord rec = w.record[unit / a.group_heads];
    T* out;
    if (!out_row<T>(a, rec, unit % a.heads_kv, r, out) || e >= a.d) return;
    float top = -INFINITY, l = 0.0f;
    f32x4 sum{0, 0, 0, 0};
    for (int s0 = 0; s0 < rec.n; s0 += 4) {
        f32x2 st[4];
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = result_row<R>(a, rec, sub, min(s0 + i, rec.n - 1), r);
            st[i] = w.stat[row];
            v[i] = *(const f32x4*)(w.out + row * a.d + e);
            if (s0 + i >= rec.n) st[i] = f32x2{-INFINITY, 0.0f};
        }
        float m = top;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, st[i][0]);
        const float base = m == -INFINITY ? 0.0f : m, fade = __builtin_amdgcn_exp2f(top - base);
        top = m;
        l *= fade;
        sum *= fade;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = __builtin_amdgcn_exp2f(st[i][0] - base);
            l += f * st[i][1];
            if (s0 + i < rec.n) sum += v[i] * f;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *(typename Vec<T>::v4*)(out + e) = from_f32<T>(sum * inv);
}
template <typename T, int R, int DP>
__global__ __launch_bounds__(256) void paged_join_few(PagedArgs a) {
    join_few<T, R, DP>(a, blockIdx.x);
}
// Where only long tiles were divided most records are empty: fewer workgroups
// look at all of them.
template <typename T, int R, int DP>
__global__ __launch_bounds__(256) void paged_join_long(PagedArgs a, uint32_t all) {
    for (uint32_t b = blockIdx.x; b < all; b += gridDim.x) join_few<T, R, DP>(a, b);
}

// Many: a workgroup a row.  The results' maxima and sums give each one's
// factor; then groups of threads, each as wide as the row, add up the outputs
// of every GROUPS-th result, four loads in flight, the first ones while the
// factors are formed, and meet in LDS.
constexpr int kMostParts = 1024;
template <typename T, int R, int DP>
__global__ __launch_bounds__(256) void paged_join_many(PagedArgs a) {
    constexpr int W = DP / 4, GROUPS = 256 / W, UN = 4;
    __shared__ float top_w[4], sum_w[4], factor[kMostParts];
    __shared__ __align__(16) f32x4 part[GROUPS][W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int unit = (int)blockIdx.x / R, r = (int)blockIdx.x % R, sub = unit % a.group_heads;
    const PagedWs w = paged_ws<R>(a);
    const PagedRecord rec = w.record[unit / a.group_heads];
    T* out;
    if (!out_row<T>(a, rec, unit % a.heads_kv, r, out)) return;
    const int grp = tid / W, e = (tid % W) * 4, e_in = min(e, a.d - 4);
    f32x2 st[kMostParts / 256];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMostParts / 256; ++i) {
        st[i] = f32x2{-INFINITY, 0.0f};
        if (tid + 256 * i < rec.n) st[i] = w.stat[result_row<R>(a, rec, sub, tid + 256 * i, r)];
    }
    f32x4 v[UN];
    const auto fetch = [&](int s0) {
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int64_t row = result_row<R>(a, rec, sub, min(s0 + i * GROUPS, rec.n - 1), r);
            v[i] = *(const f32x4*)(w.out + row * a.d + e_in);
        }
    };
    fetch(grp);
#pragma unroll
    for (int i = 0; i < kMostParts / 256; ++i) top = fmaxf(top, st[i][0]);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    if (lane == 0) top_w[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(top_w[0], top_w[1]), fmaxf(top_w[2], top_w[3]));
    float l = 0.0f;
#pragma unroll
    for (int i = 0; i < kMostParts / 256; ++i) {
        const float f = __builtin_amdgcn_exp2f(st[i][0] - (top == -INFINITY ? 0.0f : top));
        factor[tid + 256 * i] = f;
        l += f * st[i][1];
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) l += __shfl_xor(l, m, 64);
    if (lane == 0) sum_w[wave] = l;
    __syncthreads();
    l = sum_w[0] + sum_w[1] + sum_w[2] + sum_w[3];
    f32x4 sum{0, 0, 0, 0};
    for (int s0 = grp; s0 < rec.n; s0 += UN * GROUPS) {
        if (s0 != grp) fetch(s0);
#pragma unroll
        for (int i = 0; i < UN; ++i)
            if (s0 + i * GROUPS < rec.n) sum += v[i] * factor[s0 + i * GROUPS];
    }
    part[grp][tid % W] = sum;
    __syncthreads();
    if (grp != 0 || e >= a.d) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) sum += part[i][tid];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *(typename Vec<T>::v4*)(out + e) = from_f32<T>(sum * inv);
}

template <typename T, int R, int DP>
hipError_t join(const PagedArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)a.tiles * a.heads_kv;
    const int64_t few = units * (R / (256 / (DP / 4)));
    // 8 results a (tile, head group) or more: many.  (A token over 131071 keys,
    // 128 results each: 61.4 us with many, 77.8 with few; 16 sequences of 80 rows, 8
    // results each at most: 39.8 with many, 33.4 with few.)
    if (R == 16 && a.long_blocks) {
        const int64_t most = (int64_t)device_cu_count() * 8;
        paged_join_long<T, 16, DP><<<dim3((uint32_t)(few < most ? few : most)), dim3(256), 0, s>>>(a, (uint32_t)few);
    } else if (a.parts >= 8 * (int64_t)a.tiles * a.head_groups) {
        paged_join_many<T, R, DP><<<dim3((uint32_t)(units * R)), dim3(256), 0, s>>>(a);
    } else {
        paged_join_few<T, R, DP><<<dim3((uint32_t)few), dim3(256), 0, s>>>(a);
    }
    return hipGetLastError();
}

template <typename T, int R>
hipError_t join(const PagedArgs& a, hipStream_t s) {
    if (a.d <= 64) return join<T, R, 64>(a, s);
    if (a.d <= 128) return join<T, R, 128>(a, s);
    return join<T, R, 256>(a, s);
}

}  // namespace

PagedPlan plan_paged_attention(int32_t dtype, bool e4m3, const PagedArgs& a) {
    PagedPlan p{};
    const bool f32 = dtype == CONV_DTYPE_F32;
    const int64_t cus = device_cu_count(), all = (int64_t)a.tokens * a.group, seqs = a.batch < a.tokens ? a.batch : a.tokens;
    // As many rows as a sequence has on average.  (16 sequences of up to 4096 keys,
    // 4 heads of 128 bf16, 20 rows each: 32.9 us in tiles of 16, 26.6 in 64; 64
    // rows: 28.7 in 64, 29.4 in 128; 80 rows: 33.5 and 31.5.)  Beyond 128 wide, two
    // stages of 64 fp32 keys do not fit in LDS.
    p.rows = all <= 16 * seqs ? 16 : all > 64 * seqs || (f32 && a.d > 128) ? 128 : 64;
    // A sequence's rows come in groups: what its last tile may lack is a multiple
    // of what the group has in common with a tile.
    p.tiles = (int32_t)((all + seqs * (p.rows - std::gcd(a.group, p.rows))) / p.rows);
    // Workgroups that run at once, and a block's keys: as the kernels have them.
    const int size = f32 ? 4 : 2, bytes = (a.d <= 64 ? 64 : a.d <= 128 ? 128 : 256) * size;
    int64_t per_cu, keys;
    if (p.rows == 16) {
        per_cu = bytes <= 256 ? 2 : 1;
        keys = bytes > 512 ? 64 : 128;
    } else {
        keys = f32 && p.rows == 128 ? 32 : 64;
        const int64_t stage = 2 * keys * bytes;
        per_cu = stage <= 16384 ? 3 : stage <= 32768 ? 2 : 1;
    }
    // Rows of 128 bytes or less beside each other: two heads at once, so that a
    // workgroup reads 256 bytes of a token (a token of 32 sequences of up to 8192
    // keys, 8 heads of 128 E4M3: 89 us by heads, 83 by pairs).
    const int64_t row = (int64_t)a.d * (e4m3 ? 1 : size);
    const bool pair = p.rows == 16 && (e4m3 ? bytes / size : bytes) <= 128 && a.heads_kv % 2 == 0 && a.k_head == row && a.v_head == row;
    p.group_heads = pair ? 2 : 1;
    if (pair) keys /= 2;
    // Fewer (tile, group)s than two rounds of workgroups are divided.  (A prompt
    // of 8192 tokens, two rounds of them: 364 us divided, 316 whole, 450 and 369 with
    // cold inputs; one of 4096, one round: 114 and 141.  A token of 128 sequences of up to 2048 keys, two
    // rounds: 149 and 143; of 192, one and a half: 122 and 135.)
    //
    // Of more tiles of 16 rows those of more than 2048 keys are, since one sequence
    // may be longer than all others together; on half of the workgroups that run at
    // once, while the others take whole tiles.  (A token of 256 sequences of up to
    // 2048 keys, 32 heads over 8 of 128 E4M3, and of 131071 keys in one of them: 222
    // us, 3273 whole, 204 with all keys on the line.  Where no sequence is long but
    // the table has room for it, 5 to 10 us are lost: 127 and 122 at up to 1900 keys;
    // with all keys on the line 465 for 276 at up to 600 of 32 heads of 64 bf16.)
    const int64_t wgs = cus * per_cu, units = (int64_t)p.tiles * (a.heads_kv / p.group_heads);
    const int64_t blocks = ((int64_t)a.max_pages * a.page_size.d + keys - 1) / keys;
    const bool many = units >= 2 * wgs;
    const int64_t whole = many && p.rows == 16 ? 2048 / keys : 1;   // blocks
    if (p.tiles <= kPagedTiles && a.batch <= kPagedTiles && blocks > whole && (!many || p.rows == 16) && units <= 128 * wgs &&
        units * (blocks + 8) < 0x7fffffff) {
        if (many) p.long_blocks = (int32_t)whole;
        p.parts = (int32_t)(many ? wgs / 2 : wgs < units * blocks ? wgs : units * blocks);
        if (p.parts > kMostParts) p.parts = kMostParts;
        const int32_t groups = a.heads_kv / p.group_heads;
        const int64_t results = p.rows > 16 && cut_by_tiles(a.batch, p.tiles, groups, p.parts) ? p.parts : 2 * p.parts;
        p.ws_bytes = record_bytes(p.tiles, groups) + results * p.group_heads * p.rows * (a.d + 2) * 4;
    }
    return p;
}

namespace {

template <typename T, bool E4>
hipError_t launch(const PagedPlan& p, const PagedArgs& a, hipStream_t s) {
    return p.rows == 16 ? launch_paged_rows<T, E4>(a, s) : launch_paged_tile<T, E4>(a, p.rows, s);
}

template <typename T>
hipError_t join(const PagedPlan& p, const PagedArgs& a, hipStream_t s) {
    return p.rows == 16 ? join<T, 16>(a, s) : p.rows == 64 ? join<T, 64>(a, s) : join<T, 128>(a, s);
}

}  // namespace

hipError_t launch_paged_attention(int32_t dtype, bool e4m3, const PagedPlan& p, const PagedArgs& a, hipStream_t s) {
    const bool f32 = dtype == CONV_DTYPE_F32;
    const auto run = [&](const PagedArgs& c) {
        if (f32) return e4m3 ? launch<float, true>(p, c, s) : launch<float, false>(p, c, s);
        return e4m3 ? launch<bf16, true>(p, c, s) : launch<bf16, false>(p, c, s);
    };
    if (p.parts) {
        const hipError_t e = run(a);
        if (e != hipSuccess) return e;
        return f32 ? join<float>(p, a, s) : join<bf16>(p, a, s);
    }
    // A workgroup a tile and head, as many tiles as a launch's grid holds.
    const int64_t most = most_workgroups(256) / a.head_groups;
    for (int64_t t = 0; t < p.tiles; t += most) {
        PagedArgs c = a;
        c.first_tile = (int32_t)t;
        c.tiles = (int32_t)(p.tiles - t < most ? p.tiles - t : most);
        const hipError_t e = run(c);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace conv2d
