// Dispatch of linear_forward.
#include <cmath>

#include "linear_common.h"

namespace conv2d {

namespace {

// The kernel of a call, by sizes, type and alignment: the one that is expected
// to end first.
//
// linear_rows deals k among a workgroup's waves (its shape: rows_shape).  After
// some 5 us each 128-byte unit of a wave takes (us)
//   one workgroup a CU, 16 / 32 / 64 rows    bf16 0.3 / 0.25 / 0.33
//                                            fp32 0.3 / 0.55 / 0.6
//   for each workgroup a CU has, 64 rows     0.6 and 1.4
// and through registers 1.2, or 1.8 for each with 32 rows.  It takes up to 32
// rows always, and few tiles of a long k (64x4096x4096 bf16: 15.0 us against
// 23.0 in tiles; 64x4096x11264: 35.3 against 28.3).
//
// Tiles take rounds of workgroups, and in each for a step of 128 bytes (us,
// with all CUs at work), after some 6 us:
//              256    128 by pairs    128 deep    64
//   bf16       1.9    1.2             0.72        0.49, one a CU 0.30
//   fp32       -      3.85            2.07        1.1, one a CU 0.65
// (2048x4096x4096 bf16: 109 us in tiles of 256, 78 in pairs of 128, 83 in
// deep ones, 125 in tiles of 64.)
linear_tile_t pick(int32_t dtype, const LinearArgs& a) {
    if (a.m <= 32) return LINEAR_ROWS;
    const bool f32 = dtype == CONV_DTYPE_F32;
    const int64_t cus = device_cu_count();
    const auto rounds = [&](int64_t t, int64_t per_cu) {
        const int64_t tiles = ((a.m + t - 1) / t) * ((a.n + t - 1) / t);
        return (float)((tiles + cus * per_cu - 1) / (cus * per_cu));
    };
    float best = rounds(64, 1) == 1 ? (f32 ? 0.65f : 0.30f) : rounds(64, 2) * (f32 ? 1.1f : 0.49f);
    linear_tile_t tile = LINEAR_TILE_64;
    const auto offer = [&](linear_tile_t t, float cost) {
        if (cost < best) {
            best = cost;
            tile = t;
        }
    };
    offer(LINEAR_TILE_128_DEEP, rounds(128, 1) * (f32 ? 2.07f : 0.72f));
    offer(LINEAR_TILE_128, rounds(128, 2) * (f32 ? 3.85f : 1.2f));
    if (!f32) offer(LINEAR_TILE_256, rounds(256, 1) * 1.9f);
    const RowsShape sh = rows_shape(f32, a);
    const int bytes = a.k * (f32 ? 4 : 2), rows = 16 * sh.mt, waves = sh.waves;
    const float groups = (float)(((int64_t)a.m + rows - 1) / rows) * (float)((a.n + 15) / 16) / (float)cus;
    const float alone = !a.vec ? 1.2f : sh.mt == 4 ? (f32 ? 0.6f : 0.33f) : sh.mt == 2 ? (f32 ? 0.55f : 0.25f) : 0.3f;
    const float unit = fmaxf(alone, groups * (float)sh.mt * (!a.vec ? 0.9f : f32 ? 0.35f : 0.15f));
    const float step = a.vec ? best : best * 1.5f;   // through registers
    if (5.0f + (float)((bytes + 128 * waves - 1) / (128 * waves)) * unit < 6.0f + (float)((bytes + 127) / 128) * step)
        return LINEAR_ROWS;
    return tile;
}

// Whether one launch holds the call's workgroups (linear_tile.h's persistent
// ones: whether they count their tiles in 31 bits).
bool one_launch(int32_t dtype, const LinearArgs& a, linear_tile_t tile) {
    const auto blocks = [&](int64_t bm, int64_t bn) { return ((a.m + bm - 1) / bm) * ((a.n + bn - 1) / bn); };
    if (tile == LINEAR_ROWS) {
        const RowsShape sh = rows_shape(dtype == CONV_DTYPE_F32, a);
        return blocks(16 * sh.mt, 16) <= most_workgroups(64 * sh.waves);
    }
    const int t = tile == LINEAR_TILE_64 ? 64 : 128;   // or more
    return blocks(t, t) <= (a.vec ? 0x7fff0000 : most_workgroups(256));
}

}  // namespace

const char* linear_kernel_name(int32_t dtype, const LinearArgs& a) {
    static const char* const names[2][5] = {{"linear_rows_f32", "linear_tile_f32/64", "linear_tile_f32/128",
                                             "linear_tile_f32/128deep", "linear_tile_f32/256"},
                                            {"linear_rows_bf16", "linear_tile_bf16/64", "linear_tile_bf16/128",
                                             "linear_tile_bf16/128deep", "linear_tile_bf16/256"}};
    return names[dtype == CONV_DTYPE_F32 ? 0 : 1][pick(dtype, a)];
}

hipError_t launch_linear(int32_t dtype, const LinearArgs& a, hipStream_t s) {
    const linear_tile_t tile = pick(dtype, a);
    if (!one_launch(dtype, a, tile)) {
        // Halves of the rows (a few rows of any width fit).
        const int64_t es = dtype == CONV_DTYPE_F32 ? 4 : 2;
        LinearArgs lo = a, hi = a;
        lo.m = a.m / 2;
        hi.m = a.m - lo.m;
        hi.x = (const char*)a.x + lo.m * a.xs * es;
        hi.y = (char*)a.y + lo.m * a.ys * es;
        if (a.residual) hi.residual = (const char*)a.residual + lo.m * a.rs * es;
        const hipError_t e = launch_linear(dtype, lo, s);
        return e != hipSuccess ? e : launch_linear(dtype, hi, s);
    }
    if (tile == LINEAR_ROWS) return launch_linear_rows(dtype, a, s);
    return dtype == CONV_DTYPE_F32 ? launch_linear_tile<float>(a, tile, s) : launch_linear_tile<bf16>(a, tile, s);
}

}  // namespace conv2d
