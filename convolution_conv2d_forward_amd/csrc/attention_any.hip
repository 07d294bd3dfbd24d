// Softmax attention for both types and every shape: dispatch, the general
// kernel, and the join of split results.
#include "attention_common.h"
#include "linear_common.h"

namespace conv2d {

namespace {

// A workgroup of four waves takes 64 of the rows (query i, head of the group)
// that share a key head, 16 rows a wave, and walks their keys in tiles of 32.
// The product is formed transposed, S^T = K Q^T, so a lane holds scores of
// one row only: maximum and sum need two exchanges between lanes, and the
// scores are already laid out as the second operand of O^T = V^T P^T.  That
// product's sum over keys takes them in the order in which the lanes hold them,
// and V^T is read accordingly.  K and V are staged in LDS with 16 bytes of
// padding a row; the next tile is in registers meanwhile.
//
// Keys that a row does not see get weight 0 by selection.  An infinity or NaN
// in such a key's value would still spoil the row (0 * inf), so tiles that
// some row of the workgroup does not see whole are staged with those elements
// set to zero, and the rows that do see them add them one by one.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attention_any(AttnArgs a) {
    constexpr int BK = 32, C = Vec<T>::chunk, DC = DP / C;     // DC: 16-byte chunks of a row
    constexpr int KS = DP * (int)sizeof(T) / 64;               // 64-byte product steps over a row
    constexpr int LROW = DP + C;                               // LDS row, elements
    constexpr int NCH = (BK * DC + 255) / 256;                 // chunks a thread stages per operand
    __shared__ __align__(16) T lk[BK * LROW];
    __shared__ __align__(16) T lv[BK * LROW];
    __shared__ float lp[4][BK * 16];   // weights, for the one-by-one addition alone
    __shared__ int lrange[4][4];
    __shared__ int lbad;               // the last tile that held infinities or NaN

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = lane & 15, g = lane >> 4;
    uint32_t blk = blockIdx.x;
    const int bh = (int)(blk % (uint32_t)(a.batch * a.heads_kv));
    blk /= (uint32_t)(a.batch * a.heads_kv);
    const int split = (int)(blk % (uint32_t)a.splits);
    const int tile_r = a.row_tiles - 1 - (int)(blk / (uint32_t)a.splits);   // causal: the longest rows first
    const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
    const SeqLens sl = seq_lens(a, b);

    // This lane's row, and the intervals of the wave and the workgroup.
    const int row = tile_r * 64 + wave * 16 + n;
    const bool live = row < a.rows;
    const int qi = live ? row / a.group : 0, hq = hk * a.group + (live ? row - qi * a.group : 0);
    int lo = 0, hi = 0;
    row_interval(a, sl, b, qi, live, lo, hi);
    const bool empty = hi <= lo;
    int min_lo = empty ? INT32_MAX : lo, max_hi = hi;
    // Rows past the end do not count against a tile being seen whole.
    int max_lo = live ? (empty ? INT32_MAX : lo) : 0, min_hi = live ? hi : INT32_MAX;
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
        min_lo = min(min_lo, __shfl_xor(min_lo, m, 64));
        max_hi = max(max_hi, __shfl_xor(max_hi, m, 64));
        max_lo = max(max_lo, __shfl_xor(max_lo, m, 64));
        min_hi = min(min_hi, __shfl_xor(min_hi, m, 64));
    }
    if (lane == 0) {
        lrange[wave][0] = min_lo;
        lrange[wave][1] = max_hi;
        lrange[wave][2] = max_lo;
        lrange[wave][3] = min_hi;
    }
    if (tid == 0) lbad = -1;
    __syncthreads();
    int wlo = min(min(lrange[0][0], lrange[1][0]), min(lrange[2][0], lrange[3][0]));
    const int whi = max(max(lrange[0][1], lrange[1][1]), max(lrange[2][1], lrange[3][1]));
    const int full_lo = max(max(lrange[0][2], lrange[1][2]), max(lrange[2][2], lrange[3][2]));
    const int full_hi = min(min(lrange[0][3], lrange[1][3]), min(lrange[2][3], lrange[3][3]));
    if (wlo > whi) wlo = whi;

    // The tiles of this split.
    const int t0 = wlo / BK, tn = (whi + BK - 1) / BK - t0;
    const int first = t0 + (int)((int64_t)tn * split / a.splits), last = t0 + (int)((int64_t)tn * (split + 1) / a.splits);

    const T* kp = (const T*)a.k + b * a.k_s[0] + hk * a.k_s[2];
    const T* vp = (const T*)a.v + b * a.v_s[0] + hk * a.v_s[2];
    u32x4 fq[KS];
    {
        const T* qp = (const T*)a.q + b * a.q_s[0] + qi * a.q_s[1] + hq * a.q_s[2];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int e = (s * 4 + g) * C;
            fq[s] = u32x4{0, 0, 0, 0};
            if (live && e < a.d) fq[s] = *(const u32x4*)(qp + e);
        }
    }
    const ScoreP sp = score_params(a);
    const float slope = a.slopes && live ? a.slopes[hq] * kLog2e : 0.0f;
    const int pos = sl.nk - sl.nq + qi;

    u32x4 rk[NCH], rv[NCH];
    // Chunks of keys from kv_len on, and of elements from d on, are zero and not read.
    const auto fetch = [&](int tile) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * 256, key = tile * BK + c / DC, e = (c % DC) * C;
            rk[i] = rv[i] = u32x4{0, 0, 0, 0};
            if (c < BK * DC && key < sl.nk && e < a.d) {
                rk[i] = *(const u32x4*)(kp + key * a.k_s[1] + e);
                rv[i] = *(const u32x4*)(vp + key * a.v_s[1] + e);
            }
        }
    };

    f32x4 o[DP / 16] = {};
    float m_run = -INFINITY, l_run = 0.0f;
    if (first < last) fetch(first);
    for (int tile = first; tile < last; ++tile) {
        const int k0 = tile * BK;
        const bool whole = k0 >= full_lo && k0 + BK <= full_hi;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = tid + i * 256;
            if (c < BK * DC) {
                const int at = (c / DC) * LROW + (c % DC) * C;
                if (!whole && clean_chunk<T>(rv[i])) lbad = tile;
                *(u32x4*)(lk + at) = rk[i];
                *(u32x4*)(lv + at) = rv[i];
            }
        }
        __syncthreads();
        if (tile + 1 < last) fetch(tile + 1);

        f32x4 s[2] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const u32x4 fk = *(const u32x4*)(lk + (16 * t + n) * LROW + (ks * 4 + g) * C);
                s[t] = mfma_step<T>(fk, fq[ks], s[t]);
            }
        float m_new = m_run, sc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[i] = s[i >> 2][i & 3];
        scores<T>(sp, sc);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = k0 + 16 * t + 4 * g + i;
                float x = sc[4 * t + i];
                if (a.slopes) x -= slope * fabsf((float)(pos - key));
                if (!whole) x = key >= lo && key < hi ? x : -INFINITY;
                s[t][i] = x;
                m_new = fmaxf(m_new, x);
            }
        m_new = fmaxf(m_new, __shfl_xor(m_new, 16, 64));
        m_new = fmaxf(m_new, __shfl_xor(m_new, 32, 64));
        const float base = m_new == -INFINITY ? 0.0f : m_new;   // nothing seen yet: every weight is 0
        const float fade = __builtin_amdgcn_exp2f(m_run - base);
        m_run = m_new;
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(s[t][i] - base);
                sum += s[t][i];
            }
        l_run = l_run * fade + sum;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) o[d] *= fade;
        if constexpr (sizeof(T) == 2) {
            bf16x8 fp;   // rounded, as in attention_tile
#pragma unroll
            for (int i = 0; i < 8; ++i) fp[i] = (bf16)s[i >> 2][i & 3];
#pragma unroll
            for (int d = 0; d < DP / 16; ++d) {
                bf16x8 fv;
#pragma unroll
                for (int i = 0; i < 8; ++i) fv[i] = lv[(16 * (i >> 2) + 4 * g + (i & 3)) * LROW + 16 * d + n];
                o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, fp, o[d], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int d = 0; d < DP / 16; ++d)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float fv = lv[(16 * (i >> 2) + 4 * g + (i & 3)) * LROW + 16 * d + n];
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(fv, s[i >> 2][i & 3], o[d], 0, 0, 0);
                }
        }
        if (!whole && lbad == tile) {
            // The elements that were set to zero, for the rows that see them.
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) lp[wave][(16 * t + 4 * g + i) * 16 + n] = s[t][i];
            __builtin_amdgcn_wave_barrier();
            for (int j = 0; j < BK; ++j) {
                const int key = k0 + j;
                if (key < lo || key >= hi) continue;
                const float p = lp[wave][j * 16 + n];
                for (int d = 0; d < DP / 16; ++d)
                    for (int i = 0; i < 4; ++i) {
                        const int e = 16 * d + 4 * g + i;
                        if (e >= a.d) continue;
                        const float v = to_f32(vp[key * a.v_s[1] + e]);
                        if (!(fabsf(v) < INFINITY)) {
#pragma unroll
                            for (int dd = 0; dd < DP / 16; ++dd)
#pragma unroll
                                for (int ii = 0; ii < 4; ++ii)
                                    if (dd == d && ii == i) o[dd][ii] += p * v;
                        }
                    }
            }
        }
    }
    l_run += __shfl_xor(l_run, 16, 64);
    l_run += __shfl_xor(l_run, 32, 64);
    if (!live) return;
    if (a.splits == 1) {
        const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
        T* op = (T*)a.out + b * a.o_s[0] + qi * a.o_s[1] + hq * a.o_s[2];
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
            const int e = 16 * d + 4 * g;
            if (e < a.d) *(typename Vec<T>::v4*)(op + e) = from_f32<T>(o[d] * inv);
        }
        return;
    }
    const int64_t wr = ws_row(a, bh, split, row);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) {
        const int e = 16 * d + 4 * g;
        if (e < a.d) *(f32x4*)(ws_out(a, wr) + e) = o[d];
    }
    if (g == 0) *ws_stat(a, wr) = f32x2{m_run, l_run};
}

// Few splits: as many threads as the row is wide add up its outputs.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attention_join_few(AttnArgs a, uint32_t all_rows) {
    constexpr int W = DP / 4;
    const uint32_t at_row = blockIdx.x * (256 / W) + threadIdx.x / W;
    const int e = (threadIdx.x % W) * 4;
    if (at_row >= all_rows || e >= a.d) return;
    const int bh = (int)(at_row / (uint32_t)a.rows), row = (int)(at_row % (uint32_t)a.rows);
    const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
    const int qi = row / a.group, hq = hk * a.group + row % a.group;
    const int64_t at = ws_row(a, bh, 0, row);
    float top = -INFINITY, l = 0.0f;
    f32x4 sum{0, 0, 0, 0};
    for (int s0 = 0; s0 < a.splits; s0 += 4) {
        f32x2 st[4];
        f32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t wr = at + (int64_t)min(s0 + i, a.splits - 1) * a.rows;
            st[i] = *ws_stat(a, wr);
            v[i] = *(const f32x4*)(ws_out(a, wr) + e);
            if (s0 + i >= a.splits) st[i] = f32x2{-INFINITY, 0.0f};
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
            if (s0 + i < a.splits) sum += v[i] * f;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* op = (T*)a.out + b * a.o_s[0] + qi * a.o_s[1] + hq * a.o_s[2];
    *(typename Vec<T>::v4*)(op + e) = from_f32<T>(sum * inv);
}

// A workgroup per row.  The splits' maxima and sums give each split's factor;
// then groups of threads, each as wide as the row, add up the outputs of every
// GROUPS-th split, four loads in flight, and meet in LDS.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attention_join(AttnArgs a) {
    constexpr int W = DP / 4, GROUPS = 256 / W;
    __shared__ float top_w[4], sum_w[4], factor[256];
    __shared__ __align__(16) f32x4 part[GROUPS][W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bh = (int)(blockIdx.x / (uint32_t)a.rows), row = (int)(blockIdx.x % (uint32_t)a.rows);
    const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
    const int qi = row / a.group, hq = hk * a.group + row % a.group;
    const int64_t at = ws_row(a, bh, 0, row);
    const int grp = tid / W, e = (tid % W) * 4;
    f32x4 sum{0, 0, 0, 0};
    f32x2 st{-INFINITY, 0.0f};
    if (tid < a.splits) st = *ws_stat(a, at + (int64_t)tid * a.rows);
    // The first outputs are on their way while the factors are formed.
    f32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = grp + i * GROUPS;
        v[i] = f32x4{0, 0, 0, 0};
        if (s < a.splits && e < a.d) v[i] = *(const f32x4*)(ws_out(a, at + (int64_t)s * a.rows) + e);
    }
    float top = st[0];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
    if (lane == 0) top_w[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(top_w[0], top_w[1]), fmaxf(top_w[2], top_w[3]));
    const float f = __builtin_amdgcn_exp2f(st[0] - (top == -INFINITY ? 0.0f : top));
    factor[tid] = f;
    float l = f * st[1];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) l += __shfl_xor(l, m, 64);
    if (lane == 0) sum_w[wave] = l;
    __syncthreads();
    l = sum_w[0] + sum_w[1] + sum_w[2] + sum_w[3];
    for (int s0 = grp; s0 < a.splits; s0 += 4 * GROUPS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + i * GROUPS;
            if (s < a.splits) sum += v[i] * factor[s];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + (i + 4) * GROUPS;
            if (s < a.splits && e < a.d) v[i] = *(const f32x4*)(ws_out(a, at + (int64_t)s * a.rows) + e);
        }
    }
    part[grp][tid % W] = sum;
    __syncthreads();
    if (grp != 0 || e >= a.d) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) sum += part[i][tid];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* op = (T*)a.out + b * a.o_s[0] + qi * a.o_s[1] + hq * a.o_s[2];
    *(typename Vec<T>::v4*)(op + e) = from_f32<T>(sum * inv);
}

template <typename T, int DP>
hipError_t run_any(const AttnArgs& a, hipStream_t s) {
    const int64_t blocks = (int64_t)a.batch * a.heads_kv * a.row_tiles * a.splits;
    attention_any<T, DP><<<dim3((uint32_t)blocks), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t run_any(const AttnArgs& a, hipStream_t s) {
    if (a.d <= 32) return run_any<T, 32>(a, s);
    if (a.d <= 64) return run_any<T, 64>(a, s);
    if (a.d <= 96) return run_any<T, 96>(a, s);
    if (a.d <= 128) return run_any<T, 128>(a, s);
    return run_any<T, 256>(a, s);
}

}  // namespace

template <typename T, int DP>
static hipError_t run_join(const AttnArgs& a, hipStream_t s) {
    const int64_t rows = (int64_t)a.batch * a.heads_kv * a.rows;
    // 517 rows x 24 heads in 3 splits: 4 us by 8 rows a workgroup, 12 by one.
    if (a.splits <= 8) {
        constexpr int R = 256 / (DP / 4);
        attention_join_few<T, DP><<<dim3((uint32_t)((rows + R - 1) / R)), dim3(256), 0, s>>>(a, (uint32_t)rows);
    } else {
        attention_join<T, DP><<<dim3((uint32_t)rows), dim3(256), 0, s>>>(a);
    }
    return hipGetLastError();
}

template <typename T>
static hipError_t run_join(const AttnArgs& a, hipStream_t s) {
    if (a.d <= 32) return run_join<T, 32>(a, s);
    if (a.d <= 64) return run_join<T, 64>(a, s);
    if (a.d <= 128) return run_join<T, 128>(a, s);
    return run_join<T, 256>(a, s);
}

hipError_t launch_attention_join(int32_t dtype, const AttnArgs& a, hipStream_t s) {
    return dtype == CONV_DTYPE_F32 ? run_join<float>(a, s) : run_join<bf16>(a, s);
}

AttnPlan plan_attention(int32_t dtype, const AttnArgs& a) {
    AttnPlan p{};
    // A tile's keys within 32-bit byte offsets.
    const bool near = a.k_s[1] < 1 << 24 && a.v_s[1] < 1 << 24;
    // 17 to 32 rows in bf16, 32 rows of 128 over 8x4096 keys: 36.8 us in one
    // tile, 47.8 in two of 16 rows.
    p.kernel = a.rows <= (dtype == CONV_DTYPE_F32 ? 32 : 16)       ? ATTN_ROWS
               : near ? ATTN_TILE_128
                      : ATTN_ANY;
    // Heads beyond 128 leave room for one workgroup on a CU in either size:
    // 2500 causal rows of 16 heads of 256 over 4 (316 tiles of 128) take 130 us
    // in them and 149 in tiles of 64, 1300 rows (164 tiles) 69 and 53 with the
    // keys undivided.
    const int64_t cus = device_cu_count();
    if (p.kernel == ATTN_TILE_128 && !(dtype == CONV_DTYPE_F32 && a.d > 128) &&
        (int64_t)a.batch * a.heads_kv * ((a.rows + 127) / 128) < (a.d > 128 ? cus * 3 / 4 : cus * 2))
        p.kernel = ATTN_TILE_64;
    const int tile = p.kernel == ATTN_ROWS ? 16 : p.kernel == ATTN_TILE_128 ? 128 : 64;
    p.row_tiles = (a.rows + tile - 1) / tile;
    // Few row tiles leave compute units without work: the keys are then split.
    const int64_t tiles = (int64_t)a.batch * a.heads_kv * p.row_tiles;
    // Workgroups wanted, and keys for each part but the last.  Two a unit even
    // out rows of different lengths (5322 causal rows of 4 heads of 64: 63.4 us
    // undivided, 43.1 in two).  The partial results of many rows cost as much as
    // a few hundred keys: 1000 causal rows of 16 heads of 128 over 4 take 22.2 us
    // undivided, 26.9 in two; 538 of 12 fp32 heads of 128 50.1 us undivided,
    // 37.7 in two, 36.0 in three.  Keys just above a part's are divided all the
    // same, which wide bf16 heads pay for: 1300 rows of 256 73 us in two, 53
    // undivided, but 1700 72 and 92.
    const bool f32 = dtype == CONV_DTYPE_F32;
    int64_t want = 2 * cus;
    int64_t keys = f32 ? 512 : tiles * 2 >= cus ? 1024 : 256;
    if (p.kernel == ATTN_ROWS) {
        // Two workgroups fit on a unit (one where a row of K has more than 256
        // bytes); a third per unit evens out sequences of different lengths.
        const bool big = a.d * (dtype == CONV_DTYPE_F32 ? 4 : 2) > 256;
        want = big ? cus : a.batch > 1 ? 3 * cus : 2 * cus;
        keys = tiles >= cus ? 1024 : tiles * 2 >= cus ? 512 : 128;
    }
    // Of wide fp32 rows one workgroup fits on a unit: the nearest, not the next
    // number of parts (4096 causal rows of 4 heads of 128, 256 tiles: 194 us in
    // two, 203 in three).
    int64_t s = tiles < want ? (want + (f32 && p.kernel != ATTN_ROWS ? tiles / 2 : tiles - 1)) / tiles : 1;
    const int64_t most = ((int64_t)a.kv_len + keys - 1) / keys;
    if (s > most) s = most;
    if (s > ATTN_MAX_SPLITS) s = ATTN_MAX_SPLITS;
    p.splits = s < 1 ? 1 : (int32_t)s;
    if (p.splits > 1) p.ws_bytes = (int64_t)a.batch * a.heads_kv * p.splits * a.rows * (a.d + 2) * 4;
    return p;
}

hipError_t launch_attention(int32_t dtype, const AttnPlan& p, const AttnArgs& a, hipStream_t s) {
    const int64_t most = most_workgroups(256) / sequence_workgroups(a, p);
    if (a.batch > most) {
        // So many workgroups that the keys are not divided: no workspace.
        const int64_t es = dtype == CONV_DTYPE_F32 ? 4 : 2;
        for (int64_t b = 0; b < a.batch; b += most) {
            AttnArgs c = a;
            c.batch = (int32_t)(a.batch - b < most ? a.batch - b : most);
            c.q = (const char*)a.q + b * a.q_s[0] * es;
            c.k = (const char*)a.k + b * a.k_s[0] * es;
            c.v = (const char*)a.v + b * a.v_s[0] * es;
            c.out = (char*)a.out + b * a.o_s[0] * es;
            if (a.q_lens) c.q_lens = a.q_lens + b;
            if (a.kv_lens) c.kv_lens = a.kv_lens + b;
            if (a.prefix_lens) c.prefix_lens = a.prefix_lens + b;
            if (a.doc_offsets) c.doc_offsets = a.doc_offsets + b * (a.n_docs + 1);
            const hipError_t e = launch_attention(dtype, p, c, s);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
    const bool f32 = dtype == CONV_DTYPE_F32;
    const int rows = p.kernel == ATTN_TILE_128 ? 128 : 64;
    hipError_t e;
    if (p.kernel == ATTN_ROWS)
        e = launch_attention_rows(dtype, a, s);
    else if (p.kernel == ATTN_ANY)
        e = f32 ? run_any<float>(a, s) : run_any<bf16>(a, s);
    else
        e = f32 ? launch_attention_tile<float>(a, rows, s) : launch_attention_tile<bf16>(a, rows, s);
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_attention_join(dtype, a, s);
}

}  // namespace conv2d
