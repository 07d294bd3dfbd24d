// Attention of few rows over pages: single tokens, and a few drafted ones.
// Compiled once for each type and cache (paged_rows_*.hip).
#pragma once

#include "linear_common.h"
#include "paged_common.h"

namespace conv2d {

namespace {

typedef const __attribute__((address_space(1))) uint8_t* GlobalBytes;

// 16 of the rows (new token, head of the group) that share a key head a
// workgroup, whose four waves take a quarter of a block's keys each (or half of
// them, of one of two heads): straight
// from memory into the operands of the matrix cores, the next block's loads in
// flight and the one's after in the page table, no LDS or barrier between.  It
// is bound by the bytes of keys and values.
//
// S^T = K Q^T in 16x16 steps, O^T = V^T P^T with V's operands put together by
// byte permutes, as attention_rows has them.  Codes are read 16 of K's row a
// lane, whose elements Q's operand follows, and a row of V in 16 lanes; they
// become elements of T, times their scale, by one instruction for two.
//
// A lane looks up the page of one key of the wave's tile (the upper half wave
// the same keys again) and forms its place; the lanes that read a key's row get
// it by exchange.
template <typename T, int DP, bool E4, int GH>
struct PagedRows {
    static constexpr int C = Vec<T>::chunk;
    static constexpr int KS = DP * (int)sizeof(T) / 64;               // 64-byte product steps over a row
    static constexpr int PK = E4 ? 16 / C : 1, KL = KS / PK;          // steps that one load of K serves; loads
    static constexpr int VC = (DP / C + 15) / 16;                     // 16-chunk groups of a row of V
    static constexpr int BK = DP * (int)sizeof(T) > 512 ? 16 : 32, NT = BK / 16, NJ = BK / 4;
    static constexpr int OUT = VC * C;                                // 16x16 output blocks
    static constexpr int RB = DP * (int)sizeof(T), NBUF = DP <= 128 ? 2 : 1, OCC = RB <= 256 ? 2 : 1, NW = 4;
    static constexpr int KW = NW / GH, BU = KW * BK;                  // waves of a head; a block's keys
    typedef typename std::conditional<E4, typename Codes<T>::type, u32x4>::type VT;
    u32x4 k[NT][KL];
    VT v[NJ][VC];
    uint8_t scales;    // of this lane's key: K's in the lower half wave, V's in the upper
    uint32_t there;    // keys of the tile that there are

    // First element of product step s in lane group g.
    static __device__ __forceinline__ int element(int s, int g) { return E4 ? (4 * (s / PK) + g) * 16 + s % PK * C : (4 * s + g) * C; }
    // The tile's keys of a lane: row r of K's step t, row j of V in group g.
    static __device__ __forceinline__ int k_row(int t, int r) { return sizeof(T) == 2 ? 8 * (r >> 2) + 4 * t + (r & 3) : 16 * t + r; }
    static __device__ __forceinline__ int v_row(int j, int g) { return sizeof(T) == 2 ? 8 * g + j : 16 * (j >> 2) + 4 * g + (j & 3); }

    __device__ __forceinline__ void load(const PagedArgs& a, GlobalBytes scale, int entry, int k0, int nk, int h, int lane) {
        int r = lane & 15, g = lane >> 4;
        asm volatile("" : "+v"(r), "+v"(g));   // what follows from them is formed anew for each tile: it would cost registers
        const KeyPlace p = key_place(a, entry, k0 + (lane & (BK - 1)), nk);
        there = (uint32_t)__ballot(p.there) & (BK == 32 ? 0xffffffffu : 0xffffu);
        const char *kb = (const char*)a.k + h * a.k_head, *vb = (const char*)a.v + h * a.v_head;
        if (E4) scales = scale[p.s];
        // Chunks from d on are the row's first instead: no branch stands between
        // the loads, and step() makes K's zero; V's give outputs that are none.
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const char* row = kb + (uint64_t)from_lane(p.k, k_row(t, r)) * 16;
#pragma unroll
            for (int s = 0; s < KL; ++s) {
                const int e = element(s * PK, g);
                k[t][s] = *(const u32x4*)(row + (e < a.d ? e : 0) * (E4 ? 1 : (int)sizeof(T)));
            }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const char* row = vb + (uint64_t)from_lane(p.v, v_row(j, g)) * 16;
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                const int e = (16 * c + r) * C;
                v[j][c] = *(const VT*)(row + (e < a.d ? e : 0) * (E4 ? 1 : (int)sizeof(T)));
            }
        }
    }

    __device__ __forceinline__ void cut(int d, int g) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int s = 0; s < KL; ++s)
                if (element(s * PK, g) >= d) k[t][s] = u32x4{0, 0, 0, 0};
    }

    // Operand of K's step t, s.
    __device__ __forceinline__ u32x4 key(int t, int s, float scale) const {
        if constexpr (!E4) return k[t][s];
        if constexpr (sizeof(T) == 2)
            return decode(u32x2{k[t][s / PK][s % PK * 2], k[t][s / PK][s % PK * 2 + 1]}, scale, T{});
        else
            return decode(k[t][s / PK][s % PK], scale, T{});
    }
};

template <typename T, int DP, bool E4, int GH>
__global__ __launch_bounds__((64 * PagedRows<T, DP, E4, GH>::NW), (PagedRows<T, DP, E4, GH>::OCC)) void paged_rows(PagedArgs) {
    const PagedArgs& a = kernel_args();
    typedef PagedRows<T, DP, E4, GH> R;
    constexpr int C = R::C, KS = R::KS, VC = R::VC, NW = R::NW, KW = R::KW, BK = R::BK, NT = R::NT, NJ = R::NJ, OUT = R::OUT, BU = R::BU;
    __shared__ PagedLine line;
    __shared__ f32x2 stat[NW][16];
    __shared__ __align__(16) f32x4 part[NW][OUT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    ScoreP sp;
    sp.cap = a.softcap;
    sp.scale = a.softcap > 0.0f ? cap_scale(a.scale, a.softcap) : a.scale * kLog2e;

    Pieces<16, BU, 0, false> pieces;
    Piece pc;
    if (!pieces.start(a, line)) return;
    int u = pieces.begin;
    while (pieces.next(kernel_args(), line, u, pc)) {
        const PagedArgs& a = kernel_args();
        const int b = pc.b, t = pc.t, sub = wave % GH, h = pc.h * GH + sub, first = pc.k0;
        const int64_t result = (int64_t)pc.result * GH + sub;   // below 0: none
        int last = pc.k1;
        const PagedSeq sq = pc.sq;
        const int32_t* table = a.page_table + (int64_t)b * a.max_pages;
        const KeyBlocks blocks = key_blocks<16, BU>(a, sq, t * 16);
        const int row = t * 16 + r;
        const bool live = row < sq.nq * a.group;
        const int qi = live ? token_of(a, row) : 0, hq = h * a.group + (live ? row - qi * a.group : 0);
        int lo, hi;
        paged_interval(a, sq, qi, live, lo, hi);
        int f_lo = live ? lo : 0, f_hi = live ? hi : INT32_MAX;   // keys that every row sees, first tokens apart
        u32x4 fq[KS];
        const T* qp = (const T*)a.q + (int64_t)(sq.first + qi) * a.q_s + (int64_t)hq * a.d;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int e = R::element(s, g);
            fq[s] = u32x4{0, 0, 0, 0};
            if (live && e < a.d) fq[s] = *(const u32x4*)(qp + e);
        }
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) {
            f_lo = max(f_lo, __shfl_xor(f_lo, m, 64));
            f_hi = min(f_hi, __shfl_xor(f_hi, m, 64));
        }
        f_lo = __builtin_amdgcn_readfirstlane(f_lo);
        f_hi = __builtin_amdgcn_readfirstlane(f_hi);
        if (blocks.n == 0) last = first;   // no row sees a key

        f32x4 o[OUT] = {};
        float m_run = -INFINITY, l_run = 0.0f;
        const auto key0 = [&](int i) { return blocks.at(i) * BU + wave / GH * BK; };
        const auto step = [&](R& f, int i) {
            const int k0 = key0(i);
            const bool whole = k0 + BK <= f_hi && (k0 >= f_lo || k0 + BK <= a.sinks) && f.there == (BK == 32 ? 0xffffffffu : 0xffffu);
            int rr = r, gg = g;
            asm volatile("" : "+v"(rr), "+v"(gg));   // likewise
            if (a.d < DP) f.cut(a.d, gg);
            f32x4 s[NT] = {};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float scale = 1.0f;
                if (E4) scale = scale_value(from_lane(f.scales, R::k_row(t, rr)));
#pragma unroll
                for (int j = 0; j < KS; ++j) s[t] = mfma_step<T>(f.key(t, j, scale), fq[j], s[t]);
            }
            u32x4 decoded[E4 ? NJ : 1][E4 ? VC : 1];
            if constexpr (E4) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const float scale = scale_value(from_lane(f.scales, 32 + R::v_row(j, gg)));
#pragma unroll
                    for (int c = 0; c < VC; ++c) decoded[j][c] = decode(f.v[j][c], scale, T{});
                }
            }
            const auto v = [&](int j, int c) -> u32x4& {
                if constexpr (E4)
                    return decoded[j][c];
                else
                    return f.v[j][c];
            };
            // Infinities and NaN in values that some row does not see: zeros go
            // into the product, and the rows that see them get them one by one.
            bool bad = false;
            if (!whole) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int c = 0; c < VC; ++c) bad |= has_bad<T>(v(j, c));
                bad = __ballot(bad) != 0;
            }
            if (bad) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int c = 0; c < VC; ++c) clean_chunk<T>(v(j, c));
            }
            const auto sees = [&](int key) { return key < hi && (key >= lo || key < a.sinks) && (f.there >> (key - k0) & 1); };
            float top = -INFINITY, sc[4 * NT], p[NT][4];
#pragma unroll
            for (int j = 0; j < 4 * NT; ++j) sc[j] = s[j >> 2][j & 3];
            scores<T>(sp, sc);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x = sc[4 * t + j];
                    if (!whole) x = sees(k0 + (sizeof(T) == 2 ? 8 * gg + 4 * t + j : 16 * t + 4 * gg + j)) ? x : -INFINITY;
                    s[t][j] = x;
                    top = fmaxf(top, x);
                }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float m_new = fmaxf(m_run, top), base = m_new == -INFINITY ? 0.0f : m_new;
            const float fade = __builtin_amdgcn_exp2f(m_run - base);
            m_run = m_new;
            l_run *= fade;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[t][j] = __builtin_amdgcn_exp2f(s[t][j] - base);
                    l_run += p[t][j];
                }
#pragma unroll
            for (int d = 0; d < OUT; ++d) o[d] *= fade;
            if constexpr (sizeof(T) == 2) {
                bf16x8 fp, fl;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    fp[j] = (bf16)weight_part(p[j >> 2][j & 3], false);
                    fl[j] = (bf16)weight_part(p[j >> 2][j & 3], true);
                }
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        u32x4 w;   // element e of this lane's chunk, for the group's eight keys
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = __builtin_amdgcn_perm(v(2 * j + 1, c)[e >> 1], v(2 * j, c)[e >> 1],
                                                         e & 1 ? 0x07060302u : 0x05040100u);
                        o[c * 8 + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), fp,
                                                                               o[c * 8 + e], 0, 0, 0);
                        o[c * 8 + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), fl,
                                                                               o[c * 8 + e], 0, 0, 0);
                    }
            } else {
#pragma unroll
                for (int c = 0; c < VC; ++c)
#pragma unroll
                    for (int e = 0; e < C; ++e)
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            o[c * C + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __builtin_bit_cast(f32x4, v(j, c))[e], p[j >> 2][j & 3], o[c * C + e], 0, 0, 0);
            }
            if (bad) {
                // Output block (c, e) of lane l has rows 16 c C + (4 (l / 16) + i) C + e of V^T.
#pragma unroll 1
                for (int j = 0; j < BK; ++j) {
                    if (!(f.there >> j & 1)) continue;
                    const bool add = sees(k0 + j);
#pragma unroll 1
                    for (int e0 = 0; e0 < a.d; e0 += 64) {
                        const float x = e0 + lane < a.d ? value_at<T, E4>(a, table, h, k0 + j, e0 + lane) : 0.0f;
                        for (uint64_t m = __ballot(!(fabsf(x) < INFINITY)); m; m &= m - 1) {
                            const int l = (int)__builtin_ctzll(m);
                            const float y = __shfl(x, l, 64);
                            int at = e0 + l - 4 * gg * C;
                            asm volatile("" : "+v"(at));   // no comparison is kept in registers across the tiles
#pragma unroll
                            for (int i = 0; i < 4 * OUT; ++i)
                                o[i >> 2][i & 3] += add && (16 * (i / (4 * C)) + (i & 3)) * C + (i >> 2) % C == at ? y : 0.0f;
                        }
                    }
                }
            }
        };
        // A page's number is read before the loads of the block ahead of its
        // own: loads end in order, and waiting for one behind them would be
        // waiting for them.
        const auto look = [&](int i) {
            const int e = page_entry(a, table, key0(min(i, last - 1)) + (lane & (BK - 1)));
            __builtin_amdgcn_sched_barrier(0);
            return e;
        };
        // Kept as an address: made in the loop, the choice between two arguments
        // would be a load.
        uint64_t scale_at = E4 ? (uint64_t)((lane < 32 ? a.ks : a.vs) + h * a.s_head) : 0;
        asm volatile("" : "+v"(scale_at));
        const GlobalBytes scale = (GlobalBytes)scale_at;
        // The last block's loads are made again rather than left out: with a
        // branch around loads, or out of the loop between them, the compiler
        // waits for all of them.
        const auto load = [&](R& f, int i, int entry) {
            f.load(a, scale, entry, key0(min(i, last - 1)), sq.nk, h, lane);
        };
        if (first < last) {
            int e0 = look(first), e1 = look(first + 1);
            if constexpr (R::NBUF == 2) {
                R f[2];
                load(f[0], first, e0);
                for (int i = first; i + 1 < last; i += 2) {
                    e0 = look(i + 2);
                    load(f[1], i + 1, e1);
                    step(f[0], i);
                    e1 = look(i + 3);
                    load(f[0], i + 2, e0);
                    step(f[1], i + 1);
                }
                if ((last - first) & 1) step(f[0], last - 1);
            } else {
                for (int i = first; i < last; ++i) {
                    R f;
                    load(f, i, e0);
                    e0 = e1;
                    e1 = look(i + 2);
                    step(f, i);
                }
            }
        }

        wait_vmem<0>();   // or the next piece's first loads would be counted with the repeated ones

        // The results of a head's waves: the maxima and sums first, then the
        // outputs at the common maximum.  Its wave w adds up output blocks w,
        // w + KW ...
        l_run += __shfl_xor(l_run, 16, 64);
        l_run += __shfl_xor(l_run, 32, 64);
        if (g == 0) stat[wave][r] = f32x2{m_run, l_run};
        __syncthreads();
        float top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) top = fmaxf(top, stat[w * GH + sub][r][0]);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < KW; ++w) total += __builtin_amdgcn_exp2f(stat[w * GH + sub][r][0] - base) * stat[w * GH + sub][r][1];
        const float fade = __builtin_amdgcn_exp2f(m_run - base);
#pragma unroll
        for (int d = 0; d < OUT; ++d) part[wave][d][lane] = o[d] * fade;
        __syncthreads();
        if (!live) continue;
        const PagedArgs& end = kernel_args();
        T* op = (T*)end.out + (int64_t)(sq.first + qi) * end.o_s + (int64_t)hq * end.d;
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        // A lane's chunk c of its row i: C consecutive outputs, one of each of C blocks.
        for (int ci = wave / GH; ci < VC * 4; ci += KW) {
            const int c = ci >> 2, i = ci & 3, at = (16 * c + 4 * g + i) * C;
            if (at >= end.d) continue;
            float x[C];
#pragma unroll
            for (int e = 0; e < C; ++e) {
                x[e] = 0.0f;
#pragma unroll
                for (int w = 0; w < KW; ++w) x[e] += ((const float*)&part[w * GH + sub][c * C + e][lane])[i];
            }
            if (pc.result < 0) {
                T y[C];
#pragma unroll
                for (int e = 0; e < C; ++e) y[e] = from_f32<T>(x[e] * inv);
                __builtin_memcpy(op + at, y, 16);
            } else {
                float* wo = paged_ws<16>(end).out + (result * 16 + r) * end.d + at;
#pragma unroll
                for (int e = 0; e < C; ++e) wo[e] = x[e];
            }
        }
        if (pc.result >= 0 && wave < GH && g == 0) paged_ws<16>(end).stat[result * 16 + r] = f32x2{top, total};
    }
}

template <typename T, int DP, bool E4, int GH>
hipError_t run(const PagedArgs& a, hipStream_t s) {
    const uint32_t units = (uint32_t)a.tiles * (uint32_t)a.head_groups;
    const uint32_t grid = (uint32_t)a.parts + (a.parts && !a.long_blocks ? 0 : units);
    paged_rows<T, DP, E4, GH><<<dim3(grid), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int DP, bool E4>
hipError_t run(const PagedArgs& a, hipStream_t s) {
    if constexpr (DP * (E4 ? 1 : (int)sizeof(T)) <= 128)
        if (a.group_heads == 2) return run<T, DP, E4, 2>(a, s);
    return run<T, DP, E4, 1>(a, s);
}

}  // namespace

template <>
hipError_t launch_paged_rows<PAGED_T, PAGED_E4>(const PagedArgs& a, hipStream_t s) {
    if (a.d <= 64) return run<PAGED_T, 64, PAGED_E4>(a, s);
    if (a.d <= 128) return run<PAGED_T, 128, PAGED_E4>(a, s);
    return run<PAGED_T, 256, PAGED_E4>(a, s);
}

}  // namespace conv2d
