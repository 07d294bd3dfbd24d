// Attention of many rows over pages: chunks of prompts.  Compiled once for each
// type and cache (paged_tile_*.hip).
#pragma once

#include "attention_layout.h"
#include "linear_common.h"
#include "paged_common.h"

namespace conv2d {

namespace {

// The sum of lane l's and lane l ^ 16's.
__device__ __forceinline__ float both_rows(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x),
                                                    false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// attention_tile's work on pages: a workgroup of four waves takes 128 of the
// rows (new token, head of the group) that share a key head, or 64 with two
// waves a row group (KW = 2), and walks blocks of 64 keys (fp32: 32 or 64).
// Both products are transposed, S^T = K Q^T and O^T = V^T P^T, in 32x32 steps; a
// lane keeps the scores of one row; the running maximum is moved only when it
// rises by more than 8; bf16 weights are rounded before their product, but for
// sequences of up to 16 rows.
//
// A lane looks up the page of one key of a block, a block ahead, and forms its
// place; the threads that copy a key's row get it by exchange.  Pages of T go
// straight to LDS, the next block's while one is computed.  Codes come through
// registers, two blocks ahead, and are elements of T times their scale when they
// reach LDS: what reads them there is the same.
template <typename T, int DP, int KW, bool E4>
struct PagedTile : TileAttn<T, DP, KW> {
    typedef TileAttn<T, DP, KW> L;
    static constexpr int R = 32 * L::RG, S = 2, OCC = L::STAGE <= 1024 ? 3 : L::STAGE <= 2048 ? 2 : 1;
    typedef typename std::conditional<E4, typename Codes<T>::type, int>::type Code;
    static constexpr int N = E4 ? L::CP : 1;
    Code k[N], v[N];           // E4: this thread's chunks of the block that comes next
    uint32_t ks, vs;           // scales of this lane's key
};

template <typename T, int DP, int KW, int CAP, bool E4>
__global__ __launch_bounds__(256, (PagedTile<T, DP, KW, E4>::OCC)) void paged_tile(PagedArgs) {
    const PagedArgs& a = kernel_args();
    typedef PagedTile<T, DP, KW, E4> P;
    typedef TileAttn<T, DP, KW> C;
    constexpr bool HALF = C::HALF;
    constexpr int BK = C::BK, TK = C::TK, CPR = C::CPR, KS = C::KS, DT = C::DT, CP = C::CP, R = P::R;
    // A score x follows from what its register holds, u: PLAIN, x = scale u;
    // TURNED, x = cap (1 - 2 u); else x = u.
    constexpr bool PLAIN = !CAP, TURNED = CAP == kCapTurned;
    constexpr bool SIGNED = HALF && DP > 128;   // how a weight's two parts are told apart, see walk
    __shared__ __align__(1024) u32x4 lds[P::S * C::STAGE];
    __shared__ PagedLine line;
    // The last even and odd block that held infinities or NaN.
    __shared__ int lbad[2];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, g = lane >> 5, kpart = wave / C::RG;
    const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
    // A negative scale goes into Q's signs, and one of zero makes Q zero: a
    // masked score, -inf, is multiplied by the scale later (PLAIN).
    const bool flat = a.scale == 0.0f;
    const float scale = flat ? 1.0f : fabsf(a.scale) * kLog2e;
    const float cap = CAP == kCapTurned ? a.softcap * kLog2e : a.softcap;
    const float tscale = CAP == kCapTurned ? fminf(fabsf(a.scale) / a.softcap * (2.0f * kLog2e), FLT_MAX)
                         : CAP             ? cap_scale(fabsf(a.scale), a.softcap)
                                           : 0.0f;
    Pieces<R, BK, 2, true> pieces;
    Piece pc;
    if (!pieces.start(a, line)) return;
    int u = pieces.begin;
    while (pieces.next(kernel_args(), line, u, pc)) {
        const PagedArgs& a = kernel_args();
        const int chunks = a.d / C::C;
        const int h = pc.h, first = pc.k0;
        int last = pc.k1;
        const PagedSeq sq = pc.sq;
        const int32_t* table = a.page_table + (int64_t)pc.b * a.max_pages;
        const KeyBlocks blocks = key_blocks<R, BK>(a, sq, pc.t * R);
        if (blocks.n == 0) last = first;   // no row sees a key
        const int rows = sq.nq * a.group;
        // A sequence of so few rows keeps 16 bits of its weights, as in paged_rows,
        // whatever else is in the batch: lanes 16 .. 31 take rows 0 .. 15 again, with
        // the weights' second parts, and add their outputs at the end.
        const bool fine = HALF && rows <= 16;

        // This lane's row; keys that some and that all rows of the wave see
        // (first tokens apart), and those that all of the workgroup see.
        const int row = pc.t * R + wave % C::RG * 32 + (fine ? n & 15 : n);
        const bool live = row < rows;
        const int qi = live ? token_of(a, row) : 0, hq = h * a.group + (live ? row - qi * a.group : 0);
        int lo, hi, w_lo, w_hi, f_lo, f_hi, all_lo, all_hi, unused;
        paged_interval(a, sq, qi, live, lo, hi);
        {
            const int r0 = pc.t * R, rw = r0 + wave % C::RG * 32;
            const auto token = [&](int r) { return __builtin_amdgcn_readfirstlane(token_of(a, min(r, rows - 1))); };
            paged_interval(a, sq, token(rw), rw < rows, w_lo, f_hi);
            paged_interval(a, sq, token(rw + 31), rw < rows, f_lo, w_hi);
            paged_interval(a, sq, token(r0), true, unused, all_hi);
            paged_interval(a, sq, token(r0 + R - 1), true, all_lo, unused);
        }
        __syncthreads();   // the last piece's reads of LDS are over
        if (tid < 2) lbad[tid] = -1;
        if (a.d < DP)   // chunks past d stay zero: no copy touches them
            for (int i = tid; i < P::S * C::STAGE; i += 256) {
                const int r = i / CPR % BK;
                if (((i % CPR) ^ C::swizzle(r)) >= chunks) lds[i] = u32x4{0, 0, 0, 0};
            }
        u32x4 fq[KS];   // the products' second operand
        {
            const T* qp = (const T*)a.q + (int64_t)(sq.first + qi) * a.q_s + (int64_t)hq * a.d;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int e = (2 * s + g) * C::C;
                fq[s] = u32x4{0, 0, 0, 0};
                if (live && e < a.d && !flat) fq[s] = *(const u32x4*)(qp + e);
                if (a.scale < 0.0f) fq[s] ^= HALF ? 0x80008000u : 0x80000000u;
            }
        }

        const auto key0 = [&](int i) { return blocks.at(i) * BK; };
        const auto look = [&](int i) { return i < last ? page_entry(a, table, key0(i) + (lane & (BK - 1))) : 0; };
        // Keys of a block that there are, or that lie past the last one (no row
        // sees those).
        const auto on_pages = [&](int i, KeyPlace p) {
            const uint64_t m = __ballot(p.there || key0(i) + (lane & (BK - 1)) >= sq.nk);
            return BK == 64 ? m : m | 0xffffffff00000000ull;
        };
        const char *kb = (const char*)a.k + h * a.k_head, *vb = (const char*)a.v + h * a.v_head;
        const auto mixed = [&](int i, uint64_t there) {
            const int k0 = key0(i);
            return k0 + BK > all_hi || (k0 < all_lo && k0 + BK > a.sinks) || ~there != 0;
        };
        // Copies: chunks of rows tid / CPR + i * (256 / CPR) of a block.
        const auto issue = [&](KeyPlace p, int stage) {
            u32x4* dst = lds + stage * C::STAGE + wave * 64;
            int r0 = tid / CPR;
            asm volatile("" : "+v"(r0));   // the places are formed anew for each block: they would cost registers
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                const int r = r0 + i * (256 / CPR), c = (tid % CPR) ^ C::swizzle(r);
                const uint32_t pk = from_lane(p.k, r), pv = from_lane(p.v, r);
                if (c < chunks) {
                    copy16_to_lds(kb + (uint64_t)pk * 16 + c * 16, dst + i * 256);
                    copy16_to_lds(vb + (uint64_t)pv * 16 + c * 16, dst + BK * CPR + i * 256);
                }
            }
        };
        P f;
        const auto fetch = [&](KeyPlace p) {
            if constexpr (E4) {
                f.ks = a.ks[p.s + h * a.s_head];
                f.vs = a.vs[p.s + h * a.s_head];
                int r0 = tid / CPR;
                asm volatile("" : "+v"(r0));   // likewise
#pragma unroll
                for (int i = 0; i < CP; ++i) {
                    const int r = r0 + i * (256 / CPR), c = (tid % CPR) ^ C::swizzle(r);
                    const uint32_t pk = from_lane(p.k, r), pv = from_lane(p.v, r);
                    if (c < chunks) {
                        f.k[i] = *(const typename P::Code*)(kb + (uint64_t)pk * 16 + c * C::C);
                        f.v[i] = *(const typename P::Code*)(vb + (uint64_t)pv * 16 + c * C::C);
                    }
                }
            }
        };
        // A chunk of V of block i, whose infinities and NaN some row may not see.
        const auto cleaned = [&](u32x4 v, int i) {
            if (has_bad<T>(v)) {
                clean_chunk<T>(v);
                lbad[i & 1] = i;
            }
            return v;
        };
        const auto commit = [&](int i, uint64_t there, int stage) {
            if constexpr (E4) {
                const bool search = mixed(i, there);
                int r0 = tid / CPR;
                asm volatile("" : "+v"(r0));   // likewise
#pragma unroll
                for (int j = 0; j < CP; ++j) {
                    const int r = r0 + j * (256 / CPR), c = (tid % CPR) ^ C::swizzle(r);
                    const float sk = scale_value(from_lane(f.ks, r)), sv = scale_value(from_lane(f.vs, r));
                    if (c < chunks) {
                        u32x4* dst = lds + stage * C::STAGE + j * 256 + tid;
                        dst[0] = decode(f.k[j], sk, T{});
                        u32x4 v = decode(f.v[j], sv, T{});
                        if (search) v = cleaned(v, i);
                        dst[BK * CPR] = v;
                    }
                }
            }
        };

        f32x16 o[DT] = {};
        float m_run = -INFINITY, l_run = 0.0f;
        uint64_t there = ~0ull, there1 = ~0ull, there2 = ~0ull;   // of the block at hand, the next one, the one after
        int entry = look(first);
        const auto place = [&](int i, uint64_t& on) {
            const KeyPlace p = key_place(a, entry, key0(i) + (lane & (BK - 1)), sq.nk);
            on = on_pages(i, p);
            entry = look(i + 1);
            return p;
        };
        if (first < last) {
            KeyPlace p = place(first, there);
            if constexpr (E4) {
                fetch(p);
                __syncthreads();   // lbad is set
                commit(first, there, 0);
                if (first + 1 < last) {
                    p = place(first + 1, there1);
                    fetch(p);
                }
            } else {
                issue(p, 0);
            }
        }
        // The blocks.  One loop for weights of one part and one for two: with a branch
        // in the loop exponentials and products do not overlap across it (chunks
        // among single tokens 58.4 us, 56.2 with two loops, 55.2 all of one part; under a
        // window 40.8, 39.1, 38.6).
        //
        // SIGNED: two loops need more registers than 256 wide heads leave.  One
        // expression forms a weight, the first part's negative or the second part
        // (1024 tokens over 16384 keys of 16 heads over 4, E4M3: 653 us, 640 without
        // parts, 725 with two loops, 867 with a branch; bf16: 489, 470, 504, 482).
        const auto walk = [&](auto parts) {
            for (int i = first, stage = 0; i < last; ++i, stage ^= 1) {
                const int k0 = key0(i);
                // The wave's part of the block.
                const int kw = k0 + kpart * 32 * TK;
                const uint32_t at0 = lds0 + (stage * C::STAGE + kpart * 32 * TK * CPR) * 16;
                uint32_t k_at = at0 + C::k_at(lane), v_at = at0 + C::v_at(lane);
                asm volatile("" : "+v"(k_at), "+v"(v_at));   // likewise
                const bool search = mixed(i, there);
                if constexpr (!E4) {
                    wait_vmem<0>();   // this block's copies have landed
                    if (search) {
                        // This thread's own chunks of V.
                        if (i == first) __syncthreads();   // lbad is set
#pragma unroll
                        for (int j = 0; j < CP; ++j) {
                            const int r = tid / CPR + j * (256 / CPR);
                            u32x4& chunk = lds[stage * C::STAGE + BK * CPR + j * 256 + tid];
                            if (((tid % CPR) ^ C::swizzle(r)) < chunks) chunk = cleaned(chunk, i);
                        }
                    }
                }
                __syncthreads();
                const uint64_t now = there;
                if constexpr (E4) {
                    if (i + 1 < last) commit(i + 1, there1, stage ^ 1);
                    there = there1;
                    if (i + 2 < last) {
                        const KeyPlace p = place(i + 2, there2);
                        fetch(p);
                        there1 = there2;
                    }
                } else if (i + 1 < last) {
                    const KeyPlace p = place(i + 1, there);
                    issue(p, stage ^ 1);
                }
                if (kw >= w_hi || (kw + 32 * TK <= w_lo && kw >= a.sinks)) continue;   // none of the wave's rows sees a key

                f32x16 s[TK] = {};
#pragma unroll
                for (int t = 0; t < TK; ++t)
#pragma unroll
                    for (int j = 0; j < KS; ++j)
                        s[t] = mfma32_step<T>(*lds_ptr<const lds_u32x4>((k_at ^ 32 * j) + t * 512 * CPR), fq[j], s[t]);
                const float a1 = PLAIN ? scale : TURNED ? -2.0f * cap : 1.0f, a0 = TURNED ? cap : 0.0f;
                if (CAP) {
#pragma unroll
                    for (int t = 0; t < TK; ++t)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            s[t][j] = TURNED ? turned(s[t][j] * tscale) : cap * score_tanh<T>(s[t][j] * tscale) * kLog2e;
                }
                // Keys before and past what a row sees, and on no page, each where
                // some row needs it.  Score register j holds key 32 (j / 16) +
                // 8 (j / 4 % 4) + j % 4 from 4 g on.
                constexpr float NEVER = TURNED ? INFINITY : -INFINITY;
                const auto key = [](int j) { return 32 * (j >> 4) + 8 * (j >> 2 & 3) + (j & 3); };
                if (kw < f_lo && kw + 32 * TK > a.sinks) {
                    const int from = lo - kw - 4 * g, kept = a.sinks - kw - 4 * g;
#pragma unroll
                    for (int j = 0; j < 16 * TK; ++j)
                        if (key(j) < from && key(j) >= kept) s[j >> 4][j & 15] = NEVER;
                }
                if (kw + 32 * TK > f_hi) {
                    const int to = hi - kw - 4 * g;
#pragma unroll
                    for (int j = 0; j < 16 * TK; ++j)
                        if (key(j) >= to) s[j >> 4][j & 15] = NEVER;
                }
                if (~now != 0) {
                    const uint64_t mine = now >> (kpart * 32 * TK + 4 * g);
#pragma unroll
                    for (int j = 0; j < 16 * TK; ++j)
                        if (!(mine >> key(j) & 1)) s[j >> 4][j & 15] = NEVER;
                }
                float top = s[0][0];
#pragma unroll
                for (int j = 1; j < 16 * TK; ++j) {
                    const float x = s[j >> 4][j & 15];
                    top = TURNED ? fminf(top, x) : fmaxf(top, x);
                }
                {
                    float u, v;
                    both_halves(top, u, v);
                    top = (TURNED ? fminf(u, v) : fmaxf(u, v)) * a1 + a0;
                }
                if (__ballot(top > m_run + 8.0f)) {
                    const float m_new = fmaxf(m_run, top);
                    const float fade = __builtin_amdgcn_exp2f(m_run - (m_new == -INFINITY ? 0.0f : m_new));
                    m_run = m_new;
                    l_run *= fade;
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] *= fade;
                }
                const float base = a0 - (m_run == -INFINITY ? 0.0f : m_run);   // nothing seen yet: every weight is 0
#pragma unroll
                for (int t = 0; t < TK; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        s[t][j] = __builtin_amdgcn_exp2f(s[t][j] * a1 + base);
                        l_run += s[t][j];
                    }
                if constexpr (SIGNED) {
                    // w, or -(w cut off) in lanes 0 .. 15 and the rest of w in 16 .. 31.
                    const float keep = !parts ? 1.0f : n & 16 ? 1.0f + 0x1p-20f : 0.0f;
                    const uint32_t mask = parts ? 0xffff0000u : 0u;
#pragma unroll
                    for (int t = 0; t < TK; ++t)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float w = s[t][j];
                            s[t][j] = __builtin_fmaf(w, keep, -__builtin_bit_cast(float, __builtin_bit_cast(uint32_t, w) & mask));
                        }
                } else if (HALF && parts) {
#pragma unroll
                    for (int t = 0; t < TK; ++t)
#pragma unroll
                        for (int j = 0; j < 16; ++j) s[t][j] = weight_part(s[t][j], n & 16);
                }
                if constexpr (HALF) {
                    bf16x8 p[2 * TK];
#pragma unroll
                    for (int t = 0; t < 2 * TK; ++t)
#pragma unroll
                        for (int j = 0; j < 8; ++j) p[t][j] = (bf16)s[t >> 1][8 * (t & 1) + j];
#pragma unroll
                    for (int t = 0; t < 2 * TK; ++t)
#pragma unroll
                        for (int d = 0; d < DT; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(C::vt(v_at, 16 * t, 32 * d), p[t], o[d], 0, 0, 0);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
#pragma unroll
                        for (int d = 0; d < DT; ++d)
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(C::vt1(v_at, j, 32 * d), s[0][j], o[d], 0, 0, 0);
                }
                if (search && lbad[i & 1] == i) {
#pragma unroll 1
                    for (int j = 0; j < 32 * TK; ++j) {
                        if (kw + j >= sq.nk || !(now >> (kpart * 32 * TK + j) & 1)) continue;
                        bool add = kw + j < hi && (kw + j >= lo || kw + j < a.sinks);
                        if (SIGNED && fine && n < 16) add = false;   // the second part's lanes do
#pragma unroll 1
                        for (int e0 = 0; e0 < a.d; e0 += 64) {
                            const float x = e0 + lane < a.d ? value_at<T, E4>(a, table, h, kw + j, e0 + lane) : 0.0f;
                            for (uint64_t bad = __ballot(!(fabsf(x) < INFINITY)); bad; bad &= bad - 1) {
                                const int l = (int)__builtin_ctzll(bad);
                                const float y = __shfl(x, l, 64);
                                int at = e0 + l - 4 * g;
                                asm volatile("" : "+v"(at));   // no comparison is kept in registers across the blocks
#pragma unroll
                                for (int d = 0; d < DT; ++d)
#pragma unroll
                                    for (int q = 0; q < 16; ++q) o[d][q] += add && 32 * d + 8 * (q >> 2) + (q & 3) == at ? y : 0.0f;
                            }
                        }
                    }
                }
            }
        };
        if constexpr (HALF && !SIGNED) {
            if (fine)
                walk(std::true_type{});
            else
                walk(std::false_type{});
        } else {
            walk(fine);
        }
        {
            float u, v;
            both_halves(l_run, u, v);
            l_run = u + v;
        }
        if constexpr (KW == 2) {
            // The second half of the keys' results go to the first's waves.
            f32x4* part = (f32x4*)lds + wave % C::RG * (DT * 256);
            __shared__ f32x2 stat[C::RG][64];
            __syncthreads();
            if (kpart == 1) {
                stat[wave % C::RG][lane] = f32x2{m_run, l_run};
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        part[(4 * d + q) * 64 + lane] = f32x4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
            }
            __syncthreads();
            if (kpart == 1) continue;
            const f32x2 st = stat[wave][lane];
            const float m_new = fmaxf(m_run, st[0]), base = m_new == -INFINITY ? 0.0f : m_new;
            const float f0 = __builtin_amdgcn_exp2f(m_run - base), f1 = __builtin_amdgcn_exp2f(st[0] - base);
            m_run = m_new;
            l_run = l_run * f0 + st[1] * f1;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v = part[(4 * d + q) * 64 + lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[d][4 * q + j] = o[d][4 * q + j] * f0 + v[j] * f1;
                }
        }
        if (fine) {
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int q = 0; q < 16; ++q) o[d][q] = both_rows(SIGNED && n < 16 ? -o[d][q] : o[d][q]);
        }
        if (!live || (fine && n >= 16)) continue;
        const PagedArgs& end = kernel_args();
        const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
        T* op = (T*)end.out + (int64_t)(sq.first + qi) * end.o_s + (int64_t)hq * end.d;
        const int64_t wr = (int64_t)pc.result * R + row - pc.t * R;
        const PagedWs ws = paged_ws<R>(end);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int e = 32 * d + 8 * q + 4 * g;
                const f32x4 v{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
                if (e >= end.d) continue;
                if (pc.result < 0)
                    *(typename Vec<T>::v4*)(op + e) = from_f32<T>(v * inv);
                else
                    *(f32x4*)(ws.out + wr * end.d + e) = v;
            }
        if (pc.result >= 0 && g == 0) ws.stat[wr] = f32x2{m_run, l_run};
    }
}

template <typename T, int DP, int KW, bool E4>
hipError_t run(const PagedArgs& a, hipStream_t s) {
    const dim3 grid(a.parts ? (uint32_t)a.parts : (uint32_t)a.tiles * (uint32_t)a.head_groups), block(256);
    if (a.softcap == 0.0f)
        paged_tile<T, DP, KW, kCapNone, E4><<<grid, block, 0, s>>>(a);
    else if (sizeof(T) == 4 || a.softcap > kMostTurned)
        paged_tile<T, DP, KW, kCapAny, E4><<<grid, block, 0, s>>>(a);
    else if constexpr (sizeof(T) == 2)
        paged_tile<T, DP, KW, kCapTurned, E4><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T, int KW, bool E4>
hipError_t run(const PagedArgs& a, hipStream_t s) {
    if (a.d <= 64) return run<T, 64, KW, E4>(a, s);
    if (a.d <= 96) return run<T, 96, KW, E4>(a, s);
    if (a.d <= 128) return run<T, 128, KW, E4>(a, s);
    if constexpr (KW == 1 || sizeof(T) == 2) return run<T, 256, KW, E4>(a, s);
    return hipErrorInvalidValue;   // two stages of 64 fp32 keys do not fit in LDS: the plan takes 128 rows
}

}  // namespace

template <>
hipError_t launch_paged_tile<PAGED_T, PAGED_E4>(const PagedArgs& a, int rows, hipStream_t s) {
    return rows == 128 ? run<PAGED_T, 1, PAGED_E4>(a, s) : run<PAGED_T, 2, PAGED_E4>(a, s);
}

}  // namespace conv2d
