// Device helpers of the paged attention kernels: which rows and keys a
// workgroup takes, where keys lie, the join of divided results.
//
// The rows (new token, head of the group) of a sequence that share a key head
// are cut into tiles of R rows, the keys that a tile's rows see into blocks of
// BU keys: the blocks of the first tokens, then those from the window's first
// key on.  One workgroup takes a (tile, head) whole where there are many; else
// their blocks are divided (Pieces), most simply as one line, tile after tile and
// head after head, cut into equal parts, a workgroup each, whatever the
// sequences' lengths.  (A workgroup may take two heads at once: then "head" is a
// pair of them.)  A (tile, head) that is divided leaves partial results in the
// workspace, two at most a workgroup (one that its part begins with, one that it
// ends with), which a second launch joins.
//
// Lengths and offsets come from the device, so each workgroup of the first launch
// works the division out for itself; together they leave the second one a record of
// each (tile, group of heads).
#pragma once

#include "attention_common.h"
#include "decoder_internal.h"
#include "e4m3.h"

namespace conv2d {

// Tiles and sequences that a divided call may have: four a thread.
constexpr int kPagedTiles = 1024;

struct PagedSeq {
    int first, nq, nk;   // its rows of q from `first` on, its new and all its tokens
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
    PagedSeq s;
    s.first = min(max(a.q_offsets[b], 0), a.tokens);
    s.nq = max(min(max(a.q_offsets[b + 1], 0), a.tokens) - s.first, 0);
    s.nk = min(max(a.kv_lens[b], 0), a.max_pages * (int)a.page_size.d);
    return s;
}

// The kernel's argument, read anew: what is formed from it is formed where it
// is needed.  Otherwise the compiler forms it once, before the first piece, and
// keeps more in scalar registers than there are.  (With one read, 128-row tiles
// of bfloat16 have 190 lane reads for a block of 32 matrix instructions.)
__device__ __forceinline__ const PagedArgs& kernel_args() {
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const PagedArgs*)p;
}

// The new token of a row.
__device__ __forceinline__ int token_of(const PagedArgs& a, int row) { return (int)divu((uint32_t)row, a.group_div); }

// Blocks of BU keys that rows r0 .. r0 + R - 1 of a sequence see.
struct KeyBlocks {
    int ns, w0, n;   // ns from the first key on, then n - ns from block w0 on
    __device__ __forceinline__ int at(int i) const { return i < ns ? i : w0 + i - ns; }
};
template <int R, int BU>
__device__ __forceinline__ KeyBlocks key_blocks(const PagedArgs& a, PagedSeq s, int r0) {
    const int p0 = s.nk - s.nq + token_of(a, r0), p1 = s.nk - s.nq + token_of(a, min(r0 + R, s.nq * a.group) - 1);
    const int hi = min(p1 + 1, s.nk), lo = a.window && p0 >= a.window ? p0 - a.window + 1 : 0;
    KeyBlocks k{0, 0, 0};
    if (hi <= 0) return k;
    if (a.window) k.ns = (min(a.sinks, hi) + BU - 1) / BU;
    k.w0 = max(lo / BU, k.ns);
    k.n = max(k.ns, k.ns + (hi + BU - 1) / BU - k.w0);
    return k;
}

// The keys that a row sees: j < hi and (j >= lo or j < a.sinks).
__device__ __forceinline__ void paged_interval(const PagedArgs& a, PagedSeq s, int i, bool live, int& lo, int& hi) {
    const int p = s.nk - s.nq + i;
    hi = live ? max(p + 1, 0) : 0;   // p < nk
    lo = a.window && p >= a.window ? p - a.window + 1 : 0;
}

// Sums of v over the threads before this one of a workgroup of 256, and over
// all; `part` is read until the next barrier but one.
template <typename N>
__device__ __forceinline__ N sum_before(N v, N& all, N* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    N s = v;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const N o = __shfl_up(s, m, 64);
        if (lane >= m) s += o;
    }
    __syncthreads();
    if (lane == 63) part[wave] = s;
    __syncthreads();
    all = part[0] + part[1] + part[2] + part[3];
    N before = s - v;
    for (int w = 0; w < wave; ++w) before += part[w];
    return before;
}

template <int R>
__device__ __forceinline__ int tiles_of(const PagedArgs& a, int b) {
    return b < a.batch ? (paged_seq(a, b).nq * a.group + R - 1) / R : 0;
}

// The line of blocks of a divided call, in LDS.
struct PagedLine {
    int first[kPagedTiles + 1];   // a sequence's first tile
    int cum[kPagedTiles + 1];     // blocks of one head before a tile
    int part[4];
    int64_t part64[4];
};

// The last i of 0 .. n - 1 with t[i] <= x, t ascending from t[0] <= x.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, F t, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t(mid) <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Whether a tile of n blocks is on the line.
__device__ __forceinline__ bool on_line(const PagedArgs& a, int n) { return n > a.long_blocks; }

// Fills the line; returns the number of tiles.  A tile without keys counts a
// block: its rows are zeros that someone has to write.  Offsets that do not
// ascend may make more tiles than the host has counted: those are left out.
template <int R, int BU, int COST>
__device__ __forceinline__ int make_line(const PagedArgs& a, PagedLine& l) {
    const int tid = threadIdx.x;
    int n[4], sum = 0, all;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        n[i] = min(tiles_of<R>(a, 4 * tid + i), a.tiles);
        sum += n[i];
    }
    int at = sum_before(sum, all, l.part);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        l.first[4 * tid + i] = at;
        at += n[i];
    }
    const int tiles = min(all, a.tiles);
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * tid + i;
        n[i] = 0;
        if (t < tiles) {
            const int b = last_at_most(a.batch, [&](int j) { return l.first[j]; }, t);
            n[i] = max(key_blocks<R, BU>(a, paged_seq(a, b), (t - l.first[b]) * R).n, 1);
            n[i] = on_line(a, n[i]) ? n[i] + COST : 0;
        }
        sum += n[i];
    }
    at = sum_before(sum, all, l.part);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        l.cum[4 * tid + i] = at;
        at += n[i];
    }
    if (tid == 255) l.cum[kPagedTiles] = at;
    __syncthreads();
    return tiles;
}

// Tile i of the call where each is taken whole: its sequence and its place
// among the sequence's tiles; false past the last one.
template <int R>
__device__ __forceinline__ bool find_tile(const PagedArgs& a, int64_t i, int& b, int& t, int64_t* part) {
    __shared__ int found[2];
    const int tid = threadIdx.x;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 1024) {
        int64_t n[4], sum = 0, all;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[j] = tiles_of<R>(a, b0 + 4 * tid + j);
            sum += n[j];
        }
        int64_t at = before + sum_before(sum, all, part);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i >= at && i < at + n[j]) {
                found[0] = b0 + 4 * tid + j;
                found[1] = (int)(i - at);
            }
            at += n[j];
        }
        before += all;
        if (i < before) {
            __syncthreads();
            b = __builtin_amdgcn_readfirstlane(found[0]);
            t = __builtin_amdgcn_readfirstlane(found[1]);
            return true;
        }
    }
    return false;
}

// A line of `all` blocks (all heads) cut into parts: the first block of one, and
// the part that a block lies in.
__device__ __forceinline__ int part_begin(int all, int parts, int w) { return (int)((int64_t)all * w / parts); }
__device__ __forceinline__ int part_of(int all, int parts, int block) {
    return (int)((((int64_t)block + 1) * parts - 1) / all);
}

// The workspace: a record of each (tile, group of heads), then the parts' outputs, R rows
// of d for each head of each of two results, then their (running maximum, sum).
struct PagedRecord {
    int32_t n;             // results to be joined; 0: none
    int32_t slot0, slot1;  // the first one is at slot0, the i-th other at slot1 + step i
    int32_t step;
    int32_t first, rows;   // the tile's first row of q and, of the sequence's rows from it on, those that there are
    int32_t skip;          // rows of the first token that belong to the tile before
    int32_t unused;
};
struct PagedWs {
    PagedRecord* record;
    float* out;
    f32x2* stat;
};
__host__ __device__ __forceinline__ int64_t record_bytes(int64_t tiles, int head_groups) {
    return tiles * head_groups * (int64_t)sizeof(PagedRecord);
}
// Whether each tile's keys can be cut by themselves (Pieces).
__host__ __device__ __forceinline__ bool cut_by_tiles(int batch, int tiles, int head_groups, int parts) {
    return batch <= 64 && tiles <= 64 && tiles * head_groups <= parts;
}
template <int R>
__device__ __forceinline__ PagedWs paged_ws(const PagedArgs& a) {
    PagedWs w;
    w.record = (PagedRecord*)a.ws;
    w.out = (float*)((char*)a.ws + record_bytes(a.tiles, a.head_groups));
    const int results = R > 16 && cut_by_tiles(a.batch, a.tiles, a.head_groups, a.parts) ? a.parts : 2 * a.parts;
    w.stat = (f32x2*)(w.out + (int64_t)results * a.group_heads * R * a.d);
    return w;
}

// The pieces of a workgroup: blocks k0 .. k1 - 1 of a (tile, group of heads).
struct Piece {
    PagedSeq sq;
    int b, t, h;    // sequence, tile of it, group of heads
    int k0, k1;
    int result;     // in the workspace; -1 where the piece is all of its (tile, group)
};

// How keys are divided.
//
// The line is cut into equal parts, a workgroup a part: it may have the end of
// one tile's keys, tiles, and the beginning of another's.  A (tile, group) counts
// COST blocks more than it has: what it costs a workgroup to begin another one.
// (128-row tiles, chunks of prompts and single tokens, by the line: 58.2 us with
// 0, 55.5 with 2, 55.9 with 3; tiles of 16 rows share all of the memory's
// bandwidth, and 0 is best.)
//
// BY_TILES (tiles of 64 and 128 rows), where the workgroups suffice for that:
// each tile's keys are cut by themselves, into equal pieces, a workgroup a piece.
// The workgroups of an XCD then take tiles of the same head whose pieces begin at
// the same keys, and find them in its L2.  (A chunk of 2048 tokens over 32768
// keys: 677 us by the line with 9 in 100 reads found there, 624 with 96.  Tiles of
// 16 rows have no keys in common, and their pieces come out less equal: a token of
// 32 sequences of up to 8192 keys 80.6 us by the line, 82.6 by tiles.)
//
// Where there are many (tile, group)s, only tiles of more than long_blocks are on
// the line: the workgroups behind its parts take one of the others each.
//
// Up to 64 sequences and tiles are kept in the lanes of each wave, a tile a lane:
// no LDS, no barrier, each length and offset read once (a call of a token of 32
// sequences: 3 us less than by way of LDS).
template <int R, int BU, int COST, bool BY_TILES>
struct Pieces {
    PagedSeq sq;              // lane's tile: its sequence,
    int b, t;                 // number and place,
    int n, cuts, cum;         // its blocks, the pieces they are cut into, pieces (the line: blocks) of one head before
    int tiles, begin, end, w;
    int pieces;               // of one head

    static __device__ __forceinline__ bool in_lanes(const PagedArgs& a) {
        return BY_TILES && a.parts ? cut_by_tiles(a.batch, a.tiles, a.head_groups, a.parts)
                                   : a.batch <= 64 && a.tiles <= 64 && a.first_tile == 0;
    }

    static __device__ __forceinline__ int sum_before_lane(int v) {
        const int lane = threadIdx.x & 63;
        int s = v;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int o = __shfl_up(s, m, 64);
            if (lane >= m) s += o;
        }
        return s - v;
    }

    // Cuts each tile's blocks into pieces of T and less, T the least that leaves a
    // head no more than `most` pieces: a lane tries one, each 2^(1/16) of the one
    // before, from what an even division would give on; the last one cuts nothing.
    __device__ __forceinline__ void cut(int most) {
        const int lane = threadIdx.x & 63;
        const int all = __builtin_amdgcn_readlane(sum_before_lane(n) + n, 63);
        const float even = (float)all / (float)most * __builtin_amdgcn_exp2f((float)lane * 0.0625f);
        const float inv = 1.0f / (lane == 63 ? (float)all : ceilf(even));
        const auto of = [](float blocks, float inv) { return fmaxf(ceilf(__builtin_fmaf(blocks, inv, -0x1p-10f)), 1.0f); };
        float sum = 0.0f;
        const int blocks = __builtin_bit_cast(int, (float)n);
#pragma unroll 4
        for (int i = 0; i < tiles; ++i) sum += of(__builtin_bit_cast(float, __builtin_amdgcn_readlane(blocks, i)), inv);
        const int best = (int)__builtin_ctzll(__ballot(sum <= (float)most) | 1ull << 63);
        const float chosen = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, inv), best));
        cuts = lane < tiles ? (int)of((float)n, chosen) : 0;
        cum = sum_before_lane(cuts);
        pieces = __builtin_amdgcn_readlane(cum + cuts, 63);
    }

    // False: nothing to do.
    __device__ __forceinline__ bool start(const PagedArgs& a, PagedLine& l) {
        begin = 0;
        end = 1;
        if (in_lanes(a)) {
            const int lane = threadIdx.x & 63;
            PagedSeq s = paged_seq(a, min(lane, a.batch - 1));
            if (lane >= a.batch) s.nq = 0;
            const int m = min((s.nq * a.group + R - 1) / R, a.tiles), before = sum_before_lane(m);
            tiles = min(__builtin_amdgcn_readlane(before + m, 63), a.tiles);
            b = 0;
#pragma unroll
            for (int m = 32; m; m >>= 1)
                if (__shfl(before, b + m, 64) <= lane) b += m;
            t = lane - __shfl(before, b, 64);
            sq = PagedSeq{__shfl(s.first, b, 64), __shfl(s.nq, b, 64), __shfl(s.nk, b, 64)};
            n = lane < tiles ? max(key_blocks<R, BU>(a, sq, t * R).n, 1) : 0;
        }
        if (blockIdx.x >= (uint32_t)a.parts) return true;
        int blocks;   // of one head
        if (BY_TILES && in_lanes(a)) {
            cut(a.parts / a.head_groups);
            keep(a, l, 0, 0);
            const int all = pieces * a.head_groups;
            w = (int)xcd_remap(blockIdx.x, (uint32_t)all);
            return (int)blockIdx.x < all;
        } else if (in_lanes(a)) {
            const int mine = on_line(a, n) ? n + COST : 0;
            cum = sum_before_lane(mine);
            blocks = __builtin_amdgcn_readlane(cum + mine, 63);
        } else {
            tiles = make_line<R, BU, COST>(a, l);
            blocks = l.cum[tiles];
        }
        const int all = blocks * a.head_groups, least = max(a.long_blocks / 2, 1);   // blocks of a part
        const int parts = max(min(a.parts, (all + least - 1) / least), 1);
        keep(a, l, all, parts);
        w = (int)xcd_remap(blockIdx.x, (uint32_t)parts);
        begin = __builtin_amdgcn_readfirstlane(part_begin(all, parts, w));
        end = __builtin_amdgcn_readfirstlane(part_begin(all, parts, w + 1));
        return (int)blockIdx.x < parts;
    }

    // Leaves records for the join: those of every a.parts-th (tile, head), a thread
    // each.
    __device__ __forceinline__ void keep(const PagedArgs& a, const PagedLine& l, int all, int parts) {
        const int j = (int)(blockIdx.x + threadIdx.x * (uint32_t)a.parts), units = a.tiles * a.head_groups;
        const int i = j / a.head_groups, h = j - i * a.head_groups;
        if (threadIdx.x >= 64 && !a.long_blocks) return;   // fewer suffice
        PagedRecord r{};
        PagedSeq s{};
        int place = 0, blocks = 0, c = 0;
        if (in_lanes(a)) {
            const int from = min(i, 63);
            s = PagedSeq{__shfl(sq.first, from, 64), __shfl(sq.nq, from, 64), 0};
            place = __shfl(t, from, 64);
            blocks = __shfl(n, from, 64);
            c = __shfl(cum, from, 64);
            if (BY_TILES) r.n = __shfl(cuts, from, 64);   // none past the last tile
        } else if (i < tiles) {
            const int k = last_at_most(a.batch, [&](int m) { return l.first[m]; }, i);
            s = paged_seq(a, k);
            place = i - l.first[k];
            c = l.cum[i];
            blocks = l.cum[i + 1] - c - COST;
        }
        if (BY_TILES && in_lanes(a)) {
            r.slot0 = r.slot1 = h * pieces + c;
            r.step = 1;
        } else if (i < tiles && on_line(a, blocks)) {
            const int from = c * a.head_groups + h * (blocks + COST);
            const int p0 = part_of(all, parts, from + COST), p1 = part_of(all, parts, from + COST + blocks - 1);
            r.n = p1 - p0 + 1;
            r.slot0 = 2 * p0 + (part_begin(all, parts, p0) < from);
            r.slot1 = 2 * p0;
            r.step = 2;
        }
        if (j >= units) return;
        if (r.n == 1) r.n = 0;   // written whole
        const int token = token_of(a, place * R);
        r.first = s.first + token;
        r.skip = place * R - token * a.group;
        r.rows = s.nq * a.group - place * R;
        paged_ws<R>(a).record[j] = r;
    }

    __device__ __forceinline__ void from_lanes(int i, Piece& p) {
        p.b = __builtin_amdgcn_readlane(b, i);
        p.t = __builtin_amdgcn_readlane(t, i);
        p.sq = PagedSeq{__builtin_amdgcn_readlane(sq.first, i), __builtin_amdgcn_readlane(sq.nq, i),
                        __builtin_amdgcn_readlane(sq.nk, i)};
    }

    // The piece at `u` (begin at first), and where the next one is.
    __device__ __forceinline__ bool next(const PagedArgs& a, PagedLine& l, int& u, Piece& p) {
        if (u >= end) return false;
        if (blockIdx.x >= (uint32_t)a.parts) {
            // A sequence's last tiles first: they see the most keys.
            const int64_t i = (int64_t)a.first_tile + (gridDim.x - 1 - blockIdx.x) / (uint32_t)a.head_groups;
            p.h = (int)((blockIdx.x - (uint32_t)a.parts) % (uint32_t)a.head_groups);
            if (in_lanes(a)) {
                if (i >= tiles) return false;
                from_lanes((int)i, p);
            } else {
                if (!find_tile<R>(a, i, p.b, p.t, l.part64)) return false;
                p.sq = paged_seq(a, p.b);
            }
            p.k0 = 0;
            p.k1 = key_blocks<R, BU>(a, p.sq, p.t * R).n;
            p.result = -1;
            u = end;
            return a.parts == 0 || !on_line(a, p.k1);
        }
        const int heads = a.head_groups, lane = threadIdx.x & 63;
        if (BY_TILES && in_lanes(a)) {
            p.h = w / pieces;
            const int at = w - p.h * pieces, i = __builtin_popcountll(__ballot(lane < tiles && cum <= at)) - 1;
            from_lanes(i, p);
            const int of = __builtin_amdgcn_readlane(cuts, i), k = at - __builtin_amdgcn_readlane(cum, i);
            const int blocks = __builtin_amdgcn_readlane(n, i), size = blocks / of, rest = blocks - size * of;
            p.k0 = size * k + min(k, rest);
            p.k1 = p.k0 + size + (k < rest);
            p.result = of == 1 ? -1 : w;
            u = end;
            return true;
        }
        int c, blocks;
        if (in_lanes(a)) {
            const int i = __builtin_popcountll(__ballot(lane < tiles && cum * heads <= u)) - 1;
            from_lanes(i, p);
            c = __builtin_amdgcn_readlane(cum, i);
            blocks = __builtin_amdgcn_readlane(n, i);
        } else {
            const int i = __builtin_amdgcn_readfirstlane(last_at_most(tiles, [&](int j) { return l.cum[j] * heads; }, u));
            c = __builtin_amdgcn_readfirstlane(l.cum[i]);
            blocks = __builtin_amdgcn_readfirstlane(l.cum[i + 1]) - c - COST;
            p.b = __builtin_amdgcn_readfirstlane(last_at_most(a.batch, [&](int j) { return l.first[j]; }, i));
            p.t = i - __builtin_amdgcn_readfirstlane(l.first[p.b]);
            p.sq = paged_seq(a, p.b);
        }
        p.h = (u - c * heads) / (blocks + COST);
        const int at = u - c * heads - p.h * (blocks + COST), size = min(blocks + COST - at, end - u);
        p.k0 = max(at - COST, 0);
        p.k1 = at + size - COST;
        p.result = p.k0 == 0 && p.k1 == blocks ? -1 : 2 * w + (u != begin);
        u += size;
        return p.k1 > 0;   // or the part ends before the first block
    }
};

__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_ds_bpermute(lane * 4, (int)v);
}

// Where this lane's key of a tile lies.
struct KeyPlace {
    uint32_t k, v, s;   // units from a head's first page; bytes for scales
    bool there;         // before nk, on a page of the cache
};
// Entry of the page table for a key (any number), to be read well before place().
__device__ __forceinline__ int page_entry(const PagedArgs& a, const int32_t* table, int key) {
    const int n = (int)divu((uint32_t)key, a.page_size);
    return table[min(n, a.max_pages - 1)];
}
__device__ __forceinline__ KeyPlace key_place(const PagedArgs& a, int entry, int key, int nk) {
    const uint32_t token = (uint32_t)key - divu((uint32_t)key, a.page_size) * a.page_size.d;
    KeyPlace p;
    p.there = key < nk && (uint32_t)entry < (uint32_t)a.n_pages;
    const uint32_t page = p.there ? (uint32_t)entry : 0, tok = p.there ? token : 0;
    p.k = page * a.k_u.page + tok * a.k_u.token;
    p.v = page * a.v_u.page + tok * a.v_u.token;
    p.s = page * a.s_u.page + tok * a.s_u.token;
    return p;
}

// One element of a key's value, for the few that need it alone.
template <typename T, bool E4>
__device__ __forceinline__ float value_at(const PagedArgs& a, const int32_t* table, int h, int key, int e) {
    const KeyPlace p = key_place(a, page_entry(a, table, key), key, INT32_MAX);
    const char* row = (const char*)a.v + (uint64_t)p.v * 16 + h * a.v_head;
    if (E4) return decode1(((const uint8_t*)row)[e], scale_value(a.vs[p.s + h * a.s_head]));
    return to_f32(((const T*)row)[e]);
}

// 16 bits of a weight are two numbers of bf16: what one holds of it, cut off, and
// the rest, rounded.  Both are above zero where the weight is (the rest has 2^-20
// of it more), or a seen infinity would meet a zero or both signs and become NaN.
__device__ __forceinline__ float weight_part(float w, bool rest) {
    const float cut = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, w) & 0xffff0000u);
    return rest ? __builtin_fmaf(w, 0x1p-20f, w - cut) : cut;
}

// Few rows a tile (paged_rows.h) or 64 or 128 (paged_tile.h).
template <typename T, bool E4>
hipError_t launch_paged_rows(const PagedArgs& a, hipStream_t s);
template <typename T, bool E4>
hipError_t launch_paged_tile(const PagedArgs& a, int rows, hipStream_t s);
#define CONV2D_PAGED_LAUNCHES(T, E4)                                 \
    template <>                                                      \
    hipError_t launch_paged_rows<T, E4>(const PagedArgs& a, hipStream_t s); \
    template <>                                                      \
    hipError_t launch_paged_tile<T, E4>(const PagedArgs& a, int rows, hipStream_t s);
CONV2D_PAGED_LAUNCHES(float, false)
CONV2D_PAGED_LAUNCHES(float, true)
CONV2D_PAGED_LAUNCHES(bf16, false)
CONV2D_PAGED_LAUNCHES(bf16, true)
#undef CONV2D_PAGED_LAUNCHES

}  // namespace conv2d
