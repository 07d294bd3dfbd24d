// Internal declarations shared by the ABI layer of include/decoder.h and its
// kernels.
#pragma once

#include "../../include/decoder.h"
#include "attention_internal.h"

namespace conv2d {

// ----------------------------------------------------------- kv_cache ----

// Pages of keys or values, or of their scales.
struct PageStrides {
    int64_t page, token, head;   // elements
};

struct KvArgs {
    const void* k;               // dense rows: kv_cache_load writes them
    const void* v;
    const void* k_pages;         // kv_cache_store writes these
    const void* v_pages;
    const uint8_t* k_scales;     // null unless E4M3
    const uint8_t* v_scales;
    const int32_t* slots;        // store
    const int32_t* page_table;   // load
    const int32_t* kv_lens;      // load; null: all rows
    int64_t k_s, v_s;            // token strides of k and v
    int64_t k_bs, v_bs;          // their sequence strides (load)
    PageStrides ks, vs, ss;
    int32_t tokens;              // store
    int32_t batch, kv_len, max_pages;   // load
    int32_t n_pages, heads, d;
    DivU32 page_size;
};

// vec: every row of 8 elements starts at a boundary of its own size.
hipError_t launch_kv_store(int32_t dtype, bool e4m3, bool vec, const KvArgs& a, hipStream_t s);
hipError_t launch_kv_load(int32_t dtype, bool e4m3, bool vec, const KvArgs& a, hipStream_t s);

// ---------------------------------------------------- paged attention ----

// Strides of pages in units of 16 bytes, modulo 2^32: a page's and token's place
// is formed in 32 bits, since pages reach less far.
struct PageUnits {
    uint32_t page, token;
};

struct PagedArgs {
    const void* q;
    const void* k;               // pages
    const void* v;
    const uint8_t* ks;           // scales, null unless E4M3
    const uint8_t* vs;
    void* out;
    const int32_t* q_offsets;
    const int32_t* kv_lens;
    const int32_t* page_table;
    void* ws;                    // null when parts == 0
    int64_t q_s, o_s;            // token strides
    int64_t k_head, v_head;      // head strides of the pages, bytes
    PageUnits k_u, v_u, s_u;     // s_u in bytes
    int64_t s_head;
    int32_t tokens, batch, max_pages, n_pages;
    int32_t heads_q, heads_kv, group, d;
    int32_t window, sinks;
    DivU32 page_size, group_div;
    int32_t group_heads, head_groups;   // key heads that a workgroup takes at once, and how many such groups there are
    int32_t tiles;               // row tiles of all sequences, at most
    int32_t first_tile;          // of this launch, where parts == 0
    int32_t parts;               // workgroups that the keys of all tiles are divided among, at most; 0: one a tile and head
    int32_t long_blocks;         // > 0: the keys of tiles of more blocks are, and the others have one a tile and head too
    float scale, softcap;
};

// Workgroups and workspace that a call of these sizes runs with.
struct PagedPlan {
    int32_t rows;                // of a tile: 16, 64 or 128
    int32_t group_heads;
    int32_t tiles, parts, long_blocks;
    int64_t ws_bytes;
};

PagedPlan plan_paged_attention(int32_t dtype, bool e4m3, const PagedArgs& a);
hipError_t launch_paged_attention(int32_t dtype, bool e4m3, const PagedPlan& p, const PagedArgs& a, hipStream_t s);

// --------------------------------------------------------- block norm ----

constexpr int32_t NORM_MAX_WIDTH = 32768;   // a row fits in LDS in fp32

struct NormArgs {
    const void* y;
    const void* x;
    const void* gate;            // null without
    const float* post_gamma;     // null without the norm
    const float* post_beta;      // null without
    const float* pre_gamma;
    const float* pre_beta;
    void* residual;
    void* out;
    int64_t y_s, x_s, r_s, o_s, g_s;
    int32_t rows, width, post, pre;
    DivU32 gate_rows;            // of a gate row; d == 0: one gate row
    float residual_scale, block_scale, eps;
};

// vec: every row starts at a 16-byte boundary, of a multiple of 8 elements.
hipError_t launch_block_norm(int32_t dtype, bool vec, const NormArgs& a, hipStream_t s);

}  // namespace conv2d
