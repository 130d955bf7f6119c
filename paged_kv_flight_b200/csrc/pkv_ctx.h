// pkv_ctx.h -- the library context and the host-side checks and TMA map
// encoding that its entry points share (pkv_api.cu, tree_api.cu).  Not part
// of the ABI.
#pragma once

#include "pkv_internal.h"

struct pkv_ctx {
    pkv_config cfg;
    int device;
    int num_sms;
    int G;
    pkv::AttnLaunch attn;
    pkv::AttnLaunch attn_tok;     // several new tokens per request
    int workers;
    int tail_chunks;      // largest number of dynamic tail chunks per warp range
    void* ws;             // one allocation, carved below
    size_t ws_bytes;
    int* d_err;
    int* d_claim;         // chunk counter of the attention's dynamic tail
    double* d_theta;      // [head_dim / 2] rope_base^(-2i/d), fp64
    int* d_meta;
    int vmax;             // virtual requests a varlen attention call may have (bf16 pools)
    int4* d_vmap;         // [vmax] the varlen plan
    int* d_vcount;
    int prefill_rows;     // varlen requests with G x new tokens >= this go to the prefill-chunk kernel (0: none)
    int4* d_cmap;         // [vmax] its blocks
    int* d_ccount;
    float* d_part_o;
    float* d_part_ml;
    const void* tm_k_ptr;
    const void* tm_v_ptr;
    CUtensorMap tmk, tmv;
    // 16-row boxes for the several-new-tokens path where the one-token maps
    // use 32-row ones (E4M3 pools with pages of 32 tokens or more)
    const void* t16_k_ptr;
    const void* t16_v_ptr;
    CUtensorMap t16k, t16v;
    // page-high boxes (P rows) for the prefill-chunk kernel (bf16 pools) and
    // the tree attention
    const void* tp_k_ptr;
    const void* tp_v_ptr;
    CUtensorMap tpk, tpv;
    // pkv_decode_attn_tree: CTAs, the parts of items they share, the view of q
    int tree_runs;
    float* d_tree_o;
    float2* d_tree_ml;
    int4* d_tree_pos;
    const void* tq_ptr;
    int tq_tokens;
    CUtensorMap tq;
    const void* tm_w_ptr;        // QKV weight and input maps of pkv_qkv_rope_append
    int tm_w_hidden, tm_w_layout;
    int qkv_split;               // 0: automatic
    int plan_key[6];             // (x_rows, D, heads, tiles, hidden, forced split) of the cached plan
    pkv::QkvPlan plan;
    const void* tm_x_ptr;
    int tm_x_hidden, tm_x_rows;
    CUtensorMap tmw, tmx;
};

namespace pkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The checks of the arguments that every call over the pools takes.
pkv_status check_call(const pkv_ctx* ctx, int batch, int bt_stride, const void* k_pool, const void* v_pool,
                      const float* k_scale, const float* v_scale, const int32_t* block_tables,
                      const int32_t* seq_lens);

// 2-D TMA view of a pool (rows = num_pages * Hkv * P token rows of head_dim
// elements), boxes of box_rows rows x (128 or 64 bytes), swizzled.
bool encode_pool_rows(const pkv_ctx* ctx, const void* pool, int box_rows, CUtensorMap* map);

// The context's page-high maps of both pools, encoded when a pool is new.
bool page_maps(pkv_ctx* ctx, const void* k_pool, const void* v_pool);

// 3-D TMA view of q [n_tokens][Hq][head_dim] bf16, boxes of `tokens` tokens x
// one group's heads x 64 elements, 128-byte swizzle.
bool encode_q_rows(const pkv_ctx* ctx, const void* q, int n_tokens, int tokens, CUtensorMap* map);

}  // namespace pkv
