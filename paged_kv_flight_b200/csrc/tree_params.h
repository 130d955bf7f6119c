// tree_params.h -- parameters and launchers of the tree step's kernels
// (slot_map.cu, rope_axes.cu, tree_attn.cu, tree_commit.cu), shared with its
// host side (tree_api.cu).  Not part of the ABI.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// Largest cached and new tokens of a request: places in it are 32-bit.
constexpr long long kMaxTreeKeys = 0x7FFFFF00;

struct SlotMapParams {
    const int32_t* seq_lens;
    const int32_t* new_lens;
    const int32_t* parents;       // null: a chain
    int32_t* block_tables;
    const int32_t* pages_held;
    int32_t* pages_out;           // may be pages_held
    const int32_t* free_pages;
    const int32_t* free_count;
    int32_t* free_left;           // may be free_count
    int32_t* cu_q;
    int32_t* slots;
    int32_t* positions;
    uint32_t* tree_mask;
    int* err;
    int batch, bt_stride, free_cap, n_tokens, mask_words, P, page_shift, num_pages;   // P = 1 << page_shift
};
cudaError_t slot_map_prepare();
cudaError_t launch_slot_map(const SlotMapParams& p, cudaStream_t stream);

constexpr int kMaxAxes = 4;

struct RopeAxesParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_new;
    const __nv_bfloat16* v_new;
    const int32_t* positions;     // [n_axes][n_tokens]
    const int32_t* slots;
    __nv_bfloat16* q_out;         // may be q
    void* k_pool;
    void* v_pool;
    const float* k_scale;
    const float* v_scale;
    const double* theta;          // [D / 2] rope_base^(-2i/D) in fp64, from the context
    int* err;
    int n_tokens, Hq, Hkv, P, page_shift, num_pages;
    int n_axes, interleaved;
    int bound[kMaxAxes];          // consecutive: the first pair past axis a; interleaved: n_axes * sections[a]
};
cudaError_t launch_rope_axes(const RopeAxesParams& p, int head_dim, bool fp8, cudaStream_t stream);

struct TreeAttnParams {
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    const void* k_pool;
    const void* v_pool;
    const float* k_scale;
    const float* v_scale;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* cu_q;
    const uint32_t* tree_mask;
    int* err;
    float* part_o;                // [2 * runs][256][D] fp32, unnormalised: the parts of items at a run's ends
    float2* part_ml;              // [2 * runs][256] (m in log2 units, l)
    int4* pos;                    // [runs + 1] where each run starts: request, kv head, block, tile
    float scale_log2;             // log2(e) / sqrt(d)
    int batch, bt_stride, Hq, Hkv, G, P, num_pages, mask_words, n_tokens;
    int tb;                       // new tokens in the 128 rows of a stream: 128 / G
    int g_inv;                    // 65536 / G + 1: x / G = (x g_inv) >> 16 for x < 256
    unsigned long long two_inv;   // 2^37 / (2 tb) rounded up: x / (2 tb) = (x two_inv) >> 37 for x < 2^29
    unsigned long long run_inv;   // 2^64 / runs
};
constexpr int kTreeRows = 128;
constexpr int kMaxTreeRuns = 256; // CTAs of the attention at most
cudaError_t tree_attn_prepare(int head_dim, bool fp8);
// runs CTAs (one per SM), then the merge of the items they share.  tmq: q as
// [n_tokens][Hq][D], boxes of tb tokens, G heads, 64 elements.
cudaError_t launch_tree_attn(const TreeAttnParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk,
                             const CUtensorMap& tmv, int head_dim, bool fp8, int runs, cudaStream_t stream);

struct TreeCommitParams {
    void* k_pool;
    void* v_pool;
    const float* k_scale;
    const float* v_scale;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* path;
    const int32_t* path_lens;
    int32_t* lens_out;            // may be seq_lens
    int* err;
    int batch, bt_stride, path_stride, Hkv, P, page_shift, num_pages;
};
cudaError_t launch_tree_commit(const TreeCommitParams& p, int head_dim, bool fp8, cudaStream_t stream);

}  // namespace pkv
