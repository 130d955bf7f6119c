// tree_api.cu -- host side of the tree step's entry points (include/pkv.h):
// pkv_slot_map, pkv_rope_append_axes, pkv_decode_attn_tree, pkv_tree_commit.
// Arguments are checked before anything is launched; nothing here throws.
#include <math.h>

#include "pkv_ctx.h"
#include "tree_params.h"

namespace {

using pkv::aligned16;

// Rows of a call: the kernels' row counters and reciprocals.
constexpr int kMaxRows = (1 << 29) - 1;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether [a, a + an) and [b, b + bn) share a byte.
bool overlap(const void* a, size_t an, const void* b, size_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an && bn && x < y + bn && y < x + an;
}

// Kernels and the workspace belong to the context's device.
pkv_status check_device(const pkv_ctx* ctx)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    return dev == ctx->device ? PKV_OK : PKV_ERR_INVALID_ARG;
}

int page_shift(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : 6; }

pkv_status launched(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

}  // namespace

extern "C" {

pkv_status pkv_slot_map(pkv_ctx* ctx, const int32_t* seq_lens, const int32_t* new_lens, const int32_t* parents,
                        int batch, int32_t* block_tables, int bt_stride, const int32_t* pages_held,
                        int32_t* pages_out, const int32_t* free_pages, int free_cap, const int32_t* free_count,
                        int32_t* free_left, int n_tokens, int mask_words, int32_t* cu_q, int32_t* slots,
                        int32_t* positions, uint32_t* tree_mask, cudaStream_t stream)
{
    if (!ctx || batch < 0 || batch > ctx->cfg.max_batch || n_tokens < 0 || free_cap < 0) return PKV_ERR_INVALID_ARG;
    if (n_tokens > kMaxRows) return PKV_ERR_UNSUPPORTED;
    if (batch == 0) return PKV_OK;
    if (bt_stride <= 0 || bt_stride > ctx->cfg.max_blocks_per_seq) return PKV_ERR_INVALID_ARG;
    if (!seq_lens || !new_lens || !block_tables || !pages_held || !pages_out || !free_count || !free_left || !cu_q ||
        (free_cap > 0 && !free_pages) || (n_tokens > 0 && (!slots || !positions)))
        return PKV_ERR_INVALID_ARG;
    // parents and masks come together (with no row both may be NULL)
    if (parents ? !tree_mask || mask_words <= 0 : tree_mask != nullptr) return PKV_ERR_INVALID_ARG;
    const void* const all[] = {seq_lens, new_lens, parents, block_tables, pages_held, pages_out, free_pages,
                               free_count, free_left, cu_q, slots, positions, tree_mask};
    for (const void* x : all)
        if (!aligned4(x)) return PKV_ERR_INVALID_ARG;
    const size_t I = sizeof(int32_t), B = (size_t)batch * I, N = (size_t)n_tokens * I;
    const struct { const void* p; size_t n; } in[] = {{seq_lens, B}, {new_lens, B}, {parents, parents ? N : 0},
                                                      {pages_held, B}, {free_pages, (size_t)free_cap * I},
                                                      {free_count, I}},
        out[] = {{block_tables, B * (size_t)bt_stride}, {cu_q, B + I}, {slots, N}, {positions, N},
                 {tree_mask, tree_mask ? N * (size_t)mask_words : 0}, {pages_out, B}, {free_left, I}};
    const int outs = (int)(sizeof(out) / sizeof(out[0]));
    for (int i = 0; i < outs; ++i) {
        for (const auto& x : in) {
            if (out[i].p == x.p && (x.p == pages_held ? i == outs - 2 : x.p == free_count && i == outs - 1)) continue;
            if (overlap(out[i].p, out[i].n, x.p, x.n)) return PKV_ERR_INVALID_ARG;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return PKV_ERR_INVALID_ARG;
    }
    const pkv_status dev = check_device(ctx);
    if (dev != PKV_OK) return dev;

    pkv::SlotMapParams p;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.parents = parents;
    p.block_tables = block_tables;
    p.pages_held = pages_held;
    p.pages_out = pages_out;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.free_left = free_left;
    p.cu_q = cu_q;
    p.slots = slots;
    p.positions = positions;
    p.tree_mask = tree_mask;
    p.err = ctx->d_err;
    p.batch = batch;
    p.bt_stride = bt_stride;
    p.free_cap = free_cap;
    p.n_tokens = n_tokens;
    p.mask_words = mask_words;
    p.P = ctx->cfg.page_size;
    p.page_shift = page_shift(p.P);
    p.num_pages = ctx->cfg.num_pages;
    return launched(pkv::launch_slot_map(p, stream));
}

pkv_status pkv_rope_append_axes(pkv_ctx* ctx, const void* q, const void* k_new, const void* v_new, int n_tokens,
                                const int32_t* positions, int n_axes, const int* sections, int interleaved,
                                const int32_t* slots, void* q_out, void* k_pool, void* v_pool,
                                const float* k_scale, const float* v_scale, cudaStream_t stream)
{
    if (!ctx || n_tokens < 0 || n_axes < 1 || n_axes > pkv::kMaxAxes || !sections) return PKV_ERR_INVALID_ARG;
    const pkv_config& c = ctx->cfg;
    const int half = c.head_dim / 2;
    pkv::RopeAxesParams p;
    int sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0 || sections[a] > half) return PKV_ERR_INVALID_ARG;
        if (interleaved && a > 0 && sections[a] > 0 && n_axes * (sections[a] - 1) + a >= half)
            return PKV_ERR_INVALID_ARG;
        sum += sections[a];
        p.bound[a] = interleaved ? n_axes * sections[a] : sum;
    }
    if (sum != half) return PKV_ERR_INVALID_ARG;
    if (n_tokens == 0) return PKV_OK;
    if (!q || !k_new || !v_new || !q_out || !k_pool || !v_pool || !positions || !slots) return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) || !aligned16(k_pool) ||
        !aligned16(v_pool) || !aligned4(positions) || !aligned4(slots))
        return PKV_ERR_INVALID_ARG;
    const bool fp8 = c.kv_dtype == PKV_KV_FP8_E4M3;
    if (fp8 && (!k_scale || !v_scale || !aligned16(k_scale) || !aligned16(v_scale))) return PKV_ERR_INVALID_ARG;
    const size_t row = (size_t)c.head_dim * 2, qb = (size_t)n_tokens * c.num_q_heads * row,
                 kb = (size_t)n_tokens * c.num_kv_heads * row;
    if ((q_out != q && overlap(q_out, qb, q, qb)) || overlap(q_out, qb, k_new, kb) || overlap(q_out, qb, v_new, kb))
        return PKV_ERR_INVALID_ARG;
    const pkv_status dev = check_device(ctx);
    if (dev != PKV_OK) return dev;

    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_new = static_cast<const __nv_bfloat16*>(k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(v_new);
    p.positions = positions;
    p.slots = slots;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.theta = ctx->d_theta;
    p.err = ctx->d_err;
    p.n_tokens = n_tokens;
    p.Hq = c.num_q_heads;
    p.Hkv = c.num_kv_heads;
    p.P = c.page_size;
    p.page_shift = page_shift(p.P);
    p.num_pages = c.num_pages;
    p.n_axes = n_axes;
    p.interleaved = interleaved != 0;
    return launched(pkv::launch_rope_axes(p, c.head_dim, fp8, stream));
}

pkv_status pkv_decode_attn_tree(pkv_ctx* ctx, const void* q, const void* k_pool, const void* v_pool,
                                const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                int bt_stride, const int32_t* seq_lens, const int32_t* cu_q,
                                const uint32_t* tree_mask, int mask_words, int batch, int n_tokens, void* out,
                                cudaStream_t stream)
{
    const pkv_status st =
        pkv::check_call(ctx, batch, bt_stride, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens);
    if (st != PKV_OK) return st;
    if (n_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (n_tokens > kMaxRows) return PKV_ERR_UNSUPPORTED;
    if (batch == 0 || n_tokens == 0) return PKV_OK;
    if (!q || !out || !cu_q || !tree_mask || mask_words <= 0) return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(cu_q) || !aligned4(tree_mask)) return PKV_ERR_INVALID_ARG;
    const size_t bytes = (size_t)n_tokens * ctx->cfg.num_q_heads * ctx->cfg.head_dim * 2;
    if (overlap(q, bytes, out, bytes)) return PKV_ERR_INVALID_ARG;
    const pkv_status dev = check_device(ctx);
    if (dev != PKV_OK) return dev;

    const int tb = pkv::kTreeRows / ctx->G;
    if (!pkv::page_maps(ctx, k_pool, v_pool)) return PKV_ERR_CUDA;
    if (ctx->tq_ptr != q || ctx->tq_tokens != n_tokens) {
        if (!pkv::encode_q_rows(ctx, q, n_tokens, tb, &ctx->tq)) return PKV_ERR_CUDA;
        ctx->tq_ptr = q;
        ctx->tq_tokens = n_tokens;
    }

    pkv::TreeAttnParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.cu_q = cu_q;
    p.tree_mask = tree_mask;
    p.err = ctx->d_err;
    p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)ctx->cfg.head_dim));
    p.batch = batch;
    p.bt_stride = bt_stride;
    p.Hq = ctx->cfg.num_q_heads;
    p.Hkv = ctx->cfg.num_kv_heads;
    p.G = ctx->G;
    p.P = ctx->cfg.page_size;
    p.num_pages = ctx->cfg.num_pages;
    p.mask_words = mask_words;
    p.n_tokens = n_tokens;
    p.part_o = ctx->d_tree_o;
    p.part_ml = ctx->d_tree_ml;
    p.pos = ctx->d_tree_pos;
    p.tb = tb;
    p.g_inv = 65536 / ctx->G + 1;
    p.two_inv = ((1ull << 37) + 2 * tb - 1) / (2 * tb);
    p.run_inv = ~0ull / (unsigned)ctx->tree_runs;
    return launched(pkv::launch_tree_attn(p, ctx->tq, ctx->tpk, ctx->tpv, ctx->cfg.head_dim,
                                          ctx->cfg.kv_dtype == PKV_KV_FP8_E4M3, ctx->tree_runs, stream));
}

pkv_status pkv_tree_commit(pkv_ctx* ctx, void* k_pool, void* v_pool, const float* k_scale, const float* v_scale,
                           const int32_t* block_tables, int bt_stride, const int32_t* seq_lens,
                           const int32_t* path, int path_stride, const int32_t* path_lens, int batch,
                           int32_t* lens_out, cudaStream_t stream)
{
    const pkv_status st =
        pkv::check_call(ctx, batch, bt_stride, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens);
    if (st != PKV_OK || batch == 0) return st;
    if (path_stride < 0 || (path_stride > 0 && !path) || !path_lens || !lens_out) return PKV_ERR_INVALID_ARG;
    if (!aligned4(path) || !aligned4(path_lens) || !aligned4(lens_out)) return PKV_ERR_INVALID_ARG;
    const size_t B = (size_t)batch * sizeof(int32_t);
    if ((lens_out != seq_lens && overlap(lens_out, B, seq_lens, B)) || overlap(lens_out, B, path_lens, B) ||
        overlap(lens_out, B, path, B * (size_t)path_stride) || overlap(lens_out, B, block_tables, B * (size_t)bt_stride))
        return PKV_ERR_INVALID_ARG;
    const pkv_status dev = check_device(ctx);
    if (dev != PKV_OK) return dev;

    pkv::TreeCommitParams p;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.path = path;
    p.path_lens = path_lens;
    p.lens_out = lens_out;
    p.err = ctx->d_err;
    p.batch = batch;
    p.bt_stride = bt_stride;
    p.path_stride = path_stride;
    p.Hkv = ctx->cfg.num_kv_heads;
    p.P = ctx->cfg.page_size;
    p.page_shift = page_shift(p.P);
    p.num_pages = ctx->cfg.num_pages;
    return launched(pkv::launch_tree_commit(p, ctx->cfg.head_dim, ctx->cfg.kv_dtype == PKV_KV_FP8_E4M3, stream));
}

}  // extern "C"
