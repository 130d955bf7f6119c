// slot_map.cu -- the plan of a step on the device: pages for the new tokens,
// a slot and a position for each, the ancestor masks of drafted trees
// (pkv_slot_map).
//
// "TensorRT-LLM Guide: High-Throughput GPU Inference Engine", section "2.
// Paged KV Cache & Memory Virtualization" (pages allocated on demand, a table
// from logical positions to physical blocks); "Scaling TensorRT-LLM: Kernel
// Fusion and Inflight Batching in Production", section "3. Speculative
// Decoding for Tail Latency" (drafted tokens; how many were accepted is known
// on the device first).
//
// Mathematics: two prefix sums over the requests (new tokens; pages taken),
// then every token by itself: its request by a binary search of the first
// sum, its page from the table or, past the held pages, from the free stack
// at the second sum's place, its ancestors by walking the parents (strictly
// smaller places, so the walk ends).
//
// What bounds it: launch latency.  The data is a few hundred KB at most, so
// everything is one launch: every CTA repeats the scan over the batch (12
// bytes per request, from L2) instead of waiting for another kernel, and then
// takes its own rows.  pages_out and free_left may be the inputs that other
// CTAs still read, so the CTA that finishes last writes them (a counter that
// wraps by itself; no CTA waits).
#include "tree_params.h"

namespace pkv {
namespace {

constexpr int kSlotThreads = 256;
constexpr int kSlotWarps = kSlotThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

// What the plan needs of one request: pages it takes and whether its numbers
// are in range (a request out of range takes none, its tokens get no slot).
struct Request {
    long long L, n, held, take;
    bool ok;
};

__device__ __forceinline__ Request read_request(const SlotMapParams& p, int b)
{
    Request r;
    r.L = p.seq_lens[b];
    r.n = p.new_lens[b];
    r.held = p.pages_held[b];
    r.ok = r.L >= 0 && r.n >= 0 && r.held >= 0 && r.held <= p.bt_stride && r.held * p.P >= r.L &&
           r.L + r.n <= (long long)p.bt_stride * p.P && !(p.parents && r.n > 32ll * p.mask_words);
    if (r.n < 0) r.n = 0;
    const long long need = (r.L + r.n + p.P - 1) / p.P;
    r.take = r.ok && need > r.held ? need - r.held : 0;
    return r;
}

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const SlotMapParams p)
{
    extern __shared__ int s_dyn[];
    int* const s_cu = s_dyn;                   // [batch + 1] first row of each request, at most n_tokens
    int* const s_first = s_dyn + p.batch + 1;  // [batch] pages taken before it; -1: not served, or out of range
    __shared__ long long s_tok[kSlotWarps], s_pg[kSlotWarps];
    __shared__ int s_taken, s_last, s_err;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        s_taken = 0;
        s_err = 0;
    }
    int count = *p.free_count;
    if (count < 0 || count > p.free_cap) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(p.err, kErrLength);
        count = min(max(count, 0), p.free_cap);
    }

    // ---- the two prefix sums over the requests
    const int per = (p.batch + kSlotThreads - 1) / kSlotThreads;
    const int lo = min(p.batch, tid * per), hi = min(p.batch, lo + per);
    long long tok = 0, pg = 0;
    for (int b = lo; b < hi; ++b) {
        const Request r = read_request(p, b);
        tok += r.n;
        pg += r.take;
    }
    long long tok_in = tok, pg_in = pg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(kAll, tok_in, o), c = __shfl_up_sync(kAll, pg_in, o);
        if (lane >= o) {
            tok_in += a;
            pg_in += c;
        }
    }
    if (lane == 31) {
        s_tok[warp] = tok_in;
        s_pg[warp] = pg_in;
    }
    __syncthreads();
    tok = tok_in - tok;
    pg = pg_in - pg;
    for (int w = 0; w < warp; ++w) {
        tok += s_tok[w];
        pg += s_pg[w];
    }
    int err = 0, taken = 0;
    for (int b = lo; b < hi; ++b) {
        const Request r = read_request(p, b);
        const bool served = r.take == 0 || pg + r.take <= count;
        s_cu[b] = (int)min(tok, (long long)p.n_tokens);
        s_first[b] = !r.ok || !served ? -1 : (int)min(pg, (long long)count);
        if (!r.ok) err |= kErrLength;
        if (!served) err |= kErrNoPages;
        tok += r.n;
        pg += r.take;
        if (served && r.take > 0) taken = (int)pg;   // the sums only grow: the last one served is the largest
    }
    if (hi == p.batch && lo < hi) {
        s_cu[p.batch] = (int)min(tok, (long long)p.n_tokens);
        if (tok > p.n_tokens) err |= kErrLength;
    }
    if (taken) atomicMax(&s_taken, taken);
    if (err && blockIdx.x == 0) atomicOr(&s_err, err);
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int b = tid; b <= p.batch; b += kSlotThreads) p.cu_q[b] = s_cu[b];
        if (tid == 0 && s_err) atomicOr(p.err, s_err);
    }

    // ---- every row by itself
    const int total = s_cu[p.batch];
    const int stride = gridDim.x * kSlotThreads;
    int bad = 0;
    for (int row = blockIdx.x * kSlotThreads + tid; row < p.n_tokens; row += stride) {
        uint32_t* const mask = p.parents ? p.tree_mask + (size_t)row * p.mask_words : nullptr;
        int slot = -1, pos = -1, done = 0;      // done: the mask words from here up are written
        if (row < total) {
            int l = 0, h = p.batch;             // the last request with s_cu <= row
            while (h - l > 1) {
                const int mid = (l + h) >> 1;
                if (s_cu[mid] <= row) l = mid;
                else h = mid;
            }
            const int b = l, i = row - s_cu[b], L = p.seq_lens[b], held = p.pages_held[b];
            const int first = s_first[b];
            const bool in_range = first >= 0 || read_request(p, b).ok;
            int depth = i;
            bool tree_ok = true;
            if (in_range && mask) {
                depth = 0;
                int x = i, w = i >> 5;
                uint32_t acc = 1u << (i & 31);
                for (int k = p.mask_words - 1; k > w; --k) mask[k] = 0u;
                for (;;) {
                    const int parent = p.parents[row - i + x];
                    if (parent == -1) break;
                    if (parent < -1 || parent >= x) {
                        tree_ok = false;
                        break;
                    }
                    ++depth;
                    x = parent;
                    if ((x >> 5) != w) {
                        mask[w] = acc;
                        for (--w; w > (x >> 5); --w) mask[w] = 0u;
                        acc = 0u;
                    }
                    acc |= 1u << (x & 31);
                }
                if (tree_ok) {
                    mask[w] = acc;
                    for (--w; w >= 0; --w) mask[w] = 0u;
                    done = 1;
                } else {
                    bad |= kErrOrder;
                }
            }
            if (in_range && tree_ok) pos = L + depth;
            if (first >= 0) {
                const int at = L + i, lp = at / p.P, place = at - lp * p.P;
                int page;
                if (lp < held) {
                    page = p.block_tables[(size_t)b * p.bt_stride + lp];
                } else {
                    page = p.free_pages[count - 1 - (first + lp - held)];
                    // the first new token of a page enters it into the table
                    if (i == 0 || place == 0) p.block_tables[(size_t)b * p.bt_stride + lp] = page;
                }
                if ((unsigned)page >= (unsigned)p.num_pages) bad |= kErrPage;
                else if (tree_ok) slot = page * p.P + place;
            }
        }
        if (mask && !done)
            for (int k = 0; k < p.mask_words; ++k) mask[k] = 0u;
        p.slots[row] = slot;
        p.positions[row] = pos;
    }
    if (bad) atomicOr(p.err, bad);

    // ---- the outputs that may be inputs: once no CTA reads them any more
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        s_last = atomicInc(p.done, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    for (int b = tid; b < p.batch; b += kSlotThreads) {
        const Request r = read_request(p, b);
        const int first = s_first[b];
        p.pages_out[b] = (int)(r.held + (first >= 0 ? r.take : 0));
    }
    if (tid == 0) *p.free_left = count - s_taken;
}

}  // namespace

cudaError_t slot_map_prepare()
{
    return cudaFuncSetAttribute(slot_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (2 * kMaxBatch + 1) * (int)sizeof(int));
}

cudaError_t launch_slot_map(const SlotMapParams& p, cudaStream_t stream)
{
    const int want = (p.n_tokens + kSlotThreads - 1) / kSlotThreads;
    const int grid = want < 1 ? 1 : want > 296 ? 296 : want;
    slot_map_kernel<<<grid, kSlotThreads, (2 * (size_t)p.batch + 1) * sizeof(int), stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
