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
// What bounds it: latency.  The data is a few hundred KB at most, so everything
// is one launch of one cluster of up to 8 CTAs: every CTA repeats the scan over
// the batch (12 bytes per request, from L2) instead of waiting for another
// kernel, then takes its own rows.  The parents of its rows and of those before
// them are read into shared memory while the lengths are on their way, so that
// the walks up the trees do not go to L2 step by step.  pages_out and free_left
// may be the inputs that other CTAs still read: each CTA arrives at the cluster's
// barrier once it has read them, and the one that writes them waits there.  The
// sums saturate (whatever the lengths, 32 bits hold them).
//
// Measured (B200): 256 requests, 4.7 thousand tokens in trees of up to 32, 7.5 us
// a call among others (8.2 with the barrier at the end; before that 8.0 on the
// device, and 9.0 with the walks in L2 and a grid of small CTAs); 4 requests of one
// token, 5.5, most of it the host's.
#include "tree_params.h"

namespace pkv {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// What the plan needs of one request: pages it takes and whether its numbers
// are in range (a request out of range takes none, its tokens get no slot).
struct Request {
    int L, n, held, take;
    bool ok;
};

__device__ __forceinline__ Request read_request(const SlotMapParams& p, int b)
{
    Request r;
    r.L = p.seq_lens[b];
    r.n = p.new_lens[b];
    r.held = p.pages_held[b];
    const long long L = r.L, n = r.n, cap = min((long long)p.bt_stride * p.P, kMaxTreeKeys);
    r.ok = L >= 0 && n >= 0 && r.held >= 0 && r.held <= p.bt_stride && (long long)r.held * p.P >= L && L + n <= cap &&
           !(p.parents && n > 32ll * p.mask_words);
    if (r.n < 0) r.n = 0;
    r.take = 0;
    if (r.ok) r.take = max(0, (int)((L + n + p.P - 1) >> p.page_shift) - r.held);
    return r;
}

// The pages that a request lacks, as far as the table goes, also where it takes none.
__device__ __forceinline__ int wanted(const SlotMapParams& p, const Request& r)
{
    if (r.L < 0 || r.n == 0 || r.held < 0 || r.held > p.bt_stride || (long long)r.held * p.P < r.L) return 0;
    return max(0, (int)min(((long long)r.L + r.n + p.P - 1) >> p.page_shift, (long long)p.bt_stride) - r.held);
}

__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b, unsigned top) { return min(a + b, top); }

// Inclusive scan over a warp of sums that saturate at `top` (below 2^31).
__device__ __forceinline__ unsigned warp_scan(unsigned x, unsigned top, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x = sat_add(x, y, top);
    }
    return x;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) slot_map_kernel(const SlotMapParams p)
{
    constexpr int WARPS = THREADS / 32;
    extern __shared__ int s_dyn[];
    int* const s_cu = s_dyn;                   // [batch + 1] first row of each request, at most n_tokens
    int* const s_first = s_dyn + p.batch + 1;  // [batch] pages taken before it; -1: not served, -2: out of range
    int* const s_len = s_first + p.batch;      // [batch] L
    int* const s_held = s_len + p.batch;       // [batch] pages held
    __shared__ unsigned s_tok[WARPS], s_pg[WARPS];
    __shared__ int s_par[2 * THREADS];         // parents of this CTA's rows and of THREADS rows before them
    __shared__ int s_taken, s_err, s_rare;     // s_rare: the table needs more than its rows write
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, stride = gridDim.x * THREADS;

    if (tid == 0) {
        s_taken = 0;
        s_err = 0;
        s_rare = 0;
    }
    int row0 = rank * THREADS;
    int par[2] = {-1, -1};
    auto read_parents = [&] {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int row = row0 + (k - 1) * THREADS + tid;
            par[k] = p.parents && row >= 0 && row < p.n_tokens ? __ldg(&p.parents[row]) : -1;
        }
    };
    read_parents();
    const int given = *p.free_count;
    const int count = min(max(given, 0), p.free_cap);
    const unsigned tok_top = (unsigned)p.n_tokens + 1u, pg_top = (unsigned)p.free_cap + 1u;

    // ---- the two prefix sums over the requests
    const int per = (p.batch + THREADS - 1) / THREADS;
    const int lo = min(p.batch, tid * per), hi = min(p.batch, lo + per);
    unsigned tok = 0, pg = 0;
    Request r;
    for (int b = lo; b < hi; ++b) {
        r = read_request(p, b);
        tok = sat_add(tok, min((unsigned)r.n, tok_top), tok_top);
        pg = sat_add(pg, min((unsigned)r.take, pg_top), pg_top);
    }
    unsigned tok_in = warp_scan(tok, tok_top, lane), pg_in = warp_scan(pg, pg_top, lane);
    if (lane == 31) {
        s_tok[warp] = tok_in;
        s_pg[warp] = pg_in;
    }
    s_par[tid] = par[0];
    s_par[THREADS + tid] = par[1];
    __syncthreads();
    {
        // sums of the warps before, and of this thread's lanes before
        const unsigned a = warp_scan(lane < WARPS ? s_tok[lane] : 0u, tok_top, lane);
        const unsigned c = warp_scan(lane < WARPS ? s_pg[lane] : 0u, pg_top, lane);
        unsigned before_t = __shfl_up_sync(kAll, tok_in, 1), before_p = __shfl_up_sync(kAll, pg_in, 1);
        if (lane == 0) before_t = before_p = 0u;
        const unsigned wt = __shfl_sync(kAll, a, max(warp - 1, 0)), wp = __shfl_sync(kAll, c, max(warp - 1, 0));
        tok = warp ? sat_add(wt, before_t, tok_top) : before_t;
        pg = warp ? sat_add(wp, before_p, pg_top) : before_p;
    }
    int err = 0, taken = 0;
    for (int b = lo; b < hi; ++b) {
        if (per > 1) r = read_request(p, b);
        const unsigned after = sat_add(pg, min((unsigned)r.take, pg_top), pg_top);
        const bool served = r.take == 0 || after <= (unsigned)count;
        s_cu[b] = (int)min(tok, (unsigned)p.n_tokens);
        s_first[b] = !r.ok ? -2 : !served ? -1 : (int)min(pg, (unsigned)count);
        s_len[b] = r.L;
        s_held[b] = r.held;
        if (!r.ok) err |= kErrLength;
        if (!served) err |= kErrNoPages;
        if (!served || !r.ok) s_rare = 1;
        tok = sat_add(tok, min((unsigned)r.n, tok_top), tok_top);
        pg = after;
        if (served && r.take > 0) taken = (int)pg;   // the sums only grow: the last one served is the largest
    }
    if (hi == p.batch && lo < hi) {
        s_cu[p.batch] = (int)min(tok, (unsigned)p.n_tokens);
        if (tok > (unsigned)p.n_tokens) {
            err |= kErrLength;
            s_rare = 1;
        }
    }
    if (rank == 0) {
        if (given != count && tid == 0) err |= kErrLength;
        if (taken) atomicMax(&s_taken, taken);
        if (err) atomicOr(&s_err, err);
    }
    __syncthreads();
    // the inputs that may be outputs are read: whoever writes them waits for this
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    if (rank == 0) {
        for (int b = tid; b <= p.batch; b += THREADS) p.cu_q[b] = s_cu[b];
        if (tid == 0 && s_err) atomicOr(p.err, s_err);
    }

    // ---- every row by itself
    const int total = s_cu[p.batch];
    int bad = 0;
    for (;;) {
        const int row = row0 + tid;
        if (row < p.n_tokens) {
            uint32_t* const mask = p.parents ? p.tree_mask + (size_t)row * p.mask_words : nullptr;
            int slot = -1, pos = -1;
            bool done = false;                  // the mask is written
            if (row < total) {
                int l = 0, h = p.batch;         // the last request with s_cu <= row
                while (h - l > 1) {
                    const int mid = (l + h) >> 1;
                    if (s_cu[mid] <= row) l = mid;
                    else h = mid;
                }
                const int b = l, start = s_cu[b], i = row - start, L = s_len[b], held = s_held[b];
                const int first = s_first[b];
                const bool in_range = first != -2;
                const int at = (int)min((long long)L + i, kMaxTreeKeys);      // of a request in range: L + i
                const int lp = max(at, 0) >> p.page_shift, place = at & (p.P - 1);
                int page = -1;
                if (first >= 0)
                    page = lp < held ? p.block_tables[(size_t)b * p.bt_stride + lp]
                                     : __ldg(&p.free_pages[count - 1 - (first + lp - held)]);
                int depth = i;
                bool tree_ok = true;
                if (in_range && mask) {
                    depth = 0;
                    int x = i, w = i >> 5;
                    uint32_t acc = 1u << (i & 31);
                    for (int k = p.mask_words - 1; k > w; --k) mask[k] = 0u;
                    for (;;) {
                        const int from = start + x - row0 + THREADS;      // its place in the window
                        const int parent = from >= 0 ? s_par[from] : __ldg(&p.parents[start + x]);
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
                        done = true;
                    } else {
                        bad |= kErrOrder;
                    }
                }
                if (in_range && tree_ok) pos = L + depth;
                if (first >= 0) {
                    // the first new token of a page enters it into the table
                    if (lp >= held && (i == 0 || place == 0)) p.block_tables[(size_t)b * p.bt_stride + lp] = page;
                    if ((unsigned)page >= (unsigned)p.num_pages) bad |= kErrPage;
                    else if (tree_ok) slot = page * p.P + place;
                }
            }
            if (mask && !done)
                for (int k = 0; k < p.mask_words; ++k) mask[k] = 0u;
            p.slots[row] = slot;
            p.positions[row] = pos;
        }
        if (row0 + stride >= p.n_tokens) break;          // the whole CTA
        row0 += stride;
        read_parents();
        __syncthreads();
        s_par[tid] = par[0];
        s_par[THREADS + tid] = par[1];
        __syncthreads();
    }
    if (bad) atomicOr(p.err, bad);
    // Pages are entered by the rows of their first new tokens.  Where tokens were
    // dropped the pages that they were taken for are entered here (those that have
    // rows a second time, with the same number), a warp for each request: pages_out
    // and free_left count them, and the next step reads them from the table.  The
    // entries of pages that a request did not get name none, whatever was there.
    // The barrier behind it keeps pages_held, which may be pages_out, as it is read
    // here.
    if (s_rare && rank == 0) {
        for (int b = warp; b < p.batch; b += WARPS) {
            const Request x = read_request(p, b);
            const int first = s_first[b], n = wanted(p, x);
            for (int k = lane; k < n; k += 32)
                p.block_tables[(size_t)b * p.bt_stride + x.held + k] =
                    first >= 0 ? __ldg(&p.free_pages[count - 1 - (first + k)]) : -1;
        }
        __syncthreads();
    }

    // ---- the outputs that may be inputs: once no CTA reads them any more
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (rank) return;
    for (int b = lo; b < hi; ++b) {
        if (per > 1) r = read_request(p, b);
        p.pages_out[b] = r.held + (s_first[b] >= 0 ? r.take : 0);
    }
    if (tid == 0) *p.free_left = count - s_taken;
}

template <int THREADS>
cudaError_t launch_t(const SlotMapParams& p, int ctas, cudaStream_t stream)
{
    if (ctas == 1) {                 // a cluster of one needs no attribute, and starts cheaper on the host
        slot_map_kernel<THREADS><<<1, THREADS, (4 * (size_t)p.batch + 1) * sizeof(int), stream>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (4 * (size_t)p.batch + 1) * sizeof(int);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, slot_map_kernel<THREADS>, p);
}

template <int THREADS>
cudaError_t prepare_t()
{
    return cudaFuncSetAttribute(slot_map_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (4 * kMaxBatch + 1) * (int)sizeof(int));
}

}  // namespace

cudaError_t slot_map_prepare()
{
    const cudaError_t e = prepare_t<128>();
    return e != cudaSuccess ? e : prepare_t<1024>();
}

cudaError_t launch_slot_map(const SlotMapParams& p, cudaStream_t stream)
{
    // few rows and requests: a small CTA starts sooner
    if (p.n_tokens <= 128 && p.batch <= 128) return launch_t<128>(p, 1, stream);
    int ctas = 1;                    // a thread for each row, up to a portable cluster's 8 CTAs
    while (ctas < 8 && ctas * 1024 < p.n_tokens) ctas *= 2;
    return launch_t<1024>(p, ctas, stream);
}

}  // namespace pkv
