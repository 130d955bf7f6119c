// tree_attn.cu -- attention of a tree of drafted tokens over the paged cache
// on the tensor cores (pkv_decode_attn_tree): S, P and O in tensor memory
// (tcgen05), Q and the K / V pages by TMA into shared memory.
//
// "Scaling TensorRT-LLM: Kernel Fusion and Inflight Batching in Production",
// section "3. Speculative Decoding for Tail Latency" (a draft proposes tokens
// and the target model checks all of them in one forward pass); "TensorRT-LLM
// Guide: High-Throughput GPU Inference Engine", section "3. Custom Fused
// Attention Kernels: FMHA and XQA" (K / V read once for a group's heads).
//
// Mathematics: o = softmax(q K^T / sqrt(d)) V over the keys a row sees, all
// cached keys and those drafted ones whose mask bit is set.  One pass with a
// running reference m and sum l per row: S = Q K^T, P = 2^(s - m), l += P,
// O += P V; m moves only when the row's maximum passes it by more than 2^24.
//
// Work item: a request, one of its kv heads and a block of up to 2 (128 / G)
// of its new tokens; the G heads of the group times the tokens are the rows
// of the MMAs, 128 in each of two streams.  A stream has its own S / P buffer
// and O in tensor memory and its own four softmax warps, so one stream's
// softmax runs while the other's MMAs do.  With more than 128 rows the streams
// take one half of the rows each and share every K / V tile ("row mode": the
// cache is read once per 256 rows); with at most 128 they take the even and
// the odd key tiles of the same rows and are merged at the end ("key mode").
//
// The items' tiles of 128 keys, in order, are cut into as many runs as there
// are SMs, of equal cost; a run's first and last item may be parts, whose
// unnormalised O, m and l go to the workspace and are merged by tree_combine
// in a fixed order.  Nothing waits for another CTA.
//
// Warps: 0 and 2 load Q, K and V (TMA), 1 issues the MMAs, 4 .. 11 softmax and
// output, one thread per row; for E4M3 pools 12 .. 15 turn the codes into
// bf16 tiles (exact; the scales of a page and head go into the scores and the
// weights in fp32).  P goes into the matrix product as two bf16 terms, cut and
// rounded, that are off by at most 2^-15 of a weight together: with one term (half
// as many P V MMAs) each weight is off by up to 2^-8, as much again as the output's
// own rounding, and a row that sees one key does not get its V back.
//
// What bounds it, and what it measured (two B200s, us a call): the chain of a tile,
// S, softmax, P V and the handovers between them, two of which are under way at a
// time; the second term of P makes its MMAs half as many again (in brackets: with one
// term).  Long caches (8 requests of 32k to 128k tokens, 8 new ones each, 2.28 GB: 426
// and 460 [357 and 396], 76 to 83% of the measured copy), serving batches (64 requests
// of 128 to 4096, 9 to 16 new ones, 555 MB: 131 and 138 [113 and 119]), large trees (48
// requests, 33 to 64 new tokens of 64 heads: 193 and 201 [162 and 169], where the
// products alone take 78), E4M3 caches, beside the conversion (64 requests, 391 MB: 182
// and 185 [158 and 167]); a few short requests, latency (4 requests: 12.3 [11.8]).
#include "tree_params.h"
#include "pkv_device.cuh"
#include "umma.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kTRows = 128;                   // rows of a stream
constexpr int kTKeys = 128;                   // keys of a tile
constexpr int kTBlk = kTRows * 128;           // 64 columns of a 128-row tile in bf16: 16 KB
constexpr uint32_t kTCols = 512;              // tensor memory: S / P of two streams, O of two streams
constexpr uint32_t kTOcol = 2 * kTKeys;
constexpr int kMaxSlots = 8;
constexpr uint64_t kTWaitNs = 500ull * 1000ull * 1000ull;
// Cost of a tile for the cut, and of an item besides its tiles (Q, the masked
// tile, the merge of the streams, the output).  Fitted over the CTAs of three
// workloads at d = 128 in bf16, with P in one term: 3900 cycles a tile in row mode,
// 1950 in key mode, 8.7 to 12 thousand an item.  Cut by tiles alone, the slowest CTA
// took 1.5 to 2 times the mean (297 us against 184 for large trees); with 7 or 12 for
// the item they took 3 and 2% longer.  With P in two terms a tile takes about a
// quarter more in both modes, and 7, 8 and 9 for the item are alike within 1%, for
// E4M3 caches too.  Heads of 64 have the same costs, not fitted for them.
constexpr int kCostRowShift = 2, kCostKeyShift = 1, kCostItem = 9;
constexpr int kCostRow = 1 << kCostRowShift, kCostKey = 1 << kCostKeyShift;
// How far a row's maximum may pass its reference, in powers of two, before the
// reference moves: the weights are bf16 and their sums fp32, of one exponent
// range, so that nothing is lost below 2^24 (V up to 2^100); 2^8 cost E4M3
// caches 4% in moves that changed nothing.
constexpr float kSlack = 24.f;
constexpr int kSnap = 2;                      // a cut this near to an item's ends moves there

template <int D, bool FP8>
struct TreeGeo {
    static constexpr int KB = D / 64;
    static constexpr int SLOT = KB * kTBlk;                          // K or V of a tile in bf16
    static constexpr int NS = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
    static constexpr int NC = FP8 ? (D == 128 ? 4 : 6) : 0;          // tiles of codes
    static constexpr int STG = kTKeys * D;
    static constexpr int THREADS = 128 + 256 + (FP8 ? 128 : 0);
    static constexpr int BYTES = (2 + NS) * SLOT + NC * STG + 1024;
};

// A bounded wait whose clock starts late: most waits here end within some
// polls, and reading the timer first costs as much as one of them.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity)
{
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_bounded(bar, parity, kTWaitNs);
}

// ---- the cut ------------------------------------------------------------------

struct Request {
    int row0, T, L, NT;
};

// 0: nothing to do; 1: ok; 2: cu_q out of range; 3: lengths out of range
// (its rows are zero).
__device__ __forceinline__ int read_request(const TreeAttnParams& p, int b, Request& r)
{
    const int a = __ldg(&p.cu_q[b]), e = __ldg(&p.cu_q[b + 1]);
    r.L = __ldg(&p.seq_lens[b]);
    if (a < 0 || e > p.n_tokens || a > e) return 2;
    r.row0 = a;
    r.T = e - a;
    if (r.T == 0) return 0;
    const long long keys = (long long)r.L + r.T;
    if (r.L < 0 || keys > min((long long)p.bt_stride * p.P, kMaxTreeKeys) || r.T > 32ll * p.mask_words) return 3;
    r.NT = (int)((keys + kTKeys - 1) / kTKeys);
    return 1;
}

// Blocks of 2 tb tokens: those in row mode (more than tb tokens), then at
// most one in key mode.
__device__ __forceinline__ void blocks_of(const TreeAttnParams& p, int T, int& row_blocks, int& blocks)
{
    const int two = 2 * p.tb, whole = (int)(((unsigned long long)T * p.two_inv) >> 37), rest = T - whole * two;
    row_blocks = whole + (rest > p.tb ? 1 : 0);
    blocks = whole + (rest > 0 ? 1 : 0);
}

__device__ __forceinline__ long long cost_of(const TreeAttnParams& p, const Request& r)
{
    int rb, nb;
    blocks_of(p, r.T, rb, nb);
    return (long long)p.Hkv * (rb * ((long long)r.NT * kCostRow + kCostItem) + (nb - rb) * ((long long)r.NT * kCostKey + kCostItem));
}

// A place in the order of all tiles: request, kv head, block, tile.
__device__ __forceinline__ bool before(const int4& a, const int4& b)
{
    return a.x != b.x ? a.x < b.x : a.y != b.y ? a.y < b.y : a.z != b.z ? a.z < b.z : a.w < b.w;
}
__device__ __forceinline__ bool same_item(const int4& a, const int4& b) { return a.x == b.x && a.y == b.y && a.z == b.z; }

__device__ __forceinline__ int4 next_item(int b, int kvh, int blk, int blocks, int Hkv)
{
    if (++blk < blocks) return make_int4(b, kvh, blk, 0);
    if (++kvh < Hkv) return make_int4(b, kvh, 0, 0);
    return make_int4(b + 1, 0, 0, 0);
}

// The place at cost `at` of request b, moved to an item's start or end when
// it is near.
__device__ __forceinline__ int4 place_at(const TreeAttnParams& p, int b, const Request& r, long long at)
{
    int rb, nb;
    blocks_of(p, r.T, rb, nb);
    const long long row_cost = (long long)r.NT * kCostRow + kCostItem,
                    head = row_cost * rb + (nb - rb) * ((long long)r.NT * kCostKey + kCostItem);
    int kvh = 0, blk = 0;                   // a few steps: cheaper than divisions in 64 bits
    for (; at >= head; at -= head) ++kvh;
    for (; blk < rb && at >= row_cost; at -= row_cost) ++blk;
    const int tile = at <= kCostItem ? 0 : (int)((at - kCostItem) >> (blk < rb ? kCostRowShift : kCostKeyShift));
    if (tile <= kSnap) return make_int4(b, kvh, blk, 0);
    if (r.NT - tile <= kSnap) return next_item(b, kvh, blk, nb, p.Hkv);
    return make_int4(b, kvh, blk, tile);
}

// A run's share of one item: tiles t0 .. t0 + n - 1 of its NT.
struct Segment {
    int b, kvh, row0, ntok, L, T, NT, t0, n, units;
    int place;             // 0: the whole item, 1: its start, 2: a later part
    bool row_mode;
};

struct Walk {
    int4 cur, end;
    int at = -1;           // the request in r
    Request r;
    __device__ __forceinline__ bool next(const TreeAttnParams& p, Segment& s)
    {
        while (before(cur, end)) {
            if (at != cur.x) {
                at = cur.x;
                if (read_request(p, at, r) != 1) {
                    cur = make_int4(at + 1, 0, 0, 0);
                    continue;
                }
            }
            int rb, nb;
            blocks_of(p, r.T, rb, nb);
            const int first = cur.z * 2 * p.tb;
            s.b = cur.x;
            s.kvh = cur.y;
            s.row0 = r.row0 + first;
            s.ntok = min(2 * p.tb, r.T - first);
            s.L = r.L;
            s.T = r.T;
            s.NT = r.NT;
            s.row_mode = s.ntok > p.tb;
            s.t0 = cur.w;
            s.n = (same_item(cur, end) ? end.w : r.NT) - s.t0;
            s.units = s.row_mode ? 2 * s.n : s.n;
            s.place = s.n == r.NT ? 0 : s.t0 == 0 ? 1 : 2;
            cur = next_item(cur.x, cur.y, cur.z, nb, p.Hkv);
            return true;
        }
        return false;
    }
};

// Place of a segment's loads in its sequence.  Unit u is tile u of stream u %
// 2 in key mode, tile u / 2 of stream u % 2 in row mode; the MMAs go S(0),
// S(1), then P V(u), S(u + 2) for every u, and the loads in the order of
// their first use.
__device__ __forceinline__ int lead_of(const Segment& s) { return s.row_mode ? 1 : 2; }   // K tiles before the first V
__device__ __forceinline__ int k_seq(const Segment& s, int i)
{
    const int lead = lead_of(s);
    return i < lead ? i : 2 * i - lead + 1;
}
__device__ __forceinline__ int v_seq(const Segment& s, int i) { return i + min(i + lead_of(s), s.n); }

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// ---- softmax of one tile --------------------------------------------------------

// Pairs of fp32 in one 64-bit register, and their arithmetic.
__device__ __forceinline__ uint64_t two(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float first_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float second_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The scores of keys that the row does not see become -inf, whatever they
// were, before the pass below (masks in that pass would double its code for one
// tile in many).  d0: the tile's first key counted in drafted tokens; seen(i):
// word i of those the row sees; lost(k): keys 32 k .. of the tile in pages out of
// range.  This and the rest of a segment's end run once for an item, from cold
// instruction caches, where every line of code costs a fetch: short loops.
template <class Seen, class Lost>
__device__ __forceinline__ void tile_mask(uint32_t scol, int d0, Seen seen, Lost lost)
{
    uint32_t low = seen(d0 >> 5), see = 0u;
#pragma unroll 1
    for (int c0 = 0; c0 < kTKeys; c0 += 16) {
        if (c0 & 16) {
            see >>= 16;
        } else {
            const uint32_t high = seen((d0 >> 5) + c0 / 32 + 1);
            see = __funnelshift_r(low, high, d0 & 31) & ~lost(c0 / 32);
            low = high;
        }
        uint32_t x[2][8];
        tmem_ld8(scol + (uint32_t)c0, x[0]);
        tmem_ld8(scol + (uint32_t)c0 + 8u, x[1]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c >> 3][c & 7] = (see >> c) & 1u ? x[c >> 3][c & 7] : 0xFF800000u;
        tmem_st8(scol + (uint32_t)c0, x[0]);
        tmem_st8(scol + (uint32_t)c0 + 8u, x[1]);
    }
    tmem_wait_st();
}

// 16 columns of this lane times alpha: fp32, or pairs of bf16 (exact for a
// power of two).
template <bool BF16>
__device__ __forceinline__ void tmem_scale16(uint32_t col, float alpha)
{
    uint32_t x[2][8];
    tmem_ld8(col, x[0]);
    tmem_ld8(col + 8u, x[1]);
    tmem_wait_ld();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            x[h][c] = BF16 ? pack_bf16(bf16_lo(x[h][c]) * alpha, bf16_hi(x[h][c]) * alpha)
                           : __float_as_uint(__uint_as_float(x[h][c]) * alpha);
        tmem_st8(col + (uint32_t)(8 * h), x[h]);
    }
}

// Keys of a chunk of the softmax pass, and the column of the first terms of P of
// 16 keys (the second ones are half a chunk behind).
template <bool FP8>
constexpr int kChunk = FP8 ? 32 : 64;
template <bool FP8>
__device__ __forceinline__ constexpr uint32_t p_col(int kk)
{
    constexpr int N = kChunk<FP8>;
    return (uint32_t)(16 * kk / N * N + 16 * kk % N / 2);
}

constexpr float kOneUp = 1.f + 1.f / (1 << 23);

// One pass over the row's S, 64 keys (E4M3: 32) at a time in a loop that is not unrolled
// (unrolled, the code was over 64 KB, and fetching it made every warp of the SM
// several times slower).  A chunk's maximum is taken
// while its scores are in registers; the reference m, a whole number, moves
// only when some row of the warp passes it by more than 2^24, and then what was
// made with the old one (O of this stream, the tile's chunks of P, l) is
// multiplied by a power of two, which is exact.  P = 2^(s - m) goes back over the
// chunk's own S columns, just read, as two bf16 terms: of N columns the first N / 2
// hold the first terms, keys 2i and 2i + 1 in column i, the others the second.
// The first term is the weight's upper half, cut (no conversion, and the rest,
// below 2^-7 of the weight, is an exact difference); the second is the rest rounded.
// It is made larger by 2^-23 of the weight, so that it is 0 for no weight but 0: next
// to an infinity in V a second term of 0 would make NaN of it.  l is summed from the
// fp32 weights, of which the two terms leave 2^-15 at most.
//
// f: score scale in log2 units.  E4M3: `scales` of lane k holds the K scale of
// the tile's page k, of lane 8 + k its V scale; pages are 1 << shift keys.
template <int D, bool FP8>
__device__ __forceinline__ void tile_softmax(uint32_t scol, uint32_t ocol, bool first, float f, float scales, int shift,
                                             float& m, float& l)
{
    constexpr int N = kChunk<FP8>;
#pragma unroll 1
    for (int k = 0; k < kTKeys / N; ++k) {
        uint32_t x[N];
#pragma unroll
        for (int c = 0; c < N; c += 32) tmem_ld32(scol + (uint32_t)(N * k + c), *reinterpret_cast<uint32_t(*)[32]>(&x[c]));
        float fs[N / 16], vs[N / 16];
        if (FP8) {
#pragma unroll
            for (int h = 0; h < N / 16; ++h) {
                fs[h] = f * __shfl_sync(0xffffffffu, scales, (N * k + 16 * h) >> shift);
                vs[h] = __shfl_sync(0xffffffffu, scales, 8 + ((N * k + 16 * h) >> shift));
            }
        }
        tmem_wait_ld();
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < N / 16; ++h) {                     // short chains: one warp alone has to fill its pipes
            float g[4];
#pragma unroll
            for (int k2 = 0; k2 < 4; ++k2) {
                const float* y = reinterpret_cast<const float*>(&x[16 * h + 4 * k2]);
                g[k2] = fmaxf(max3(y[0], y[1], y[2]), y[3]);
            }
            const float y = fmaxf(max3(g[0], g[1], g[2]), g[3]);
            mx = fmaxf(mx, FP8 ? y * fs[h] : y);
        }
        if (!FP8) mx *= f;
        if (__any_sync(0xffffffffu, mx > m + kSlack)) {
            const float mn = fmaxf(m, ceilf(mx)), alpha = m == mn ? 1.f : ex2(m - mn);
            if (!first) {          // S of this tile was issued after the last P V of the stream: O is settled
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) tmem_scale16<false>(ocol + (uint32_t)c0, alpha);
            }
            tmem_wait_st();
#pragma unroll 1
            for (int c0 = 0; c0 < N * k; c0 += 16) tmem_scale16<true>(scol + (uint32_t)c0, alpha);
            l *= alpha;
            m = mn;
        }
        const float mref = m == -INFINITY ? 0.f : m;
        const uint64_t m2 = two(-mref, -mref);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < N / 16; ++h) {                     // 16 keys: 8 columns
            const uint64_t f2 = FP8 ? two(fs[h], fs[h]) : two(f, f);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = 16 * h + 2 * i;
                const uint64_t z = fma2(two(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), f2, m2);
                uint64_t e = two(ex2(first_of(z)), ex2(second_of(z)));
                sum[i & 1] = add2(sum[i & 1], e);
                if (FP8) e = mul2(e, two(vs[h], vs[h]));       // the V scale goes into what P V takes, not into the sum
                x[c] = (uint32_t)e;
                x[c + 1] = (uint32_t)(e >> 32);
                w[i] = __byte_perm(x[c], x[c + 1], 0x7632);
            }
            tmem_st8(scol + (uint32_t)(N * k + 8 * h), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = 16 * h + 2 * i;
                const float r0 = fmaf(__uint_as_float(x[c]), kOneUp, -__uint_as_float(x[c] & 0xFFFF0000u)),
                            r1 = fmaf(__uint_as_float(x[c + 1]), kOneUp, -__uint_as_float(x[c + 1] & 0xFFFF0000u));
                w[i] = pack_bf16(r0, r1);
            }
            tmem_st8(scol + (uint32_t)(N * k + N / 2 + 8 * h), w);
        }
        const uint64_t all = add2(sum[0], sum[1]);
        l += first_of(all) + second_of(all);
    }
    tmem_wait_st();
}

// ---- the kernel -------------------------------------------------------------------

template <int D, bool FP8>
__global__ void __launch_bounds__(TreeGeo<D, FP8>::THREADS, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv, const TreeAttnParams p)
{
    using Gm = TreeGeo<D, FP8>;
    constexpr int KB = Gm::KB, NS = Gm::NS, NCX = FP8 ? Gm::NC : 1, SLOT = Gm::SLOT;
    constexpr int THREADS = Gm::THREADS, WARPS = THREADS / 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[NS], s_empty[NS], s_cfull[NCX], s_cempty[NCX];
    __shared__ __align__(8) uint64_t s_qfull[2], s_qempty[2], s_sfull[2], s_pfull[2], s_ofin[2], s_drain;
    __shared__ float2 s_ml[kTRows];
    __shared__ long long s_scan[WARPS];
    __shared__ int4 s_pos[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad, s_fail, s_odd;
    __shared__ int s_issued[kMaxSlots + 2];       // loads issued into each slot, and of each Q

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, W = gridDim.x;
    grid_launch_dependents();

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t q0 = base, ring = base + 2u * SLOT, stage = ring + (uint32_t)(NS * SLOT);
    const uint32_t full = smem_u32(s_full), empty = smem_u32(s_empty), cfull = smem_u32(s_cfull),
                   cempty = smem_u32(s_cempty), qfull = smem_u32(s_qfull), qempty = smem_u32(s_qempty),
                   sfull = smem_u32(s_sfull), pfull = smem_u32(s_pfull), ofin = smem_u32(s_ofin),
                   drain = smem_u32(&s_drain);

    // ---- set up, while the lengths are read
    if (tid == 0) {
        s_bad = 0;
        s_fail = 0;
        s_odd = 0;
        for (int i = 0; i < kMaxSlots + 2; ++i) s_issued[i] = 0;
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + 8u * i, FP8 ? 4u : 1u);
            mbar_init(empty + 8u * i, 1u);
        }
        for (int i = 0; FP8 && i < NCX; ++i) {
            mbar_init(cfull + 8u * i, 1u);
            mbar_init(cempty + 8u * i, 4u);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(qfull + 8u * i, 1u);
            mbar_init(qempty + 8u * i, 1u);
            mbar_init(sfull + 8u * i, 1u);
            mbar_init(pfull + 8u * i, 4u);
            mbar_init(ofin + 8u * i, 1u);
        }
        mbar_init(drain, 1u);
        fence_mbar_init();
    }

    if (warp == 1) {
        __syncwarp();
        tmem_alloc(smem_u32(&s_tmem), kTCols);
    }

    // ---- where this CTA's run starts and ends
    {
        const int per = (p.batch + THREADS - 1) / THREADS;
        const int lo = min(p.batch, tid * per), hi = min(p.batch, lo + per);
        long long mine = 0;
        int err = 0, zero = 0;
        Request r;
        for (int b = lo; b < hi; ++b) {
            const int st = read_request(p, b, r);
            if (st == 1) mine += cost_of(p, r);
            else if (st) err = kErrLength;
            zero |= st == 3;
        }
        if (err && cta == 0) atomicOr(p.err, err);
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) s_scan[warp] = incl;
        if (tid < 2) s_pos[tid] = make_int4(p.batch, 0, 0, 0);
        tmem_fence_before();
        zero = __syncthreads_or(zero);
        tmem_fence_after();
        long long pre = incl - mine, total = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const long long x = s_scan[w];
            if (w < warp) pre += x;
            total += x;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int cut = cta + k;             // total * cut / W, all CTAs by the same arithmetic
            const long long x = cut == W ? total : (long long)__umul64hi((unsigned long long)total, p.run_inv * (unsigned)cut);
            if (x < pre || x >= pre + mine) continue;
            long long at = pre;
            for (int b = lo; b < hi; ++b) {
                if (per > 1 && read_request(p, b, r) != 1) continue;      // with one request a thread, r is it
                const long long c = cost_of(p, r);
                if (x < at + c) {
                    s_pos[k] = place_at(p, b, r, x - at);
                    break;
                }
                at += c;
            }
        }
        __syncthreads();
        if (tid < 2 && (tid == 0 || cta == W - 1)) p.pos[cta + tid] = s_pos[tid];
        // rows of requests whose lengths are out of range
        for (int b = cta; zero && b < p.batch; b += W) {
            if (read_request(p, b, r) != 3) continue;
            uint4* dst = reinterpret_cast<uint4*>(p.out + (size_t)r.row0 * p.Hq * D);
            const size_t n = (size_t)r.T * p.Hq * D / 8;
            for (size_t i = tid; i < n; i += THREADS) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    Walk walk;
    walk.cur = s_pos[0];
    walk.end = s_pos[1];
    const uint32_t tmem = s_tmem;
    if (!before(walk.cur, walk.end)) {            // nothing for the whole CTA
        if (warp == 1) {
            __syncwarp();
            tmem_dealloc(tmem, kTCols);
        }
        return;
    }
    Segment s;

    if (warp < 4) {
        if (warp == 0 || warp == 2) {
            // ---- loads: warp 0 those of Q and K, warp 2 those of V (a box takes
            // about 100 cycles to issue: one warp alone was what bounded pages of
            // 16 tokens).  A warp waits for its own places of the ring only.  A
            // parity tells two phases apart, so that needs its last place within
            // a ring before the next one: they are at most 3 apart.
            const bool is_k = warp == 0;
            constexpr int N = FP8 ? NCX : NS;
            constexpr int ROWB = FP8 ? D : 2 * D;                // bytes of a row in the pool
            const uint32_t lfull = FP8 ? cfull : full, lempty = FP8 ? cempty : empty, dst0 = FP8 ? stage : ring;
            constexpr int LSLOT = FP8 ? Gm::STG : SLOT;
            constexpr int LB = FP8 ? 1 : KB;                     // TMA boxes across a row
            const int ppt = kTKeys / p.P;
            int rb = 0, qc0 = 0, qc1 = 0, qsel = 0;
            bool ok = true;
            auto wait = [&](uint32_t bar, int phase) {
                ok = ok && __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(phase & 1))) != 0;
            };
            while (ok && walk.next(p, s)) {
                const int n_keys = s.L + s.T;
                const int32_t* bt = p.block_tables + (size_t)s.b * p.bt_stride;
                auto page_of = [&](int i) {                      // this lane's page of tile i; -1: out of range, -2: none
                    const int at = (s.t0 + i) * ppt + lane;
                    if (i >= s.n || lane >= ppt || at * p.P >= n_keys) return -2;
                    const int page = __ldg(&bt[at]);
                    return (unsigned)page < (unsigned)p.num_pages ? page : -1;
                };
                auto load_q = [&](int buf, int& count, int token) {
                    if (count > 0) wait(qempty + 8u * buf, count - 1);
                    if (!ok) return;
                    if (elect_one()) {
                        s_issued[kMaxSlots + buf] = count + 1;
                        mbar_arrive_expect_tx(qfull + 8u * buf, (uint32_t)(KB * 128 * p.tb * p.G));
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb)
                            tma_load_3d(q0 + (uint32_t)(buf * SLOT + kb * kTBlk), &tmq, 64 * kb, s.kvh * p.G, token, qfull + 8u * buf);
                    }
                    __syncwarp();
                    ++count;
                };
                int page = page_of(0);
                for (int i = 0; ok && i < s.n; ++i) {
                    const int seq = rb + (is_k ? k_seq(s, i) : v_seq(s, i)), cur = page;
                    page = page_of(i + 1);
                    const int j = seq % N;
                    if (seq >= N) wait(lempty + 8u * j, seq / N - 1);
                    if (!ok) break;
                    if (cur == -1) {                             // its keys are masked, and rows above the pool read as zero
                        s_bad = 1;
                        atomicOr(p.err, kErrPage);
                    }
                    const int np = __popc(__ballot_sync(0xffffffffu, cur != -2));
                    const int y = cur < 0 ? -p.P : (cur * p.Hkv + s.kvh) * p.P;
                    if (elect_one()) {
                        s_issued[j] = seq / N + 1;
                        mbar_arrive_expect_tx(lfull + 8u * j, (uint32_t)(np * p.P * ROWB));
                    }
                    const CUtensorMap* const map = is_k ? &tmk : &tmv;
                    uint32_t dst = dst0 + (uint32_t)(j * LSLOT);
                    for (int k = 0; k < np; ++k) {
                        const int yk = __shfl_sync(0xffffffffu, y, k);
                        if (elect_one()) {
#pragma unroll
                            for (int kb = 0; kb < LB; ++kb) tma_load_2d(dst + (uint32_t)(kb * kTBlk), map, 64 * kb, yk, lfull + 8u * j);
                        }
                        dst += (uint32_t)(p.P * (FP8 ? D : 128));
                    }
                    __syncwarp();
                    if (is_k && i == 0) {                        // the first tile is under way: now Q, once it is free
                        if (s.row_mode) {
                            load_q(0, qc0, s.row0);
                            load_q(1, qc1, s.row0 + p.tb);
                        } else {
                            if (qsel == 0) load_q(0, qc0, s.row0);
                            else load_q(1, qc1, s.row0);
                            qsel ^= 1;
                        }
                    }
                }
                rb += 2 * s.n;
            }
            if (!ok) s_fail = 1;
        } else if (warp == 1) {
            // ---- MMA issue: the warp together, one elected lane for each instruction
            constexpr uint32_t idS = umma_idesc_bf16<kTRows, kTKeys>();
            constexpr uint32_t idO = umma_idesc_bf16<kTRows, D, true>();
            int rb = 0, qsel = 0, qc0 = 0, qc1 = 0, pc0 = 0, pc1 = 0;
            bool ok = true;
            auto wait = [&](uint32_t bar, int phase) {
                ok = ok && __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(phase & 1))) != 0;
            };
            while (ok && walk.next(p, s)) {
                const int qb0 = s.row_mode ? 0 : qsel, qb1 = s.row_mode ? 1 : qsel;
                auto tile_of = [&](int u) { return s.row_mode ? u >> 1 : u; };
                auto k_bar = [&](int u, int& phase) {
                    const int seq = rb + k_seq(s, tile_of(u));
                    phase = seq / NS;
                    return seq % NS;
                };
                // the instructions of S(u), by the elected lane
                auto score = [&](int u, int slot) {
                    const int st = u & 1, qb = st ? qb1 : qb0;
                    const uint64_t qa = sw128_kmajor_desc(q0 + (uint32_t)(qb * SLOT)),
                                   ka = sw128_kmajor_desc(ring + (uint32_t)(slot * SLOT));
                    const uint32_t dcol = tmem + (uint32_t)(st * kTKeys);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t off = (uint64_t)(((kk >> 2) * kTBlk + (kk & 3) * 32) >> 4);
                        umma_bf16_all(dcol, qa + off, ka + off, idS, kk ? 1u : 0u);
                    }
                    umma_commit(sfull + 8u * st);
                    if (!s.row_mode || st) umma_commit(empty + 8u * slot);
                    if (s.row_mode ? u >= s.units - 2 : u == s.units - 1) umma_commit(qempty + 8u * qb);
                };
                wait(qfull + 8u * qb0, qb0 ? qc1 : qc0);
                if (s.row_mode) wait(qfull + 8u, qc1);
                if (s.row_mode || qb0) ++qc1;
                if (s.row_mode || !qb0) ++qc0;
                for (int u = 0; u < 2 && u < s.units; ++u) {
                    int phase;
                    const int slot = k_bar(u, phase);
                    wait(full + 8u * slot, phase);
                    if (!ok) break;
                    tmem_fence_after();
                    if (elect_one()) score(u, slot);
                    __syncwarp();
                }
                // P V(u) and S(u + 2) go out together once P(u) is written; that K
                // has landed is looked at while P is awaited
                for (int u = 0; ok && u < s.units; ++u) {
                    const int st = u & 1, i = tile_of(u);
                    const int vseq = rb + v_seq(s, i), vslot = vseq % NS;
                    const bool next = u + 2 < s.units;
                    int kphase = 0, kslot = 0;
                    if (next) kslot = k_bar(u + 2, kphase);
                    wait(full + 8u * vslot, vseq / NS);
                    const bool k_here = next && __all_sync(0xffffffffu, mbar_try_wait(full + 8u * kslot, (uint32_t)(kphase & 1)));
                    const int steps = (min(kTKeys, s.L + s.T - (s.t0 + i) * kTKeys) + 15) / 16;
                    const uint64_t va = sw128_mnmajor_desc(ring + (uint32_t)(vslot * SLOT), (uint32_t)kTBlk, 1024u);
                    const uint32_t pcol = tmem + (uint32_t)(st * kTKeys), ocol = tmem + kTOcol + (uint32_t)(st * 128);
                    const uint32_t later = u >= 2 ? 1u : 0u;
                    wait(pfull + 8u * st, st ? pc1 : pc0);
                    if (st) ++pc1;
                    else ++pc0;
                    if (!ok) break;
                    tmem_fence_after();
                    if (elect_one()) {
                        // 16 keys each: both terms of P over the same V
                        auto step = [&](int kk) {
                            const uint32_t at = pcol + p_col<FP8>(kk);
                            const uint64_t v = va + (uint64_t)(kk * 128);
                            umma_bf16_ts_all(ocol, at, v, idO, kk ? 1u : later);
                            umma_bf16_ts_all(ocol, at + (uint32_t)(kChunk<FP8> / 2), v, idO, 1u);
                        };
                        if (steps == kTKeys / 16) {
#pragma unroll
                            for (int kk = 0; kk < kTKeys / 16; ++kk) step(kk);
                        } else {
#pragma unroll 1
                            for (int kk = 0; kk < steps; ++kk) step(kk);
                        }
                        if (!s.row_mode || st) umma_commit(empty + 8u * vslot);
                        if (!next) umma_commit(ofin + 8u * st);
                        if (k_here) score(u + 2, kslot);
                    }
                    __syncwarp();
                    if (next && !k_here) {
                        wait(full + 8u * kslot, kphase);
                        if (!ok) break;
                        if (elect_one()) score(u + 2, kslot);
                        __syncwarp();
                    }
                }
                if (!s.row_mode) qsel ^= 1;
                rb += 2 * s.n;
            }
            if (!ok) s_fail = 1;
            if (elect_one()) umma_commit(drain);                   // every MMA has ended before the tensor memory is given back
            (void)mbar_wait_bounded(drain, 0u, kTWaitNs);
            __syncwarp();
        }
    } else if (warp < 12) {
        // ---- softmax and output: row r of stream st
        const int st = (warp - 4) >> 2, quarter = warp & 3, r = 32 * quarter + lane;
        const int rtok = (r * p.g_inv) >> 16, g = r - rtok * p.G;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t scol = lanes + (uint32_t)(st * kTKeys);
        const int shift = 31 - __clz(p.P);
        int rb = 0, sc = 0, oc0 = 0, oc1 = 0;
        bool ok = true;
        auto wait = [&](uint32_t bar, int phase) {
            ok = ok && __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(phase & 1))) != 0;
        };
        auto pair = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory"); };   // the two warps of these lanes
        while (walk.next(p, s)) {
            const int tok0 = s.row_mode ? st * p.tb : 0;
            const int rows = min(p.tb, s.ntok - tok0) * p.G;
            const bool valid = r < rows, act = 32 * quarter < rows;
            const int n_keys = s.L + s.T;
            const int32_t* bt = p.block_tables + (size_t)s.b * p.bt_stride;
            const size_t trow = (size_t)s.row0 + tok0 + rtok;
            const uint32_t* mrow = p.tree_mask + (valid ? trow : (size_t)s.row0) * p.mask_words;
            // word i of the drafted keys this row sees; all cached keys before
            // them.  Those of the first 64 are read ahead.
            auto word = [&](int i) -> uint32_t {
                if (!valid || 32 * i >= s.T) return 0u;
                return __ldg(&mrow[i]) & (s.T - 32 * i < 32 ? (1u << (s.T - 32 * i)) - 1u : ~0u);
            };
            const uint32_t word0 = word(0), word1 = word(1);
            auto seen = [&](int i) -> uint32_t { return i < 0 ? ~0u : i == 0 ? word0 : i == 1 ? word1 : word(i); };
            // E4M3: lanes 0 .. 7 hold the K scales of a tile's pages, 8 .. 15 the V scales, one tile ahead
            const int step = s.row_mode ? 1 : 2, first = s.row_mode ? 0 : st;
            auto page_of = [&](int i) {
                const int at = ((s.t0 + i) << (7 - shift)) + (lane & 7);
                return FP8 && i < s.n && lane < 16 && at * p.P < n_keys && (lane & 7) < (kTKeys >> shift) ? __ldg(&bt[at]) : -1;
            };
            // 1 where there is no page.  K scales of 0 and next to it are made 1e-30
            // (-inf, a masked score, x 0 is no number; scores move by less than
            // 2^-60); V scales stay as they are
            auto scale_of = [&](int page) {
                if (!FP8 || (unsigned)page >= (unsigned)p.num_pages) return 1.f;
                const float x = __ldg(&(lane < 8 ? p.k_scale : p.v_scale)[(size_t)page * p.Hkv + s.kvh]);
                return lane < 8 && x < 1e-30f ? 1e-30f : x;
            };
            float scale_next = 0.f;
            int page_next = -1;
            if (FP8) {
                scale_next = scale_of(page_of(first));
                page_next = page_of(first + step);
            }
            float m = -INFINITY, l = 0.f;
            for (int u = st; u < s.units; u += 2) {
                const int i = s.row_mode ? u >> 1 : u, key0 = (s.t0 + i) * kTKeys;
                float scales = 0.f;
                if (FP8) {
                    scales = scale_next;
                    scale_next = scale_of(page_next);
                    page_next = page_of(i + 2 * step);
                }
                wait(sfull + 8u * st, sc++);
                tmem_fence_after();
                const bool bad = *(volatile int*)&s_bad != 0;
                const bool tail = key0 + kTKeys > s.L;
                if (ok && act) {
                    if (tail || bad) {
                        auto lost = [&](int k) {
                            uint32_t gone = 0u;
#pragma unroll 1
                            for (int c = 0; bad && c < 32; c += 16) {
                                const int at = (key0 + 32 * k + c) >> shift;
                                if (at * p.P < n_keys && (unsigned)__ldg(&bt[at]) >= (unsigned)p.num_pages) gone |= 0xFFFFu << c;
                            }
                            return gone;
                        };
                        tile_mask(scol, key0 - s.L, seen, lost);
                    }
                    tile_softmax<D, FP8>(scol, lanes + kTOcol + (uint32_t)(st * 128), u < 2, p.scale_log2, scales, shift, m, l);
                }
                if (tail && (!s.row_mode || st == 0)) {
                    // V rows behind the last key hold anything: zero them, so that
                    // 0 x V stays 0; and the numbers of drafted tokens that are not
                    // finite, which rows that see them take back at the end
                    const int seq = rb + v_seq(s, i), slot = seq % NS;
                    wait(full + 8u * slot, seq / NS);
                    const uint32_t va = ring + (uint32_t)(slot * SLOT);
                    const int z0 = n_keys - key0, d0 = max(0, s.L - key0);
                    if (ok) {
                        bool wrote = false;
                        const int pieces = (min(kTKeys, (z0 + 15) & ~15) - d0) * KB * 8;      // up to the last step of P V
#pragma unroll 1
                        for (int x = 32 * quarter + lane; x < pieces; x += 128) {
                            const int row = d0 + x / (KB * 8), rem = x % (KB * 8);
                            const uint32_t addr = va + (uint32_t)((rem >> 3) * kTBlk + row * 128 + (rem & 7) * 16);
                            const uint4 v = lds128(addr);
                            uint32_t w[4] = {v.x, v.y, v.z, v.w}, odd[4], any = 0u;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {          // bit 15 of a half: its exponent is all ones
                                odd[k] = ((w[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                                any |= odd[k];
                            }
                            if (row < z0 && !any) continue;
                            if (row < z0) s_odd = 1;
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[k] = row < z0 ? w[k] & ~((odd[k] >> 15) * 0xFFFFu) : 0u;
                            sts128(addr, make_uint4(w[0], w[1], w[2], w[3]));
                            wrote = true;
                        }
                        if (wrote) fence_proxy_async_smem();
                    }
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + 8u * st);
            }

            // ---- the end of the segment
            if (s.row_mode) {
                wait(ofin + 8u * st, st ? oc1 : oc0);
                ++oc0;
                ++oc1;
            } else {
                wait(ofin, oc0++);
                if (s.n > 1) wait(ofin + 8u, oc1++);
            }
            tmem_fence_after();
            float a0 = st == 0 ? 1.f : 0.f, a1 = 1.f - a0;
            if (!s.row_mode) {
                float2 other;
                if (st == 1) s_ml[r] = make_float2(m, l);
                pair();
                if (st == 0) other = s_ml[r];
                pair();
                if (st == 0) s_ml[r] = make_float2(m, l);
                pair();
                if (st == 1) other = s_ml[r];
                const float m0 = st == 0 ? m : other.x, m1 = st == 0 ? other.x : m;
                const float l0 = st == 0 ? l : other.y, l1 = st == 0 ? other.y : l;
                m = fmaxf(m0, m1);
                a0 = m0 == -INFINITY ? 0.f : ex2(m0 - m);
                a1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
                l = l0 * a0 + l1 * a1;
            }
            if (ok && act) {
                const bool both = !s.row_mode && s.n > 1;
                const int cols = s.row_mode ? D : D / 2, col0 = s.row_mode ? 0 : st * (D / 2);
                const float inv = m == -INFINITY ? 0.f : 1.f / l;      // -inf: the row sees nothing
                const bool odd = *(volatile int*)&s_odd != 0;
                const size_t slot_row = ((size_t)(2 * cta + (s.place == 1)) * 2 * kTRows) + (s.row_mode ? st * kTRows : 0) + r;
                __nv_bfloat16* const orow = p.out + (trow * p.Hq + (size_t)s.kvh * p.G + g) * D;
                if (valid && s.place && (s.row_mode || st == 0)) p.part_ml[slot_row] = make_float2(m, l);
#pragma unroll 1
                for (int c0 = col0; c0 < col0 + cols; c0 += 16) {
                    uint32_t x[2][8];
                    float o[16];
                    const uint32_t oc = lanes + kTOcol + (uint32_t)((s.row_mode ? st * 128 : 0) + c0);
                    tmem_ld8(oc, x[0]);
                    tmem_ld8(oc + 8u, x[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) o[c] = __uint_as_float(x[c >> 3][c & 7]) * (s.row_mode ? 1.f : a0);
                    if (both) {
                        tmem_ld8(oc + 128u, x[0]);
                        tmem_ld8(oc + 136u, x[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] = fmaf(a1, __uint_as_float(x[c >> 3][c & 7]), o[c]);
                    }
                    if (!valid) continue;
                    if (s.place == 0) {
#pragma unroll
                        for (int c = 0; c < 16; c += 8)
                            *reinterpret_cast<uint4*>(orow + c0 + c) =
                                make_uint4(pack_bf16(o[c] * inv, o[c + 1] * inv), pack_bf16(o[c + 2] * inv, o[c + 3] * inv),
                                           pack_bf16(o[c + 4] * inv, o[c + 5] * inv), pack_bf16(o[c + 6] * inv, o[c + 7] * inv));
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; c += 4)
                            *reinterpret_cast<float4*>(p.part_o + slot_row * D + c0 + c) =
                                make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                }
                // numbers that are not finite in V of the drafted tokens this row sees
                const int j1 = min(s.T, (s.t0 + s.n) * kTKeys - s.L);
#pragma unroll 1
                for (int j = max(0, s.t0 * kTKeys - s.L); odd && valid && j < j1; ++j) {
                    if (!((seen(j >> 5) >> (j & 31)) & 1u)) continue;
                    const int page = bt[(s.L + j) >> shift];
                    if ((unsigned)page >= (unsigned)p.num_pages) continue;
                    const size_t at = (((size_t)page * p.Hkv + s.kvh) * p.P + ((s.L + j) & (p.P - 1))) * D;
#pragma unroll 1
                    for (int c = col0; c < col0 + cols; ++c) {
                        float v;
                        if (FP8) {
                            const __nv_fp8_storage_t code = reinterpret_cast<const uint8_t*>(p.v_pool)[at + c];
                            v = __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
                        } else {
                            v = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v_pool)[at + c]);
                        }
                        if (isfinite(v)) continue;
                        if (s.place == 0) orow[c] = __float2bfloat16_rn(__bfloat162float(orow[c]) + v);
                        else p.part_o[slot_row * D + c] += v;
                    }
                }
            }
            tmem_fence_before();
            if (!s.row_mode) pair();         // both warps have read both streams' O
            rb += 2 * s.n;
        }
        if (!ok) s_fail = 1;
    } else if (FP8) {
        // ---- codes to bf16: lane l of a warp takes rows 8 k + l % 8, 16 codes l / 8
        // + 4 j.  Eight warps, with the registers of the others, were slower (177
        // us against 169): they take issue slots and instruction fetches from the
        // softmax, whose chain the tiles wait for
        const int w = warp & 3;
        int rb = 0;
        bool ok = true;
        while (ok && walk.next(p, s)) {
            const int end = rb + 2 * s.n;
            for (int q = rb; q < end; ++q) {
                const int c = q % NCX, slot = q % NS;
                ok = __all_sync(0xffffffffu, wait_bar(cfull + 8u * c, (uint32_t)((q / NCX) & 1))) != 0;
                if (ok && q >= NS) ok = __all_sync(0xffffffffu, wait_bar(empty + 8u * slot, (uint32_t)((q / NS - 1) & 1))) != 0;
                if (!ok) break;
                const uint32_t src = stage + (uint32_t)(c * Gm::STG), dst = ring + (uint32_t)(slot * SLOT);
#pragma unroll 1
                for (int j = 0; j < D / 64; ++j) {
                    const int ch = (lane >> 3) + 4 * j;                  // 16 codes: d 16 ch ..
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = 32 * w + 8 * k + (lane & 7);
                        v[k] = lds128(src + (D == 128 ? (uint32_t)(row * 128 + ((ch ^ (row & 7)) << 4))
                                                      : (uint32_t)(row * 64 + ((ch ^ ((row >> 1) & 3)) << 4))));
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = 32 * w + 8 * k + (lane & 7);
                        const uint32_t in[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                        uint32_t o[8];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float2 a = f16x2_to_f32(cvt_lo(in[x])), b = f16x2_to_f32(cvt_hi(in[x]));
                            o[2 * x] = pack_bf16(a.x, a.y);
                            o[2 * x + 1] = pack_bf16(b.x, b.y);
                        }
                        const uint32_t row_at = dst + (uint32_t)((ch >> 2) * kTBlk + row * 128);
                        const int c16 = 2 * (ch & 3);
                        sts128(row_at + (uint32_t)((c16 ^ (row & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
                        sts128(row_at + (uint32_t)(((c16 + 1) ^ (row & 7)) << 4), make_uint4(o[4], o[5], o[6], o[7]));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full + 8u * slot);
                    mbar_arrive(cempty + 8u * c);
                }
            }
            rb = end;
        }
        if (!ok) s_fail = 1;
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, kTCols);
        if (lane == 0 && s_fail) {
            // copies under way land before the CTA's memory is given back
            atomicOr(p.err, kErrTimeout);
            for (int i = 0; i < (FP8 ? NCX : NS); ++i)
                if (s_issued[i]) (void)mbar_wait_bounded((FP8 ? cfull : full) + 8u * i, (uint32_t)((s_issued[i] - 1) & 1), kTWaitNs);
            for (int i = 0; i < 2; ++i)
                if (s_issued[kMaxSlots + i]) (void)mbar_wait_bounded(qfull + 8u * i, (uint32_t)((s_issued[kMaxSlots + i] - 1) & 1), kTWaitNs);
        }
    }
}

// ---- merge of the items that the cut went through -----------------------------------

constexpr int kCombineThreads = 128;
constexpr int kCombineGroups = 8;       // blocks per cut, each a share of the item's rows
constexpr int kRowLanes = 16;           // lanes of a row

// Block (i, y): if cut i + 1 is the first inside its item, the parts of that
// item: the last segment of run i, then the first segments of the runs behind.
// Bound by a chain of dependent loads (places, lengths, parts): 16 lanes take a
// row, and what they need of four parts is under way together.
template <int D>
__global__ void __launch_bounds__(kCombineThreads) tree_combine_kernel(const TreeAttnParams p, int W)
{
    constexpr int E = D / kRowLanes, ROWS = kCombineThreads / kRowLanes;
    __shared__ int4 s_pos[kMaxTreeRuns + 2];
    __shared__ int s_slot[kMaxTreeRuns + 1];
    __shared__ int s_n;
    grid_dependency_wait();
    const int cut = blockIdx.x + 1;
    for (int c = cut - 1 + threadIdx.x; c <= W; c += kCombineThreads) s_pos[c - (cut - 1)] = p.pos[c];
    __syncthreads();
    const int4 a = s_pos[0], x = s_pos[1];
    if (x.w == 0 || (a.w != 0 && same_item(a, x))) return;
    if (threadIdx.x == 0) {
        int n = 0;
        s_slot[n++] = 2 * (cut - 1) + 1;
        for (int c = cut; c < W; ++c) {
            const int4 at = s_pos[c - cut + 1];
            if (at.w == 0 || !same_item(at, x)) break;
            if (before(at, s_pos[c - cut + 2])) s_slot[n++] = 2 * c;
        }
        s_n = n;
    }
    Request r;
    if (read_request(p, x.x, r) != 1) return;         // the same for all
    __syncthreads();
    const int n = s_n, first = x.z * 2 * p.tb, ntok = min(2 * p.tb, r.T - first), rows = ntok * p.G;
    const int lane = threadIdx.x % kRowLanes;
    for (int q = blockIdx.y * ROWS + threadIdx.x / kRowLanes; q < rows; q += kCombineGroups * ROWS) {
        // row q: its token and head, and its place among the parts' rows
        const int half = ntok > p.tb && q >= p.tb * p.G ? 1 : 0, in_half = q - half * p.tb * p.G;
        const int tok_in = (in_half * p.g_inv) >> 16, g = in_half - tok_in * p.G, tok = half * p.tb + tok_in;
        const size_t row = (size_t)(half * kTRows + in_half);
        float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < n; c0 += 4) {
            float2 ml[4];
            float4 v[4][E / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const size_t at = (size_t)s_slot[min(c0 + k, n - 1)] * 2 * kTRows + row;
                ml[k] = p.part_ml[at];
#pragma unroll
                for (int e = 0; e < E / 4; ++e) v[k][e] = *reinterpret_cast<const float4*>(p.part_o + at * D + lane * E + 4 * e);
            }
            // (the last part stands in for those behind it: the maximum is the same)
            const float mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m);
            const float old = m == -INFINITY ? 0.f : ex2(m - mn);
            l *= old;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= old;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (c0 + k >= n) break;
                // A part in which the row sees nothing is (-inf, 0) and O = 0.  One whose
                // scores are no numbers has m = -inf too, as the maximum leaves NaN out,
                // but l and O are NaN, and stay so times 0
                const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - mn);
                l = fmaf(f, ml[k].y, l);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(f, reinterpret_cast<const float*>(v[k])[e], acc[e]);
            }
            m = mn;
        }
        const float inv = m == -INFINITY ? 0.f : 1.f / l;
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) w[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
        __nv_bfloat16* dst = p.out + (((size_t)r.row0 + first + tok) * p.Hq + (size_t)x.y * p.G + g) * D + lane * E;
        if (E == 8) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(w);
        else *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(w);
    }
}

template <int D, bool FP8>
cudaError_t launch_t(const TreeAttnParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                     int runs, cudaStream_t stream)
{
    tree_attn_kernel<D, FP8><<<runs, TreeGeo<D, FP8>::THREADS, TreeGeo<D, FP8>::BYTES, stream>>>(tmq, tmk, tmv, p);
    cudaError_t e = cudaGetLastError();
    // tables of up to 2 kSnap + 1 tiles: every cut lies near an item's end and
    // has moved there, so that nothing is left to merge (4 requests, 14.0 us a
    // call with the launch, 12.3 without)
    if (e != cudaSuccess || runs < 2 || (long long)p.bt_stride * p.P <= (2 * kSnap + 1) * kTKeys) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(runs - 1), kCombineGroups);
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<D>, p, runs);
}

template <int D, bool FP8>
cudaError_t prepare_t()
{
    return cudaFuncSetAttribute(tree_attn_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                TreeGeo<D, FP8>::BYTES);
}

}  // namespace

cudaError_t tree_attn_prepare(int head_dim, bool fp8)
{
    if (head_dim == 128) return fp8 ? prepare_t<128, true>() : prepare_t<128, false>();
    return fp8 ? prepare_t<64, true>() : prepare_t<64, false>();
}

cudaError_t launch_tree_attn(const TreeAttnParams& p, const CUtensorMap& tmq, const CUtensorMap& tmk,
                             const CUtensorMap& tmv, int head_dim, bool fp8, int runs, cudaStream_t stream)
{
    if (head_dim == 128)
        return fp8 ? launch_t<128, true>(p, tmq, tmk, tmv, runs, stream) : launch_t<128, false>(p, tmq, tmk, tmv, runs, stream);
    return fp8 ? launch_t<64, true>(p, tmq, tmk, tmv, runs, stream) : launch_t<64, false>(p, tmq, tmk, tmv, runs, stream);
}

}  // namespace pkv
