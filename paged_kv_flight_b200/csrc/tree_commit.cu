// tree_commit.cu -- the accepted path of a verified tree moved to the front
// of its drafted slots (pkv_tree_commit).
//
// "Scaling TensorRT-LLM: Kernel Fusion and Inflight Batching in Production",
// section "3. Speculative Decoding for Tail Latency" (the accepted prefix of
// the drafted tokens is kept); section "The Paged KV-Cache".
//
// K and V of slot L + path[j] go to slot L + j.  path is strictly increasing
// from 0 up, so path[j] >= j: a row is never overwritten by the rows before
// it.  The rows go in waves: every thread holds its 16 bytes of K and of V in
// registers, a barrier, then the stores; a later wave's sources lie behind
// all destinations so far, so one barrier per wave is enough.
//
// What bounds it: latency (the moved rows are a few MB at most: a chain of
// dependent loads, lengths and path, table entries, rows, and one launch).  The
// places of the first 128 moves stay in shared memory from the check to the
// move.  One CTA takes 8 kv heads of a request (with a CTA for each head the
// launch of 2048 of them bounded a batch of 256), the CTAs of a request are a
// cluster: each arrives at its barrier once it has read seq_lens, and one waits
// there before it writes lens_out, which may be the same.
//
// Measured (B200, a call among others): 256 requests, paths of 8, 8 kv heads, E4M3,
// 6.2 us (8.2 with a CTA a head); 4 requests, paths of 5, bf16, 4.9, the host.
#include "tree_params.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitHeads = 8;             // kv heads of a CTA
constexpr int kCommitRows = 4;              // rows that a thread holds at once

// 4 E4M3 codes of one scale stored under another: fl32(code * from) / to.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float from, float to)
{
    const float2 a = dev::f16x2_to_f32(dev::cvt_lo(w)), b = dev::f16x2_to_f32(dev::cvt_hi(w));
    return (uint32_t)dev::e4m3_satfinite(__fdiv_rn(__fmul_rn(a.x, from), to)) |
           ((uint32_t)dev::e4m3_satfinite(__fdiv_rn(__fmul_rn(a.y, from), to)) << 8) |
           ((uint32_t)dev::e4m3_satfinite(__fdiv_rn(__fmul_rn(b.x, from), to)) << 16) |
           ((uint32_t)dev::e4m3_satfinite(__fdiv_rn(__fmul_rn(b.y, from), to)) << 24);
}

__device__ __forceinline__ uint4 rescale16(uint4 v, float from, float to)
{
    return make_uint4(rescale4(v.x, from, to), rescale4(v.y, from, to), rescale4(v.z, from, to),
                      rescale4(v.w, from, to));
}

// Grid (cluster size, batch): rank blockIdx.x of request blockIdx.y takes the
// kv heads 8 rank .., 8 (rank + cluster size) .., and so on.
template <int D, bool FP8>
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const TreeCommitParams p)
{
    constexpr int CHUNKS = D * (FP8 ? 1 : 2) / 16;          // 16-byte pieces of a row
    constexpr int STEP = kCommitThreads / CHUNKS / kCommitHeads;     // rows of all threads together
    constexpr int ROWS = STEP * kCommitRows;                // rows per wave
    __shared__ int2 s_move[kCommitThreads];                 // rows (page x P + place) that entry j goes from and to
    const int b = blockIdx.y, tid = threadIdx.x;
    const int32_t* path = p.path + (size_t)b * p.path_stride;
    const int32_t* table = p.block_tables + (size_t)b * p.bt_stride;
    int a = tid < p.path_stride ? __ldg(&path[tid]) : 0;    // on its way with the lengths
    int before = tid > 0 && tid < p.path_stride ? __ldg(&path[tid - 1]) : -1;
    const int L = p.seq_lens[b], n = p.path_lens[b];
    const long long cap = min((long long)p.bt_stride * p.P, kMaxTreeKeys);
    int bad = L < 0 || n < 0 || n > p.path_stride || (long long)L + n > cap ? kErrLength : 0;
    if (!bad) {
        for (int j = tid; j < n; j += kCommitThreads) {
            if (j != tid) {
                a = path[j];
                before = path[j - 1];
            }
            if (a <= before || before < -1) {
                bad |= kErrOrder;
            } else if ((long long)L + a >= cap) {
                bad |= kErrLength;
            } else {
                const int p0 = table[(L + a) >> p.page_shift], p1 = table[(L + j) >> p.page_shift];
                if ((unsigned)p0 >= (unsigned)p.num_pages || (unsigned)p1 >= (unsigned)p.num_pages) bad |= kErrPage;
                if (j == tid) s_move[j] = make_int2(p0 * p.P + ((L + a) & (p.P - 1)), p1 * p.P + ((L + j) & (p.P - 1)));
            }
        }
    }
    const bool good = !__syncthreads_or(bad);
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    if (bad && blockIdx.x == 0) atomicOr(p.err, bad);
    if (good) {
        const int chunk = tid % CHUNKS, head = tid / CHUNKS % kCommitHeads, r = tid / CHUNKS / kCommitHeads;
        for (int h0 = blockIdx.x * kCommitHeads; h0 < p.Hkv; h0 += gridDim.x * kCommitHeads) {
            const int kvh = h0 + head;
            for (int j0 = 0; j0 < n; j0 += ROWS) {
                uint4 k[kCommitRows], v[kCommitRows];
                size_t to[kCommitRows];
                bool moves[kCommitRows];
#pragma unroll
                for (int i = 0; i < kCommitRows; ++i) {
                    const int j = j0 + r + i * STEP;
                    int2 at = make_int2(0, 0);
                    if (j < n && kvh < p.Hkv) {
                        if (j < kCommitThreads) {
                            at = s_move[j];
                        } else {
                            const int src = L + path[j], dst = L + j;
                            at = make_int2(table[src >> p.page_shift] * p.P + (src & (p.P - 1)),
                                           table[dst >> p.page_shift] * p.P + (dst & (p.P - 1)));
                        }
                    }
                    moves[i] = at.x != at.y;
                    if (!moves[i]) continue;
                    const int p0 = at.x >> p.page_shift, p1 = at.y >> p.page_shift;
                    const size_t from = (((size_t)p0 * p.Hkv + kvh) * p.P + (at.x & (p.P - 1))) * CHUNKS + chunk;
                    to[i] = (((size_t)p1 * p.Hkv + kvh) * p.P + (at.y & (p.P - 1))) * CHUNKS + chunk;
                    k[i] = reinterpret_cast<const uint4*>(p.k_pool)[from];
                    v[i] = reinterpret_cast<const uint4*>(p.v_pool)[from];
                    if (FP8 && p0 != p1) {
                        const size_t s0 = (size_t)p0 * p.Hkv + kvh, s1 = (size_t)p1 * p.Hkv + kvh;
                        const float k0 = __ldg(&p.k_scale[s0]), k1 = __ldg(&p.k_scale[s1]), v0 = __ldg(&p.v_scale[s0]),
                                    v1 = __ldg(&p.v_scale[s1]);
                        if (k0 != k1) k[i] = rescale16(k[i], k0, k1);
                        if (v0 != v1) v[i] = rescale16(v[i], v0, v1);
                    }
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kCommitRows; ++i) {
                    if (!moves[i]) continue;
                    reinterpret_cast<uint4*>(p.k_pool)[to[i]] = k[i];
                    reinterpret_cast<uint4*>(p.v_pool)[to[i]] = v[i];
                }
            }
        }
    }
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (blockIdx.x == 0 && tid == 0) p.lens_out[b] = good ? L + n : L;
}

template <int D, bool FP8>
cudaError_t launch_t(const TreeCommitParams& p, cudaStream_t stream)
{
    int size = 1;                       // CTAs per request: a power of two, at most 8
    while (size < 8 && size * kCommitHeads < p.Hkv) size *= 2;
    if (size == 1) {                    // a cluster of one needs no attribute
        tree_commit_kernel<D, FP8><<<dim3(1, (unsigned)p.batch), kCommitThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size, (unsigned)p.batch);
    cfg.blockDim = dim3(kCommitThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_commit_kernel<D, FP8>, p);
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitParams& p, int head_dim, bool fp8, cudaStream_t stream)
{
    if (head_dim == 128) return fp8 ? launch_t<128, true>(p, stream) : launch_t<128, false>(p, stream);
    return fp8 ? launch_t<64, true>(p, stream) : launch_t<64, false>(p, stream);
}

}  // namespace pkv
