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
// dependent loads, table entry to row, and one launch).  One CTA per request
// and kv head; the CTAs of a request are a cluster, whose barrier lets one of
// them write lens_out after all have read seq_lens, which may be the same.
#include "tree_params.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kCommitThreads = 128;

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
// kv heads rank, rank + cluster size, ...
template <int D, bool FP8>
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const TreeCommitParams p)
{
    constexpr int CHUNKS = D * (FP8 ? 1 : 2) / 16;          // 16-byte pieces of a row
    constexpr int ROWS = kCommitThreads / CHUNKS;           // rows per wave
    const int b = blockIdx.y, tid = threadIdx.x;
    const int L = p.seq_lens[b], n = p.path_lens[b];
    const int32_t* path = p.path + (size_t)b * p.path_stride;
    const int32_t* table = p.block_tables + (size_t)b * p.bt_stride;
    const long long cap = (long long)p.bt_stride * p.P;
    int bad = L < 0 || n < 0 || n > p.path_stride || (long long)L + n > cap ? kErrLength : 0;
    if (!bad) {
        for (int j = tid; j < n; j += kCommitThreads) {
            const int a = path[j], before = j ? path[j - 1] : -1;
            if (a <= before || before < -1) bad |= kErrOrder;
            else if ((long long)L + a >= cap) bad |= kErrLength;
            else if ((unsigned)table[(L + a) / p.P] >= (unsigned)p.num_pages ||
                     (unsigned)table[(L + j) / p.P] >= (unsigned)p.num_pages)
                bad |= kErrPage;
        }
    }
    const bool good = !__syncthreads_or(bad);
    if (bad && blockIdx.x == 0) atomicOr(p.err, bad);
    if (good) {
        const int chunk = tid % CHUNKS, r = tid / CHUNKS;
        for (int kvh = blockIdx.x; kvh < p.Hkv; kvh += gridDim.x) {
            for (int j0 = 0; j0 < n; j0 += ROWS) {
                const int j = j0 + r;
                const int a = j < n ? path[j] : j;
                uint4 k, v;
                size_t to = 0;
                if (a != j) {
                    const int p0 = table[(L + a) / p.P], p1 = table[(L + j) / p.P];
                    const size_t from = (((size_t)p0 * p.Hkv + kvh) * p.P + (L + a) % p.P) * CHUNKS + chunk;
                    to = (((size_t)p1 * p.Hkv + kvh) * p.P + (L + j) % p.P) * CHUNKS + chunk;
                    k = reinterpret_cast<const uint4*>(p.k_pool)[from];
                    v = reinterpret_cast<const uint4*>(p.v_pool)[from];
                    if (FP8 && p0 != p1) {
                        const size_t s0 = (size_t)p0 * p.Hkv + kvh, s1 = (size_t)p1 * p.Hkv + kvh;
                        const float k0 = p.k_scale[s0], k1 = p.k_scale[s1], v0 = p.v_scale[s0], v1 = p.v_scale[s1];
                        if (k0 != k1) k = rescale16(k, k0, k1);
                        if (v0 != v1) v = rescale16(v, v0, v1);
                    }
                }
                __syncthreads();
                if (a != j) {
                    reinterpret_cast<uint4*>(p.k_pool)[to] = k;
                    reinterpret_cast<uint4*>(p.v_pool)[to] = v;
                }
            }
        }
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (blockIdx.x == 0 && tid == 0) p.lens_out[b] = good ? L + n : L;
}

template <int D, bool FP8>
cudaError_t launch_t(const TreeCommitParams& p, cudaStream_t stream)
{
    int size = 1;                       // CTAs per request: a power of two up to the kv heads, at most 8
    while (size * 2 <= p.Hkv && size < 8) size *= 2;
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
