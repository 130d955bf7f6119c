// tree_attn.cu -- attention of a tree of drafted tokens over the paged cache
// (pkv_decode_attn_tree).
//
// "Scaling TensorRT-LLM: Kernel Fusion and Inflight Batching in Production",
// section "3. Speculative Decoding for Tail Latency" (a draft proposes tokens
// and the target model checks all of them in one forward pass).
//
// One CTA per (new token, kv head), the G query heads of the group together;
// its warps take the keys in turn, each with a running maximum and sum per
// head, and are merged at the end.
#include "tree_params.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

using namespace dev;

constexpr int kTreeWarps = 4;

template <int D, bool FP8>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_attn_kernel(const TreeAttnParams p)
{
    constexpr int E = D / 32;            // elements of a row per lane
    __shared__ float s_o[kTreeWarps][kMaxGroup][D], s_m[kTreeWarps][kMaxGroup], s_l[kTreeWarps][kMaxGroup];
    const int row = blockIdx.x, kvh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_q[mid] <= row) lo = mid;
        else hi = mid;
    }
    const int b = lo, a = p.cu_q[b], e = p.cu_q[b + 1];
    if (a < 0 || e > p.n_tokens || a > e) {
        if (tid == 0) atomicOr(p.err, kErrLength);
        return;
    }
    if (row < a || row >= e) return;
    const int L = p.seq_lens[b], T = e - a;
    const bool ok = L >= 0 && (long long)L + T <= (long long)p.bt_stride * p.P && T <= 32 * p.mask_words;
    if (!ok && tid == 0) atomicOr(p.err, kErrLength);
    const int keys = ok ? L + T : 0;
    float q[kMaxGroup][E], o[kMaxGroup][E], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            o[g][i] = 0.f;
            q[g][i] = g < p.G ? __bfloat162float(p.q[((size_t)row * p.Hq + kvh * p.G + g) * D + lane + 32 * i]) : 0.f;
        }
    }
    for (int j = warp; j < keys; j += kTreeWarps) {
        const int d = j - L;
        if (d >= 0 && !((p.tree_mask[(size_t)row * p.mask_words + d / 32] >> (d & 31)) & 1u)) continue;
        const int page = p.block_tables[(size_t)b * p.bt_stride + j / p.P];
        if ((unsigned)page >= (unsigned)p.num_pages) {
            if (lane == 0) atomicOr(p.err, kErrPage);
            continue;
        }
        const size_t at = (((size_t)page * p.Hkv + kvh) * p.P + j % p.P) * D;
        float k[E], v[E], ks = 1.f, vs = 1.f;
        if (FP8) {
            ks = p.k_scale[(size_t)page * p.Hkv + kvh];
            vs = p.v_scale[(size_t)page * p.Hkv + kvh];
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (FP8) {
                const __nv_fp8_storage_t kc = reinterpret_cast<const uint8_t*>(p.k_pool)[at + lane + 32 * i];
                const __nv_fp8_storage_t vc = reinterpret_cast<const uint8_t*>(p.v_pool)[at + lane + 32 * i];
                k[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(kc, __NV_E4M3))) * ks;
                v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(vc, __NV_E4M3))) * vs;
            } else {
                k[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.k_pool)[at + lane + 32 * i]);
                v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.v_pool)[at + lane + 32 * i]);
            }
        }
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
            if (g >= p.G) break;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) s += q[g][i] * k[i];
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, w);
            s *= p.scale_log2;
            const float mn = fmaxf(m[g], s), al = exp2f(m[g] - mn), pr = exp2f(s - mn);
            m[g] = mn;
            l[g] = l[g] * al + pr;
#pragma unroll
            for (int i = 0; i < E; ++i) o[g][i] = o[g][i] * al + pr * v[i];
        }
    }
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
#pragma unroll
        for (int i = 0; i < E; ++i) s_o[warp][g][lane + 32 * i] = o[g][i];
        if (lane == 0) {
            s_m[warp][g] = m[g];
            s_l[warp][g] = l[g];
        }
    }
    __syncthreads();
    for (int x = tid; x < p.G * D; x += kTreeWarps * 32) {
        const int g = x / D, c = x - g * D;
        float mx = -INFINITY, sum = 0.f, acc = 0.f;
        for (int w = 0; w < kTreeWarps; ++w) mx = fmaxf(mx, s_m[w][g]);
        for (int w = 0; w < kTreeWarps; ++w) {
            const float f = s_m[w][g] == -INFINITY ? 0.f : exp2f(s_m[w][g] - mx);
            sum += s_l[w][g] * f;
            acc += s_o[w][g][c] * f;
        }
        p.out[((size_t)row * p.Hq + kvh * p.G + g) * D + c] = __float2bfloat16_rn(mx == -INFINITY ? 0.f : acc / sum);
    }
}

}  // namespace

cudaError_t launch_tree_attn(const TreeAttnParams& p, int head_dim, bool fp8, cudaStream_t stream)
{
    const dim3 grid((unsigned)p.n_tokens, (unsigned)p.Hkv), block(kTreeWarps * 32);
    if (head_dim == 128) {
        if (fp8) tree_attn_kernel<128, true><<<grid, block, 0, stream>>>(p);
        else tree_attn_kernel<128, false><<<grid, block, 0, stream>>>(p);
    } else {
        if (fp8) tree_attn_kernel<64, true><<<grid, block, 0, stream>>>(p);
        else tree_attn_kernel<64, false><<<grid, block, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace pkv
