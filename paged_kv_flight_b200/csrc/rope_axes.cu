// rope_axes.cu -- rotary embedding at given positions with several axes, and
// the append of k / v at given slots (pkv_rope_append_axes).
//
// "Scaling TensorRT-LLM: Kernel Fusion and Inflight Batching in Production",
// section "What Gets Fused" (RoPE and the cache write in one kernel) and
// section "The Paged KV-Cache"; "TensorRT-LLM Guide: High-Throughput GPU
// Inference Engine", section "4. Native FP8 Quantization" (E4M3 storage).
//
// Mathematics: pair (x_i, x_{i+d/2}) of a head turns by the angle phi_i =
// positions[axis(i)] theta_i: (a cos - b sin, b cos + a sin).  What is stored is
// what pkv_rope_append stores (rope_common.cuh): everything in fp64 from the angle
// on, rounded once, so that caches filled by both calls agree bit for bit.
//
// Most of it is done in fp32 all the same, with the fp64 sine and cosine rounded:
// with u = 2^-24, that is u |a c| + u |b s| for the two roundings, u |b s| for a
// product and u |y| for the fused sum, 3 u (|a| + |b|) at most in all, and 4 u with
// the rounding of the interval's ends below.  Where y - delta and y + delta, delta =
// 5 u (|a| + |b|), round to the same number of the storage type, so does the fp64
// form, which lies between.  The others (some in ten thousand) are done in fp64.
// (All of it in fp64, the conversions from and to bf16 alone, at a quarter of a
// warp a cycle, would take as long as the memory.)
#include "tree_params.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

// One CTA per token; a thread takes 8 pairs of a head at a time (two 16-byte
// loads, neighbouring lanes side by side), the first of them ahead of the angles.
//
// What bounds it: for long calls memory and the instructions (issue slots 69% taken,
// by ncu).  Measured (two B200s): 8192 tokens of 64 + 8 heads of 128, 59.9 and 62.7
// us, 82 to 87% of the measured copy (57.5 in fp32 alone; on the slower one 65.0 with
// every load behind the angles, 83 with no table, the rare values taking their own
// fp64 angles, 93 with 12 CTAs an SM by spilling registers).  64 tokens, 6.1 us a call
// among others: a launch and three dependent loads.
constexpr int kAxesThreads = 128;

constexpr float kDelta = 5.f / (1 << 24);
constexpr float kLeast = 5.6e-45f;             // 2^-147: the roundings next to 0, where fp32 has no more digits

// Element k of 8 as fp32.
__device__ __forceinline__ float element(const uint4& v, int k)
{
    const uint32_t w = k < 4 ? (k < 2 ? v.x : v.y) : (k < 6 ? v.z : v.w);
    return (k & 1) ? dev::bf16_hi(w) : dev::bf16_lo(w);
}

// The largest difference from the fp64 form; 0 for zeros, whose signs are right.
__device__ __forceinline__ float delta_of(float a, float b)
{
    const float size = fabsf(a) + fabsf(b);
    return fminf(size, fmaf(size, kDelta, kLeast));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kAxesThreads) rope_axes_kernel(const RopeAxesParams p)
{
    constexpr int HALF = D / 2;
    constexpr int PIECES = HALF / 8;
    __shared__ float s_cos[HALF], s_sin[HALF];
    __shared__ double s_cos64[HALF], s_sin64[HALF];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int slot = p.slots[t];
    if (slot == -1) return;
    const int page = slot >> p.page_shift, place = slot & (p.P - 1);
    if (slot < 0 || page >= p.num_pages) {
        if (tid == 0) atomicOr(p.err, kErrPage);
        return;
    }
    const int items = (p.Hq + p.Hkv) * PIECES;
    uint4 xa = make_uint4(0u, 0u, 0u, 0u), xb = xa;
    auto load = [&](int it) {
        const int r = it / PIECES, i0 = (it - r * PIECES) * 8;
        const __nv_bfloat16* src = r < p.Hq ? p.q + ((size_t)t * p.Hq + r) * D : p.k_new + ((size_t)t * p.Hkv + r - p.Hq) * D;
        xa = *reinterpret_cast<const uint4*>(src + i0);
        xb = *reinterpret_cast<const uint4*>(src + i0 + HALF);
    };
    if (tid < items) load(tid);
    for (int i = tid; i < HALF; i += kAxesThreads) {
        int a;
        if (p.interleaved) {
            a = i % p.n_axes;
            if (i >= p.bound[a]) a = 0;
        } else {
            a = 0;
            while (i >= p.bound[a]) ++a;        // the last bound is HALF
        }
        double s, c;
        dev::rope_sincos((double)p.positions[(size_t)a * p.n_tokens + t] * p.theta[i], &s, &c);
        s_cos64[i] = c;
        s_sin64[i] = s;
        s_cos[i] = (float)c;
        s_sin[i] = (float)s;
    }
    __syncthreads();
    for (int it = tid; it < items; it += kAxesThreads) {
        const int r = it / PIECES, i0 = (it - r * PIECES) * 8;
        const bool is_q = r < p.Hq;
        const int kvh = r - p.Hq;
        if (it != tid) load(it);
        float ya[8], yb[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float a = element(xa, k), b = element(xb, k);
            const float c = s_cos[i0 + k], s = s_sin[i0 + k];
            ya[k] = a * c - b * s;
            yb[k] = b * c + a * s;
        }
        // both values of pair k in fp64
        auto exact = [&](int k, double& a64, double& b64) {
            dev::rope_rotate((double)element(xa, k), (double)element(xb, k), s_cos64[i0 + k], s_sin64[i0 + k], &a64, &b64);
        };
        const size_t row = ((size_t)page * p.Hkv + kvh) * p.P + place;
        uint32_t again = 0u;                    // bit k: pair k may round another way
        if (is_q || !FP8) {
            __nv_bfloat16* dst =
                is_q ? p.q_out + ((size_t)t * p.Hq + r) * D : reinterpret_cast<__nv_bfloat16*>(p.k_pool) + row * D;
            uint32_t wa[4], wb[4];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const float d0 = delta_of(element(xa, k), element(xb, k)), d1 = delta_of(element(xa, k + 1), element(xb, k + 1));
                wa[k / 2] = dev::pack_bf16(ya[k] - d0, ya[k + 1] - d1);
                wb[k / 2] = dev::pack_bf16(yb[k] - d0, yb[k + 1] - d1);
                const uint32_t ha = dev::pack_bf16(ya[k] + d0, ya[k + 1] + d1), hb = dev::pack_bf16(yb[k] + d0, yb[k + 1] + d1);
                if ((wa[k / 2] ^ ha) | (wb[k / 2] ^ hb)) again |= 3u << k;
            }
            *reinterpret_cast<uint4*>(dst + i0) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
            *reinterpret_cast<uint4*>(dst + i0 + HALF) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
            asm volatile("" ::: "memory");      // single values over them, of another type
#pragma unroll 1
            for (; again; again &= again - 1u) {
                const int k = __ffs(again) - 1;
                double a64, b64;
                exact(k, a64, b64);
                dst[i0 + k] = dev::bf16_from_f64(a64);
                dst[i0 + HALF + k] = dev::bf16_from_f64(b64);
            }
        }
        if (is_q) continue;
        const __nv_bfloat16* vsrc = p.v_new + ((size_t)t * p.Hkv + kvh) * D;
        const uint4 va = *reinterpret_cast<const uint4*>(vsrc + i0), vb = *reinterpret_cast<const uint4*>(vsrc + i0 + HALF);
        if (!FP8) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.v_pool) + row * D;
            *reinterpret_cast<uint4*>(dst + i0) = va;
            *reinterpret_cast<uint4*>(dst + i0 + HALF) = vb;
        } else {
            const float sk = p.k_scale[(size_t)page * p.Hkv + kvh], sv = p.v_scale[(size_t)page * p.Hkv + kvh];
            // y / sk by the reciprocal: 2 u for its rounding and the product's, u for
            // that of the quotient
            const float inv = 1.f / sk;
            if (!(inv < INFINITY)) again = 0xFFu;        // a scale of 0 or next to it
            uint8_t ka[8], kb[8], oa[8], ob[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float za = ya[k] * inv, zb = yb[k] * inv,
                            d = fmaf(4.f * delta_of(element(xa, k), element(xb, k)), inv, kLeast);
                ka[k] = dev::e4m3_satfinite(za - d);
                kb[k] = dev::e4m3_satfinite(zb - d);
                if (ka[k] != dev::e4m3_satfinite(za + d) || kb[k] != dev::e4m3_satfinite(zb + d)) again |= 1u << k;
                oa[k] = dev::e4m3_satfinite(__fdiv_rn(element(va, k), sv));
                ob[k] = dev::e4m3_satfinite(__fdiv_rn(element(vb, k), sv));
            }
            uint8_t* kd = reinterpret_cast<uint8_t*>(p.k_pool) + row * D + i0;
            uint8_t* vd = reinterpret_cast<uint8_t*>(p.v_pool) + row * D + i0;
            *reinterpret_cast<uint2*>(kd) = *reinterpret_cast<const uint2*>(ka);
            *reinterpret_cast<uint2*>(kd + HALF) = *reinterpret_cast<const uint2*>(kb);
            *reinterpret_cast<uint2*>(vd) = *reinterpret_cast<const uint2*>(oa);
            *reinterpret_cast<uint2*>(vd + HALF) = *reinterpret_cast<const uint2*>(ob);
            asm volatile("" ::: "memory");
#pragma unroll 1
            for (; again; again &= again - 1u) {
                const int k = __ffs(again) - 1;
                double a64, b64;
                exact(k, a64, b64);
                kd[k] = dev::e4m3_satfinite(__double2float_rn(__ddiv_rn(a64, (double)sk)));
                kd[HALF + k] = dev::e4m3_satfinite(__double2float_rn(__ddiv_rn(b64, (double)sk)));
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxesParams& p, int head_dim, bool fp8, cudaStream_t stream)
{
    const unsigned grid = (unsigned)p.n_tokens;
    if (head_dim == 128) {
        if (fp8) rope_axes_kernel<128, true><<<grid, kAxesThreads, 0, stream>>>(p);
        else rope_axes_kernel<128, false><<<grid, kAxesThreads, 0, stream>>>(p);
    } else {
        if (fp8) rope_axes_kernel<64, true><<<grid, kAxesThreads, 0, stream>>>(p);
        else rope_axes_kernel<64, false><<<grid, kAxesThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace pkv
