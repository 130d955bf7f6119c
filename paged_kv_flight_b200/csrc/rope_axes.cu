// rope_axes.cu -- rotary embedding at given positions with several axes, and
// the append of k / v at given slots (pkv_rope_append_axes).
//
// "Scaling TensorRT-LLM: Kernel Fusion and Inflight Batching in Production",
// section "What Gets Fused" (RoPE and the cache write in one kernel) and
// section "The Paged KV-Cache"; "TensorRT-LLM Guide: High-Throughput GPU
// Inference Engine", section "4. Native FP8 Quantization" (E4M3 storage).
//
// Mathematics: pair (x_i, x_{i+d/2}) of a head turns by the angle phi_i =
// positions[axis(i)] theta_i: (a cos - b sin, b cos + a sin).  The angle is
// taken in turns, pos * (theta_i / 2 pi) in fp64, and its whole turns are
// dropped exactly there, so that far positions keep their fraction (an fp32
// product would lose it: 2^-24 of 60000 radians is 4e-3 radians); what is left
// is at most half a turn and goes on in fp32, as does the rotation (errors of
// 2^-23, far below the 2^-9 of the bf16 that it is rounded to, once).
#include "tree_params.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

// One CTA per token; a thread takes 8 pairs of a head at a time (two 16-byte
// loads, neighbouring lanes side by side).
//
// What bounds it: memory for long calls.  Measured (B200): 8192 tokens of 64 + 8
// heads of 128, 57.5 us, 90% of the measured copy (with 64 threads a CTA 58.0,
// 192 58.9, 288 70.5; with the first loads ahead of the angles 59.5, their
// registers cost more than the wait that the other CTAs hide anyway).  64
// tokens, 6.8 us on the device: a launch and three dependent loads.
constexpr int kAxesThreads = 128;

template <int D, bool FP8>
__global__ void __launch_bounds__(kAxesThreads) rope_axes_kernel(const RopeAxesParams p)
{
    constexpr int HALF = D / 2;
    constexpr int PIECES = HALF / 8;
    constexpr double kInvTwoPi = 0.15915494309189535;
    __shared__ float s_cos[HALF], s_sin[HALF];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int slot = p.slots[t];
    if (slot == -1) return;
    const int page = slot >> p.page_shift, place = slot & (p.P - 1);
    if (slot < 0 || page >= p.num_pages) {
        if (tid == 0) atomicOr(p.err, kErrPage);
        return;
    }
    for (int i = tid; i < HALF; i += kAxesThreads) {
        int a;
        if (p.interleaved) {
            a = i % p.n_axes;
            if (i >= p.bound[a]) a = 0;
        } else {
            a = 0;
            while (i >= p.bound[a]) ++a;        // the last bound is HALF
        }
        const double turns = (double)p.positions[(size_t)a * p.n_tokens + t] * (p.theta[i] * kInvTwoPi);
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        s_cos[i] = c;
        s_sin[i] = s;
    }
    __syncthreads();
    const int items = (p.Hq + p.Hkv) * PIECES;
    for (int it = tid; it < items; it += kAxesThreads) {
        const int r = it / PIECES, i0 = (it - r * PIECES) * 8;
        const bool is_q = r < p.Hq;
        const int kvh = r - p.Hq;
        const __nv_bfloat16* src = is_q ? p.q + ((size_t)t * p.Hq + r) * D : p.k_new + ((size_t)t * p.Hkv + kvh) * D;
        const uint4 xa = *reinterpret_cast<const uint4*>(src + i0), xb = *reinterpret_cast<const uint4*>(src + i0 + HALF);
        const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
        float ya[8], yb[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float a = (k & 1) ? dev::bf16_hi(wa[k >> 1]) : dev::bf16_lo(wa[k >> 1]);
            const float b = (k & 1) ? dev::bf16_hi(wb[k >> 1]) : dev::bf16_lo(wb[k >> 1]);
            const float c = s_cos[i0 + k], s = s_sin[i0 + k];
            ya[k] = a * c - b * s;
            yb[k] = b * c + a * s;
        }
        const size_t row = ((size_t)page * p.Hkv + kvh) * p.P + place;
        if (is_q || !FP8) {
            __nv_bfloat16* dst =
                is_q ? p.q_out + ((size_t)t * p.Hq + r) * D : reinterpret_cast<__nv_bfloat16*>(p.k_pool) + row * D;
            *reinterpret_cast<uint4*>(dst + i0) =
                make_uint4(dev::pack_bf16(ya[0], ya[1]), dev::pack_bf16(ya[2], ya[3]), dev::pack_bf16(ya[4], ya[5]),
                           dev::pack_bf16(ya[6], ya[7]));
            *reinterpret_cast<uint4*>(dst + i0 + HALF) =
                make_uint4(dev::pack_bf16(yb[0], yb[1]), dev::pack_bf16(yb[2], yb[3]), dev::pack_bf16(yb[4], yb[5]),
                           dev::pack_bf16(yb[6], yb[7]));
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
            const uint32_t va4[4] = {va.x, va.y, va.z, va.w}, vb4[4] = {vb.x, vb.y, vb.z, vb.w};
            uint8_t ka[8], kb[8], oa[8], ob[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float a = (k & 1) ? dev::bf16_hi(va4[k >> 1]) : dev::bf16_lo(va4[k >> 1]);
                const float b = (k & 1) ? dev::bf16_hi(vb4[k >> 1]) : dev::bf16_lo(vb4[k >> 1]);
                ka[k] = dev::e4m3_satfinite(__fdiv_rn(ya[k], sk));
                kb[k] = dev::e4m3_satfinite(__fdiv_rn(yb[k], sk));
                oa[k] = dev::e4m3_satfinite(__fdiv_rn(a, sv));
                ob[k] = dev::e4m3_satfinite(__fdiv_rn(b, sv));
            }
            uint8_t* kd = reinterpret_cast<uint8_t*>(p.k_pool) + row * D + i0;
            uint8_t* vd = reinterpret_cast<uint8_t*>(p.v_pool) + row * D + i0;
            *reinterpret_cast<uint2*>(kd) = *reinterpret_cast<const uint2*>(ka);
            *reinterpret_cast<uint2*>(kd + HALF) = *reinterpret_cast<const uint2*>(kb);
            *reinterpret_cast<uint2*>(vd) = *reinterpret_cast<const uint2*>(oa);
            *reinterpret_cast<uint2*>(vd + HALF) = *reinterpret_cast<const uint2*>(ob);
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
