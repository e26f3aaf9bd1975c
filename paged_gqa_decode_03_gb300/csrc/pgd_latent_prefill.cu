// Causal attention over packed prompts with keys and values expanded from latent vectors
// (packed_latent_prefill).  A warp per query row and head, one pass over the tokens with a
// running maximum and sum.
#include "pgd_device.cuh"
#include "pgd_internal.h"

namespace pgd {

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x += __shfl_xor_sync(~0u, x, o);
    return x;
}

__global__ void __launch_bounds__(128) packed_latent_prefill_kernel(const LatentPrefillParams p)
{
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * 4 + (threadIdx.x >> 5), row = blockIdx.x;
    if (h >= p.H)
        return;
    int s = -1, row0 = 0;
    for (int i = 0; i < p.S; ++i) {
        const int a = __ldg(p.cu_seqlens + i), n = __ldg(p.cu_seqlens + i + 1) - a;
        if (n < 0 || n > p.max_len || a < 0 || a > p.total - n) {
            if (row == 0 && h == 0 && lane == 0)
                atomicOr(p.err, kErrQueryLen);
        } else if (row >= a && row < a + n) {
            s = i;
            row0 = a;
        }
    }
    if (s < 0)
        return;
    float q[4], qr[2], o[4];
    const __half *qp = p.q + (size_t)row * p.q_token + (size_t)h * p.q_head;
    for (int k = 0; k < 4; ++k) {
        const int d = lane + 32 * k;
        q[k] = d < p.D ? __half2float(qp[d]) : 0.f;
        o[k] = 0.f;
    }
    for (int k = 0; k < 2; ++k)
        qr[k] = lane + 32 * k < p.P ? __half2float(qp[p.D + lane + 32 * k]) : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int t = row0; t <= row; ++t) {
        const __half *kp = p.k + (size_t)t * p.k_token + (size_t)h * p.k_head;
        const __half *vp = p.v + (size_t)t * p.v_token + (size_t)h * p.v_head;
        float dot = 0.f;
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < p.D)
                dot += q[k] * __half2float(kp[lane + 32 * k]);
        for (int k = 0; k < 2; ++k)
            if (lane + 32 * k < p.P)
                dot += qr[k] * __half2float(p.k_rope[(size_t)t * p.kr_token + lane + 32 * k]);
        const float x = warp_sum(dot) * p.scale_log2, top = fmaxf(m, x);
        const float keep = ex2(m - top), w = ex2(x - top);
        l = l * keep + w;
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < p.D)
                o[k] = o[k] * keep + w * __half2float(vp[lane + 32 * k]);
        m = top;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int k = 0; k < 4; ++k) {
        const int d = lane + 32 * k;
        const size_t at = ((size_t)row * p.H + h) * p.D + d;
        if (d >= p.D)
            continue;
        if (p.out_half)
            p.out_half[at] = __float2half_rn(o[k] * inv);
        else
            p.out[at] = o[k] * inv;
    }
}

cudaError_t launch_latent_prefill(const LatentPrefillParams &p, cudaStream_t stream)
{
    packed_latent_prefill_kernel<<<dim3(p.total, (p.H + 3) / 4), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pgd
