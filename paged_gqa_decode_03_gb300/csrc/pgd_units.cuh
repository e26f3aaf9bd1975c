// What the kernels over packed prompts share: their turns over the list of units, the
// causal border, a row's maximum.
#pragma once

#include "pgd_device.cuh"
#include "pgd_internal.h"

namespace pgd {

// Turn k of CTA b takes unit k * grid + b, every other turn in the opposite
// direction.
__device__ __forceinline__ int unit_of(int k)
{
    const int b = (int)blockIdx.x, grid = (int)gridDim.x;
    return k * grid + ((k & 1) ? grid - 1 - b : b);
}

// (A plain load: the order kernel may still be writing the list while this
// kernel already runs, up to griddep_wait, so it is not read-only here.)
__device__ __forceinline__ int4 unit_at(const PrefillParams &p, int k, int units)
{
    const int ui = unit_of(k);
    return ui < units ? p.units[ui] : make_int4(0, 0, 0, 0);
}

// The lowest n bits (none for n <= 0, all 32 for n >= 32).
__device__ __forceinline__ uint32_t first_bits(int n)
{
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// The largest of a row's 128 scores: four independent chains of three-input
// maxima.
__device__ __forceinline__ float max128(const float (&v)[4][32])
{
    float e[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        e[c] = fmaxf(v[c][0], v[c][1]);
#pragma unroll
        for (int i = 2; i < 32; i += 2)
            e[c] = fmax3(e[c], v[c][i], v[c][i + 1]);
    }
    return fmax3(e[0], e[1], fmaxf(e[2], e[3]));
}

}  // namespace pgd
