// Rotary positions where a step's rows meet the cache: queries rotated in place or
// into their output, rotated keys and the values (or a latent cache's rows) into
// their pages, in one launch.
//
// Pair i of a head turns by angle = position * f_i: (a, b) -> m (a cos - b sin,
// b cos + a sin), the pair being values (i, i + rot / 2) or (2i, 2i + 1) of the
// head's first rot.  f_i is fp32 as the caller gives it and the product is taken
// exactly: a position is a whole number, so whole turns of f_i / 2 pi drop out of
// it and what is left is a 64-bit fraction of a turn, F_i = frac(f_i / 2 pi) 2^64;
// position * F_i mod 2^64 is the place on the circle, whatever the position (an
// fp32 product at position 10^6 is off by up to 0.03 radians).  f_i / 2 pi is the
// product with a rounded 1 / 2 pi in 53 bits and F_i whole: position * (f_i 2^-52 +
// 2 pi 2^-64) radians at most (f_i below 0: 2^-54, one rounding next to 1).  The place goes
// on as 32 bits and an fp32 number of half turns: 1.1e-7 radians more, at any position.
//
// Every value moves once, so the call is a copy, bound by HBM, with a few
// operations a value: the sines and cosines of a row are worked out once, in shared
// memory, for all its heads.
#include <algorithm>

#include "pgd_device.cuh"
#include "pgd_internal.h"

namespace pgd {

namespace {

constexpr int kRopeThreads = 256;
// Items of a thread in flight, and CTAs an SM with them: two and six where blocks of rows
// fill two items a thread at least as well as three, else three and four.  65536 rows of 32
// / 8 heads x 128 (384 items a row) take 249 us with three, 270 with two; 10007 of 24 / 4 x
// 256 (512) 52.6 and 51.0; 30011 of a latent cache with 16 heads (100) 36.6 and 34.7.  Others:
// three and five 257, 60.4, 37.0; four and three 269, 53.5, 38.1.
constexpr int rope_ctas(int ahead) { return ahead == 2 ? 6 : 4; }

__device__ __forceinline__ void rotate2(uint32_t &a, uint32_t &b, const float2 &c0, const float2 &c1)
{
    const float2 x = unpack_half2(a), y = unpack_half2(b);
    a = pack_half2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
    b = pack_half2(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
}
// the pair within one word
__device__ __forceinline__ uint32_t rotate1(uint32_t w, const float2 &c)
{
    const float2 x = unpack_half2(w);
    return pack_half2(x.x * c.x - x.y * c.y, x.y * c.x + x.x * c.y);
}

}  // namespace

// An item is 32 bytes of a head, as two pieces of 16: of the rotated values the
// pieces that belong together (a piece of either half, or two adjacent ones of
// interleaved pairs: 8 pairs in either case), of the others two adjacent pieces.  A
// CTA goes from block of rows to block of rows: a block's loads go out first, and come
// while its sines and cosines are worked out.
template <int AHEAD>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas(AHEAD))
    paged_rope_write_kernel(const RopeParams p)
{
    extern __shared__ uint8_t rope_smem[];
    const int pairs = p.rot / 2;
    uint64_t *turn = reinterpret_cast<uint64_t *>(rope_smem);  // [pairs] F_i
    float2 *cs = reinterpret_cast<float2 *>(turn + pairs);     // [2][rows][pairs] (cos, sin) m
    // (in 64 bits, which are slow here: once a CTA)
    for (int i = threadIdx.x; i < pairs; i += kRopeThreads) {
        const double t = (double)__ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / 2 pi
        turn[i] = (uint64_t)((t - floor(t)) * 18446744073709551616.0);
    }
    __syncthreads();

    const int q_items = p.Hq << p.log2q, k_items = p.Hkv << p.log2k;
    const int per_row = q_items + k_items + (p.Hkv << p.log2v);
    const int rot_items = p.rot / 16;
    int turns = 0;
    for (int n0 = blockIdx.x * p.rows_per_cta; n0 < p.rows; n0 += gridDim.x * p.rows_per_cta, ++turns) {
        const int rows = min(p.rows_per_cta, p.rows - n0);
        const int count = rows * per_row;
        float2 *const table = cs + (turns & 1) * p.rows_per_cta * pairs;
        for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < count; i0 += AHEAD * kRopeThreads) {
            uint4 a[AHEAD], b[AHEAD];
            uint16_t *dst[AHEAD];
            int second[AHEAD], turned[AHEAD];  // the second piece's place; first of its pairs or -1
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = i0 + u * kRopeThreads;
                dst[u] = nullptr;
                if (i >= count)
                    continue;
                // (by the reciprocal: exact for blocks of several rows, of 768 items at most)
                const int dn = p.rows_per_cta == 1 ? 0 : (int)__umulhi(i, p.row_inverse), n = n0 + dn;
                const int pos = __ldg(p.positions + n);
                if (pos < 0)
                    continue;
                int j = i - dn * per_row;
                const bool is_q = j < q_items, is_v = j >= q_items + k_items;
                j -= is_q ? 0 : is_v ? q_items + k_items : q_items;
                const int log2d = is_q ? p.log2q : is_v ? p.log2v : p.log2k;
                const int h = j >> log2d, c = j & ((1 << log2d) - 1);
                const bool rotated = !is_v && c < rot_items;
                const int first = rotated && !p.interleaved ? 8 * c : 16 * c;
                second[u] = rotated && !p.interleaved ? pairs : 8;
                turned[u] = rotated ? dn * pairs + 8 * c : -1;
                const uint16_t *src;
                if (is_q) {
                    if (!rotated && p.in_place)
                        continue;
                    src = p.q + (size_t)n * p.q_token + (size_t)h * p.q_head;
                    dst[u] = p.q_out + (size_t)n * p.qo_token + (size_t)h * p.qo_head + first;
                } else {
                    const int slot = __ldg(p.slots + n);
                    if (slot < 0)
                        continue;
                    const int page = slot >> p.log2BS, row = slot & ((1 << p.log2BS) - 1);
                    if (page >= p.NB) {
                        if (j == 0)
                            atomicOr(p.err, kErrPageRange);
                        continue;
                    }
                    src = is_v ? p.v_new + (size_t)n * p.v_token + (size_t)h * p.v_head
                               : p.k_new + (size_t)n * p.k_token + (size_t)h * p.k_head;
                    dst[u] = (is_v ? p.v_cache : p.k_cache) + (size_t)page * p.page_stride +
                             (size_t)h * p.head_stride + (size_t)row * p.token_stride + first;
                }
                src += first;
                a[u] = *reinterpret_cast<const uint4 *>(src);
                b[u] = *reinterpret_cast<const uint4 *>(src + second[u]);
            }
            if (i0 == (int)threadIdx.x) {
                for (int i = threadIdx.x; i < rows * pairs; i += kRopeThreads) {
                    const int n = (int)__umulhi(i, p.pair_inverse);
                    const int pos = __ldg(p.positions + n0 + n);
                    if (pos < 0)
                        continue;
                    const uint64_t at = (uint64_t)(uint32_t)pos * turn[i - n * pairs];
                    float s, c;
                    sincospif((float)(int32_t)(at >> 32) * 0x1p-31f, &s, &c);
                    table[i] = make_float2(c * p.magnitude, s * p.magnitude);
                }
                // (one barrier a block: the other table is written only behind the next)
                __syncthreads();
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                if (!dst[u])
                    continue;
                if (turned[u] >= 0) {
                    const float2 *t = table + turned[u];
                    if (p.interleaved) {
                        a[u].x = rotate1(a[u].x, t[0]);
                        a[u].y = rotate1(a[u].y, t[1]);
                        a[u].z = rotate1(a[u].z, t[2]);
                        a[u].w = rotate1(a[u].w, t[3]);
                        b[u].x = rotate1(b[u].x, t[4]);
                        b[u].y = rotate1(b[u].y, t[5]);
                        b[u].z = rotate1(b[u].z, t[6]);
                        b[u].w = rotate1(b[u].w, t[7]);
                    } else {
                        rotate2(a[u].x, b[u].x, t[0], t[1]);
                        rotate2(a[u].y, b[u].y, t[2], t[3]);
                        rotate2(a[u].z, b[u].z, t[4], t[5]);
                        rotate2(a[u].w, b[u].w, t[6], t[7]);
                    }
                }
                *reinterpret_cast<uint4 *>(dst[u]) = a[u];
                *reinterpret_cast<uint4 *>(dst[u] + second[u]) = b[u];
            }
        }
    }
}

cudaError_t launch_rope_write(RopeParams p, int num_sms, cudaStream_t stream)
{
    const int per_row = (p.Hq << p.log2q) + (p.Hkv << p.log2k) + (p.Hkv << p.log2v);
    // the rows that a block's items hold, and the share of them that these fill
    auto rows_of = [&](int ahead) { return std::max(1, std::min(ahead * kRopeThreads / per_row, 16)); };
    auto fill = [&](int ahead) {
        const int items = rows_of(ahead) * per_row, at_once = ahead * kRopeThreads;
        return (double)items / ((items + at_once - 1) / at_once * at_once);
    };
    const int ahead = fill(2) >= fill(3) ? 2 : 3;
    // rows enough for a CTA's threads, but CTAs enough for every SM first
    p.rows_per_cta = std::max(1, std::min(rows_of(ahead), p.rows / (2 * num_sms)));
    const long long blocks = (p.rows + (long long)p.rows_per_cta - 1) / p.rows_per_cta;
    const unsigned grid = (unsigned)std::min<long long>(blocks, (long long)rope_ctas(ahead) * num_sms);
    // i / d = umulhi(i, 2^32 / d rounded up) while i d < 2^32
    p.row_inverse = (uint32_t)((0xFFFFFFFFull + per_row) / per_row);
    p.pair_inverse = (uint32_t)((0xFFFFFFFFull + p.rot / 2) / (p.rot / 2));
    const size_t smem = (size_t)(p.rot / 2) * 8 * (1 + 2 * p.rows_per_cta);  // 34 KB at most
    if (ahead == 2)
        paged_rope_write_kernel<2><<<grid, kRopeThreads, smem, stream>>>(p);
    else
        paged_rope_write_kernel<3><<<grid, kRopeThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pgd
