// Rows of an attention output from tensor memory to global memory.
#pragma once

#include "pgd_device.cuh"

namespace pgd {

// Rows of the output from the registers of a warp: lane r holds 32 words (fp32
// values, or pairs of fp16) of row r.  Written as they are, every store would
// touch 32 rows, a line each; so each four lanes first exchange eight-word
// pieces (a 4 x 4 transpose by two butterflies), after which the four hold one
// row's 128 bytes, of four rows in turn, and a store touches 8 lines.
struct RowOut {
    char *at[4];   // where rows 4 * (lane / 4) + 0 .. 3 of the warp begin, or null
};

__device__ __forceinline__ void store_words(const RowOut &o, uint32_t (&w)[32], int byte, int lane,
                                            bool wide)
{
    const bool odd = lane & 1, high = lane & 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int q = 0; q < 4; q += 2) {  // pieces (0, 1) and (2, 3) with lane ^ 1
            const uint32_t got =
                __shfl_xor_sync(~0u, odd ? w[8 * q + i] : w[8 * (q + 1) + i], 1);
            w[8 * q + i] = odd ? got : w[8 * q + i];
            w[8 * (q + 1) + i] = odd ? w[8 * (q + 1) + i] : got;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {     // pieces (0, 2) and (1, 3) with lane ^ 2
            const uint32_t got =
                __shfl_xor_sync(~0u, high ? w[8 * q + i] : w[8 * (q + 2) + i], 2);
            w[8 * q + i] = high ? got : w[8 * q + i];
            w[8 * (q + 2) + i] = high ? w[8 * (q + 2) + i] : got;
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (o.at[q]) {
            char *dst = o.at[q] + byte + 32 * (lane & 3);
            if (wide) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst),
                             "r"(w[8 * q]), "r"(w[8 * q + 1]), "r"(w[8 * q + 2]), "r"(w[8 * q + 3]),
                             "r"(w[8 * q + 4]), "r"(w[8 * q + 5]), "r"(w[8 * q + 6]),
                             "r"(w[8 * q + 7])
                             : "memory");
            } else {  // an output that starts on 16 bytes only
                *reinterpret_cast<uint4 *>(dst) =
                    make_uint4(w[8 * q], w[8 * q + 1], w[8 * q + 2], w[8 * q + 3]);
                *reinterpret_cast<uint4 *>(dst + 16) =
                    make_uint4(w[8 * q + 4], w[8 * q + 5], w[8 * q + 6], w[8 * q + 7]);
            }
        }
}

// COLS columns of O from tensor memory (from column `col` of the tile's O on,
// at `taddr`), scaled by the row's 1 / l, to the output; `last` runs once
// the last value has been read.
template <int COLS, class F>
__device__ __forceinline__ void write_rows(const RowOut &o, bool half, bool wide, uint32_t taddr,
                                           int col, float inv, int lane, F &&last)
{
    static_assert(COLS % 64 == 0, "an fp16 store takes 64 columns");
    float v[32];
    uint32_t w[32];
    if (half) {
#pragma unroll 1
        for (int c = 0; c < COLS; c += 64) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                tc_ld32(taddr + c + 32 * h, v);
                tc_wait_ld();
                tc_ld_ready(v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[16 * h + i] = pack_half2(v[2 * i] * inv, v[2 * i + 1] * inv);
            }
            if (c + 64 == COLS)
                last();
            store_words(o, w, (col + c) * 2, lane, wide);
        }
    } else {
#pragma unroll 1
        for (int c = 0; c < COLS; c += 32) {
            tc_ld32(taddr + c, v);
            tc_wait_ld();
            tc_ld_ready(v);
            if (c + 32 == COLS)
                last();
#pragma unroll
            for (int i = 0; i < 32; ++i)
                w[i] = __float_as_uint(v[i] * inv);
            store_words(o, w, (col + c) * 4, lane, wide);
        }
    }
}

// Where the rows of a warp's quarter of a tile (TQ tokens x the G heads of a KV
// head) lie in out [tokens][Hq][row_bytes], from the tile's first token and head
// on: the same for every tile, so worked out once.
struct RowPlaces {
    uint32_t off[4];  // bytes, in units of 16
    uint32_t token;   // the rows' tokens within the tile, a byte each (255: none)
    __device__ __forceinline__ RowPlaces(size_t row_bytes, int Hq, int G, int TQ, int quarter,
                                         int lane)
    {
        int r = 32 * quarter + (lane & ~3);
        int ti = r / G, h = r - ti * G;
        token = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q, ++r) {
            off[q] = (uint32_t)(((size_t)ti * Hq + h) * row_bytes / 16);
            token |= (r < TQ * G ? (uint32_t)ti : 255u) << (8 * q);
            if (++h == G) {
                h = 0;
                ++ti;
            }
        }
    }
    // the rows of a tile of `left` tokens (at most 128) that begins at `first`
    __device__ __forceinline__ RowOut at(char *first, int left) const
    {
        RowOut o;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o.at[q] = (int)((token >> (8 * q)) & 255u) < left ? first + 16 * (size_t)off[q] : nullptr;
        return o;
    }
};

}  // namespace pgd
