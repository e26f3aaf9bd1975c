// The bookkeeping and the writes of a serving step over the paged cache: the
// step's page tables, slots, positions and lengths from the requests' token
// counts, and the step's K and V rows into their pages.  Times are of a call in
// a captured graph of such calls, unless "a call" is said.
#include <algorithm>
#include <climits>

#include "pgd_device.cuh"
#include "pgd_internal.h"

namespace pgd {

// ---------------------------------------------------------------- paged_kv_slots
// Request s has C_s cached tokens and gets n_s more.  With owned_s =
// ceil(C_s / BS), need_s = ceil((C_s + n_s) / BS) - owned_s and the exclusive
// sums cu_s of n and a_s of need, row r of request s is token t = C_s + r -
// cu_s, on page j = t / BS: the request's own page table[s][j] where j <
// owned_s, else free page number start + a_s + j - owned_s, which the row that
// opens the page (t % BS == 0) also enters into the table.  So every output is
// a function of the counts: no claim, no atomic, the same pages every time.
//
// A launch moves little (8 bytes a row and some 20 a request: a thousand of both
// are 4 ns of HBM time) and is bound by latency: one launch, in which every CTA
// scans the counts itself (two loads, one block scan, one barrier: cheaper than a
// second launch or a wait across CTAs) and then takes four consecutive rows per
// thread, which share one search of the request in shared memory.  On the
// device 4.9 us for 64 requests of one token, 5.6 for 257 with 17 prompt
// chunks, 8.1 for 2048 with 2000 prompts of up to 511 tokens (the 4 requests that
// a thread scans twice, one load at a time, then 6.5 rows a thread); a call from
// Python takes the host 8.2 to 9 us.  Sums saturate (min(a + b, cap) is
// associative on non-negative numbers), so no count can overflow them.
constexpr int kSlotThreads = 512;
constexpr int kSlotRows = 4;  // rows per thread and turn

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b)
{
    return min(a + b, (uint32_t)kSlotCountCap);
}

__global__ void __launch_bounds__(kSlotThreads) paged_kv_slots_kernel(const SlotParams p)
{
    extern __shared__ int slot_smem[];
    int *cu = slot_smem;               // [S + 1] first row of each request
    int *first = slot_smem + p.S + 1;  // [S] first free-list entry of each request
    __shared__ uint2 warp_sum[kSlotThreads / 32];

    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int BS = 1 << p.log2BS;
    const long long maxlen = (long long)p.MB << p.log2BS;
    const int start = p.free_start ? __ldg(p.free_start) : 0;
    const uint32_t start_ok = (uint32_t)min(max(start, 0), kSlotCountCap);
    unsigned err = start < 0 ? kErrNoPage : 0u;

    // each thread owns a contiguous run of requests
    const int per = (p.S + kSlotThreads - 1) / kSlotThreads;
    const int s0 = min(t * per, p.S), s1 = min(s0 + per, p.S);
    // the counts as they are used: not negative, the context inside the table
    auto context = [&](int s) -> int {
        const int c = __ldg(p.context_lens + s);
        if (c < 0 || c > maxlen)
            err |= kErrSeqLen;
        return (int)min((long long)max(c, 0), maxlen);
    };
    auto queries = [&](int s) -> int {
        const int n = __ldg(p.query_lens + s);
        if (n < 0)
            err |= kErrQueryLen;
        return min(max(n, 0), kSlotCountCap);
    };
    auto pages_needed = [&](int c, int n) -> int {
        const long long len = min((long long)c + n, maxlen);
        return (int)((len + BS - 1) >> p.log2BS) - ((c + BS - 1) >> p.log2BS);
    };
    uint2 total = make_uint2(0, 0);
    // a second round only when the rows do not fit: the requests past row N
    // then count as having only the rows that do (cu keeps the first round's
    // sums, clamped to N wherever it is read)
    for (int round = 0; round < 2; ++round) {
        uint2 mine = make_uint2(0, 0);
        for (int s = s0; s < s1; ++s) {
            const int c = context(s);
            const int n = round ? min(cu[s + 1], p.N) - min(cu[s], p.N) : queries(s);
            mine.x = sat_add(mine.x, n);
            mine.y = sat_add(mine.y, pages_needed(c, n));
        }
        uint2 inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t x = __shfl_up_sync(~0u, inc.x, off), y = __shfl_up_sync(~0u, inc.y, off);
            if (lane >= off) {
                inc.x = sat_add(inc.x, x);
                inc.y = sat_add(inc.y, y);
            }
        }
        uint2 at = make_uint2(__shfl_up_sync(~0u, inc.x, 1), __shfl_up_sync(~0u, inc.y, 1));
        if (lane == 0)
            at = make_uint2(0, 0);
        if (lane == 31)
            warp_sum[w] = inc;
        __syncthreads();
        total = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < kSlotThreads / 32; ++i) {
            if (i == w) {
                at.x = sat_add(at.x, total.x);
                at.y = sat_add(at.y, total.y);
            }
            total.x = sat_add(total.x, warp_sum[i].x);
            total.y = sat_add(total.y, warp_sum[i].y);
        }
        __syncthreads();  // warp_sum is read: the next round may write it
        for (int s = s0; s < s1; ++s) {
            const int n = round ? min(cu[s + 1], p.N) - min(cu[s], p.N) : queries(s);
            if (round == 0)
                cu[s] = at.x;
            first[s] = (int)(start_ok + at.y);
            at.x = sat_add(at.x, n);
            at.y = sat_add(at.y, pages_needed(context(s), n));
        }
        if (round == 0 && t == 0)
            cu[p.S] = total.x;
        __syncthreads();
        if (round == 0 && cu[p.S] <= p.N)
            break;
        err |= kErrQueryLen;
    }
    const int rows_used = min(cu[p.S], p.N);

    if (blockIdx.x == 0) {
        for (int s = t; s <= p.S; s += kSlotThreads)
            p.cu_seqlens_q[s] = min(cu[s], p.N);
        for (int s = t; s < p.S; s += kSlotThreads) {
            const long long len =
                (long long)context(s) + (min(cu[s + 1], p.N) - min(cu[s], p.N));
            if (len > maxlen)
                err |= kErrSeqLen;
            p.seq_lens[s] = (int)min(len, maxlen);
        }
        if (t == 0) {
            *p.free_end = (int)(start_ok + total.y);
            if ((long long)start_ok + total.y > p.num_free)
                err |= kErrNoPage;
        }
    }

    const int groups = (p.N + kSlotRows - 1) / kSlotRows;
    for (int i = blockIdx.x * kSlotThreads + t; i < groups; i += gridDim.x * kSlotThreads) {
        const int r0 = i * kSlotRows;
        int slot[kSlotRows], pos[kSlotRows];
        int s = 0;
        if (r0 < rows_used) {  // the last request whose first row is at or before r0
            int lo = 0, hi = p.S - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= r0)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            s = lo;
        }
#pragma unroll
        for (int k = 0; k < kSlotRows; ++k) {
            const int r = r0 + k;
            slot[k] = pos[k] = -1;
            if (r < rows_used) {
                while (cu[s + 1] <= r)
                    ++s;
                const int c = (int)min((long long)max(__ldg(p.context_lens + s), 0), maxlen);
                const long long tok = (long long)c + (r - cu[s]);
                pos[k] = (int)min(tok, (long long)INT_MAX);
                if (tok < maxlen) {
                    const int j = (int)(tok >> p.log2BS), in_page = (int)tok & (BS - 1);
                    const int owned = (c + BS - 1) >> p.log2BS;
                    int32_t *entry = p.block_tables + (size_t)s * p.MB + j;
                    int id;
                    if (j < owned) {
                        id = *entry;
                        if ((unsigned)id >= (unsigned)p.NB) {
                            err |= kErrPageRange;
                            id = -1;
                        }
                    } else {
                        const long long at = (long long)first[s] + (j - owned);
                        id = at < p.num_free ? __ldg(p.free_pages + at) : -1;
                        if (at < p.num_free && (unsigned)id >= (unsigned)p.NB) {
                            err |= kErrPageRange;
                            id = -1;
                        }
                        if (in_page == 0)
                            *entry = id;
                    }
                    slot[k] = id < 0 ? -1 : (id << p.log2BS) + in_page;
                }
            }
        }
        const bool whole = r0 + kSlotRows <= p.N;
        if (whole && p.vector_slots)
            *reinterpret_cast<int4 *>(p.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        else
            for (int k = 0; k < kSlotRows; ++k)
                if (r0 + k < p.N)
                    p.slots[r0 + k] = slot[k];
        if (p.positions) {
            if (whole && p.vector_positions)
                *reinterpret_cast<int4 *>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            else
                for (int k = 0; k < kSlotRows; ++k)
                    if (r0 + k < p.N)
                        p.positions[r0 + k] = pos[k];
        }
    }
    if (err)
        atomicOr(p.err, err);
}

cudaError_t launch_kv_slots(const SlotParams &p, int num_sms, cudaStream_t stream)
{
    const size_t smem = (2 * (size_t)p.S + 1) * sizeof(int);
    // a launch that has not asked for more gets 48 KB, the kernel's static
    // arrays included: ask well before
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            paged_kv_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSlotSmemMax);
        if (e != cudaSuccess)
            return e;
    }
    const long long groups = ((long long)p.N + kSlotRows - 1) / kSlotRows;
    const long long blocks = (groups + kSlotThreads - 1) / kSlotThreads;
    const int grid = (int)std::max(1ll, std::min<long long>(blocks, num_sms));
    paged_kv_slots_kernel<<<grid, kSlotThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------- paged_kv_write
// Row n of k_new / v_new goes to cache row slots[n] = page * BS + row of every
// KV head: a scatter of whole rows of head_dim halves, so it is a copy, bound
// by HBM (each byte read once and written once).  A CTA takes `rows_per_cta`
// tokens; a thread moves 16-byte pieces, of K and of V, consecutive threads
// consecutive pieces of a token's heads (runs of head_dim halves on both
// sides).  131072 rows of 8 heads x 128: 162 us, 6.6 TB/s of reads and writes
// (a plain copy: 6.8); 64 rows: 2.0.  10007 rows of 4 x 256 into 8-row pages,
// token-major: 16.4 us a call in turn with other work, 4.8 TB/s (a copy's rate
// would give 11.5): 5004 short CTAs, each with a slot to read before its one
// load of K and of V.  (The same call over and over takes 9.0 us, with its 39 MB
// of rows and most of its writes in the L2: no measure of HBM.)
constexpr int kWriteThreads = 256;

// SAME: K's and V's rows lie at the same strides, so one address calculation
// serves both (with two, 64 rows take 2.15 us instead of 2.07, 10007 rows 9.35
// instead of 9.1, 131072 rows 163.8 instead of 163.1).
template <bool SAME>
__global__ void __launch_bounds__(kWriteThreads) paged_kv_write_kernel(const WriteParams p)
{
    const int pieces = p.Hkv * p.vec;  // 16-byte pieces of one token's K (or V)
    const int n0 = blockIdx.x * p.rows_per_cta;
    const int count = min(p.rows_per_cta, p.rows - n0) * pieces;
    for (int i = threadIdx.x; i < count; i += kWriteThreads) {
        const int dn = i / pieces, in_row = i - dn * pieces, n = n0 + dn;
        const int h = in_row / p.vec, c = in_row - h * p.vec;
        const int slot = __ldg(p.slots + n);
        if (slot < 0)
            continue;
        const int page = slot >> p.log2BS, row = slot & ((1 << p.log2BS) - 1);
        if (page >= p.NB) {
            if (in_row == 0)
                atomicOr(p.err, kErrPageRange);
            continue;
        }
        const size_t k_at = (size_t)n * p.k_token_stride + (size_t)h * p.k_head_stride + 8 * c;
        const size_t v_at =
            SAME ? k_at : (size_t)n * p.v_token_stride + (size_t)h * p.v_head_stride + 8 * c;
        const size_t to = (size_t)page * p.page_stride + (size_t)h * p.head_stride +
                          (size_t)row * p.token_stride + 8 * c;
        const uint4 k = __ldg(reinterpret_cast<const uint4 *>(p.k_new + k_at));
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p.v_new + v_at));
        *reinterpret_cast<uint4 *>(p.k_cache + to) = k;
        *reinterpret_cast<uint4 *>(p.v_cache + to) = v;
    }
}

cudaError_t launch_kv_write(WriteParams p, cudaStream_t stream)
{
    const int pieces = p.Hkv * p.vec;
    p.rows_per_cta = std::max(1, kWriteThreads / pieces);
    const unsigned blocks = (unsigned)((p.rows + (long long)p.rows_per_cta - 1) / p.rows_per_cta);
    const bool same = p.k_token_stride == p.v_token_stride && p.k_head_stride == p.v_head_stride;
    if (same)
        paged_kv_write_kernel<true><<<blocks, kWriteThreads, 0, stream>>>(p);
    else
        paged_kv_write_kernel<false><<<blocks, kWriteThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pgd
