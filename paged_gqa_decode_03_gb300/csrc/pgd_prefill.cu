// Causal attention over whole packed prompts whose K and V are still rows of
// the projection's output, not yet pages of a cache (packed_gqa_prefill), on
// the 5th-generation tensor cores.
//
// For query head h of KV head g = h / G and the token at position t of its
// prompt, out = sum_{u <= t} p_u v_u / sum_u p_u with p_u = exp2(s_u - m), s_u =
// q . k_u * scale * log2(e): one pass over the keys with a running maximum m
// and sum.  A tile is 128 rows: TQ = 128 / G tokens x the G heads of one KV
// head, so that every K and V byte serves the group.  Work is 4 D operations
// per row and key on operands that come from L2 almost always: the tensor
// cores are what bounds a long prompt.  Times are of calls in a captured graph,
// unless "a call" is said: called from Python in turn with other work.
#include <algorithm>

#include "pgd_device.cuh"
#include "pgd_internal.h"
#include "pgd_rows.cuh"
#include "pgd_units.cuh"

namespace pgd {

namespace {

constexpr int kNT = 128;               // keys per stage
constexpr int kSlab = 128 * 128;       // bytes of 128 rows of one 64-wide slab of head_dim
// Of the products' descriptor: -A for A.  With a negative scale the scores are
// those of -q, and the softmax goes by |scale|: its loop then looks for the
// largest score whatever the sign (a second loop for the smallest, although it
// was not run, cost 4 x 2048 tokens 115 us instead of 111 by its place in the
// code).
constexpr uint32_t kNegateA = 1u << 13;

// The units of a call in decreasing order of their stages (a counting sort):
// {first row of q, position of that row, rows left in the prompt, KV head} per
// tile (or pair of tiles) of `span` tokens and KV head.  The CTAs of the
// attention kernel deal them out like cards, back and forth, so the long ones are
// spread evenly and the short ones fill the end.
__global__ void __launch_bounds__(kPrefillOrderKeys)
    packed_prefill_order_kernel(const PrefillParams p)
{
    __shared__ int cnt[kPrefillOrderKeys];
    __shared__ int warp_tot[kPrefillOrderKeys / 32];
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    griddep_launch_dependents();  // their set-up may pass meanwhile
    cnt[t] = 0;
    __syncthreads();
    // calls f(key, i0, n, row0) for every tile, a warp per prompt
    auto each = [&](auto &&f) {
        for (int s = w; s < p.S; s += kPrefillOrderKeys / 32) {
            const int row0 = __ldg(p.cu_seqlens + s);
            const int n = __ldg(p.cu_seqlens + s + 1) - row0;
            if (n < 0 || n > p.max_len || row0 < 0 || row0 > p.total - n) {
                if (lane == 0)
                    atomicOr(p.err, kErrQueryLen);
                continue;
            }
            for (int i0 = lane * p.span; i0 < n; i0 += 32 * p.span)
                f(min((min(i0 + p.span, n) + kNT - 1) / kNT, kPrefillOrderKeys - 1), i0, n, row0);
        }
    };
    each([&](int key, int, int, int) { atomicAdd(&cnt[key], p.Hkv); });
    __syncthreads();
    // exclusive prefix sum over the keys from the largest down: thread t owns
    // key kPrefillOrderKeys - 1 - t
    const int k = kPrefillOrderKeys - 1 - t;
    const int c = cnt[k];
    int inc = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(~0u, inc, off);
        if (lane >= off)
            inc += y;
    }
    if (lane == 31)
        warp_tot[w] = inc;
    __syncthreads();
    if (w == 0) {
        const int own = warp_tot[lane];
        int x = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(~0u, x, off);
            if (lane >= off)
                x += y;
        }
        warp_tot[lane] = x - own;
        if (lane == 31) {
            // prompts that overlap can have more units than the rows allow
            if ((unsigned)x > (unsigned)p.max_units)
                atomicOr(p.err, kErrQueryLen);
            *p.num_units = max(0, min(x, p.max_units));
        }
    }
    __syncthreads();
    cnt[k] = warp_tot[w] + inc - c;
    __syncthreads();
    each([&](int key, int i0, int n, int row0) {
        const int at = atomicAdd(&cnt[key], p.Hkv);
        for (int g = 0; g < p.Hkv; ++g)
            if ((unsigned)(at + g) < (unsigned)p.max_units)
                p.units[at + g] = make_int4(row0 + i0, i0, n - i0, g);
    });
}

}  // namespace

// packed_prefill_pair_kernel<D> (head_dim 64, 128) — persistent, one CTA per
// SM, each unit a pair of consecutive 128-row tiles A and B of one KV head that
// share every K and V stage.
//
// Tensor memory (512 columns): O of A and B (2 D), P of A and B as fp16 (2 x
// 64), and the scores: 128 columns a buffer.  At head_dim 128 that leaves ONE
// score buffer for both tiles, and that is enough: a tile's softmax reads its
// 128 scores into registers in one round trip (~300 cycles) and hands the
// buffer back, long before its exponentials are done, and the tensor pipe has
// a P V product (512 cycles) to do meanwhile.  So the pipe runs S_A(j+1),
// P_A(j) V_j, S_B(j+1), P_B(j) V_j without a gap: S(j+1) does not wait for P(j)
// V_j, nor P V for a softmax that has just begun.  Where a stage's cycles go,
// by clock stamps: a period of 3150 for both tiles, of which the products take
// 2048; between a tile's scores being whole and the other's being whole lie
// 330 cycles of reading, 250 until the next product is issued and the 512 of
// it behind what the pipe still holds.  A tile's softmax takes 2400 of the
// period (reading 330, maximum 400, exponentials 900, P 200, barriers).
// One prompt of 16381 tokens, 32 / 8 heads x 128: 1450 to 1530 us by the GPU's
// clock at the time, a call 1504, 1460 TFLOP/s; 4 x 2048 tokens: 111 us, a call
// 122.  Tried
// and slower: part of the exponentials as polynomials on the FMA pipes (a
// quarter of them: 1450 -> 1690 us: the issue slots, not the special-function
// unit, are short); two threads per row (16 softmax warps: 1630); the rows'
// way out by four warps of their own (4 x 2048: 115 -> 127, O has no second
// place to go on in); polling for o_done instead of waiting (1580).
//   * warp 0, one thread: Q tiles, K and V stages by tensor copies (one per
//     stage; K and V in rings of their own)
//   * warp 1, one thread: the scores; warp 2, one thread: the outputs.  The pipe
//     queues only a few products and a thread spends about 70 cycles on each
//     barrier it tests, so one thread for both kept the pipe idle half the
//     time (a period of 4150 cycles; a thread per tile: 3300, S_A(j+1)'s wait
//     for the buffer holding up P_A(j) V_j).
//   * warps 4-7 / 8-11: softmax of tile A / B, a thread per row
template <int D> struct PairShape;
template <> struct PairShape<64> {
    static constexpr int NK = 4, NV = 4, SBUF = 2;
};
template <> struct PairShape<128> {
    static constexpr int NK = 2, NV = 3, SBUF = 1;
};
constexpr int kPairThreads = 384;

template <int D> constexpr size_t pair_smem_bytes()
{
    return size_t(2) * 128 * D * 2 + size_t(PairShape<D>::NK + PairShape<D>::NV) * kNT * D * 2 + 1024;
}

template <int D>
__global__ void __launch_bounds__(kPairThreads, 1)
    packed_prefill_pair_kernel(const __grid_constant__ CUtensorMap tmap_q,
                               const __grid_constant__ CUtensorMap tmap_k,
                               const __grid_constant__ CUtensorMap tmap_v, const PrefillParams p)
{
    constexpr int NK = PairShape<D>::NK, NV = PairShape<D>::NV, SBUF = PairShape<D>::SBUF;
    constexpr int SLABS = D / 64;
    constexpr int KV_TILE = kNT * D * 2;
    constexpr int Q_TILE = 128 * D * 2;
    constexpr uint32_t S_COL = 2 * D, P_COL = S_COL + SBUF * kNT;
    static_assert(P_COL + 128 <= 512, "tensor memory");
    constexpr uint32_t IDESC_S = tc_idesc_f16(128, kNT, 0, 0);
    constexpr uint32_t IDESC_O = tc_idesc_f16(128, D, 0, 1);

    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV],
        v_empty[NV], s_full[2], s_free[2], p_full[2], o_done[2], o_free[2], mma_done;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_flag;
    __shared__ volatile int s_issued[2];  // S products issued for each tile

    const uint32_t dyn_base = smem_addr(dyn_smem);
    const uint32_t base = (dyn_base + 1023u) & ~1023u;
    uint8_t *const base_ptr = dyn_smem + (base - dyn_base);
    const uint32_t q_s = base, k_s = q_s + 2 * Q_TILE, v_s = k_s + NK * KV_TILE;
    uint8_t *const v_ptr = base_ptr + 2 * Q_TILE + NK * KV_TILE;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&q_full), 1);
        mbar_init(smem_addr(&q_empty), 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_addr(&k_full[i]), 1);
            mbar_init(smem_addr(&k_empty[i]), 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_addr(&v_full[i]), 1);
            mbar_init(smem_addr(&v_empty[i]), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_addr(&s_full[x]), 1);
            mbar_init(smem_addr(&s_free[x]), 4);
            mbar_init(smem_addr(&p_full[x]), 4);
            mbar_init(smem_addr(&o_done[x]), 1);
            mbar_init(smem_addr(&o_free[x]), 4);
        }
        mbar_init(smem_addr(&mma_done), 2);
        s_issued[0] = s_issued[1] = 0;
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (warp == 1)
        tc_alloc(smem_addr(&tmem_base_s), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    griddep_wait();  // the list of units
    const int units = *p.num_units;
    const int turns = (units + (int)gridDim.x - 1) / (int)gridDim.x;

    const bool half_out = p.out_half != nullptr;
    char *const out = half_out ? reinterpret_cast<char *>(p.out_half) : reinterpret_cast<char *>(p.out);
    const size_t row_bytes = (size_t)D * (half_out ? 2 : 4);
    auto give_up = [&]() {
        if (!abort_flag)
            atomicOr(p.err, kErrTimeout);
        abort_flag = 1;
    };
    // stages of the two tiles of a unit: tile A holds tokens i0 .. i0+TQ-1 of
    // the prompt, B the next TQ; left: the prompt's tokens from i0 on
    auto stages = [&](const int4 &u, int x) {
        const int from = x * p.TQ;
        return u.z > from ? (u.y + min(u.z, from + p.TQ) + kNT - 1) / kNT : 0;
    };
    // Steps of 16 keys that the output's product takes of the tile's last stage: at
    // head_dim 64 up to its last key, by twos (8192 tokens: 341 us, with the
    // whole stage 358), at 128 the whole stage (16381 tokens: 1462 us, by
    // twos 1477; 190 prompts of 128 tokens: 96 and 95)
    constexpr int PART = D == 64 ? 2 : kNT / 16;
    auto last_steps = [&](const int4 &u, int x) {
        return ((u.y + min(u.z, (x + 1) * p.TQ) - 1) % kNT / (16 * PART) + 1) * PART;
    };

    // the softmax warps hold a row's 128 scores and half of its weights: they
    // take registers that the copying and issuing warps do not need (128 x 80 +
    // 256 x 208 of the 384 x 168 of the launch)
    if (warp < 4) {
      regs_give<80>();
      if (warp == 0) {
        if (lane == 0) {
            // ======================================================== copies
            const uint64_t pol = l2_evict_last_policy();
            int nk = 0, nv = 0, nq = 0;   // copies issued so far
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                return mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns);
            };
            auto load_k = [&](int row, int g) {
                const int st = nk % NK;
                if (!wait(&k_empty[st], ((nk / NK) & 1) ^ 1))
                    return false;
                const uint32_t bar = smem_addr(&k_full[st]);
                mbar_arrive_expect_tx(bar, KV_TILE);
                tma_load_4d(k_s + st * KV_TILE, &tmap_k, 0, row, 0, g, bar, pol);
                ++nk;
                return true;
            };
            auto load_v = [&](int row, int g) {
                const int st = nv % NV;
                if (!wait(&v_empty[st], ((nv / NV) & 1) ^ 1))
                    return false;
                const uint32_t bar = smem_addr(&v_full[st]);
                mbar_arrive_expect_tx(bar, KV_TILE);
                tma_load_4d(v_s + st * KV_TILE, &tmap_v, 0, row, 0, g, bar, pol);
                ++nv;
                return true;
            };
            int4 next = unit_at(p, 0, units);
            for (int k = 0; k < turns && ok; ++k) {
                const int ui = unit_of(k);
                const int4 u = next;
                next = unit_at(p, k + 1, units);
                if (ui >= units)
                    continue;
                const int g = u.w, row0 = u.x - u.y;  // KV head, the prompt's first row
                const int nt = max(stages(u, 0), stages(u, 1));
                // the unit's first K goes out before its Q, whose place is
                // free only after the last unit's last S
                ok = load_k(row0, g) && wait(&q_empty, (nq & 1) ^ 1);
                if (!ok)
                    break;
                const int ntq = u.z > p.TQ ? 2 : 1;
                const uint32_t bar = smem_addr(&q_full);
                mbar_arrive_expect_tx(bar, ntq * SLABS * p.TQ * p.G * 128);
                for (int x = 0; x < ntq; ++x)
                    for (int sl = 0; sl < SLABS; ++sl)
                        tma_load_4d(q_s + x * Q_TILE + sl * kSlab, &tmap_q, 0, g * p.G,
                                    u.x + x * p.TQ, sl, bar);
                ++nq;
                ok = load_v(row0, g);
                for (int j = 1; j < nt && ok; ++j)
                    ok = load_k(row0 + j * kNT, g) && load_v(row0 + j * kNT, g);
            }
            if (!ok) {
                give_up();
                // let the copies in flight land before the CTA exits
                if (nq)
                    mbar_wait_bounded(smem_addr(&q_full), (nq - 1) & 1, nullptr, p.wait_budget_ns);
                for (int i = max(0, nk - NK); i < nk; ++i)
                    mbar_wait_bounded(smem_addr(&k_full[i % NK]), (i / NK) & 1, nullptr,
                                      p.wait_budget_ns);
                for (int i = max(0, nv - NV); i < nv; ++i)
                    mbar_wait_bounded(smem_addr(&v_full[i % NV]), (i / NV) & 1, nullptr,
                                      p.wait_budget_ns);
            }
        }
        __syncwarp();
      } else if (warp == 1) {
        if (lane == 0) {
            // ======================================================== scores
            const uint32_t idesc_s = IDESC_S | (p.scale_log2 < 0.f ? kNegateA : 0u);
            const uint64_t q_desc = tc_sdesc(q_s, 16, 1024);
            const uint64_t k_desc = tc_sdesc(k_s, 16, 1024);
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                if (ok && !mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns))
                    ok = false;
                return ok;
            };
            int nk = 0, nq = 0;        // K stages, Q pairs used up
            int uses[2] = {0, 0};      // of each score buffer
            int ns[2] = {0, 0};        // S products of each tile
            int4 next = unit_at(p, 0, units);
            for (int k = 0; k < turns && ok; ++k) {
                const int ui = unit_of(k);
                const int4 u = next;
                next = unit_at(p, k + 1, units);
                if (ui >= units)
                    continue;
                const int nt0 = stages(u, 0), nt1 = stages(u, 1), nmax = max(nt0, nt1);
                wait(&q_full, nq & 1);
                ++nq;
                for (int j = 0; j < nmax && ok; ++j, ++nk) {
                    const int st = nk % NK;
                    wait(&k_full[st], (nk / NK) & 1);
                    const uint64_t ks = k_desc + ((st * KV_TILE) >> 4);
                    for (int x = 0; x < 2; ++x) {
                        if (j >= (x ? nt1 : nt0))
                            continue;
                        // the buffer's last scores have been read
                        const int b = SBUF == 2 ? x : 0;
                        if (uses[b] && !wait(&s_free[b], (uses[b] - 1) & 1))
                            break;
                        ++uses[b];
                        tc_fence_after();
                        const uint64_t qx = q_desc + ((x * Q_TILE) >> 4);
                        const uint32_t d = tmem + S_COL + b * kNT;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma(d, qx + (((kk / 4) * kSlab + (kk % 4) * 32) >> 4),
                                   ks + (((kk / 4) * kSlab + (kk % 4) * 32) >> 4), idesc_s, kk > 0);
                        tc_commit(smem_addr(&s_full[x]));
                        s_issued[x] = ++ns[x];
                    }
                    tc_commit(smem_addr(&k_empty[st]));
                }
                tc_commit(smem_addr(&q_empty));
            }
            if (!ok)
                give_up();
            // every product issued has completed before the memory is freed
            tc_commit(smem_addr(&mma_done));
            mbar_wait_bounded(smem_addr(&mma_done), 0, nullptr, p.wait_budget_ns);
        }
        __syncwarp();
      } else if (warp == 2) {
        if (lane == 0) {
            // ======================================================== outputs
            const uint64_t v_desc = tc_sdesc(v_s, kSlab, 1024);
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                if (ok && !mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns))
                    ok = false;
                return ok;
            };
            int nv = 0;                           // V stages used up
            int np[2] = {0, 0}, no[2] = {0, 0};   // P V products, units of each tile
            int4 next = unit_at(p, 0, units);
            for (int k = 0; k < turns && ok; ++k) {
                const int ui = unit_of(k);
                const int4 u = next;
                next = unit_at(p, k + 1, units);
                if (ui >= units)
                    continue;
                const int nt0 = stages(u, 0), nt1 = stages(u, 1), nmax = max(nt0, nt1);
                for (int j = 0; j < nmax && ok; ++j, ++nv) {
                    const int st = nv % NV;
                    wait(&v_full[st], (nv / NV) & 1);
                    const uint64_t vs = v_desc + ((st * KV_TILE) >> 4);
                    for (int x = 0; x < 2; ++x) {
                        if (j >= (x ? nt1 : nt0))
                            continue;
                        // the last unit's output has been read
                        if (j == 0 && no[x]++ && !wait(&o_free[x], no[x] & 1))
                            break;
                        if (!wait(&p_full[x], np[x] & 1))
                            break;
                        ++np[x];
                        // let the tile's next scores go first: they are on the
                        // path that sets the period, this product is not.  Only
                        // a matter of order, so the look is short and goes on
                        // either way.
                        if (j + 1 < (x ? nt1 : nt0))
                            for (int i = 0; i < 16 && s_issued[x] <= np[x]; ++i)
                                ;
                        tc_fence_after();
                        const uint32_t o = tmem + x * D, a = tmem + P_COL + x * 64;
                        const int steps = j + 1 < (x ? nt1 : nt0) ? kNT / 16 : last_steps(u, x);
#pragma unroll
                        for (int part = 0; part < kNT / 16; part += PART) {
                            if (part >= steps)
                                break;
#pragma unroll
                            for (int kk = part; kk < part + PART; ++kk)
                                tc_mma_ta(o, a + kk * 8, vs + ((kk * 2048) >> 4), IDESC_O,
                                          j > 0 || kk > 0);
                        }
                        tc_commit(smem_addr(&o_done[x]));
                    }
                    tc_commit(smem_addr(&v_empty[st]));
                }
            }
            if (!ok)
                give_up();
            tc_commit(smem_addr(&mma_done));
            mbar_wait_bounded(smem_addr(&mma_done), 0, nullptr, p.wait_budget_ns);
        }
        __syncwarp();
      }
    } else {
        regs_take<208>();
        // ============================================================ softmax
        const int x = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int r = 32 * quarter + lane;  // this thread's row of the tile
        const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t s_col = S_COL + (SBUF == 2 ? x : 0) * kNT, o_col = x * D,
                       p_col = P_COL + x * 64;
        const int ti = r / p.G;
        // a scale of 0 runs as 1e-30: exp2 of every score is then 1 in fp32
        // (the mean over the range, as for 0) while masked scores, -inf, still
        // give 0
        const float sc = p.scale_log2 == 0.f ? 1e-30f : fabsf(p.scale_log2);
        const float2 sc2 = make_float2(sc, sc);
        const RowPlaces places(row_bytes, p.Hq, p.G, p.TQ, quarter, lane);
        int ns = 0, nv = 0;  // S tiles of this tile, V stages of the CTA, so far
        bool ok = true;
        int4 next = unit_at(p, 0, units);
        for (int k = 0; k < turns && ok; ++k) {
            const int ui = unit_of(k);
            const int4 u = next;
            next = unit_at(p, k + 1, units);  // a turn ahead: its latency passes meanwhile
            if (ui >= units)
                continue;
            const int g = u.w;
            const int nt0 = stages(u, 0), nt1 = stages(u, 1), ntx = x ? nt1 : nt0;
            const int left = min(p.TQ, u.z - x * p.TQ);  // tokens of this tile
            const int n = u.y + u.z;                     // tokens of the prompt
            const bool row_ok = r < p.TQ * p.G && ti < left;
            const int lo = u.y + x * p.TQ;          // position of the tile's first token
            const int lim = row_ok ? lo + ti : -1;  // and of this row's
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < ntx; ++j, ++ns) {
                const int t0 = j * kNT;
                // wait outcomes are warp-uniform: tensor-memory loads and
                // stores are warp-collective
                if (!__all_sync(~0u, mbar_wait_bounded(smem_addr(&s_full[x]), ns & 1, &abort_flag,
                                                       p.wait_budget_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tc_ld32(t_lane + s_col + 32 * c, v[c]);
                tc_wait_ld();
                // the scores are in registers: the buffer takes the next ones
                tc_fence_before();
                if (lane == 0)
                    mbar_arrive(smem_addr(&s_free[SBUF == 2 ? x : 0]));
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tc_ld_ready(v[c]);
                // where the causal border crosses this stage: 32 keys at a time
                if (t0 + kNT - 1 > lo) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (t0 + 32 * c + 31 > lo) {
                            const uint32_t seen = first_bits(lim + 1 - (t0 + 32 * c));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[c][i] = (seen >> i) & 1u ? v[c][i] : -INFINITY;
                        }
                }
                // has this tile's last P V ended?  (asked here, used below)
                const bool pv_over =
                    j == 0 || mbar_try_wait(smem_addr(&o_done[x]), (ns - 1) & 1);
                const float mt = max128(v) * sc;
                // the reference moves only when the maximum has grown by more
                // than 8 (log2 units): O is rescaled rarely
                bool rescale = false;
                float alpha = 1.f;
                if (mt > m_ref + kRefRoom) {
                    const float ref = mt - kRefBelow;
                    rescale = row_ok && m_ref != -INFINITY;
                    alpha = rescale ? ex2(m_ref - ref) : 1.f;
                    m_ref = ref;
                }
                const float off = m_ref == -INFINITY ? 0.f : -m_ref;
                const float2 off2 = make_float2(off, off);
                float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float2 a = ffma2(make_float2(v[2 * h + c][i], v[2 * h + c][i + 1]), sc2,
                                             off2);
                            a.x = ex2(a.x);
                            a.y = ex2(a.y);
                            pk[16 * c + i / 2] = pack_half2(a.x, a.y);
                            sum2 = fadd2(sum2, a);
                        }
                    }
                    if (h == 0 && j > 0) {
                        // this tile's last P V is done with P (and O may be rescaled)
                        if (!__all_sync(~0u, pv_over) &&
                            !__all_sync(~0u, mbar_wait_bounded(smem_addr(&o_done[x]), (ns - 1) & 1,
                                                               &abort_flag, p.wait_budget_ns))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    tc_st32u(t_lane + p_col + 32 * h, pk);
                }
                if (!ok)
                    break;
                if (j > 0 && __any_sync(~0u, rescale)) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tc_ld32(t_lane + o_col + 32 * c, o);
                        tc_wait_ld();
                        tc_ld_ready(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] *= alpha;
                        tc_st32(t_lane + o_col + 32 * c, o);
                    }
                }
                // rows behind the prompt belong to the next one and may hold
                // anything: zero those of them in V that the tile's last product
                // takes in (their weights are 0, which does not hide a NaN).
                // Each tile does so before its own product; the other's writes
                // the same zeros.
                const int za = n - t0, ze = j + 1 < ntx ? 0 : 16 * last_steps(u, x);
                const bool zero_v = za < ze;
                if (zero_v) {
                    const int st = (nv + j) % NV;
                    mbar_wait_bounded(smem_addr(&v_full[st]), ((nv + j) / NV) & 1, nullptr,
                                      p.wait_budget_ns);
                    uint8_t *vs = v_ptr + st * KV_TILE;
                    for (int idx = r; idx < (ze - za) * SLABS * 8; idx += 128) {
                        const int row = za + idx / (SLABS * 8), c = idx % (SLABS * 8);
                        *reinterpret_cast<uint4 *>(vs + (c >> 3) * kSlab + row * 128 +
                                                   (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                tc_wait_st();
                if (zero_v)
                    fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&p_full[x]));
                l = l * alpha + (sum2.x + sum2.y);
            }
            // ---- out = O / l
            if (ok && ntx > 0) {
                ok = __all_sync(~0u, mbar_wait_bounded(smem_addr(&o_done[x]), (ns - 1) & 1,
                                                       &abort_flag, p.wait_budget_ns));
                if (ok) {
                    tc_fence_after();
                    const float inv = l > 0.f ? 1.f / l : 0.f;
                    const RowOut rows =
                        places.at(out + ((size_t)(u.x + x * p.TQ) * p.Hq + (size_t)g * p.G) *
                                            row_bytes, left);
                    write_rows<D>(rows, half_out, p.wide_rows, t_lane + o_col, 0, inv, lane, [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_addr(&o_free[x]));
                    });
                }
            }
            nv += max(nt0, nt1);
        }
        if (!ok)
            give_up();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

// packed_prefill_wide_kernel (head_dim 256) — persistent, one tile per unit: O
// takes 256 tensor-memory columns, two score buffers the other 256 (P over the
// scores it came from), so S(j+1) runs while the softmax works on S(j).  K and
// V move in pieces of 16 KB, K by 64-wide slabs of its 128 keys, V by 32 keys of
// all of head_dim, so that beside the 64 KB of Q nine of them fit and each is
// free again after its own products: a stage's copies are never waited for as
// a whole.  Eight softmax warps: rows r by halves of a stage's keys.
// A prompt of 8192 tokens, 16 / 2 heads: 396 to 405 us, 1360 to 1390 TFLOP/s.  37
// prompts of 1 to 512 tokens, 24 / 4 heads: 29 to 32 us, a call 32, of which a
// unit's start and end are the larger part: a unit of one token costs 3.8 us of
// its CTA's time.  The output's product of a unit's last stage ends at the tile's
// last key, rounded up to 16, so that of the rows behind a prompt 15 at most have
// to be zeroed (the whole stage: 34.5 us).  Ending its copies and scores there as
// well added 5 % to the long prompt: not taken.
constexpr int kWideThreads = 384;
constexpr int kWideNK = 5, kWideNV = 4;  // pieces
constexpr int kWideD = 256;
constexpr size_t kWideSmem = size_t(4) * kSlab + size_t(kWideNK + kWideNV) * kSlab + 1024;

__global__ void __launch_bounds__(kWideThreads, 1)
    packed_prefill_wide_kernel(const __grid_constant__ CUtensorMap tmap_q,
                               const __grid_constant__ CUtensorMap tmap_k,
                               const __grid_constant__ CUtensorMap tmap_v, const PrefillParams p)
{
    constexpr int D = kWideD, NK = kWideNK, NV = kWideNV, SLABS = 4, VP = 4;
    constexpr int PIECE = kSlab, VKEYS = kNT / VP;
    constexpr uint32_t S_COL = 256;
    constexpr uint32_t IDESC_S = tc_idesc_f16(128, kNT, 0, 0);
    constexpr uint32_t IDESC_O = tc_idesc_f16(128, D, 0, 1);

    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV],
        v_empty[NV], s_full[2], p_full, o_done[2], o_free, mma_done;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_flag;
    __shared__ float pair_red[2][2][128];  // [parity][half][row]: the halves' exchange

    const uint32_t dyn_base = smem_addr(dyn_smem);
    const uint32_t base = (dyn_base + 1023u) & ~1023u;
    uint8_t *const base_ptr = dyn_smem + (base - dyn_base);
    const uint32_t q_s = base, k_s = q_s + SLABS * kSlab, v_s = k_s + NK * PIECE;
    uint8_t *const v_ptr = base_ptr + SLABS * kSlab + NK * PIECE;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&q_full), 1);
        mbar_init(smem_addr(&q_empty), 1);
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_addr(&k_full[i]), 1);
            mbar_init(smem_addr(&k_empty[i]), 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_addr(&v_full[i]), 1);
            mbar_init(smem_addr(&v_empty[i]), 1);
        }
        mbar_init(smem_addr(&s_full[0]), 1);
        mbar_init(smem_addr(&s_full[1]), 1);
        mbar_init(smem_addr(&p_full), 8);
        mbar_init(smem_addr(&o_done[0]), 1);
        mbar_init(smem_addr(&o_done[1]), 1);
        mbar_init(smem_addr(&o_free), 8);
        mbar_init(smem_addr(&mma_done), 2);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (warp == 1)
        tc_alloc(smem_addr(&tmem_base_s), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    griddep_wait();  // the list of units
    const int units = *p.num_units;
    const int turns = (units + (int)gridDim.x - 1) / (int)gridDim.x;

    const bool half_out = p.out_half != nullptr;
    char *const out = half_out ? reinterpret_cast<char *>(p.out_half) : reinterpret_cast<char *>(p.out);
    const size_t row_bytes = (size_t)D * (half_out ? 2 : 4);
    auto give_up = [&]() {
        if (!abort_flag)
            atomicOr(p.err, kErrTimeout);
        abort_flag = 1;
    };
    auto stages = [&](const int4 &u) { return (u.y + min(u.z, p.TQ) + kNT - 1) / kNT; };
    auto last_steps = [&](const int4 &u) {
        return (u.y + min(u.z, p.TQ) - 1) % kNT / 16 + 1;
    };

    // (384 x 168 at the launch: 128 x 120 and 256 x 192, with which no role
    // spills; 8192 tokens 396 us instead of 406, short prompts 31 instead of 32)
    if (warp < 4) {
      regs_give<120>();
      if (warp == 0) {
        if (lane == 0) {
            // ======================================================== copies
            const uint64_t pol = l2_evict_last_policy();
            int nk = 0, nv = 0, nq = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                return mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns);
            };
            auto load_k = [&](int row, int g, int slab) {
                const int st = nk % NK;
                if (!wait(&k_empty[st], ((nk / NK) & 1) ^ 1))
                    return false;
                const uint32_t bar = smem_addr(&k_full[st]);
                mbar_arrive_expect_tx(bar, PIECE);
                tma_load_4d(k_s + st * PIECE, &tmap_k, 0, row, slab, g, bar, pol);
                ++nk;
                return true;
            };
            auto load_v = [&](int row, int g) {
                const int st = nv % NV;
                if (!wait(&v_empty[st], ((nv / NV) & 1) ^ 1))
                    return false;
                const uint32_t bar = smem_addr(&v_full[st]);
                mbar_arrive_expect_tx(bar, PIECE);
                tma_load_4d(v_s + st * PIECE, &tmap_v, 0, row, 0, g, bar, pol);
                ++nv;
                return true;
            };
            int4 next = unit_at(p, 0, units);
            for (int k = 0; k < turns && ok; ++k) {
                const int ui = unit_of(k);
                const int4 u = next;
                next = unit_at(p, k + 1, units);
                if (ui >= units)
                    continue;
                const int g = u.w, nt = stages(u), row0 = u.x - u.y;
                for (int sl = 0; sl < SLABS && ok; ++sl)
                    ok = load_k(row0, g, sl);
                ok = ok && wait(&q_empty, (nq & 1) ^ 1);
                if (!ok)
                    break;
                const uint32_t bar = smem_addr(&q_full);
                mbar_arrive_expect_tx(bar, SLABS * p.TQ * p.G * 128);
                for (int sl = 0; sl < SLABS; ++sl)
                    tma_load_4d(q_s + sl * kSlab, &tmap_q, 0, g * p.G, u.x, sl, bar);
                ++nq;
                // in the order of use: K of stage j + 1 before V of stage j
                for (int j = 0; j < nt && ok; ++j) {
                    for (int sl = 0; j + 1 < nt && sl < SLABS && ok; ++sl)
                        ok = load_k(row0 + (j + 1) * kNT, g, sl);
                    for (int i = 0; i < VP && ok; ++i)
                        ok = load_v(row0 + j * kNT + i * VKEYS, g);
                }
            }
            if (!ok) {
                give_up();
                if (nq)
                    mbar_wait_bounded(smem_addr(&q_full), (nq - 1) & 1, nullptr, p.wait_budget_ns);
                for (int i = max(0, nk - NK); i < nk; ++i)
                    mbar_wait_bounded(smem_addr(&k_full[i % NK]), (i / NK) & 1, nullptr,
                                      p.wait_budget_ns);
                for (int i = max(0, nv - NV); i < nv; ++i)
                    mbar_wait_bounded(smem_addr(&v_full[i % NV]), (i / NV) & 1, nullptr,
                                      p.wait_budget_ns);
            }
        }
        __syncwarp();
      } else if (warp == 1 || warp == 2) {
        if (lane == 0) {
            // ======================================================== products
            // (scores and outputs by a thread each, as in the pair kernel)
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                if (ok && !mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns))
                    ok = false;
                return ok;
            };
            int4 next = unit_at(p, 0, units);
            if (warp == 1) {
                const uint32_t idesc_s = IDESC_S | (p.scale_log2 < 0.f ? kNegateA : 0u);
                const uint64_t q_desc = tc_sdesc(q_s, 16, 1024);
                const uint64_t k_desc = tc_sdesc(k_s, 16, 1024);
                int nk = 0, nq = 0, ns = 0;
                for (int k = 0; k < turns && ok; ++k) {
                    const int ui = unit_of(k);
                    const int4 u = next;
                    next = unit_at(p, k + 1, units);
                    if (ui >= units)
                        continue;
                    const int nt = stages(u);
                    wait(&q_full, nq & 1);
                    ++nq;
                    for (int j = 0; j < nt && ok; ++j, ++ns) {
                        // into the buffer of P(ns - 2), once its product is over
                        if (ns >= 2)
                            wait(&o_done[ns & 1], ((ns >> 1) & 1) ^ 1);
                        const uint32_t d = tmem + S_COL + (ns & 1) * kNT;
                        for (int sl = 0; sl < SLABS; ++sl, ++nk) {
                            const int st = nk % NK;
                            if (!wait(&k_full[st], (nk / NK) & 1))
                                break;
                            tc_fence_after();
                            const uint64_t ks = k_desc + ((st * PIECE) >> 4);
                            const uint64_t qs = q_desc + ((sl * kSlab) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma(d, qs + ((kk * 32) >> 4), ks + ((kk * 32) >> 4), idesc_s,
                                       sl > 0 || kk > 0);
                            tc_commit(smem_addr(&k_empty[st]));
                        }
                        tc_commit(smem_addr(&s_full[ns & 1]));
                    }
                    tc_commit(smem_addr(&q_empty));
                }
            } else {
                const uint64_t v_desc = tc_sdesc(v_s, VKEYS * 128, 1024);
                int nv = 0, np = 0, no = 0;
                for (int k = 0; k < turns && ok; ++k) {
                    const int ui = unit_of(k);
                    const int4 u = next;
                    next = unit_at(p, k + 1, units);
                    if (ui >= units)
                        continue;
                    const int nt = stages(u);
                    // the last unit's output has been read
                    if (no++ && !wait(&o_free, no & 1))
                        break;
                    for (int j = 0; j < nt && ok; ++j, ++np) {
                        if (!wait(&p_full, np & 1))
                            break;
                        const uint32_t a = tmem + S_COL + (np & 1) * kNT;
                        const int steps = j + 1 < nt ? kNT / 16 : last_steps(u);
                        for (int i = 0; i < VP; ++i, ++nv) {
                            const int st = nv % NV;
                            if (!wait(&v_full[st], (nv / NV) & 1))
                                break;
                            tc_fence_after();
                            const uint64_t vs = v_desc + ((st * PIECE) >> 4);
#pragma unroll
                            for (int kk = 0; kk < VKEYS / 16; ++kk)
                                if (i * (VKEYS / 16) + kk < steps)
                                    tc_mma_ta(tmem, a + (i * (VKEYS / 16) + kk) * 8,
                                          vs + ((kk * 2048) >> 4), IDESC_O, j > 0 || i > 0 || kk > 0);
                            tc_commit(smem_addr(&v_empty[st]));
                        }
                        tc_commit(smem_addr(&o_done[np & 1]));
                    }
                }
            }
            if (!ok)
                give_up();
            // every product issued has completed before the memory is freed
            tc_commit(smem_addr(&mma_done));
            mbar_wait_bounded(smem_addr(&mma_done), 0, nullptr, p.wait_budget_ns);
        }
        __syncwarp();
      }
    } else {
        // ============================================================ softmax
        regs_take<192>();
        constexpr int HC = kNT / 2, HD = D / 2;
        const int quarter = warp & 3;
        const int half = (warp - 4) >> 2;
        const int r = 32 * quarter + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t pair_bar = 1 + quarter;
        const int ti = r / p.G;
        const float sc = p.scale_log2 == 0.f ? 1e-30f : fabsf(p.scale_log2);
        const float2 sc2 = make_float2(sc, sc);
        const RowPlaces places(row_bytes, p.Hq, p.G, p.TQ, quarter, lane);
        int ns = 0, nv = 0;
        bool ok = true;
        // after a failed wait the loops keep running without doing work, so
        // that the two warps of a pair meet at every named barrier
        auto wait = [&](uint64_t *bar, int parity) {
            if (ok && !__all_sync(~0u, mbar_wait_bounded(smem_addr(bar), parity, &abort_flag,
                                                         p.wait_budget_ns))) {
                ok = false;
                give_up();
            }
        };
        int4 next = unit_at(p, 0, units);
        for (int k = 0; k < turns; ++k) {
            const int ui = unit_of(k);
            const int4 u = next;
            next = unit_at(p, k + 1, units);
            if (ui >= units)
                continue;
            const int g = u.w, nt = stages(u), n = u.y + u.z;
            const bool row_ok = r < p.TQ * p.G && ti < min(p.TQ, u.z);
            const int lim = row_ok ? u.y + ti : -1;
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < nt; ++j, ++ns, nv += VP) {
                const int t0 = j * kNT, c0 = t0 + half * HC;
                const uint32_t s_col = S_COL + (ns & 1) * kNT;
                wait(&s_full[ns & 1], (ns >> 1) & 1);
                float v[2][32];
                float e = -INFINITY;
                if (ok) {
                    tc_fence_after();
                    tc_ld32(t_lane + s_col + half * HC, v[0]);
                    tc_ld32(t_lane + s_col + half * HC + 32, v[1]);
                    tc_wait_ld();
                    tc_ld_ready(v[0]);
                    tc_ld_ready(v[1]);
                    if (c0 + HC - 1 > lim) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[c][i] = c0 + 32 * c + i > lim ? -INFINITY : v[c][i];
                    }
                    float ec[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        ec[c] = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float a = v[c >> 1][16 * (c & 1) + i],
                                        b = v[c >> 1][16 * (c & 1) + i + 1];
                            ec[c] = fmax3(ec[c], a, b);
                        }
                    }
                    e = fmax3(ec[0], ec[1], fmaxf(ec[2], ec[3]));
                }
                pair_red[ns & 1][half][r] = e;
                tc_fence_before();
                named_barrier_sync(pair_bar, 64);
                tc_fence_after();
                const float e2 = pair_red[ns & 1][half ^ 1][r];
                if (!ok)
                    continue;
                const float mt = fmaxf(e, e2) * sc;
                bool rescale = false;
                float alpha = 1.f;
                if (mt > m_ref + kRefRoom) {
                    const float ref = mt - kRefBelow;
                    rescale = m_ref != -INFINITY;
                    alpha = rescale ? ex2(m_ref - ref) : 1.f;
                    m_ref = ref;
                }
                const float off = m_ref == -INFINITY ? 0.f : -m_ref;
                const float2 off2 = make_float2(off, off);
                float2 sum2 = make_float2(0.f, 0.f);
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 a = ffma2(make_float2(v[c][i], v[c][i + 1]), sc2, off2);
                        a.x = ex2(a.x);
                        a.y = ex2(a.y);
                        pk[16 * c + i / 2] = pack_half2(a.x, a.y);
                        sum2 = fadd2(sum2, a);
                    }
                l = l * alpha + (sum2.x + sum2.y);
                // both halves have read their scores (the barrier above): P over them
                tc_st32u(t_lane + s_col + half * 32, pk);
                if (j > 0) {
                    wait(&o_done[(ns - 1) & 1], ((ns - 1) >> 1) & 1);  // O may be rescaled
                    if (!ok)
                        continue;
                    tc_fence_after();
                    if (__any_sync(~0u, rescale)) {
#pragma unroll 1
                        for (int c = 0; c < HD / 32; ++c) {
                            float o[32];
                            tc_ld32(t_lane + half * HD + 32 * c, o);
                            tc_wait_ld();
                            tc_ld_ready(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] *= alpha;
                            tc_st32(t_lane + half * HD + 32 * c, o);
                        }
                    }
                }
                const int za = n - t0, ze = j + 1 < nt ? 0 : 16 * last_steps(u);
                const bool zero_v = za < ze;  // (as in the pair kernel)
                if (zero_v) {
                    mbar_wait_bounded(smem_addr(&v_full[(nv + za / VKEYS) % NV]),
                                      ((nv + za / VKEYS) / NV) & 1, nullptr, p.wait_budget_ns);
                    for (int idx = half * 128 + r; idx < (ze - za) * SLABS * 8; idx += 256) {
                        const int key = za + idx / (SLABS * 8), c = idx % (SLABS * 8);
                        const int st = (nv + key / VKEYS) % NV, row = key % VKEYS;
                        *reinterpret_cast<uint4 *>(v_ptr + st * PIECE + (c >> 3) * (VKEYS * 128) +
                                                   row * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                tc_wait_st();
                if (zero_v)
                    fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&p_full));
            }
            wait(&o_done[(ns - 1) & 1], ((ns - 1) >> 1) & 1);
            // the row's exp-sum from both halves, then each half writes its columns
            // (through the last stage's slot: its readers are done, since o_done
            // came after every warp's p_full, and the next stage takes the other)
            pair_red[(ns & 1) ^ 1][half][r] = l;
            named_barrier_sync(pair_bar, 64);
            const float lt = l + pair_red[(ns & 1) ^ 1][half ^ 1][r];
            if (!ok)
                continue;
            tc_fence_after();
            const float inv = lt > 0.f ? 1.f / lt : 0.f;
            const RowOut rows = places.at(
                out + ((size_t)u.x * p.Hq + (size_t)g * p.G) * row_bytes, min(p.TQ, u.z));
            write_rows<HD>(rows, half_out, p.wide_rows, t_lane + half * HD, half * HD, inv, lane, [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&o_free));
            });
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

cudaError_t prefill_set_up(int head_dim)
{
    const cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    return head_dim == 64    ? cudaFuncSetAttribute(packed_prefill_pair_kernel<64>, most,
                                                    (int)pair_smem_bytes<64>())
           : head_dim == 128 ? cudaFuncSetAttribute(packed_prefill_pair_kernel<128>, most,
                                                    (int)pair_smem_bytes<128>())
                             : cudaFuncSetAttribute(packed_prefill_wide_kernel, most,
                                                    (int)kWideSmem);
}

cudaError_t launch_prefill_order(const PrefillParams &p, cudaStream_t stream)
{
    packed_prefill_order_kernel<<<1, kPrefillOrderKeys, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_prefill(int head_dim, const CUtensorMap &tq, const CUtensorMap &tk,
                           const CUtensorMap &tv, const PrefillParams &p, int grid,
                           cudaStream_t stream)
{
    auto kernel = head_dim == 64    ? packed_prefill_pair_kernel<64>
                  : head_dim == 128 ? packed_prefill_pair_kernel<128>
                                    : packed_prefill_wide_kernel;
    const size_t smem = head_dim == 64    ? pair_smem_bytes<64>()
                        : head_dim == 128 ? pair_smem_bytes<128>()
                                          : kWideSmem;
    cudaError_t e;
    if ((e = launch_prefill_order(p, stream)) != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(head_dim == 256 ? kWideThreads : kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, p);
}

}  // namespace pgd
