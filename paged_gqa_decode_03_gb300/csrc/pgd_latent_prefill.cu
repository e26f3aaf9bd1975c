// Causal attention over packed prompts whose keys and values have been expanded from
// latent vectors (packed_latent_prefill), on the 5th-generation tensor cores.
//
// Head h has keys k[t][h] and values v[t][h] of its own (head_dim each) and, behind the
// keys, one rotated key k_rope[t] that all heads share: out = sum_{u <= t} p_u v_u /
// sum_u p_u with p_u = exp2((q . [k_u | k_rope_u]) scale log2(e) - m), one pass over the
// keys with a running reference m and sum.  2 (2 head_dim + rope_dim) operations a row
// and key, a head's keys read by its rows alone: the tensor cores bound a long prompt.
//
// The shape is that of packed_gqa_prefill's pair kernel: a unit is two tiles of 128
// tokens of one head that share every stage of 128 keys, a warp each for copies (K,
// V), scores and outputs, a softmax thread a row; the units are the order kernel's,
// longest first.  What differs:
//   * The queries of two tiles, head_dim 128 with its rotary part, take 96 KB, so K and
//     V move in pieces of 16 KB, K by 64-wide slabs (the last of them the rotary keys,
//     from a tensor without heads), V by 64 keys: eight places, five for K, three for V.
//     Each tile's queries come as soon as its own last scores of the unit before are done.
//   * Products, copies and commits are issued by an elected lane (see elect_one), all of
//     a product's together: a wait between them costs more than a piece's products.
//   * What runs once a unit (the causal border, the zeroed tail, the output) is short
//     loops outside the loop over stages: long unrolled code is fetched anew each time.
//     The border written into the loop's 128 scores took a tile's last stage 3900 cycles
//     where a stage takes 1300, and slowed the loop by its mere presence.
//
// Measured, head_dim 128 (rope_dim 64): one prompt of 16381 tokens x 16 heads 815 to 935 us
// (1685 to 1470 TFLOP/s: few calls to sustained ones, by the power limit), 4 x 2048 x 32 heads
// 159 to 169 a call and 155 in a graph, 37 prompts of 1 to 512 tokens x 16 heads 31 to 33 and
// 28.5.  By clock stamps a period of both tiles takes
// 3200 to 3450 cycles, of which the products take 2560.  They are there in time (a tile's
// weights 400 cycles before the other's scores are whole), so what is lost lies between the
// four groups of a period, 150 to 200 cycles each; shared memory is read at a quarter of
// its rate.  A short unit is bound by its chain instead (queries and first keys, scores,
// softmax, product, output: 6000 cycles), a call by the order kernel and the first copies
// in front (5 us).
#include <algorithm>

#include "pgd_device.cuh"
#include "pgd_internal.h"
#include "pgd_rows.cuh"
#include "pgd_units.cuh"

namespace pgd {

namespace {

constexpr int kNT = 128;               // keys per stage
constexpr int kTile = 128;             // tokens per tile
constexpr int kSlab = 128 * 128;       // bytes of 128 rows of one 64-wide slab
constexpr uint32_t kNegateA = 1u << 13;  // of the products' descriptor: -A for A (a negative scale)
constexpr int kExpandedThreads = 384;

// Pieces of K and V in the rings, score buffers.
template <int D> struct ExpandedShape;
template <> struct ExpandedShape<64> {
    static constexpr int NK = 6, NV = 3, SBUF = 2;
};
template <> struct ExpandedShape<128> {
    static constexpr int NK = 5, NV = 3, SBUF = 1;
};
template <int D> constexpr size_t expanded_smem_bytes()
{
    return size_t(2) * (D / 64 + 1) * kSlab +
           size_t(ExpandedShape<D>::NK + ExpandedShape<D>::NV) * kSlab + 1024;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kExpandedThreads, 1)
    packed_latent_prefill_kernel(const __grid_constant__ CUtensorMap tmap_q,
                                 const __grid_constant__ CUtensorMap tmap_qr,
                                 const __grid_constant__ CUtensorMap tmap_k,
                                 const __grid_constant__ CUtensorMap tmap_kr,
                                 const __grid_constant__ CUtensorMap tmap_v, const PrefillParams p)
{
    using X = ExpandedShape<D>;
    constexpr int NK = X::NK, NV = X::NV, SBUF = X::SBUF;
    constexpr int SLABS = D / 64, KP = SLABS + 1, VP = SLABS, VKEYS = kNT / VP;
    constexpr int PIECE = kSlab;
    constexpr int Q_TILE = KP * kSlab;
    constexpr uint32_t S_COL = 2 * D, P_COL = S_COL + SBUF * kNT;
    static_assert(P_COL + 128 <= 512, "tensor memory");
    constexpr uint32_t IDESC_S = tc_idesc_f16(128, kNT, 0, 0);
    constexpr uint32_t IDESC_O = tc_idesc_f16(128, D, 0, 1);

    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t q_full[2], q_empty[2], k_full[NK], k_empty[NK], v_full[NV],
        v_empty[NV], s_full[2], s_free[2], p_full[2], z_go[2], z_full[2], o_done[2], o_free[2], mma_done;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_flag;

    const uint32_t dyn_base = smem_addr(dyn_smem);
    const uint32_t base = (dyn_base + 1023u) & ~1023u;
    uint8_t *const base_ptr = dyn_smem + (base - dyn_base);
    const uint32_t q_s = base, k_s = q_s + 2 * Q_TILE, v_s = k_s + NK * PIECE;
    uint8_t *const v_ptr = base_ptr + 2 * Q_TILE + NK * PIECE;

    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_addr(&k_full[i]), 1);
            mbar_init(smem_addr(&k_empty[i]), 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_addr(&v_full[i]), 1);
            mbar_init(smem_addr(&v_empty[i]), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_addr(&q_full[x]), 1);
            mbar_init(smem_addr(&q_empty[x]), 1);
            mbar_init(smem_addr(&s_full[x]), 1);
            mbar_init(smem_addr(&s_free[x]), 4);
            mbar_init(smem_addr(&p_full[x]), 4);
            mbar_init(smem_addr(&z_go[x]), 1);
            mbar_init(smem_addr(&z_full[x]), 4);
            mbar_init(smem_addr(&o_done[x]), 1);
            mbar_init(smem_addr(&o_free[x]), 4);
        }
        mbar_init(smem_addr(&mma_done), 2);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_qr);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_kr);
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
        const int from = x * kTile;
        return u.z > from ? (u.y + min(u.z, from + kTile) + kNT - 1) / kNT : 0;
    };
    // Steps of 16 keys that the output's product takes of a tile's last stage: up to its
    // last key
    auto last_steps = [&](const int4 &u, int x) {
        return (u.y + min(u.z, (x + 1) * kTile) - 1) % kNT / 16 + 1;
    };

    // the softmax warps hold a row's 128 scores and half of its weights: they
    // take registers that the copying and issuing warps do not need (128 x 104
    // + 256 x 200 of the 384 x 168 of the launch)
    if (warp < 4) {
      regs_give<104>();
      if (warp == 0 || warp == 3) {
        if (elect_one()) {
            // ======================================================== copies
            // warp 0: Q tiles, K by 64-wide slabs and the rotary keys; warp 3: V
            const bool is_v = warp == 3;
            const uint64_t pol = l2_evict_last_policy();
            uint64_t *full = is_v ? v_full : k_full;
            const int slots = is_v ? NV : NK;
            int n = 0, nq[2] = {0, 0};   // copies issued so far
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                return mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns);
            };
            auto load_k = [&](int row, int head, int from, int to) {
                for (int kp = from; kp < to; ++kp, ++n) {
                    const int st = n % NK;
                    if (!wait(&k_empty[st], ((n / NK) & 1) ^ 1))
                        return false;
                    const uint32_t bar = smem_addr(&k_full[st]);
                    mbar_arrive_expect_tx(bar, PIECE);
                    if (kp < SLABS)
                        tma_load_4d(k_s + st * PIECE, &tmap_k, 0, row, kp, head, bar, pol);
                    else
                        tma_load_4d(k_s + st * PIECE, &tmap_kr, 0, row, 0, 0, bar, pol);
                }
                return true;
            };
            auto load_v = [&](int row, int head) {
                for (int vp = 0; vp < VP; ++vp, ++n) {
                    const int st = n % NV;
                    if (!wait(&v_empty[st], ((n / NV) & 1) ^ 1))
                        return false;
                    const uint32_t bar = smem_addr(&v_full[st]);
                    mbar_arrive_expect_tx(bar, PIECE);
                    tma_load_4d(v_s + st * PIECE, &tmap_v, 0, row + vp * VKEYS, 0, head, bar, pol);
                }
                return true;
            };
            int4 next = unit_at(p, 0, units);
            for (int k = 0; k < turns && ok; ++k) {
                const int ui = unit_of(k);
                const int4 u = next;
                next = unit_at(p, k + 1, units);
                if (ui >= units)
                    continue;
                const int head = u.w, row0 = u.x - u.y;  // the prompt's first row
                const int nt = max(stages(u, 0), stages(u, 1));
                if (is_v) {
                    for (int j = 0; j < nt && ok; ++j)
                        ok = load_v(row0 + j * kNT, head);
                    continue;
                }
                // A tile's place for Q is free after the last unit's last scores of that
                // tile: tile A's comes before the last of the first K, tile B's behind it
                auto load_q = [&](int x) {
                    if (!wait(&q_empty[x], (nq[x] & 1) ^ 1))
                        return false;
                    const uint32_t bar = smem_addr(&q_full[x]);
                    mbar_arrive_expect_tx(bar, Q_TILE);
                    tma_load_4d(q_s + x * Q_TILE, &tmap_q, 0, u.x + x * kTile, 0, head, bar);
                    tma_load_4d(q_s + x * Q_TILE + SLABS * kSlab, &tmap_qr, 0, u.x + x * kTile, 0, head,
                                bar);
                    ++nq[x];
                    return true;
                };
                ok = load_k(row0, head, 0, KP - 1) && load_q(0) && load_k(row0, head, KP - 1, KP) &&
                     (u.z <= kTile || load_q(1));
                for (int j = 1; j < nt && ok; ++j)
                    ok = load_k(row0 + j * kNT, head, 0, KP);
            }
            if (!ok) {
                give_up();
                // let the copies in flight land before the CTA exits
                for (int x = 0; x < 2; ++x)
                    if (nq[x])
                        mbar_wait_bounded(smem_addr(&q_full[x]), (nq[x] - 1) & 1, nullptr,
                                          p.wait_budget_ns);
                for (int i = max(0, n - slots); i < n; ++i)
                    mbar_wait_bounded(smem_addr(&full[i % slots]), (i / slots) & 1, nullptr,
                                      p.wait_budget_ns);
            }
        }
        __syncwarp();
      } else {
        // ============================================================ products
        // warp 1: scores, warp 2: outputs.  The warp stays together: barriers are tested by
        // all lanes (34 cycles each; 88 by a lane alone), products issued by an elected one.
        bool ok = true;
        auto wait = [&](uint64_t *bar, int parity) {
            if (ok && !__all_sync(~0u, mbar_wait_bounded(smem_addr(bar), parity, &abort_flag,
                                                         p.wait_budget_ns)))
                ok = false;
            return ok;
        };
        int4 next = unit_at(p, 0, units);
        if (warp == 1) {
            const uint32_t idesc_s = IDESC_S | (p.scale_log2 < 0.f ? kNegateA : 0u);
            const uint64_t q_desc = tc_sdesc(q_s, 16, 1024);
            const uint64_t k_desc = tc_sdesc(k_s, 16, 1024);
            int nk = 0, nq[2] = {0, 0};  // K pieces, Q tiles used up
            int uses[2] = {0, 0};      // of each score buffer
            for (int k = 0; k < turns && ok; ++k) {
                const int ui = unit_of(k);
                const int4 u = next;
                next = unit_at(p, k + 1, units);
                if (ui >= units)
                    continue;
                const int nt0 = stages(u, 0), nt1 = stages(u, 1), nmax = max(nt0, nt1);
                for (int j = 0; j < nmax && ok; ++j, nk += KP) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const bool last_user = x == 1 || j >= nt1;
                        if (j >= (x ? nt1 : nt0) || !ok)
                            continue;
                        // (all waits come first: groups of products with a wait between them
                        // reach the pipe 300 cycles apart, more than a group's 256)
                        if (j == 0 && !wait(&q_full[x], nq[x]++ & 1))
                            continue;
                        if (x == 0 || j >= nt0)
                            for (int kp = 0; kp < KP; ++kp)
                                wait(&k_full[(nk + kp) % NK], ((nk + kp) / NK) & 1);
                        // the buffer's last scores have been read
                        const int b = SBUF == 2 ? x : 0;
                        if (uses[b] && !wait(&s_free[b], (uses[b] - 1) & 1))
                            continue;
                        ++uses[b];
                        if (!ok)
                            continue;
                        const uint64_t qx = q_desc + ((x * Q_TILE) >> 4);
                        const uint32_t d = tmem + S_COL + b * kNT;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kp = 0; kp < KP; ++kp) {
                                const int st = (nk + kp) % NK;
                                const uint64_t ks = k_desc + ((st * PIECE) >> 4);
                                const uint64_t qs = qx + ((kp * kSlab) >> 4);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc_mma(d, qs + ((kk * 32) >> 4), ks + ((kk * 32) >> 4), idesc_s,
                                           kp > 0 || kk > 0);
                                if (kp == KP - 1)
                                    tc_commit(smem_addr(&s_full[x]));
                                if (last_user)
                                    tc_commit(smem_addr(&k_empty[st]));
                            }
                            if (j == (x ? nt1 : nt0) - 1)
                                tc_commit(smem_addr(&q_empty[x]));
                        }
                        __syncwarp();
                    }
                }
            }
        } else {
            const uint64_t v_desc = tc_sdesc(v_s, VKEYS * 128, 1024);
            int nv = 0;                           // V pieces used up
            // P V products, units, zeroed tails of each tile
            int np[2] = {0, 0}, no[2] = {0, 0}, nz[2] = {0, 0};
            for (int k = 0; k < turns && ok; ++k) {
                const int ui = unit_of(k);
                const int4 u = next;
                next = unit_at(p, k + 1, units);
                if (ui >= units)
                    continue;
                const int nt0 = stages(u, 0), nt1 = stages(u, 1), nmax = max(nt0, nt1);
                for (int j = 0; j < nmax && ok; ++j, nv += VP) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int nt = x ? nt1 : nt0;
                        const bool last_user = x == 1 || j >= nt1;
                        if (j >= nt || !ok)
                            continue;
                        // the last unit's output has been read
                        if (j == 0 && no[x]++ && !wait(&o_free[x], no[x] & 1))
                            continue;
                        if (!wait(&p_full[x], np[x] & 1))
                            continue;
                        ++np[x];
                        const uint32_t o = tmem + x * D, a = tmem + P_COL + x * 64;
                        const bool last = j + 1 == nt;
                        const int steps = last ? last_steps(u, x) : kNT / 16;
                        // keys behind the prompt in the last step: zeroed in V first
                        const bool tail = last && u.y + u.z - j * kNT < 16 * steps;
                        if (steps == kNT / 16 && !tail) {
                            for (int vp = 0; vp < VP; ++vp)
                                wait(&v_full[(nv + vp) % NV], ((nv + vp) / NV) & 1);
                            if (!ok)
                                continue;
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int vp = 0; vp < VP; ++vp) {
                                    const int st = (nv + vp) % NV;
                                    const uint64_t vs = v_desc + ((st * PIECE) >> 4);
#pragma unroll
                                    for (int kk = 0; kk < VKEYS / 16; ++kk)
                                        tc_mma_ta(o, a + (vp * (VKEYS / 16) + kk) * 8,
                                                  vs + ((kk * 2048) >> 4), IDESC_O,
                                                  j > 0 || vp > 0 || kk > 0);
                                    if (last_user)
                                        tc_commit(smem_addr(&v_empty[st]));
                                }
                                tc_commit(smem_addr(&o_done[x]));
                            }
                            __syncwarp();
                            continue;
                        }
                        for (int vp = 0; vp < VP && ok; ++vp) {
                            const int st = (nv + vp) % NV, k0 = vp * (VKEYS / 16);
                            if (!wait(&v_full[st], ((nv + vp) / NV) & 1))
                                break;
                            tc_fence_after();
                            const uint64_t vs = v_desc + ((st * PIECE) >> 4);
                            const int here = min(VKEYS / 16, steps - k0);
                            if (here > 0 && steps <= k0 + VKEYS / 16 && tail) {
                                if (lane == 0)
                                    mbar_arrive(smem_addr(&z_go[x]));
                                __syncwarp();
                                if (!wait(&z_full[x], nz[x]++ & 1))
                                    break;
                                tc_fence_after();
                            }
                            if (elect_one()) {
#pragma unroll 1
                                for (int kk = 0; kk < here; ++kk)
                                    tc_mma_ta(o, a + (k0 + kk) * 8, vs + ((kk * 2048) >> 4), IDESC_O,
                                              j > 0 || vp > 0 || kk > 0);
                                if (last_user)
                                    tc_commit(smem_addr(&v_empty[st]));
                                if (vp == VP - 1)
                                    tc_commit(smem_addr(&o_done[x]));
                            }
                            __syncwarp();
                        }
                    }
                }
            }
        }
        if (!ok && lane == 0)
            give_up();
        // every product issued has completed before the memory is freed
        if (elect_one())
            tc_commit(smem_addr(&mma_done));
        __syncwarp();
        mbar_wait_bounded(smem_addr(&mma_done), 0, nullptr, p.wait_budget_ns);
      }
    } else {
        regs_take<200>();
        // ============================================================ softmax
        const int x = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int r = 32 * quarter + lane;  // this thread's row of the tile
        const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t s_col = S_COL + (SBUF == 2 ? x : 0) * kNT, o_col = x * D,
                       p_col = P_COL + x * 64;
        // a scale of 0 runs as 1e-30: exp2 of every score is then 1 in fp32
        // (the mean over the range, as for 0) while masked scores, -inf, still
        // give 0
        const float sc = p.scale_log2 == 0.f ? 1e-30f : fabsf(p.scale_log2);
        const float2 sc2 = make_float2(sc, sc);
        int ns = 0, nv = 0, nz = 0;  // S tiles of this tile, V pieces of the CTA, zeroed tails so far
        bool ok = true;
        int4 next = unit_at(p, 0, units);
        for (int k = 0; k < turns && ok; ++k) {
            const int ui = unit_of(k);
            const int4 u = next;
            next = unit_at(p, k + 1, units);  // a turn ahead: its latency passes meanwhile
            if (ui >= units)
                continue;
            const int head = u.w;
            const int nt0 = stages(u, 0), nt1 = stages(u, 1), ntx = x ? nt1 : nt0;
            const int left = min(kTile, u.z - x * kTile);  // tokens of this tile
            const int n = u.y + u.z;                     // tokens of the prompt
            const bool row_ok = r < left;
            const int lo = u.y + x * kTile;          // position of the tile's first token
            float m_ref = -INFINITY, l = 0.f;
            int j = 0;
#pragma unroll 1
            for (int part = 0; part < 2 && ok && ntx > 0; ++part) {
                if (part == 1) {
                    // The causal border crosses a tile's last stage alone (tiles and stages begin at
                    // multiples of 128): of a warp's 32 rows it cuts the warp's own 32 keys, the rows
                    // see all keys before and none behind.  The scores behind it are replaced where
                    // they lie, in a loop of few instructions: they run once a unit, cold.
                    if (!__all_sync(~0u, mbar_wait_bounded(smem_addr(&s_full[x]), ns & 1, &abort_flag,
                                                           p.wait_budget_ns))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = quarter; c < 4; ++c) {
                        const int seen = 32 * (quarter - c) + lane;
                        float w[32];
                        tc_ld32(t_lane + s_col + 32 * c, w);
                        tc_wait_ld();
                        tc_ld_ready(w);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            w[i] = i <= seen ? w[i] : -INFINITY;
                        tc_st32(t_lane + s_col + 32 * c, w);
                    }
                    tc_wait_st();
                }
                for (const int end = ntx - 1 + part; j < end; ++j, ++ns) {
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
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&p_full[x]));
                    l = l * alpha + (sum2.x + sum2.y);
                }
            }
            // Rows behind the prompt belong to the next one and may hold anything: those
            // that the tile's last step takes in are zeroed in V (their weights are 0,
            // which does not hide a NaN), when the products have come to their piece.
            const int za = n - lo, ze = 16 * last_steps(u, x);
            if (ok && ntx > 0 && za < ze) {
                if (!__all_sync(~0u, mbar_wait_bounded(smem_addr(&z_go[x]), nz++ & 1, &abort_flag,
                                                       p.wait_budget_ns))) {
                    ok = false;
                } else {
                    const int vp = za / VKEYS, st = (nv + (ntx - 1) * VP + vp) % NV;
                    uint8_t *vs = v_ptr + st * PIECE;
                    for (int idx = r; idx < (ze - za) * SLABS * 8; idx += 128) {
                        const int row = za - vp * VKEYS + idx / (SLABS * 8), c = idx % (SLABS * 8);
                        *reinterpret_cast<uint4 *>(vs + (c >> 3) * (VKEYS * 128) + row * 128 +
                                                   (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&z_full[x]));
                }
            }
            // ---- out = O / l
            if (ok && ntx > 0) {
                ok = __all_sync(~0u, mbar_wait_bounded(smem_addr(&o_done[x]), (ns - 1) & 1,
                                                       &abort_flag, p.wait_budget_ns));
                if (ok) {
                    tc_fence_after();
                    const float inv = l > 0.f ? 1.f / l : 0.f;
                    auto read = [&] {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_addr(&o_free[x]));
                    };
                    char *const dst =
                        out + ((size_t)(u.x + x * kTile + r) * p.Hq + head) * row_bytes;
                    write_own_row<D>(row_ok ? dst : nullptr, half_out, p.wide_rows, t_lane + o_col,
                                     inv, read);
                }
            }
            nv += VP * max(nt0, nt1);
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

cudaError_t latent_prefill_set_up(int head_dim)
{
    const cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    return head_dim == 64 ? cudaFuncSetAttribute(packed_latent_prefill_kernel<64>, most,
                                                 (int)expanded_smem_bytes<64>())
                          : cudaFuncSetAttribute(packed_latent_prefill_kernel<128>, most,
                                                 (int)expanded_smem_bytes<128>());
}

cudaError_t launch_latent_prefill(int head_dim, const LatentPrefillMaps &m, const PrefillParams &p,
                                  int grid, cudaStream_t stream)
{
    auto kernel = head_dim == 64 ? packed_latent_prefill_kernel<64> : packed_latent_prefill_kernel<128>;
    cudaError_t e;
    if ((e = launch_prefill_order(p, stream)) != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kExpandedThreads);
    cfg.dynamicSmemBytes = head_dim == 64 ? expanded_smem_bytes<64>() : expanded_smem_bytes<128>();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, m.q, m.qr, m.k, m.kr, m.v, p);
}

}  // namespace pgd
