// Attention over a latent cache, absorbed queries (paged_latent_attention), on the
// 5th-generation tensor cores: every head reads the same rows, whose latent part is
// key and value at once.
//
// For row r of the queries and cached token t, s_t = (q_r . c_t + q_rope_r . k_t)
// scale log2(e); out_r = sum p_t c_t / sum p_t over the tokens that r sees, p_t =
// exp2(s_t - m), in one pass with a running reference m and sum.
//
// A cached row of 2 (R + P) bytes serves all rows of its sequence with 2 (2 R + P)
// operations each: at R 512, P 64 and 128 rows 242 operations a byte, just below what
// the GPU has (284), so HBM bounds a decode step with up to 128 heads, if nothing
// else does.  What decides the shape of the work:
//   * Output: 128 rows x 512 fp32 would fill an SM's tensor memory and leave no room
//     for scores, and the 128 x 576 queries take 147 KB of its shared memory.  So two
//     CTAs (a pair of the tensor cores, cta_group::2, M 128) share a tile of 128 rows:
//     64 rows of queries, weights and outputs in each.
//   * A stage is 128 tokens.  Scores: each CTA copies 64 of them (all R + P values):
//     B, split over the pair by tokens.  Outputs: each CTA copies all 128, of half of
//     the R values: B, split by values.  That takes the latent part in twice, the
//     second time from L2: every byte comes from HBM once, and an SM takes in from L2
//     two to three times what HBM gives it (130 GB/s and more in copies of 32 KB).
//   * A product of a pair takes 32 cycles (scores, N 128: 36 a stage) or 64 (outputs,
//     N 256: 16), 2176 cycles a stage at R 512, against 3150 in which HBM brings its
//     147 KB.  Fewer rows cost the same; HBM still bounds.  They run at that rate only
//     when an elected lane of a converged warp issues them: `if (lane == 0)` costs 50
//     cycles a product and 300 a turn (32 requests of 8 k to 32 k tokens took 231 us that
//     way, 139 this way).
//   * The stages of all units (sequence, tile of rows) are cut into equal runs, one
//     per resident pair, whatever the lengths; a unit that is cut leaves pieces
//     (reference maximum, exp-sum, unscaled output; two per run at most), which a
//     second kernel joins.  Rings run on from unit to unit.
//   * Weights go to tensor memory as fp16, two stages of them, next to two score
//     buffers.  A row of A lies there twice (lanes r and 64 + r), and its scores come
//     split over the same lanes: the two warps of a row exchange their halves through
//     16 KB of shared memory.  (In shared memory, as the products would take them too,
//     they need a release of plain writes to the pair each stage: 1500 cycles or more.)
//
// Measured in a graph (a call: 0.5 to 4 us more): 32 requests of 8 k to 32 k tokens with 16
// heads 122 to 125 us (655 MB: 5.3 TB/s; HBM's floor 97), 64 of 512 to 4096 tokens with 128
// heads 61.5, 24 of up to 8 k tokens with up to 5 rows of 32 heads 47, one of 1000 tokens 15
// (nearly all of it in every call: the runs' division 2, the first pages, copies and Q 4, the
// last softmax and outputs 3, the joining kernel 4).  What bounds a long run is not settled.
// It is not the bytes in flight alone: other divisions of the same memory, against 126, gave
// 133 with five places for K and three for V, 132 with Q's place cut to a tile's rows where
// they are few and longer rings, 143 with two pieces of 32 KB for K.  The latent part comes
// into shared memory twice, 139 KB a stage and SM, which is the likelier cause.
//
// A unit's stages are its sequence's, also for tiles of earlier rows that see none of the
// last: a chunk of 4096 rows takes 375 us with 16 heads, 3046 with 128 (1540 TFLOP/s of
// which half are of use), behind 8192 cached tokens 1130 and 9267 (1530, 1/1.2 of use).
#include <type_traits>

#include "pgd_device.cuh"
#include "pgd_internal.h"
#include "pgd_rows.cuh"

namespace pgd {

namespace {

// warp 0 Q, K and rotary-key copies, 1 V copies, 2 scores, 3 outputs, 4-11 softmax
constexpr int kLatentThreads = 384;
constexpr uint32_t kLatentNegateA = 1u << 13;  // of the products' descriptor: -A for A

// What a sequence asks for: its length, first query row, rows (0 where its numbers do
// not fit together), stages per unit and units (tiles of two half tiles).  (Plain
// loads: the kernel starts while the one before it may still be writing, up to
// griddep_wait, so its inputs are not read-only here.)
struct LatentSeq {
    int L, row0, n, T, tiles;
    unsigned bad;
};

__device__ __forceinline__ LatentSeq latent_seq(const LatentParams &p, int s)
{
    LatentSeq q;
    const int maxlen = p.MB << p.log2BS;
    q.L = p.seq_lens[s];
    q.row0 = p.cu_q ? p.cu_q[s] : s;
    q.n = p.cu_q ? p.cu_q[s + 1] - q.row0 : 1;
    q.bad = 0;
    if (q.L < 0 || q.L > maxlen)
        q.bad = kErrSeqLen;
    else if (q.n < 0 || q.n > (p.cu_q ? q.L : 1) || q.n > p.max_q || q.row0 < 0 ||
             q.row0 > p.total_q - q.n)
        q.bad = kErrQueryLen;
    if (q.bad)
        q.n = 0;
    // (a row of a sequence without tokens: one stage, in which it sees nothing)
    q.T = q.n ? max(1, (q.L + kLatentNT - 1) / kLatentNT) : 0;
    q.tiles = (p.half_tiles(q.n) + 1) / 2;
    return q;
}
__device__ __forceinline__ int latent_cost(const LatentSeq &q)
{
    return q.tiles * (q.T + kLatentUnitCost);
}

// A run [x0, x1) of the cost of all units, a unit (or the part of it that the run
// holds) at a time: stage t of a unit that begins at cost c lies at c +
// kLatentUnitCost + t.  Every role walks its own copy.
struct LatentWalk {
    LatentSeq q;
    int s, v, t, t_end;  // sequence, its tile, stages [t, t_end)
    int at, x1;          // where unit v begins, and the run's end

    __device__ __forceinline__ LatentWalk(const LatentParams &p, int s0, int begin, int x0, int x1_)
    {
        s = s0;
        x1 = at = x1_;
        v = t = t_end = 0;
        if (x0 >= x1)
            return;
        q = latent_seq(p, s);
        v = (x0 - begin) / (q.T + kLatentUnitCost);
        at = begin + v * (q.T + kLatentUnitCost);
        t = max(0, x0 - at - kLatentUnitCost);
        set_end();
    }
    __device__ __forceinline__ void set_end()
    {
        t_end = min(q.T, x1 - at - kLatentUnitCost);
        if (t_end <= t)  // the run ends before the unit's first stage
            at = x1;
    }
    __device__ __forceinline__ bool more() const { return at < x1; }
    __device__ __forceinline__ void next(const LatentParams &p)
    {
        at += q.T + kLatentUnitCost;
        if (at >= x1)
            return;
        t = 0;
        if (++v == q.tiles) {
            v = 0;
            do
                q = latent_seq(p, ++s);
            while (latent_cost(q) == 0);
        }
        set_end();
    }
    // the run that holds the unit's last stage, of `runs` equal ones of `total`
    __device__ __forceinline__ int last_run(int total, int runs) const
    {
        return (int)(((long long)(at + q.T + kLatentUnitCost) * runs - 1) / total);
    }
};

// A half tile: the rows of one CTA.  Heads up to 64 go together with as many tokens as
// fit, more heads in blocks of 64 of one token.
struct HalfTile {
    int token, head;  // of its first row, within the sequence
    __device__ __forceinline__ HalfTile(const LatentParams &p, int index)
    {
        token = p.HB == 1 ? index * p.TQ : index / p.HB;
        head = p.HB == 1 ? 0 : (index - token * p.HB) * 64;
    }
};

// Sum over the CTA's threads before this one of `x`, and over all in *total.
__device__ __forceinline__ int latent_prefix(int x, int *warp_sum, int *total)
{
    constexpr int WARPS = kLatentThreads / 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(~0u, inc, off);
        if (lane >= off)
            inc += y;
    }
    if (lane == 31)
        warp_sum[w] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < w)
            before += warp_sum[i];
        all += warp_sum[i];
    }
    __syncthreads();
    *total = all;
    return before + inc - x;
}

}  // namespace

// In front of calls whose rows, if they overlap (offsets that decrease, of which some sequences
// are flagged), may cost more than 32 bits count: *allowed is then 0 instead of S, and nothing
// is run.  (A look in the main kernel instead took every call 0.3 to 0.5 us.)
constexpr int kLatentCheckThreads = 1024;
__global__ void __launch_bounds__(kLatentCheckThreads) paged_latent_check_kernel(const LatentParams p)
{
    __shared__ unsigned long long all;
    if (threadIdx.x == 0)
        all = 0;
    __syncthreads();
    unsigned long long cost = 0;
    for (int s = threadIdx.x; s < p.S; s += kLatentCheckThreads) {
        const LatentSeq q = latent_seq(p, s);
        if (q.bad)
            atomicOr(p.err, q.bad);
        cost += (unsigned)latent_cost(q);
    }
    atomicAdd(&all, cost);
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool fits = all < 1ull << 31;
        if (!fits)
            atomicOr(p.err, kErrQueryLen);
        *p.allowed = fits ? p.S : 0;
    }
}

template <int R>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLatentThreads, 1)
    paged_latent_kernel(const __grid_constant__ CUtensorMap tmap_q,
                        const __grid_constant__ CUtensorMap tmap_qr,
                        const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_kr,
                        const __grid_constant__ CUtensorMap tmap_v, const LatentParams p)
{
    using X = LatentShape<R>;
    constexpr int NT = kLatentNT, NK = X::NK, NV = X::NV, KP = X::KP, VP = X::VP, NS = X::NS,
                  NR = X::NR;
    constexpr int KSLABS = X::KSLABS, VSLABS = X::VSLABS, VKEYS = X::VKEYS;
    constexpr int PIECE = kLatentPiece, KGROUP = KSLABS * 1024, VGROUP = VSLABS * 1024;
    constexpr int SLABS = R / 64, ROWS = kLatentRows, Q_SLAB = ROWS * 128, X_BYTES = 8 * 32 * 64;
    // a CTA's columns: outputs and scores (N / 2 of a pair's product), two stages' weights
    constexpr uint32_t O_COL = 0, S_COL = R / 2, P_COL = S_COL + NS * NT / 2;
    static_assert(P_COL + 2 * NT / 2 <= 512, "tensor memory");
    constexpr int ON = R >= 256 ? 256 : R;        // N of an output's product
    constexpr uint32_t IDESC_S = tc_idesc_f16(128, NT, 0, 0);
    constexpr uint32_t IDESC_O = tc_idesc_f16(128, ON, 0, 1);

    extern __shared__ __align__(1024) uint8_t dyn_smem[];
    // (the even CTA's q_full, k_full, v_full, s_free, z_full, p_full and o_free count for both)
    __shared__ __align__(8) uint64_t q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV],
        v_empty[NV], z_go, z_full, s_full[NS], s_free[NS], p_full[2], o_done[2], o_free, mma_done;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_flag;
    __shared__ float red[2][4][ROWS];  // [parity][quarter of a stage's tokens][row]
    __shared__ int warp_sum[kLatentThreads / 32], run_begin, run_seq;

    const uint32_t q_s = smem_addr(dyn_smem), x_s = q_s + (SLABS + 1) * Q_SLAB, r_s = x_s + X_BYTES,
                   k_s = r_s + NR * ROWS * 128, v_s = k_s + NK * PIECE;
    uint8_t *const x_ptr = dyn_smem + (x_s - q_s);
    uint8_t *const v_ptr = dyn_smem + (v_s - q_s);

    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int run = (int)blockIdx.x / 2;
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
        mbar_init(smem_addr(&z_go), 1);
        mbar_init(smem_addr(&z_full), 16);
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_addr(&s_full[i]), 1);
            mbar_init(smem_addr(&s_free[i]), 16);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&p_full[i]), 16);
            mbar_init(smem_addr(&o_done[i]), 1);
        }
        mbar_init(smem_addr(&o_free), 16);
        mbar_init(smem_addr(&mma_done), 2);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_qr);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_kr);
        prefetch_tensormap(&tmap_v);
    }
    if (warp == 0)
        tc_alloc_pair(smem_addr(&tmem_base_s), 512);

    griddep_wait();  // what the launches before wrote
    // ---- the run: [x0, x1) of the cost of all units; the sequence that holds x0
    const int S = p.allowed ? *p.allowed : p.S;
    int total = 0, mine = 0, before = 0;  // before: this thread's (last) sequence
    for (int s0 = 0; s0 < S; s0 += kLatentThreads) {
        const int s = s0 + (int)threadIdx.x;
        int all;
        mine = 0;
        if (s < S) {
            const LatentSeq q = latent_seq(p, s);
            if (q.bad && blockIdx.x == 0)
                atomicOr(p.err, q.bad);
            mine = latent_cost(q);
        }
        before = total + latent_prefix(mine, warp_sum, &all);
        total += all;
    }
    const int x0 = (int)((long long)total * run / p.runs);
    const int x1 = (int)((long long)total * (run + 1) / p.runs);
    if (x1 > x0 && S <= kLatentThreads) {
        if (mine > 0 && before <= x0 && x0 < before + mine) {
            run_seq = (int)threadIdx.x;
            run_begin = before;
        }
    } else if (x1 > x0) {
        int past = 0;
        for (int s0 = 0; s0 < S && past <= x0; s0 += kLatentThreads) {
            const int s = s0 + (int)threadIdx.x;
            const int here = s < S ? latent_cost(latent_seq(p, s)) : 0;
            int all;
            const int at = past + latent_prefix(here, warp_sum, &all);
            if (here > 0 && at <= x0 && x0 < at + here) {
                run_seq = s;
                run_begin = at;
            }
            past += all;
        }
    }
    tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    griddep_launch_dependents();
    LatentWalk walk(p, x1 > x0 ? run_seq : 0, x1 > x0 ? run_begin : 0, x0, x1);

    auto give_up = [&]() {
        if (!abort_flag)
            atomicOr(p.err, kErrTimeout);
        abort_flag = 1;
    };
    // a barrier of the CTA that issues the products
    auto lead = [&](uint64_t *bar) { return cluster_addr(smem_addr(bar), 0); };

    if (warp < 2) {
        // ============================================================ copies
        // warp 0: Q, the latent part as K by slabs of this CTA's 64 tokens, the rotary
        // keys; warp 1: the latent part as V, tokens of this CTA's half of the values.
        // A piece is a copy per page (or one copy, where pages are longer).
        // (barriers are tested by all lanes, copies issued by an elected one, a piece's all
        // together, their pages handed round: whatever a single lane does by itself costs
        // it hundreds of cycles, and each choice of one some tens)
        const bool is_v = warp == 1;
        const int rows = is_v ? p.v_rows : p.k_rows;
        const int copies = (is_v ? VKEYS : ROWS) / rows;
        const int from = lane * rows + (is_v ? 0 : rank * ROWS);
        const uint32_t copy_bytes = (rows / 8) * (is_v ? VGROUP : KGROUP);
        int nst = 0, nq = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, int parity) {
            ok = __all_sync(~0u, mbar_wait_bounded(smem_addr(bar), parity, &abort_flag,
                                                   p.wait_budget_ns));
            return ok;
        };
        // The page of this lane's copy of the tokens from `token` on: looked up (page_at),
        // and a turn later, when the value has come, checked (-1: none, reads zeros).
        auto page_at = [&](const LatentWalk &w, int token, bool &there) -> int {
            const int pg = (token + from) >> p.log2BS;
            there = lane < copies && pg < (w.q.L + p.BS - 1) >> p.log2BS;
            return ld_if(there, p.block_tables + (size_t)w.s * p.MB + (there ? pg : 0));
        };
        auto checked = [&](int id, bool there) -> int {
            const bool good = (unsigned)id < (unsigned)p.NB;
            if (there && !good)
                atomicOr(p.err, kErrPageRange);
            return there && good ? id : -1;
        };
        if (is_v) {
            const uint64_t last_use = l2_evict_first_policy();
            for (; walk.more() && ok; walk.next(p)) {
                const int end = walk.t_end * NT;
                bool there;
                int id = page_at(walk, walk.t * NT, there);
                for (int token = walk.t * NT; token < end; token += VKEYS, ++nst) {
                    const int page = checked(id, there);
                    id = page_at(walk, token + VKEYS, there);
                    const int grp = (token & (p.BS - 1)) >> 3;     // (0 where there are more copies)
                    const int st = nst % NV;
                    if (!wait(&v_empty[st], ((nst / NV) & 1) ^ 1))
                        break;
                    const uint32_t bar = lead(&v_full[st]);
                    int pages[VKEYS / 8];
#pragma unroll
                    for (int c = 0; c < VKEYS / 8; ++c)
                        pages[c] = __shfl_sync(~0u, page, c);
                    if (elect_one()) {
                        if (rank == 0)  // for both CTAs' copies
                            mbar_arrive_expect_tx(smem_addr(&v_full[st]), 2 * PIECE);
#pragma unroll
                        for (int c = 0; c < VKEYS / 8; ++c)
                            if (c < copies)
                                tma_load_5d_pair(v_s + st * PIECE + c * copy_bytes, &tmap_v, 0, 0,
                                                 rank * VSLABS, grp, pages[c], bar, last_use);
                    }
                    __syncwarp();
                }
            }
        } else {
            const uint64_t pol = l2_evict_last_policy();
            const uint32_t lead_k = lead(k_full);
            const int grp = p.BS == 2 * ROWS ? rank * (ROWS / 8) : 0;
            auto load_q = [&] {
                if (!wait(&q_empty, (nq & 1) ^ 1))
                    return false;
                ++nq;
                const int bytes = p.TQ * p.hb * 128;
                const HalfTile half(p, walk.v * 2 + rank);
                const int row = walk.q.row0 + half.token;
                const uint32_t q_bar = lead(&q_full);
                if (elect_one()) {
                    if (rank == 0)
                        mbar_arrive_expect_tx(smem_addr(&q_full), 2 * (SLABS + 1) * bytes);
                    for (int sl = 0; sl < SLABS; ++sl)
                        tma_load_4d_pair(q_s + sl * Q_SLAB, &tmap_q, 0, half.head, row, sl, q_bar);
                    tma_load_4d_pair(q_s + SLABS * Q_SLAB, &tmap_qr, 0, half.head, row, 0, q_bar);
                }
                __syncwarp();
                return true;
            };
            int nq_from = 0;  // K pieces in front of the unit
            for (; walk.more() && ok; walk.next(p)) {
                bool there;
                int id = page_at(walk, walk.t * NT, there);
                nq_from = nst;
                if (nst == 0 && !load_q())  // the run's first, while the page comes
                    break;
                for (int t = walk.t; t < walk.t_end; ++t) {
                    const int page = checked(id, there);
                    id = page_at(walk, (t + 1) * NT, there);
                    int made = 0;
                    // (copies of a piece as a constant, so that their code has no tests: pages of
                    // 16 rows 54.7 -> 48.1 us for 24 requests of up to 5 rows)
                    auto stage = [&](auto n) {
                        constexpr int C = decltype(n)::value;
                        int pages[C];
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            pages[c] = __shfl_sync(~0u, page, c);
#pragma unroll
                        for (int kp = 0; kp < KP; ++kp) {
                            // (a stage's pieces lie in the ring's first or second half, or all of it)
                            const int st = KP == NK ? kp : (nst + kp) % NK;
                            const uint32_t parity = ((KP == NK ? nst / NK : (nst + kp) / NK) & 1) ^ 1;
                            if (!ok || !wait(&k_empty[st], parity))
                                continue;
                            ++made;
                            const uint32_t bar = lead_k + 8 * st;
                            if (rank == 0 && elect_one())
                                mbar_arrive_expect_tx(smem_addr(k_full) + 8 * st,
                                                      2 * (PIECE + (kp == 0 ? ROWS * 128 : 0)));
                            if (elect_one()) {
                                // (the rotary keys with the stage's first piece)
#pragma unroll
                                for (int c = 0; c < C; ++c) {
                                    if (kp == 0)
                                        tma_load_4d_pair(r_s + (st / KP * ROWS + c * (ROWS / C)) * 128,
                                                         &tmap_kr, 0, 0, grp, pages[c], bar);
                                    tma_load_5d_pair(k_s + st * PIECE + c * (PIECE / C), &tmap_k, 0, 0,
                                                     kp * KSLABS, grp, pages[c], bar, pol);
                                }
                            }
                            __syncwarp();
                            // Q after the unit's first K: its place is free only after the last
                            // unit's last scores, and no place for K comes free before it
                            if (kp == (KP < NK ? KP : NK) - 1 && nq_from > 0 && t == walk.t)
                                load_q();
                        }
                    };
                    if (copies == 1)
                        stage(std::integral_constant<int, 1>{});
                    else if (copies == 2)
                        stage(std::integral_constant<int, 2>{});
                    else if (copies == 4)
                        stage(std::integral_constant<int, 4>{});
                    else
                        stage(std::integral_constant<int, 8>{});
                    nst += made;
                    if (!ok)
                        break;
                }
            }
        }
        if (!ok && lane == 0) {
            give_up();
            // let the copies in flight land before the CTA exits (the even CTA's
            // barriers count both CTAs' copies, and neither leaves alone)
            if (rank == 0) {
                if (nq)
                    mbar_wait_bounded(smem_addr(&q_full), (nq - 1) & 1, nullptr, p.wait_budget_ns);
                uint64_t *full = is_v ? v_full : k_full;
                const int slots = is_v ? NV : NK;
                for (int i = max(0, nst - slots); i < nst; ++i)
                    mbar_wait_bounded(smem_addr(&full[i % slots]), (i / slots) & 1, nullptr,
                                      p.wait_budget_ns);
            }
        }
    } else if (warp < 4) {
        if (rank == 0 && elect_one()) {
            // ======================================================== products
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                if (ok && !mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns))
                    ok = false;
                return ok;
            };
            if (warp == 2) {
                // (a negative scale: -q for q)
                const uint32_t idesc_s = IDESC_S | (p.scale_log2 < 0.f ? kLatentNegateA : 0u);
                const uint64_t q_desc = tc_sdesc(q_s, 16, 1024);
                const uint64_t k_desc = tc_sdesc(k_s, 16, KGROUP);
                const uint64_t r_desc = tc_sdesc(r_s, 16, 1024);
                const uint64_t qr_desc = q_desc + ((SLABS * Q_SLAB) >> 4);
                int nk = 0, ns = 0, nq = 0;  // K pieces, score products, Q tiles
                for (; walk.more() && ok; walk.next(p)) {
                    wait(&q_full, nq & 1);
                    ++nq;
                    for (int t = walk.t; t < walk.t_end && ok; ++t, ++ns) {
                        // the buffer's last scores have been read
                        const int b = ns % NS;
                        if (ns >= NS)
                            wait(&s_free[b], ((ns / NS) & 1) ^ 1);
                        const uint32_t d = tmem + S_COL + b * (NT / 2);
                        for (int kp = 0; kp < KP; ++kp, ++nk) {
                            const int st = nk % NK;
                            if (!wait(&k_full[st], (nk / NK) & 1))
                                break;
                            tc_fence_after();
                            if (kp == 0) {
                                // (of rope_dim 32 the other half of both rows is zeros)
                                const uint64_t rs = r_desc + ((st / KP * ROWS * 128) >> 4);
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    tc_mma_pair(d, qr_desc + ((kk * 32) >> 4), rs + ((kk * 32) >> 4),
                                                idesc_s, kk > 0);
                            }
                            const uint64_t ks = k_desc + ((st * PIECE) >> 4);
                            const uint64_t qs = q_desc + ((kp * KSLABS * Q_SLAB) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4 * KSLABS; ++kk)
                                tc_mma_pair(d, qs + (((kk / 4) * Q_SLAB + (kk % 4) * 32) >> 4),
                                            ks + (((kk / 4) * 1024 + (kk % 4) * 32) >> 4), idesc_s,
                                            true);
                            tc_commit_pair(smem_addr(&k_empty[st]));
                        }
                        tc_commit_pair(smem_addr(&s_full[b]));
                    }
                    tc_commit_pair(smem_addr(&q_empty));
                }
            } else {
                const uint64_t v_desc = tc_sdesc(v_s, 1024, VGROUP);
                int nv = 0, np = 0, no = 0, nz = 0;  // V pieces, output products, units, zeroed tails
                for (; walk.more() && ok; walk.next(p)) {
                    // the last unit's output has been read
                    if (no++ && !wait(&o_free, no & 1))
                        break;
                    for (int t = walk.t; t < walk.t_end && ok; ++t, ++np) {
                        if (!wait(&p_full[np & 1], (np >> 1) & 1))
                            break;
                        const uint32_t ps = tmem + P_COL + (np & 1) * (NT / 2);
                        // steps of 16 tokens: up to the sequence's last (one at least)
                        const int rows = walk.q.L - t * NT;
                        const int steps = max(1, (rows + 15) / 16);
                        for (int vp = 0; vp < VP; ++vp, ++nv) {
                            const int st = nv % NV, k0 = vp * (VKEYS / 16);
                            if (!wait(&v_full[st], (nv / NV) & 1))
                                break;
                            tc_fence_after();
                            const uint64_t vs = v_desc + ((st * PIECE) >> 4);
                            auto step = [&](int kk, bool more) {
#pragma unroll
                                for (int n = 0; n < R / ON; ++n)
                                    tc_mma_ta_pair(tmem + O_COL + n * (ON / 2), ps + (k0 + kk) * 8,
                                                vs + ((kk * 2 * VGROUP + n * 2048) >> 4), IDESC_O,
                                                more);
                            };
                            if (rows >= NT) {
#pragma unroll
                                for (int kk = 0; kk < VKEYS / 16; ++kk)
                                    step(kk, t > walk.t || vp > 0 || kk > 0);
                            } else {
                                const int here = min(VKEYS / 16, steps - k0);
                                if (here > 0 && steps <= k0 + VKEYS / 16 && rows < 16 * steps) {
                                    // the last step's rows behind the sequence are zeroed first
                                    mbar_arrive_cluster<true>(cluster_addr(smem_addr(&z_go), 1));
                                    mbar_arrive(smem_addr(&z_go));
                                    if (!wait(&z_full, nz++ & 1))
                                        break;
                                    tc_fence_after();
                                }
#pragma unroll 1
                                for (int kk = 0; kk < here; ++kk)
                                    step(kk, t > walk.t || vp > 0 || kk > 0);
                            }
                            tc_commit_pair(smem_addr(&v_empty[st]));
                        }
                        tc_commit_pair(smem_addr(&o_done[np & 1]));
                    }
                }
            }
            if (!ok)
                give_up();
            // every product issued here has completed before the memory is freed
            tc_commit_pair(smem_addr(&mma_done));
            mbar_wait_bounded(smem_addr(&mma_done), 0, nullptr, p.wait_budget_ns);
        }
        __syncwarp();
    } else {
        // ============================================================ softmax
        // A pair's product leaves in each CTA 64 rows over 128 lanes: lanes 64 h + r
        // hold row r, of its columns the half h (of the scores: the CTA h's tokens,
        // of the outputs: the CTA h's half of the values).  Warps 4-7 take the first
        // half of a lane's columns, warps 8-11 the second: four threads a row.
        constexpr int SC = NT / 4, OC = R / 4;  // columns of a thread
        const int quarter = warp & 3, ch = (warp - 4) >> 2;
        const int h = quarter >> 1, r = 32 * (quarter & 1) + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t row_bar = 1 + (quarter & 1);  // the four warps of 32 rows
        const int part = 2 * h + ch;                 // which quarter of a stage's tokens
        const uint32_t swap_bar = 3 + 2 * (quarter & 1) + ch;  // this warp and the one of quarter ^ 2
        const int swap = (lane >> 1) & 3;
        uint8_t *const mine_x = x_ptr + ((warp - 4) * 32 + lane) * 64;
        const uint8_t *const other_x = x_ptr + (((warp - 4) ^ 2) * 32 + lane) * 64;
        const int ti = r / p.hb, hh = r - ti * p.hb;
        // a scale of 0 runs as 1e-30: exp2 of every score is then 1 in fp32 (the mean,
        // as for 0) while masked scores, -inf, still give 0
        const float sc = p.scale_log2 == 0.f ? 1e-30f : fabsf(p.scale_log2);
        const float2 sc2 = make_float2(sc, sc);
        const bool scribe = threadIdx.x == 128 && rank == 0;
        if (scribe)
            p.cut[run] = make_int4(-1, 0, 0, 0);
        if (!walk.more() && part == 0)  // a run without a stage, perhaps between a unit's pieces
            p.part_ml[((size_t)(2 * run) * 2 + rank) * ROWS + r] = make_float2(-INFINITY, 0.f);
        const size_t row_bytes = (size_t)R * (p.out_half ? 2 : 4);
        int ns = 0;
        bool ok = true;
        // after a failed wait the loops keep running without doing work, so that warps
        // meet at every named barrier; outcomes are made warp-uniform (tensor-memory
        // loads and stores are warp-collective)
        auto wait = [&](uint64_t *bar, int parity) {
            if (ok && !__all_sync(~0u, mbar_wait_bounded(smem_addr(bar), parity, &abort_flag,
                                                         p.wait_budget_ns))) {
                ok = false;
                give_up();
            }
        };
        int nz = 0;  // tails zeroed
        for (; walk.more(); walk.next(p)) {
            const LatentSeq &q = walk.q;
            const HalfTile half(p, walk.v * 2 + rank);
            const int token = half.token + ti;  // this row's, within the sequence's new ones
            const bool row_ok = ti < p.TQ && token < q.n && half.head + hh < p.H;
            const int lim = row_ok ? q.L - q.n + token : -1;  // the last token it sees
            float m_ref = -INFINITY, l = 0.f;
            for (int t = walk.t; t < walk.t_end; ++t, ++ns) {
                const int t0 = t * NT, c0 = t0 + part * SC, b = ns % NS;
                wait(&s_full[b], (ns / NS) & 1);
                float v[SC];
                float e = -INFINITY;
                if (ok) {
                    tc_fence_after();
                    tc_ld32(t_lane + S_COL + b * (NT / 2) + ch * SC, v);
                    tc_wait_ld();
                    tc_ld_ready(v);
                    // the buffer takes other scores
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster<false>(lead(&s_free[b]));
                    if (c0 + SC - 1 > lim) {
#pragma unroll
                        for (int i = 0; i < SC; ++i)
                            v[i] = c0 + i > lim ? -INFINITY : v[i];
                    }
                    float ec[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        ec[c] = fmaxf(v[8 * c], v[8 * c + 1]);
#pragma unroll
                        for (int i = 2; i < 8; i += 2)
                            ec[c] = fmax3(ec[c], v[8 * c + i], v[8 * c + i + 1]);
                    }
                    e = fmax3(ec[0], ec[1], fmaxf(ec[2], ec[3]));
                }
                red[ns & 1][part][r] = e;
                named_barrier_sync(row_bar, 128);
                if (!ok) {
                    named_barrier_sync(swap_bar, 64);
                    continue;
                }
                const float mt = fmax3(fmaxf(red[ns & 1][0][r], red[ns & 1][1][r]),
                                       red[ns & 1][2][r], red[ns & 1][3][r]) * sc;
                // the reference moves only when the maximum has grown by more than 8
                // (log2 units): O is rescaled rarely
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
                uint32_t pk[SC / 2];
#pragma unroll
                for (int i = 0; i < SC; i += 2) {
                    float2 a = ffma2(make_float2(v[i], v[i + 1]), sc2, off2);
                    a.x = ex2(a.x);
                    a.y = ex2(a.y);
                    pk[i / 2] = pack_half2(a.x, a.y);
                    sum2 = fadd2(sum2, a);
                }
                l = l * alpha + (sum2.x + sum2.y);
                if (ns > 1) {  // the product before the last has read its weights
                    wait(&o_done[ns & 1], ((ns >> 1) & 1) ^ 1);
                    tc_fence_after();
                }
                // A (weights) of a pair's product of 128 rows lies twice in tensor memory:
                // lanes r and 64 + r both hold row r, for their halves of the outputs.  So
                // the two warps of a row exchange what they have.
#pragma unroll
                for (int c = 0; c < SC / 8; ++c)
                    *reinterpret_cast<uint4 *>(mine_x + ((c ^ swap) << 4)) =
                        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                named_barrier_sync(swap_bar, 64);
                const uint32_t p_col = t_lane + P_COL + (ns & 1) * (NT / 2) + ch * (SC / 2);
                tc_st16u(p_col + h * (NT / 4), pk);
#pragma unroll
                for (int c = 0; c < SC / 8; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(other_x + ((c ^ swap) << 4));
                    pk[4 * c] = w.x;
                    pk[4 * c + 1] = w.y;
                    pk[4 * c + 2] = w.z;
                    pk[4 * c + 3] = w.w;
                }
                tc_st16u(p_col + (h ^ 1) * (NT / 4), pk);
                if (t > walk.t && __any_sync(~0u, rescale)) {
                    wait(&o_done[(ns - 1) & 1], ((ns - 1) >> 1) & 1);  // O is whole
                    if (!ok)
                        continue;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < OC; c += 32) {
                        float o[32];
                        tc_ld32(t_lane + O_COL + ch * OC + c, o);
                        tc_wait_ld();
                        tc_ld_ready(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] *= alpha;
                        tc_st32(t_lane + O_COL + ch * OC + c, o);
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster<false>(lead(&p_full[ns & 1]));
                // Rows of the last step behind the sequence may hold anything: they are zeroed
                // in V (their weights are 0, which does not hide a NaN), when the products
                // have come to their piece.
                const int za = q.L - t0, ze = max(16, (za + 15) & ~15);
                if (t0 + NT > q.L && za < ze) {
                    wait(&z_go, nz++ & 1);
                    if (!ok)
                        continue;
                    for (int i = threadIdx.x - 128; i < (ze - za) * VSLABS * 8; i += 256) {
                        const int row = za + i / (VSLABS * 8), c = i % (VSLABS * 8);
                        const int st = (ns * VP + row / VKEYS) % NV, in = row % VKEYS;
                        *reinterpret_cast<uint4 *>(v_ptr + st * PIECE + (in / 8) * VGROUP +
                                                   (c >> 3) * 1024 + (in % 8) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank)
                            mbar_arrive_cluster<true>(lead(&z_full));
                        else
                            mbar_arrive(smem_addr(&z_full));
                    }
                }
            }
            // The row's exp-sum from its four threads (through the last stage's slot: its
            // readers are past it, since o_done came after every warp's weights, and the
            // next stage takes the other), then each writes its columns.
            wait(&o_done[(ns - 1) & 1], ((ns - 1) >> 1) & 1);
            red[(ns & 1) ^ 1][part][r] = l;
            named_barrier_sync(row_bar, 128);
            const float *lr = &red[(ns & 1) ^ 1][0][r];
            const float lt = (lr[0] + lr[ROWS]) + (lr[2 * ROWS] + lr[3 * ROWS]);
            // (and all of its readers are past it before the stage after the next)
            if (!ok)
                continue;
            tc_fence_after();
            const bool whole = walk.t == 0 && walk.t_end == q.T;
            const size_t piece = (size_t)(2 * run + (walk.t == 0)) * 2 + rank;
            auto read = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster<false>(lead(&o_free));
            };
            const size_t row =
                whole ? (size_t)(q.row0 + token) * p.H + half.head + hh : piece * ROWS + r;
            char *const dst = whole ? static_cast<char *>(p.out) + row * row_bytes
                                    : reinterpret_cast<char *>(p.part_o) + row * R * 4;
            const bool half_out = whole && p.out_half;
            write_own_row<OC>(row_ok ? dst + (h * (R / 2) + ch * OC) * (half_out ? 2 : 4) : nullptr,
                              half_out, !whole || p.wide_rows, t_lane + O_COL + ch * OC,
                              !whole ? 1.f : lt > 0.f ? 1.f / lt : 0.f, read);
            if (!whole) {
                // (-inf says that there is nothing to join; scores that are all NaN leave
                // it too, with a sum of NaN, which is to reach the output)
                if (row_ok && part == 0)
                    p.part_ml[piece * ROWS + r] =
                        make_float2(m_ref == -INFINITY && lt != 0.f ? 0.f : m_ref, lt);
                if (scribe && walk.t == 0)
                    p.cut[run] = make_int4(walk.s, walk.v, walk.last_run(total, p.runs), 0);
            }
        }
    }
    tc_fence_before();
    cluster_sync();  // neither CTA leaves while the other may still use its memory
    if (warp == 0) {
        tc_fence_after();
        tc_dealloc_pair(tmem, 512);
    }
    cluster_sync();  // the memory is given back by both while both are there
}

// Joins the pieces of the unit that is cut at the end of run blockIdx.x (if one is):
// its piece 1 there, then piece 0 of every later run up to the last.  A row's output
// is sum_i w_i o_i / sum_i w_i l_i with w_i = exp2(m_i - max m).  A warp per row, a
// row's pieces loaded several at a time.
constexpr int kLatentJoinThreads = 256;
constexpr int kLatentJoinRows = kLatentJoinThreads / 32;

template <int R>
__global__ void __launch_bounds__(kLatentJoinThreads) paged_latent_join_kernel(const LatentParams p)
{
    constexpr int VPL = R / 32, V4 = VPL / 4;  // values per lane
    constexpr int AHEAD = 4;
    const int run = blockIdx.x, rank = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = kLatentJoinRows * blockIdx.z + warp;
    const int ti = r / p.hb, hh = r - ti * p.hb;
    griddep_launch_dependents();  // a next call's kernel may set itself up
    griddep_wait();
    const int4 cut = p.cut[run];
    if (cut.x < 0 || ti >= p.TQ)
        return;
    const int row0 = p.cu_q ? p.cu_q[cut.x] : cut.x;
    const int n = p.cu_q ? p.cu_q[cut.x + 1] - row0 : 1;
    const HalfTile half(p, cut.y * 2 + rank);
    if (half.token + ti >= n || half.head + hh >= p.H)
        return;
    auto piece = [&](int i) -> size_t {
        return ((size_t)(i == run ? 2 * run + 1 : 2 * i) * 2 + rank) * kLatentRows + r;
    };
    float4 acc[V4];
    float den = 0.f, top = -INFINITY;
#pragma unroll
    for (int k = 0; k < V4; ++k)
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = run; i0 <= cut.z; i0 += AHEAD) {
        float2 ml[AHEAD];
        float4 x[AHEAD][V4];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            ml[a] = make_float2(-INFINITY, 0.f);
            if (i0 + a > cut.z)
                continue;
            const size_t at = piece(i0 + a);
            ml[a] = p.part_ml[at];
#pragma unroll
            for (int k = 0; k < V4; ++k)
                x[a][k] = *reinterpret_cast<const float4 *>(p.part_o + at * R + 128 * k + 4 * lane);
        }
        float m = top;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            m = fmaxf(m, ml[a].x);
        if (m == -INFINITY)
            continue;
        const float keep = ex2(top - m);
        den *= keep;
#pragma unroll
        for (int k = 0; k < V4; ++k) {
            acc[k].x *= keep;
            acc[k].y *= keep;
            acc[k].z *= keep;
            acc[k].w *= keep;
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            if (ml[a].x == -INFINITY)  // nothing there, or nothing that the row sees
                continue;
            const float w = ex2(ml[a].x - m);
            den += w * ml[a].y;
#pragma unroll
            for (int k = 0; k < V4; ++k) {
                acc[k].x += w * x[a][k].x;
                acc[k].y += w * x[a][k].y;
                acc[k].z += w * x[a][k].z;
                acc[k].w += w * x[a][k].w;
            }
        }
        top = m;
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
    const size_t at = ((size_t)(row0 + half.token + ti) * p.H + half.head + hh) * R + 4 * lane;
#pragma unroll
    for (int k = 0; k < V4; ++k) {
        const float4 o = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
        if (p.out_half)
            *reinterpret_cast<uint2 *>(static_cast<__half *>(p.out) + at + 128 * k) =
                make_uint2(pack_half2(o.x, o.y), pack_half2(o.z, o.w));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + 128 * k) = o;
    }
}

namespace {

template <int R> cudaError_t latent_resident_of(int *runs)
{
    const int smem = (int)latent_smem_bytes<R>();
    cudaError_t e = cudaFuncSetAttribute(paged_latent_kernel<R>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kLatentThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(runs, paged_latent_kernel<R>, &cfg);
}

template <int R>
cudaError_t launch_latent_of(const LatentMaps &m, const LatentParams &p, cudaStream_t stream)
{
    // (the main kernel too sets itself up under the launch before it: 4 us less a call)
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * p.runs));  // (pairs by the kernel's cluster size)
    cfg.blockDim = dim3(kLatentThreads);
    cfg.dynamicSmemBytes = latent_smem_bytes<R>();
    cfg.stream = stream;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, paged_latent_kernel<R>, m.q, m.qr, m.k, m.kr, m.v, p);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t join = {};
    join.gridDim = dim3((unsigned)p.runs, 2, kLatentRows / kLatentJoinRows);
    join.blockDim = dim3(kLatentJoinThreads);
    join.stream = stream;
    join.attrs = &overlap;
    join.numAttrs = 1;
    return cudaLaunchKernelEx(&join, paged_latent_join_kernel<R>, p);
}

}  // namespace

cudaError_t latent_resident(int latent_dim, int *runs)
{
    *runs = 0;
    return latent_dim == 128   ? latent_resident_of<128>(runs)
           : latent_dim == 256 ? latent_resident_of<256>(runs)
                               : latent_resident_of<512>(runs);
}

cudaError_t launch_latent(const LatentMaps &m, const LatentParams &p, cudaStream_t stream)
{
    if (p.allowed) {
        paged_latent_check_kernel<<<1, kLatentCheckThreads, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return p.R == 128   ? launch_latent_of<128>(m, p, stream)
           : p.R == 256 ? launch_latent_of<256>(m, p, stream)
                        : launch_latent_of<512>(m, p, stream);
}

}  // namespace pgd
