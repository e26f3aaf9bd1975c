// Attention of trees of drafted tokens over the paged cache (paged_gqa_tree) on
// the 5th-generation tensor cores: the verification step of speculative decoding
// with several continuations per sequence.
//
// A sequence's newest n_s tokens are the nodes of a tree; row i attends the tokens
// before the tree, its ancestors and itself: out = sum p_u v_u / sum p_u over those
// tokens, p_u = exp2(s_u - m), in one pass with a running maximum and sum.  A
// node's ancestors have smaller indices, so the mask only matters in the
// stages that reach into the tree, where each row looks tokens up in its
// ancestor bits.
//
// Every K and V byte serves at most a few hundred rows, so the call is bound by
// the K and V bytes from HBM; everything below is about keeping all SMs reading
// until the end.  (Times are of calls in a captured graph, unless "a call" is
// said: called from Python in turn with other work.)
//   * A unit is one (sequence, KV head, one or two tiles); a tile is 128 rows (TQ =
//     128 / G nodes x the G heads of the KV head).  An SM takes in some 55 GB/s
//     whatever the copies, 152 of them 8.3 TB/s: little more than HBM gives, so a
//     byte must not go to two SMs.  Where trees have more rows than one tile,
//     two CTAs work on two tiles as a pair (tcgen05 cta_group::2): one product of
//     256 rows, whose B operand is split over the two, so that each copies half of
//     every stage (half of K's tokens, half of V's head_dim) and both use all of it.
//     32 sequences of 8 k to 32 k tokens, 16 / 2 heads x 256: 268 to 290 us by the
//     machine, a call 297 us, 4.6 TB/s (two CTAs of a cluster that each hold all
//     of a stage, copied by multicast: 338 us); 64 of 512 to 4096 tokens, 32 / 8
//     heads x 128, single CTAs: 107 us, a call 115 us, 5.6 TB/s; one of 1000:
//     12.5 us, a call 15.7, latency.
//   * The stages of all units, one after the other, are cut into equal runs, one
//     per resident CTA or pair: no run has more than another, whatever the
//     lengths.  A unit that is cut leaves pieces (reference maximum, exp-sum,
//     unscaled output; at most two per run, so the scratch does not grow with the
//     batch), which a second kernel joins.
//   * The K and V rings run on from unit to unit, so a unit's start and end
//     pass while the next unit's stages are already coming in.
//   * Scores and outputs are issued by a thread each: a thread spends some 1400
//     cycles a stage on its barriers and commits, the products of a stage take
//     about as long, and one thread for both was slower than the copies
//     (2900 cycles a stage at head_dim 128, of which HBM leaves 3040).
#include "pgd_device.cuh"
#include "pgd_internal.h"
#include "pgd_rows.cuh"

namespace pgd {

namespace {

// warp 0 Q and K copies, 1 V copies, 2 scores, 3 outputs, 4-11 softmax
constexpr int kTreeThreads = 384;
constexpr uint32_t kTreeNegateA = 1u << 13;  // of the products' descriptor: -A for A
constexpr int kTreeVWarp = 1, kTreeSWarp = 2;
constexpr int kTreeWords = kTreeMaxNodes / 32;

template <int D, bool PAIR> constexpr size_t tree_smem_bytes()
{
    return size_t(128) * D * 2 + size_t(TreeShape<D, PAIR>::NK) * TreePieces<D, PAIR>::K_BYTES +
           size_t(TreeShape<D, PAIR>::NV) * TreePieces<D, PAIR>::V_BYTES + 1024;
}

// Ancestor bits: bit j of row i is set where node i sees node j.  Nine words a
// row: the ninth stays zero for the funnel shift, and the odd stride spreads the
// rows over the banks.
struct TreeBits {
    uint32_t bits[kTreeMaxNodes][kTreeWords + 1];
    int16_t up[kTreeMaxNodes];  // the doubled parent link, -1 past the root
};

// Built by the 256 softmax threads (thread = node) together by pointer
// doubling: ceil(log2 n) rounds, whatever the tree's depth.  A parent that is not
// an earlier node counts as none and is flagged (negative: none).
__device__ __forceinline__ void build_tree_bits(TreeBits &tree, const int32_t *parents, int n,
                                                int tid, uint32_t bar, unsigned *err)
{
    named_barrier_sync(bar, 256);  // the last tree's readers are done
    if (tid < n) {
        int up = __ldg(parents + tid);
        if (up >= tid) {
            atomicOr(err, kErrTree);
            up = -1;
        }
        tree.up[tid] = (int16_t)max(up, -1);
#pragma unroll
        for (int w = 0; w <= kTreeWords; ++w)
            tree.bits[tid][w] = w == (tid >> 5) ? 1u << (tid & 31) : 0u;
    }
    named_barrier_sync(bar, 256);
    const int words = (n + 31) >> 5;
    for (int reach = 1; reach < n; reach <<= 1) {
        const int up = tid < n ? tree.up[tid] : -1;
        uint32_t other[kTreeWords];
        int next = -1;
        if (up >= 0) {
            next = tree.up[up];
#pragma unroll
            for (int w = 0; w < kTreeWords; ++w)
                other[w] = w < words ? tree.bits[up][w] : 0u;
        }
        named_barrier_sync(bar, 256);
        if (up >= 0) {
            tree.up[tid] = (int16_t)next;
#pragma unroll
            for (int w = 0; w < kTreeWords; ++w)
                if (w < words)
                    tree.bits[tid][w] |= other[w];
        }
        named_barrier_sync(bar, 256);
    }
}

// Which of the 32 tokens from node index j0 on (negative: before the tree,
// where every token is seen) node i sees.
__device__ __forceinline__ uint32_t tree_word(const TreeBits &tree, int i, int j0)
{
    if (j0 <= -32)
        return ~0u;
    if (j0 < 0)
        return (tree.bits[i][0] << -j0) | ((1u << -j0) - 1u);
    if (j0 >= kTreeMaxNodes)
        return 0u;
    return __funnelshift_r(tree.bits[i][j0 >> 5], tree.bits[i][(j0 >> 5) + 1], j0 & 31);
}

// What a sequence asks for: its length, first row, nodes (0 where its numbers do
// not fit together or the table cannot hold its length: its tree is at the
// length's end, so no other length will do), stages per unit and units.
struct TreeSeq {
    int L, row0, n, T, groups;
    unsigned bad;  // the device error bit of a sequence that is left out
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int s)
{
    TreeSeq q;
    const int maxlen = p.MB << p.log2BS;
    q.L = __ldg(p.seq_lens + s);
    q.row0 = __ldg(p.cu_q + s);
    q.n = __ldg(p.cu_q + s + 1) - q.row0;
    q.bad = 0;
    if (q.L < 0 || q.L > maxlen)
        q.bad = kErrSeqLen;
    else if (q.n < 0 || q.n > q.L || q.n > p.max_q || q.row0 < 0 || q.row0 > p.total_q - q.n)
        q.bad = kErrQueryLen;
    if (q.bad)
        q.L = q.n = 0;
    q.T = (q.L + kTreeNT - 1) / kTreeNT;
    q.groups = ((q.n + p.TQ - 1) / p.TQ + p.cs - 1) / p.cs;
    return q;
}
// What a unit counts in the division of the work: its stages, and what it costs
// beside them (its start and end), in stages: with 1, 2, 3, 4 a batch of 64
// requests of 512 to 4096 tokens takes 106.6, 106.4, 106.5, 107 us (with 0 it
// took 8 us more), 32 of 8 k to 32 k tokens 275 with any.
constexpr int kTreeUnitCost = 2;
__device__ __forceinline__ int tree_cost(const TreeParams &p, const TreeSeq &q)
{
    return q.T ? q.groups * p.Hkv * (q.T + kTreeUnitCost) : 0;
}

// A run [x0, x1) of the cost of all units, a unit (or the part of it that the
// run holds) at a time: stage t of a unit that begins at cost c lies at c +
// kTreeUnitCost + t, so a cut before it begins the unit in the next run.  Every
// role walks its own copy.
struct TreeWalk {
    TreeSeq q;
    int s, v, t, t_end;  // sequence, unit within it, stages [t, t_end)
    int at, x1;          // where unit v begins, and the run's end

    __device__ __forceinline__ TreeWalk(const TreeParams &p, int s0, int begin, int x0, int x1_)
    {
        s = s0;
        x1 = at = x1_;
        v = t = t_end = 0;
        if (x0 >= x1)
            return;
        q = tree_seq(p, s);  // begin: where the sequence's first unit begins
        v = (x0 - begin) / (q.T + kTreeUnitCost);
        at = begin + v * (q.T + kTreeUnitCost);
        t = max(0, x0 - at - kTreeUnitCost);
        set_end();
    }
    __device__ __forceinline__ void set_end()
    {
        t_end = min(q.T, x1 - at - kTreeUnitCost);
        if (t_end <= t)  // the run ends before the unit's first stage
            at = x1;
    }
    __device__ __forceinline__ bool more() const { return at < x1; }
    __device__ __forceinline__ int head() const { return v / q.groups; }
    __device__ __forceinline__ int group() const { return v % q.groups; }
    __device__ __forceinline__ void next(const TreeParams &p)
    {
        at += q.T + kTreeUnitCost;
        if (at >= x1)
            return;
        t = 0;
        if (++v == q.groups * p.Hkv) {
            v = 0;
            do
                q = tree_seq(p, ++s);
            while (tree_cost(p, q) == 0);
        }
        set_end();
    }
    // the run that holds the unit's last stage, of `runs` equal ones of `total`
    __device__ __forceinline__ int last_run(int total, int runs) const
    {
        return (int)(((long long)(at + q.T + kTreeUnitCost) * runs - 1) / total);
    }
};

// Sum over the CTA's threads before this one of `x`, and over all in *total.
__device__ __forceinline__ int block_prefix(int x, int *warp_sum, int *total)
{
    constexpr int WARPS = kTreeThreads / 32;
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

template <int D, bool PAIR>
__global__ void __launch_bounds__(kTreeThreads, 1)
    paged_tree_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const TreeParams p)
{
    using P = TreePieces<D, PAIR>;
    constexpr int NT = kTreeNT, CS = PAIR ? 2 : 1;
    constexpr int NK = TreeShape<D, PAIR>::NK, NV = TreeShape<D, PAIR>::NV;
    constexpr int KP = TreeShape<D, PAIR>::KP, VP = TreeShape<D, PAIR>::VP;
    static_assert(NK >= KP && NV >= VP, "a stage's pieces fit the rings");
    constexpr int KKEYS = P::KKEYS, KSLABS = P::KSLABS, VKEYS = P::VKEYS, VSLABS = P::VSLABS;
    constexpr int K_BYTES = P::K_BYTES, V_BYTES = P::V_BYTES;
    constexpr int KGROUP = KSLABS * 1024, VGROUP = VSLABS * 1024;  // 8 rows of a piece
    constexpr int SLABS = D / 64, Q_SLAB = 128 * 128;
    constexpr uint32_t O_COL = 0, S_COL = D;  // tensor memory: O, two score buffers
    static_assert(S_COL + 2 * NT <= 512, "tensor memory");
    constexpr uint32_t IDESC_S = tc_idesc_f16(128 * CS, NT, 0, 0);
    constexpr uint32_t IDESC_O = tc_idesc_f16(128 * CS, D, 0, 1);

    extern __shared__ uint8_t dyn_smem[];
    // (of a pair, the even CTA's q_full, k_full, v_full, p_full and o_free count for both)
    __shared__ __align__(8) uint64_t q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV],
        v_empty[NV], v_here, s_full[2], p_full, o_done[2], o_free, mma_done;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_flag;
    __shared__ float pair_red[2][2][128];  // [parity][half][row]: the halves' exchange
    __shared__ TreeBits tree;
    __shared__ int warp_sum[kTreeThreads / 32], run_begin, run_seq;

    const uint32_t dyn_base = smem_addr(dyn_smem);
    const uint32_t base = (dyn_base + 1023u) & ~1023u;
    uint8_t *const base_ptr = dyn_smem + (base - dyn_base);
    const uint32_t q_s = base, k_s = q_s + 128 * D * 2, v_s = k_s + NK * K_BYTES;
    uint8_t *const v_ptr = base_ptr + 128 * D * 2 + NK * K_BYTES;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    const int run = (int)blockIdx.x / CS;
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
        mbar_init(smem_addr(&p_full), 8 * CS);
        mbar_init(smem_addr(&o_done[0]), 1);
        mbar_init(smem_addr(&o_done[1]), 1);
        mbar_init(smem_addr(&o_free), 8 * CS);
        mbar_init(smem_addr(&mma_done), 2);
        mbar_init(smem_addr(&v_here), 1);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    if (warp == 0) {
        if constexpr (PAIR)
            tc_alloc_pair(smem_addr(&tmem_base_s), 512);
        else
            tc_alloc(smem_addr(&tmem_base_s), 512);
    }

    // ---- the run: [x0, x1) of the cost of all units; the sequence that holds x0
    int total = 0, mine = 0, before = 0;  // before: this thread's (last) sequence
    for (int s0 = 0; s0 < p.S; s0 += kTreeThreads) {
        const int s = s0 + (int)threadIdx.x;
        int all;
        mine = 0;
        if (s < p.S) {
            const TreeSeq q = tree_seq(p, s);
            if (q.bad && blockIdx.x == 0)
                atomicOr(p.err, q.bad);
            mine = tree_cost(p, q);
        }
        before = total + block_prefix(mine, warp_sum, &all);
        total += all;
    }
    const int x0 = (int)((long long)total * run / p.runs);
    const int x1 = (int)((long long)total * (run + 1) / p.runs);
    if (x1 > x0 && p.S <= kTreeThreads) {
        if (mine > 0 && before <= x0 && x0 < before + mine) {
            run_seq = (int)threadIdx.x;
            run_begin = before;
        }
    } else if (x1 > x0) {
        int past = 0;
        for (int s0 = 0; s0 < p.S && past <= x0; s0 += kTreeThreads) {
            const int s = s0 + (int)threadIdx.x;
            const int here = s < p.S ? tree_cost(p, tree_seq(p, s)) : 0;
            int all;
            const int at = past + block_prefix(here, warp_sum, &all);
            if (here > 0 && at <= x0 && x0 < at + here) {
                run_seq = s;
                run_begin = at;
            }
            past += all;
        }
    }
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync();  // both CTAs' barriers exist
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    griddep_launch_dependents();
    TreeWalk walk(p, x1 > x0 ? run_seq : 0, x1 > x0 ? run_begin : 0, x0, x1);

    auto give_up = [&]() {
        if (!abort_flag)
            atomicOr(p.err, kErrTimeout);
        abort_flag = 1;
    };
    // a barrier of the CTA that issues the products
    auto lead = [&](uint64_t *bar) {
        return PAIR ? cluster_addr(smem_addr(bar), 0) : smem_addr(bar);
    };

    if (warp < 4) {
      // to the softmax warps (128 x 152 + 256 x 176 of the launch's 384 x 168): at
      // head_dim 64 and 128 nothing spills but 8 bytes in the pairs.  (With 104
      // and 200 the copying warps did: 64 requests 111.5 us instead of 107.9.)
      regs_give<152>();
      if (warp == 0 || warp == kTreeVWarp) {
        // ============================================================ copies
        // warp 0: Q tiles and K, warp 1: V.  A piece is a copy per page (or one
        // copy, where pages are longer): lane c issues copy c.
        const bool is_v = warp == kTreeVWarp;
        const uint64_t pol = l2_evict_first_policy();
        const CUtensorMap *map = is_v ? &tmap_v : &tmap_k;
        uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
        const int slots = is_v ? NV : NK, bytes = is_v ? V_BYTES : K_BYTES;
        const uint32_t ring = is_v ? v_s : k_s;
        const int rows = is_v ? p.v_rows : p.k_rows;
        const int copies = (is_v ? VKEYS : KKEYS) / rows;
        // this lane's first token of a piece, and its place there; of a pair, K's
        // second half of the tokens belongs to the odd CTA
        const int row = lane * rows, from = row + (is_v ? 0 : rank * KKEYS % NT);
        const uint32_t place = (row / 8) * (is_v ? VGROUP : KGROUP);
        int nst = 0, nq = 0;
        bool ok = true;
        for (; walk.more() && ok; walk.next(p)) {
            const TreeSeq &q = walk.q;
            const int g = walk.head();
            const int npages = (q.L + p.BS - 1) >> p.log2BS;
            const int32_t *bt = p.block_tables + (size_t)walk.s * p.MB;
            auto block_of = [&](int token) -> int {  // block coordinate, -1: none (reads zeros)
                const int pg = (token + from) >> p.log2BS;
                int b = -1;
                if (lane < copies && pg < npages) {
                    const int id = __ldg(bt + pg);
                    if ((unsigned)id < (unsigned)p.NB)
                        b = id * p.blk_page + g * p.blk_head;
                    else
                        atomicOr(p.err, kErrPageRange);
                }
                return b;
            };
            // K's pieces are slabs of a stage's tokens, V's are tokens
            const int step = is_v ? VKEYS : NT, end = walk.t_end * NT;
            int blk_next = block_of(walk.t * NT);
            for (int token = walk.t * NT; token < end && ok; token += step) {
                const int blk = blk_next;
                if (token + step < end)
                    blk_next = block_of(token + step);  // in flight while this one waits
                const int grp = ((token + from) & (p.BS - 1)) >> 3;
                for (int kp = 0; kp < (is_v ? 1 : KP); ++kp, ++nst) {
                    const int st = nst % slots;
                    bool w = true;
                    if (lane == 0)
                        w = mbar_wait_bounded(smem_addr(&empty[st]), ((nst / slots) & 1) ^ 1,
                                              &abort_flag, p.wait_budget_ns);
                    ok = __shfl_sync(~0u, w, 0);
                    if (!ok)
                        break;
                    if (lane == 0 && rank == 0)  // for both CTAs' copies
                        mbar_arrive_expect_tx(smem_addr(&full[st]), CS * bytes);
                    __syncwarp();
                    if (lane < copies) {
                        const uint32_t dst = ring + st * bytes + place;
                        const int slab = is_v ? rank * VSLABS : kp * KSLABS;
                        if constexpr (PAIR)
                            tma_load_5d_pair(dst, map, 0, 0, slab, grp, blk, lead(&full[st]), pol);
                        else
                            tma_load_5d(dst, map, 0, 0, slab, grp, blk, smem_addr(&full[st]), pol);
                    }
                }
                if (ok && !is_v && token == walk.t * NT) {
                    // Q after the unit's first K: its place is free only after
                    // the last unit's last scores
                    bool w = true;
                    if (lane == 0) {
                        w = mbar_wait_bounded(smem_addr(&q_empty), (nq & 1) ^ 1, &abort_flag,
                                              p.wait_budget_ns);
                        if (w) {
                            if (rank == 0)
                                mbar_arrive_expect_tx(smem_addr(&q_full),
                                                      CS * SLABS * p.TQ * p.G * 128);
                            const int first = q.row0 + (walk.group() * CS + rank) * p.TQ;
                            for (int sl = 0; sl < SLABS; ++sl) {
                                if constexpr (PAIR)
                                    tma_load_4d_pair(q_s + sl * Q_SLAB, &tmap_q, 0, g * p.G, first,
                                                     sl, lead(&q_full));
                                else
                                    tma_load_4d(q_s + sl * Q_SLAB, &tmap_q, 0, g * p.G, first, sl,
                                                smem_addr(&q_full));
                            }
                        }
                    }
                    ok = __shfl_sync(~0u, w, 0);
                    if (ok)
                        ++nq;
                }
            }
        }
        if (!ok && lane == 0) {
            give_up();
            // let the copies in flight land before the CTA exits (of a pair, the
            // even CTA's barriers count both CTAs' copies, and neither leaves alone)
            if (nq && rank == 0)
                mbar_wait_bounded(smem_addr(&q_full), (nq - 1) & 1, nullptr, p.wait_budget_ns);
            for (int i = max(0, nst - slots); i < nst && rank == 0; ++i)
                mbar_wait_bounded(smem_addr(&full[i % slots]), (i / slots) & 1, nullptr,
                                  p.wait_budget_ns);
        }
      } else if (lane == 0 && rank == 0) {
        // ============================================================ products
        bool ok = true;
        auto wait = [&](uint64_t *bar, int parity) {
            if (ok && !mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns))
                ok = false;
            return ok;
        };
        auto commit = [&](uint64_t *bar) {  // in both CTAs of a pair
            if constexpr (PAIR)
                tc_commit_pair(smem_addr(bar));
            else
                tc_commit(smem_addr(bar));
        };
        if (warp == kTreeSWarp) {
            // (a negative scale: -q for q)
            const uint32_t idesc_s = IDESC_S | (p.scale_log2 < 0.f ? kTreeNegateA : 0u);
            const uint64_t q_desc = tc_sdesc(q_s, 16, 1024);
            const uint64_t k_desc = tc_sdesc(k_s, 16, KGROUP);
            int nk = 0, ns = 0, nq = 0;  // K pieces, S products, Q tiles
            for (; walk.more() && ok; walk.next(p)) {
                wait(&q_full, nq & 1);
                ++nq;
                for (int t = walk.t; t < walk.t_end && ok; ++t, ++ns) {
                    // into the buffer of P(ns - 2), once its product is over
                    if (ns >= 2)
                        wait(&o_done[ns & 1], ((ns >> 1) & 1) ^ 1);
                    const uint32_t d = tmem + S_COL + (ns & 1) * NT;
                    for (int kp = 0; kp < KP; ++kp, ++nk) {
                        const int st = nk % NK;
                        if (!wait(&k_full[st], (nk / NK) & 1))
                            break;
                        tc_fence_after();
                        const uint64_t ks = k_desc + ((st * K_BYTES) >> 4);
                        const uint64_t qs = q_desc + ((kp * KSLABS * Q_SLAB) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4 * KSLABS; ++kk) {
                            const uint64_t a = qs + (((kk / 4) * Q_SLAB + (kk % 4) * 32) >> 4);
                            const uint64_t b = ks + (((kk / 4) * 1024 + (kk % 4) * 32) >> 4);
                            if constexpr (PAIR)
                                tc_mma_pair(d, a, b, idesc_s, kp > 0 || kk > 0);
                            else
                                tc_mma(d, a, b, idesc_s, kp > 0 || kk > 0);
                        }
                        commit(&k_empty[st]);
                    }
                    commit(&s_full[ns & 1]);
                }
                commit(&q_empty);
            }
        } else {
            const uint64_t v_desc = tc_sdesc(v_s, 1024, VGROUP);
            int nv = 0, np = 0, no = 0;  // V pieces, P V products, units
            for (; walk.more() && ok; walk.next(p)) {
                // the last unit's output has been read
                if (no++ && !wait(&o_free, no & 1))
                    break;
                for (int t = walk.t; t < walk.t_end && ok; ++t, ++np) {
                    if (!wait(&p_full, np & 1))
                        break;
                    const uint32_t a = tmem + S_COL + (np & 1) * NT;
                    for (int vp = 0; vp < VP; ++vp, ++nv) {
                        const int st = nv % NV;
                        if (!wait(&v_full[st], (nv / NV) & 1))
                            break;
                        tc_fence_after();
                        const uint64_t vs = v_desc + ((st * V_BYTES) >> 4);
#pragma unroll
                        for (int kk = 0; kk < VKEYS / 16; ++kk) {
                            const uint32_t pa = a + (vp * (VKEYS / 16) + kk) * 8;
                            const uint64_t b = vs + ((kk * 2 * VGROUP) >> 4);
                            const bool more = t > walk.t || vp > 0 || kk > 0;
                            if constexpr (PAIR)
                                tc_mma_ta_pair(tmem + O_COL, pa, b, IDESC_O, more);
                            else
                                tc_mma_ta(tmem + O_COL, pa, b, IDESC_O, more);
                        }
                        commit(&v_empty[st]);
                    }
                    commit(&o_done[np & 1]);
                }
            }
        }
        if (!ok)
            give_up();
        // every product issued here has completed before the memory is freed
        commit(&mma_done);
        mbar_wait_bounded(smem_addr(&mma_done), 0, nullptr, p.wait_budget_ns);
      }
      __syncwarp();
    } else {
        // ============================================================ softmax
        // warps 4-7 take the first half of a stage's tokens, warps 8-11 the
        // second, for the same rows: warp w reads tensor-memory quarter w & 3
        regs_take<176>();
        constexpr int HC = NT / 2, HD = D / 2;
        const int quarter = warp & 3;
        const int half = (warp - 4) >> 2;
        const int r = 32 * quarter + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t pair_bar = 1 + quarter;
        const int ti = r / p.G;
        // a scale of 0 runs as 1e-30: exp2 of every score is then 1 in fp32
        // (the mean, as for 0) while masked scores, -inf, still give 0; with a
        // negative one the scores are those of -q
        const float sc = p.scale_log2 == 0.f ? 1e-30f : fabsf(p.scale_log2);
        const float2 sc2 = make_float2(sc, sc);
        const bool scribe = threadIdx.x == 128 && rank == 0;
        if (scribe)
            p.cut[run] = make_int4(-1, 0, 0, 0);
        if (!walk.more() && half == 0)  // a run without a stage, perhaps between a unit's pieces
            p.part_ml[((size_t)(2 * run) * CS + rank) * 128 + r] = make_float2(-INFINITY, 0.f);
        const size_t row_bytes = (size_t)D * (p.out_half ? 2 : 4);
        const RowPlaces places(row_bytes, p.Hq, p.G, p.TQ, quarter, lane);
        int ns = 0, built = -1;
        bool ok = true;
        // after a failed wait the loops keep running without doing work, so
        // that warps meet at every named barrier; outcomes are made
        // warp-uniform (tensor-memory loads and stores are warp-collective)
        auto wait = [&](uint64_t *bar, int parity) {
            if (ok && !__all_sync(~0u, mbar_wait_bounded(smem_addr(bar), parity, &abort_flag,
                                                         p.wait_budget_ns))) {
                ok = false;
                give_up();
            }
        };
        // to the thread that issues the outputs (far: also what was written to V)
        auto signal = [&](uint64_t *bar, bool far) {
            if (PAIR && far)
                mbar_arrive_cluster<true>(lead(bar));
            else if (PAIR)
                mbar_arrive_cluster<false>(lead(bar));
            else
                mbar_arrive(smem_addr(bar));
        };
        // waits for V's pieces [a, b); of a pair, the even CTA's barriers count
        // both CTAs' copies, and it tells the odd one
        int told = 0;
        auto wait_v = [&](int a, int b) {
            if (PAIR && rank == 1) {
                mbar_wait_bounded(smem_addr(&v_here), told++ & 1, &abort_flag, p.wait_budget_ns);
                return;
            }
            for (int i = a; i < b; ++i)
                mbar_wait_bounded(smem_addr(&v_full[i % NV]), (i / NV) & 1, &abort_flag,
                                  p.wait_budget_ns);
            if (PAIR && threadIdx.x == 128)
                mbar_arrive_cluster<true>(cluster_addr(smem_addr(&v_here), 1));
        };
        for (; walk.more(); walk.next(p)) {
            const TreeSeq &q = walk.q;
            const int g = walk.head(), tile = walk.group() * CS + rank;
            const int left = min(p.TQ, q.n - tile * p.TQ);  // nodes of this tile (or none)
            const bool row_ok = r < p.TQ * p.G && ti < left;
            const int node = tile * p.TQ + ti;
            const int prefix = q.L - q.n;
            if (walk.t_end * NT > prefix && built != walk.s) {
                build_tree_bits(tree, p.parents + q.row0, q.n, threadIdx.x - 128, 5, p.err);
                built = walk.s;
            }
            float m_ref = -INFINITY, l = 0.f;
            for (int t = walk.t; t < walk.t_end; ++t, ++ns) {
                const int t0 = t * NT, c0 = t0 + half * HC;
                const uint32_t s_col = S_COL + (ns & 1) * NT;
                wait(&s_full[ns & 1], (ns >> 1) & 1);
                float v[HC / 32][32];
                float e = -INFINITY;
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < HC / 32; ++c)
                        tc_ld32(t_lane + s_col + half * HC + 32 * c, v[c]);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < HC / 32; ++c)
                        tc_ld_ready(v[c]);
                    if (c0 + HC > prefix) {
                        // (what lies behind the sequence has no bit either)
#pragma unroll
                        for (int c = 0; c < HC / 32; ++c) {
                            const uint32_t seen =
                                row_ok ? tree_word(tree, node, c0 + 32 * c - prefix) : 0u;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[c][i] = (seen >> i) & 1u ? v[c][i] : -INFINITY;
                        }
                    }
                    float ec[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        ec[c] = fmaxf(v[c >> 1][16 * (c & 1)], v[c >> 1][16 * (c & 1) + 1]);
#pragma unroll
                        for (int i = 2; i < 16; i += 2)
                            ec[c] = fmax3(ec[c], v[c >> 1][16 * (c & 1) + i],
                                          v[c >> 1][16 * (c & 1) + i + 1]);
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
                uint32_t pk[HC / 2];
#pragma unroll
                for (int c = 0; c < HC / 32; ++c)
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
                if (t > walk.t) {
                    wait(&o_done[(ns - 1) & 1], ((ns - 1) >> 1) & 1);  // O may be rescaled
                    if (!ok)
                        continue;
                    tc_fence_after();
                    if (__any_sync(~0u, rescale)) {
#pragma unroll 1
                        for (int c = 0; c < HD / 32; ++c) {
                            float o[32];
                            tc_ld32(t_lane + O_COL + half * HD + 32 * c, o);
                            tc_wait_ld();
                            tc_ld_ready(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] *= alpha;
                            tc_st32(t_lane + O_COL + half * HD + 32 * c, o);
                        }
                    }
                }
                // rows of the stage behind the sequence may hold anything: zero
                // them in V (their weights are 0, which does not hide a NaN)
                const bool zero_v = t0 + NT > q.L;
                if (zero_v) {
                    const int za = q.L - t0;  // first row behind it
                    wait_v(ns * VP + za / VKEYS, ns * VP + VP);
                    for (int idx = half * 128 + r; idx < (NT - za) * VSLABS * 8; idx += 256) {
                        const int row = za + idx / (VSLABS * 8), c = idx % (VSLABS * 8);
                        const int st = (ns * VP + row / VKEYS) % NV, in = row % VKEYS;
                        *reinterpret_cast<uint4 *>(v_ptr + st * V_BYTES + (in / 8) * VGROUP +
                                                   (c >> 3) * 1024 + (in % 8) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                tc_wait_st();
                if (zero_v)
                    fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    signal(&p_full, zero_v);
            }
            wait(&o_done[(ns - 1) & 1], ((ns - 1) >> 1) & 1);
            // the row's exp-sum from both halves, then each half writes its
            // columns (through the last stage's slot: its readers are done,
            // since o_done came after every warp's p_full, and the next stage
            // takes the other).  No warp goes on to the next unit before that
            // product is over: p_full, v_here and the V ring count on it (a
            // phase further on would pass for the one before).
            pair_red[(ns & 1) ^ 1][half][r] = l;
            named_barrier_sync(pair_bar, 64);
            const float lt = l + pair_red[(ns & 1) ^ 1][half ^ 1][r];
            if (!ok)
                continue;
            tc_fence_after();
            const bool whole = walk.t == 0 && walk.t_end == q.T;
            auto read = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    signal(&o_free, false);
            };
            // a store takes 64 columns at least: at head_dim 64 the first
            // half's warps write whole rows
            constexpr int WC = D == 64 ? 64 : HD;
            const int col = D == 64 ? 0 : half * HD;
            if (D == 64 && half == 1) {
                read();
            } else if (whole) {
                const RowOut rows = places.at(
                    static_cast<char *>(p.out) +
                        ((size_t)(q.row0 + tile * p.TQ) * p.Hq + (size_t)g * p.G) * row_bytes, left);
                write_rows<WC>(rows, p.out_half, p.wide_rows, t_lane + O_COL + col, col,
                               lt > 0.f ? 1.f / lt : 0.f, lane, read);
            } else {
                // a piece: 0 where the unit began in an earlier run, else 1
                const size_t piece = (size_t)(2 * run + (walk.t == 0)) * CS + rank;
                RowOut rows;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 32 * quarter + (lane & ~3) + i;
                    rows.at[i] = row < p.TQ * p.G && row / p.G < left
                                     ? reinterpret_cast<char *>(p.part_o + (piece * 128 + row) * D)
                                     : nullptr;
                }
                write_rows<WC>(rows, false, true, t_lane + O_COL + col, col, 1.f, lane, read);
                // (-inf says that there is nothing to join; scores that are all NaN
                // leave it too, with a sum of NaN, which is to reach the output)
                if (row_ok && half == 0)
                    p.part_ml[piece * 128 + r] =
                        make_float2(m_ref == -INFINITY && lt != 0.f ? 0.f : m_ref, lt);
                if (scribe && walk.t == 0)
                    p.cut[run] = make_int4(walk.s, g, walk.group(), walk.last_run(total, p.runs));
            }
        }
    }
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync();  // neither CTA leaves while the other may still use its memory
    else
        __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        if constexpr (PAIR)
            tc_dealloc_pair(tmem, 512);
        else
            tc_dealloc(tmem, 512);
    }
    if constexpr (PAIR)
        cluster_sync();  // the memory is given back by both while both are there
}

// Joins the pieces of the unit that is cut at the end of run blockIdx.x (if one
// is): its piece 1 there, then piece 0 of every later run up to the last.  A
// row's output is sum_i w_i o_i / sum_i w_i l_i with w_i = exp2(m_i - max m).
// A warp per row: what it waits for is latency, so the rows go to as many warps
// as there are and a row's pieces are loaded eight at a time (11 to 15 us with
// 32 rows and one piece at a time per CTA of eight warps, 4 to 6 now).
constexpr int kTreeJoinThreads = 256;
constexpr int kTreeJoinRows = kTreeJoinThreads / 32;

template <int D>
__global__ void __launch_bounds__(kTreeJoinThreads) paged_tree_join_kernel(const TreeParams p)
{
    constexpr int VPL = D / 32;  // values per lane
    constexpr int AHEAD = 8;
    const int run = blockIdx.x, rank = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = kTreeJoinRows * blockIdx.z + warp, ti = r / p.G;
    griddep_wait();
    const int4 cut = p.cut[run];
    if (cut.x < 0 || r >= p.TQ * p.G)
        return;
    const int row0 = __ldg(p.cu_q + cut.x), n = __ldg(p.cu_q + cut.x + 1) - row0;
    const int node = (cut.z * p.cs + rank) * p.TQ + ti;
    if (node >= n)
        return;
    auto piece = [&](int i) -> size_t {
        return ((size_t)(i == run ? 2 * run + 1 : 2 * i) * p.cs + rank) * 128 + r;
    };
    float acc[VPL], den = 0.f, top = -INFINITY;
#pragma unroll
    for (int k = 0; k < VPL; ++k)
        acc[k] = 0.f;
    for (int i0 = run; i0 <= cut.w; i0 += AHEAD) {
        float2 ml[AHEAD], x[AHEAD][VPL / 2];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            ml[a] = make_float2(-INFINITY, 0.f);
            if (i0 + a > cut.w)
                continue;
            const size_t at = piece(i0 + a);
            ml[a] = p.part_ml[at];
#pragma unroll
            for (int k = 0; k < VPL / 2; ++k)
                x[a][k] = *reinterpret_cast<const float2 *>(p.part_o + at * D + VPL * lane + 2 * k);
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
        for (int k = 0; k < VPL; ++k)
            acc[k] *= keep;
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            if (ml[a].x == -INFINITY)  // nothing there, or nothing that the row sees
                continue;
            const float w = ex2(ml[a].x - m);
            den += w * ml[a].y;
#pragma unroll
            for (int k = 0; k < VPL / 2; ++k) {
                acc[2 * k] += w * x[a][k].x;
                acc[2 * k + 1] += w * x[a][k].y;
            }
        }
        top = m;
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
    const size_t at =
        ((size_t)(row0 + node) * p.Hq + (size_t)cut.y * p.G + (r - ti * p.G)) * D + VPL * lane;
#pragma unroll
    for (int k = 0; k < VPL; k += 2) {
        if (p.out_half)
            *reinterpret_cast<uint32_t *>(static_cast<__half *>(p.out) + at + k) =
                pack_half2(acc[k] * inv, acc[k + 1] * inv);
        else
            *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at + k) =
                make_float2(acc[k] * inv, acc[k + 1] * inv);
    }
}

namespace {

template <int D, bool PAIR> void tree_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr)
{
    *cfg = {};
    cfg->blockDim = dim3(kTreeThreads);
    cfg->dynamicSmemBytes = tree_smem_bytes<D, PAIR>();
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = 2;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = PAIR ? 1 : 0;
}

template <int D, bool PAIR> cudaError_t tree_resident_of(int *runs)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    tree_config<D, PAIR>(&cfg, &attr);
    cudaError_t e = cudaFuncSetAttribute(paged_tree_kernel<D, PAIR>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess)
        return e;
    if (PAIR) {
        cfg.gridDim = dim3(2);
        return cudaOccupancyMaxActiveClusters(runs, paged_tree_kernel<D, PAIR>, &cfg);
    }
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess)
        return e;
    return cudaDeviceGetAttribute(runs, cudaDevAttrMultiProcessorCount, dev);
}

template <int D, bool PAIR>
cudaError_t launch_tree_of(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                           const TreeParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    tree_config<D, PAIR>(&cfg, &attr);
    cfg.gridDim = dim3((unsigned)(p.runs * p.cs));
    cfg.stream = stream;
    cudaError_t e;
    if ((e = cudaLaunchKernelEx(&cfg, paged_tree_kernel<D, PAIR>, tq, tk, tv, p)) != cudaSuccess)
        return e;
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t join = {};
    join.gridDim = dim3((unsigned)p.runs, (unsigned)p.cs, 128 / kTreeJoinRows);
    join.blockDim = dim3(kTreeJoinThreads);
    join.stream = stream;
    join.attrs = &overlap;
    join.numAttrs = 1;
    return cudaLaunchKernelEx(&join, paged_tree_join_kernel<D>, p);
}

}  // namespace

cudaError_t tree_resident(int head_dim, bool pair, int *runs)
{
    *runs = 0;
    switch (head_dim) {
    case 64:
        return pair ? cudaSuccess : tree_resident_of<64, false>(runs);
    case 128:
        return pair ? tree_resident_of<128, true>(runs) : tree_resident_of<128, false>(runs);
    default:
        return pair ? tree_resident_of<256, true>(runs) : tree_resident_of<256, false>(runs);
    }
}

cudaError_t launch_tree(int head_dim, const CUtensorMap &tq, const CUtensorMap &tk,
                        const CUtensorMap &tv, const TreeParams &p, cudaStream_t stream)
{
    const bool pair = p.cs == 2;
    switch (head_dim) {
    case 64:
        return launch_tree_of<64, false>(tq, tk, tv, p, stream);
    case 128:
        return pair ? launch_tree_of<128, true>(tq, tk, tv, p, stream)
                    : launch_tree_of<128, false>(tq, tk, tv, p, stream);
    default:
        return pair ? launch_tree_of<256, true>(tq, tk, tv, p, stream)
                    : launch_tree_of<256, false>(tq, tk, tv, p, stream);
    }
}

}  // namespace pgd
