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
// until the end:
//   * A unit is one (sequence, KV head, group of tiles); a tile is 128 rows (TQ =
//     128 / G nodes x the G heads of the KV head).  Where trees have more rows
//     than one tile, the tiles of a group are the CTAs of a cluster: each loads
//     its share of every stage and multicasts it to all, so that a byte leaves
//     L2 once for the group.
//   * The stages of all units, one after the other, are cut into equal runs, one
//     per resident cluster: no cluster has more than a stage more than another,
//     whatever the lengths.  A unit that is cut leaves pieces (reference maximum,
//     exp-sum, unscaled output; at most two per cluster, so the scratch does not
//     grow with the batch), which a second kernel joins.
//   * The K and V rings run on from unit to unit, so a unit's start and end
//     pass while the next unit's stages are already coming in.
#include "pgd_device.cuh"
#include "pgd_internal.h"
#include "pgd_rows.cuh"

namespace pgd {

namespace {

// warp 0 K copies, 1 scores, 2-9 softmax, 10 V copies, 11 outputs
constexpr int kTreeThreads = 384;
constexpr int kTreeVWarp = 10, kTreeOWarp = 11;
constexpr int kTreeWords = kTreeMaxNodes / 32;

template <int D> constexpr size_t tree_smem_bytes()
{
    return size_t(128) * D * 2 +
           size_t(TreeShape<D>::NK + TreeShape<D>::NV) * TreeShape<D>::NT * D * 2 + 1024;
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
// not fit together), stages per unit and units.
struct TreeSeq {
    int L, row0, n, T, groups;
    bool bad;
};

template <int NT> __device__ __forceinline__ TreeSeq tree_seq(const TreeParams &p, int s)
{
    TreeSeq q;
    const int maxlen = p.MB << p.log2BS;
    const int L = __ldg(p.seq_lens + s);
    q.L = min(max(L, 0), maxlen);
    q.row0 = __ldg(p.cu_q + s);
    q.n = __ldg(p.cu_q + s + 1) - q.row0;
    q.bad = q.n < 0 || q.n > q.L || q.n > p.max_q || q.row0 < 0 || q.row0 > p.total_q - q.n;
    if (q.bad)
        q.n = 0;
    q.T = (q.L + NT - 1) / NT;
    q.groups = ((q.n + p.TQ - 1) / p.TQ + p.cs - 1) / p.cs;
    return q;
}
__device__ __forceinline__ long long tree_stages(const TreeParams &p, const TreeSeq &q)
{
    return (long long)q.groups * p.Hkv * q.T;
}

// The cluster's run through the stages of all units, a unit (or the part of it
// that the run holds) at a time.  Every role walks its own copy.
template <int NT> struct TreeWalk {
    TreeSeq q;
    int s, v, t, t_end;      // sequence, unit within it, stages [t, t_end)
    long long left;          // stages of the run from t on

    __device__ __forceinline__ TreeWalk(const TreeParams &p, int s0, long long skip, long long run)
    {
        s = s0;
        left = run;
        t = t_end = v = 0;
        if (left <= 0)
            return;
        q = tree_seq<NT>(p, s);
        v = (int)(skip / q.T);
        t = (int)(skip - (long long)v * q.T);
        t_end = (int)min((long long)q.T, t + left);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ int head() const { return v / q.groups; }
    __device__ __forceinline__ int group() const { return v % q.groups; }
    __device__ __forceinline__ void next(const TreeParams &p)
    {
        left -= t_end - t;
        if (left <= 0)
            return;
        t = 0;  // stages are left, so the unit has ended
        if (++v == q.groups * p.Hkv) {
            v = 0;
            do
                q = tree_seq<NT>(p, ++s);
            while (tree_stages(p, q) == 0);
        }
        t_end = (int)min((long long)q.T, left);
    }
};

// Sum over the CTA's threads before this one of `x`, and over all in *total.
__device__ __forceinline__ long long block_prefix(long long x, long long *warp_sum, long long *total)
{
    constexpr int WARPS = kTreeThreads / 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(~0u, inc, off);
        if (lane >= off)
            inc += y;
    }
    if (lane == 31)
        warp_sum[w] = inc;
    __syncthreads();
    long long before = 0, all = 0;
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

template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
    paged_tree_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const TreeParams p)
{
    constexpr int NT = TreeShape<D>::NT, NK = TreeShape<D>::NK, NV = TreeShape<D>::NV;
    constexpr int SLABS = D / 64;
    constexpr int GROUP = SLABS * 1024;  // one 8-row group of K or V, all slabs
    constexpr int KV_TILE = NT * D * 2;
    constexpr int Q_SLAB = 128 * 128;
    constexpr uint32_t O_COL = 0, S_COL = D;  // tensor memory: O, two score buffers
    static_assert(S_COL + 2 * NT <= 512, "tensor memory");
    constexpr uint32_t IDESC_S = tc_idesc_f16(128, NT, 0, 0);
    constexpr uint32_t IDESC_O = tc_idesc_f16(128, D, 0, 1);

    extern __shared__ uint8_t dyn_smem[];
    __shared__ __align__(8) uint64_t q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV],
        v_empty[NV], s_full[2], p_full, o_done[2], o_free, mma_done;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_flag;
    __shared__ float pair_red[2][2][128];  // [parity][half][row]: the halves' exchange
    __shared__ TreeBits tree;
    __shared__ long long warp_sum[kTreeThreads / 32], run_skip;
    __shared__ int run_seq;

    const uint32_t dyn_base = smem_addr(dyn_smem);
    const uint32_t base = (dyn_base + 1023u) & ~1023u;
    uint8_t *const base_ptr = dyn_smem + (base - dyn_base);
    const uint32_t q_s = base, k_s = q_s + 128 * D * 2, v_s = k_s + NK * KV_TILE;
    uint8_t *const v_ptr = base_ptr + 128 * D * 2 + NK * KV_TILE;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.cs > 1 ? (int)cluster_rank() : 0;
    const int cluster = (int)blockIdx.x / p.cs;
    const uint16_t everyone = (uint16_t)((1u << p.cs) - 1u);
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&q_full), 1);
        mbar_init(smem_addr(&q_empty), 1);
        // a stage's place is free once every CTA that it is copied to has used it
        for (int i = 0; i < NK; ++i) {
            mbar_init(smem_addr(&k_full[i]), 1);
            mbar_init(smem_addr(&k_empty[i]), p.cs);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(smem_addr(&v_full[i]), 1);
            mbar_init(smem_addr(&v_empty[i]), p.cs);
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

    // ---- the run: stages [x0, x1) of all; the sequence that holds x0
    long long total = 0;
    for (int s0 = 0; s0 < p.S; s0 += kTreeThreads) {
        const int s = s0 + (int)threadIdx.x;
        long long mine = 0, all;
        if (s < p.S) {
            const TreeSeq q = tree_seq<NT>(p, s);
            if (q.bad && blockIdx.x == 0)
                atomicOr(p.err, kErrQueryLen);
            mine = tree_stages(p, q);
        }
        block_prefix(mine, warp_sum, &all);
        total += all;
    }
    const long long x0 = total * cluster / p.clusters, x1 = total * (cluster + 1) / p.clusters;
    if (x1 > x0) {
        long long before = 0;
        for (int s0 = 0; s0 < p.S && before <= x0; s0 += kTreeThreads) {
            const int s = s0 + (int)threadIdx.x;
            const long long mine = s < p.S ? tree_stages(p, tree_seq<NT>(p, s)) : 0;
            long long all;
            const long long at = before + block_prefix(mine, warp_sum, &all);
            if (mine > 0 && at <= x0 && x0 < at + mine) {
                run_seq = s;
                run_skip = x0 - at;
            }
            before += all;
        }
    }
    tc_fence_before();
    if (p.cs > 1)
        cluster_sync();  // every CTA's barriers exist
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    griddep_launch_dependents();
    TreeWalk<NT> walk(p, x1 > x0 ? run_seq : 0, x1 > x0 ? run_skip : 0, x1 - x0);

    auto give_up = [&]() {
        if (!abort_flag)
            atomicOr(p.err, kErrTimeout);
        abort_flag = 1;
    };

    if (warp == 0 || warp == kTreeVWarp) {
        // ============================================================ copies
        // warp 0: Q tiles and K, warp 10: V.  A stage is a copy per page (or
        // part of one); the cluster's CTAs take equal shares of them, lane c
        // the share's copy c.
        const bool is_v = warp == kTreeVWarp;
        const uint64_t pol = l2_evict_first_policy();
        const CUtensorMap *map = is_v ? &tmap_v : &tmap_k;
        uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
        const int slots = is_v ? NV : NK;
        const uint32_t ring = is_v ? v_s : k_s;
        const int share = NT / p.box_rows / p.cs;
        const int copy = rank * share + lane;  // this lane's copy
        const int from = copy * p.box_rows;    // its first token within a stage
        int nst = 0, nq = 0;
        bool ok = true;
        for (; walk.more() && ok; walk.next(p)) {
            const TreeSeq &q = walk.q;
            const int g = walk.head();
            const int npages = (q.L + p.BS - 1) >> p.log2BS;
            const int32_t *bt = p.block_tables + (size_t)walk.s * p.MB;
            auto block_of = [&](int t) -> int {  // block coordinate, -1: none (reads zeros)
                const int pg = (t * NT + from) >> p.log2BS;
                int b = -1;
                if (lane < share && pg < npages) {
                    const int id = __ldg(bt + pg);
                    if ((unsigned)id < (unsigned)p.NB)
                        b = id * p.blk_page + g * p.blk_head;
                    else if (!is_v)
                        atomicOr(p.err, kErrPageRange);
                }
                return b;
            };
            int blk_next = block_of(walk.t);
            for (int t = walk.t; t < walk.t_end; ++t) {
                const int st = nst % slots;
                const int blk = blk_next;
                if (t + 1 < walk.t_end)
                    blk_next = block_of(t + 1);  // in flight while this stage waits
                bool w = true;
                if (lane == 0)
                    w = mbar_wait_bounded(smem_addr(&empty[st]), ((nst / slots) & 1) ^ 1,
                                          &abort_flag, p.wait_budget_ns);
                ok = __shfl_sync(~0u, w, 0);
                if (!ok)
                    break;
                const uint32_t bar = smem_addr(&full[st]);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, KV_TILE);
                __syncwarp();
                if (lane < share) {
                    const uint32_t dst = ring + st * KV_TILE + (from / 8) * GROUP;
                    const int grp = ((t * NT + from) & (p.BS - 1)) >> 3;
                    if (p.cs > 1)
                        tma_load_5d_multicast(dst, map, 0, 0, 0, grp, blk, bar, everyone, pol);
                    else
                        tma_load_5d(dst, map, 0, 0, 0, grp, blk, bar, pol);
                }
                ++nst;
                if (!is_v && t == walk.t) {
                    // Q after the unit's first K: its place is free only after
                    // the last unit's last scores
                    if (lane == 0) {
                        w = mbar_wait_bounded(smem_addr(&q_empty), (nq & 1) ^ 1, &abort_flag,
                                              p.wait_budget_ns);
                        if (w) {
                            const uint32_t qb = smem_addr(&q_full);
                            mbar_arrive_expect_tx(qb, SLABS * p.TQ * p.G * 128);
                            const int tile = walk.group() * p.cs + rank;
                            for (int sl = 0; sl < SLABS; ++sl)
                                tma_load_4d(q_s + sl * Q_SLAB, &tmap_q, 0, g * p.G,
                                            q.row0 + tile * p.TQ, sl, qb);
                        }
                    }
                    ok = __shfl_sync(~0u, w, 0);
                    if (!ok)
                        break;
                    ++nq;
                }
            }
        }
        if (!ok && lane == 0) {
            give_up();
            // let the copies in flight land before the CTA exits
            if (nq)
                mbar_wait_bounded(smem_addr(&q_full), (nq - 1) & 1, nullptr, p.wait_budget_ns);
            for (int i = max(0, nst - slots); i < nst; ++i)
                mbar_wait_bounded(smem_addr(&full[i % slots]), (i / slots) & 1, nullptr,
                                  p.wait_budget_ns);
        }
        __syncwarp();
    } else if (warp == 1 || warp == kTreeOWarp) {
        if (lane == 0) {
            // ======================================================== products
            // scores by one thread, outputs by another: a thread spends some
            // 1400 cycles a stage on its barriers and commits, the products of
            // a stage take about as long, and one thread for both would be
            // slower than the copies
            bool ok = true;
            auto wait = [&](uint64_t *bar, int parity) {
                if (ok && !mbar_wait_bounded(smem_addr(bar), parity, &abort_flag, p.wait_budget_ns))
                    ok = false;
                return ok;
            };
            auto release = [&](uint64_t *bar) {
                if (p.cs > 1)
                    tc_commit_multicast(smem_addr(bar), everyone);
                else
                    tc_commit(smem_addr(bar));
            };
            if (warp == 1) {
                const uint64_t q_desc = tc_sdesc(q_s, 16, 1024);
                const uint64_t k_desc = tc_sdesc(k_s, 16, GROUP);
                int ns = 0, nq = 0;  // S products, Q tiles
                for (; walk.more() && ok; walk.next(p)) {
                    wait(&q_full, nq & 1);
                    ++nq;
                    for (int t = walk.t; t < walk.t_end; ++t, ++ns) {
                        // into the buffer of P(ns - 2), once its product is over
                        const int st = ns % NK;
                        if ((ns >= 2 && !wait(&o_done[ns & 1], ((ns >> 1) & 1) ^ 1)) ||
                            !wait(&k_full[st], (ns / NK) & 1))
                            break;
                        tc_fence_after();
                        const uint64_t ks = k_desc + ((st * KV_TILE) >> 4);
                        const uint32_t d = tmem + S_COL + (ns & 1) * NT;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma(d, q_desc + (((kk / 4) * Q_SLAB + (kk % 4) * 32) >> 4),
                                   ks + (((kk / 4) * 1024 + (kk % 4) * 32) >> 4), IDESC_S, kk > 0);
                        tc_commit(smem_addr(&s_full[ns & 1]));
                        release(&k_empty[st]);
                    }
                    tc_commit(smem_addr(&q_empty));
                }
            } else {
                const uint64_t v_desc = tc_sdesc(v_s, 1024, GROUP);
                int np = 0, no = 0;  // P V products, units
                for (; walk.more() && ok; walk.next(p)) {
                    // the last unit's output has been read
                    if (no++ && !wait(&o_free, no & 1))
                        break;
                    for (int t = walk.t; t < walk.t_end; ++t, ++np) {
                        const int st = np % NV;
                        if (!wait(&v_full[st], (np / NV) & 1) || !wait(&p_full, np & 1))
                            break;
                        tc_fence_after();
                        const uint64_t vs = v_desc + ((st * KV_TILE) >> 4);
                        const uint32_t a = tmem + S_COL + (np & 1) * NT;
#pragma unroll
                        for (int kk = 0; kk < NT / 16; ++kk)
                            tc_mma_ta(tmem + O_COL, a + kk * 8, vs + ((kk * 2 * GROUP) >> 4),
                                      IDESC_O, t > walk.t || kk > 0);
                        tc_commit(smem_addr(&o_done[np & 1]));
                        release(&v_empty[st]);
                    }
                }
            }
            if (!ok)
                give_up();
            // every product issued here has completed before the memory is freed
            tc_commit(smem_addr(&mma_done));
            mbar_wait_bounded(smem_addr(&mma_done), 0, nullptr, p.wait_budget_ns);
        }
        __syncwarp();
    } else {
        // ============================================================ softmax
        // warps 2-5 take the first half of a stage's tokens, warps 6-9 the
        // second, for the same rows: warp w reads tensor-memory quarter w & 3
        constexpr int HC = NT / 2, HD = D / 2;
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const int r = 32 * quarter + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t pair_bar = 1 + quarter;
        const int ti = r / p.G;
        // a scale of 0 runs as 1e-30: exp2 of every score is then 1 in fp32
        // (the mean, as for 0) while masked scores, infinite with the sign that
        // scales to -inf, still give 0
        const float sc = p.scale_log2 == 0.f ? 1e-30f : p.scale_log2;
        const bool neg = sc < 0.f;
        const float masked = neg ? INFINITY : -INFINITY;
        const float2 sc2 = make_float2(sc, sc);
        const bool scribe = threadIdx.x == 64 && rank == 0;
        if (scribe)
            p.cut[cluster] = make_int4(-1, 0, 0, 0);
        if (!walk.more() && half == 0)  // an empty run (fewer stages than runs) between a unit's pieces
            p.part_ml[((size_t)(2 * cluster) * p.cs + rank) * 128 + r] = make_float2(-INFINITY, 0.f);
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
        for (; walk.more(); walk.next(p)) {
            const TreeSeq &q = walk.q;
            const int g = walk.head(), tile = walk.group() * p.cs + rank;
            const int left = min(p.TQ, q.n - tile * p.TQ);  // nodes of this tile (or none)
            const bool row_ok = r < p.TQ * p.G && ti < left;
            const int node = tile * p.TQ + ti;
            const int prefix = q.L - q.n;
            if (walk.t_end * NT > prefix && built != walk.s) {
                build_tree_bits(tree, p.parents + q.row0, q.n, threadIdx.x - 64, 5, p.err);
                built = walk.s;
            }
            float m_ref = -INFINITY, l = 0.f;
            for (int t = walk.t; t < walk.t_end; ++t, ++ns) {
                const int t0 = t * NT, c0 = t0 + half * HC;
                const uint32_t s_col = S_COL + (ns & 1) * NT;
                wait(&s_full[ns & 1], (ns >> 1) & 1);
                float v[HC / 32][32];
                float e = masked;
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
                                v[c][i] = (seen >> i) & 1u ? v[c][i] : masked;
                        }
                    }
                    // the extreme: the sign is the call's, a branch around two loops
                    float ec[2 * (HC / 32)];
                    if (!neg) {
#pragma unroll
                        for (int c = 0; c < 2 * (HC / 32); ++c) {
                            ec[c] = v[c >> 1][16 * (c & 1)];
#pragma unroll
                            for (int i = 1; i < 15; i += 2)
                                ec[c] = fmax3(ec[c], v[c >> 1][16 * (c & 1) + i],
                                              v[c >> 1][16 * (c & 1) + i + 1]);
                            ec[c] = fmaxf(ec[c], v[c >> 1][16 * (c & 1) + 15]);
                        }
                        e = fmaxf(ec[0], ec[1]);
                        if constexpr (HC == 64)
                            e = fmax3(e, ec[2], ec[3]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 2 * (HC / 32); ++c) {
                            ec[c] = v[c >> 1][16 * (c & 1)];
#pragma unroll
                            for (int i = 1; i < 15; i += 2)
                                ec[c] = fmin3(ec[c], v[c >> 1][16 * (c & 1) + i],
                                              v[c >> 1][16 * (c & 1) + i + 1]);
                            ec[c] = fminf(ec[c], v[c >> 1][16 * (c & 1) + 15]);
                        }
                        e = fminf(ec[0], ec[1]);
                        if constexpr (HC == 64)
                            e = fmin3(e, ec[2], ec[3]);
                    }
                }
                pair_red[ns & 1][half][r] = e;
                tc_fence_before();
                named_barrier_sync(pair_bar, 64);
                tc_fence_after();
                const float e2 = pair_red[ns & 1][half ^ 1][r];
                if (!ok)
                    continue;
                e = neg ? fminf(e, e2) : fmaxf(e, e2);
                const float mt = e == masked ? -INFINITY : e * sc;
                // the reference maximum moves only by more than 8 (log2 units):
                // p stays below 2^8, well inside fp16, and O is rescaled rarely
                bool rescale = false;
                float alpha = 1.f;
                if (mt > m_ref + 8.f) {
                    rescale = row_ok && m_ref != -INFINITY;
                    alpha = rescale ? ex2(m_ref - mt) : 1.f;
                    m_ref = mt;
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
                if constexpr (HC == 64)
                    tc_st32u(t_lane + s_col + half * 32, pk);
                else
                    tc_st16u(t_lane + s_col + half * 16, pk);
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
                    const int st = ns % NV;
                    mbar_wait_bounded(smem_addr(&v_full[st]), (ns / NV) & 1, nullptr,
                                      p.wait_budget_ns);
                    uint8_t *vs = v_ptr + st * KV_TILE;
                    const int za = q.L - t0;
                    for (int idx = half * 128 + r; idx < (NT - za) * SLABS * 8; idx += 256) {
                        const int row = za + idx / (SLABS * 8), c = idx % (SLABS * 8);
                        *reinterpret_cast<uint4 *>(vs + (row / 8) * GROUP + (c >> 3) * 1024 +
                                                   (row % 8) * 128 + (c & 7) * 16) =
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
            // the row's exp-sum from both halves, then each half writes its
            // columns (through the last stage's slot: its readers are done,
            // since o_done came after every warp's p_full, and the next stage
            // takes the other)
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
                    mbar_arrive(smem_addr(&o_free));
            };
            // a store takes 64 columns at least: at head_dim 64 the first
            // half's warps write whole rows
            constexpr int WC = D == 64 ? 64 : HD;
            const int col = D == 64 ? 0 : half * HD;
            if (D == 64 && half == 1) {
                read();
            } else if (whole) {
                const RowOut rows =
                    rows_out(p.out, (size_t)D * (p.out_half ? 2 : 4), p.Hq, p.G, p.TQ,
                             q.row0 + tile * p.TQ, left, g, quarter, lane);
                write_rows<WC>(rows, p.out_half, p.wide_rows, t_lane + O_COL + col, col,
                               lt > 0.f ? 1.f / lt : 0.f, lane, read);
            } else {
                // a piece: 0 where the unit began in an earlier run, else 1
                const size_t piece = (size_t)(2 * cluster + (walk.t == 0)) * p.cs + rank;
                RowOut rows;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 32 * quarter + (lane & ~3) + i;
                    rows.at[i] = row < p.TQ * p.G && row / p.G < left
                                     ? reinterpret_cast<char *>(p.part_o + (piece * 128 + row) * D)
                                     : nullptr;
                }
                write_rows<WC>(rows, false, true, t_lane + O_COL + col, col, 1.f, lane, read);
                if (row_ok && half == 0)
                    p.part_ml[piece * 128 + r] = make_float2(m_ref, lt);
                if (scribe && walk.t == 0) {
                    // the run that holds the unit's last stage
                    const long long end = x1 - walk.left + q.T;  // one past it
                    p.cut[cluster] = make_int4(walk.s, g, walk.group(),
                                               (int)((end * p.clusters - 1) / total));
                }
            }
        }
    }
    tc_fence_before();
    if (p.cs > 1)
        cluster_sync();  // no CTA leaves while another may still signal it
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

// Joins the pieces of the unit that is cut at the end of run blockIdx.x (if one
// is): its piece 1 there, then piece 0 of every later run up to the last.  A
// row's output is sum_i w_i o_i / sum_i w_i l_i with w_i = exp2(m_i - max m).
// CTA (run, tile, quarter): 32 rows, a warp per row in turn.
constexpr int kTreeJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kTreeJoinThreads) paged_tree_join_kernel(const TreeParams p)
{
    constexpr int VPL = D / 32;  // values per lane
    const int run = blockIdx.x, rank = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    const int4 cut = p.cut[run];
    if (cut.x < 0)
        return;
    const int row0 = __ldg(p.cu_q + cut.x), n = __ldg(p.cu_q + cut.x + 1) - row0;
    const int tile = cut.z * p.cs + rank;
    for (int r = 32 * blockIdx.z + warp; r < 32 * (int)blockIdx.z + 32; r += kTreeJoinThreads / 32) {
        const int ti = r / p.G, node = tile * p.TQ + ti;
        if (r >= p.TQ * p.G || node >= n)
            break;  // (rows in order: none after it either)
        auto piece = [&](int i) -> size_t {
            return ((size_t)(i == run ? 2 * run + 1 : 2 * i) * p.cs + rank) * 128 + r;
        };
        float top = -INFINITY;
        for (int i = run + lane; i <= cut.w; i += 32)
            top = fmaxf(top, p.part_ml[piece(i)].x);
#pragma unroll
        for (int off = 16; off; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(~0u, top, off));
        float acc[VPL], den = 0.f;
#pragma unroll
        for (int k = 0; k < VPL; ++k)
            acc[k] = 0.f;
        for (int i = run; i <= cut.w; ++i) {
            const float2 ml = p.part_ml[piece(i)];
            if (ml.x == -INFINITY)  // the row sees nothing there
                continue;
            const float *o = p.part_o + piece(i) * D + VPL * lane;
            const float w = ex2(ml.x - top);
            den += w * ml.y;
#pragma unroll
            for (int k = 0; k < VPL; k += 2) {
                const float2 x = *reinterpret_cast<const float2 *>(o + k);
                acc[k] += w * x.x;
                acc[k + 1] += w * x.y;
            }
        }
        const float inv = den > 0.f ? 1.f / den : 0.f;
        const size_t at = ((size_t)(row0 + node) * p.Hq + (size_t)cut.y * p.G + (r - ti * p.G)) * D +
                          VPL * lane;
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
}

namespace {

template <int D> void tree_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int cs)
{
    *cfg = {};
    cfg->blockDim = dim3(kTreeThreads);
    cfg->dynamicSmemBytes = tree_smem_bytes<D>();
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)cs;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = cs > 1 ? 1 : 0;
}

template <int D> cudaError_t tree_clusters_dim(int cs, int *clusters)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    tree_config<D>(&cfg, &attr, cs);
    cudaError_t e = cudaFuncSetAttribute(paged_tree_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess)
        return e;
    if (cs == 1) {
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess)
            return e;
        return cudaDeviceGetAttribute(clusters, cudaDevAttrMultiProcessorCount, dev);
    }
    cfg.gridDim = dim3((unsigned)cs);
    return cudaOccupancyMaxActiveClusters(clusters, paged_tree_kernel<D>, &cfg);
}

template <int D>
cudaError_t launch_tree_dim(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const TreeParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    tree_config<D>(&cfg, &attr, p.cs);
    cfg.gridDim = dim3((unsigned)(p.clusters * p.cs));
    cfg.stream = stream;
    cudaError_t e;
    if ((e = cudaLaunchKernelEx(&cfg, paged_tree_kernel<D>, tq, tk, tv, p)) != cudaSuccess)
        return e;
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t join = {};
    join.gridDim = dim3((unsigned)p.clusters, (unsigned)p.cs, 4);
    join.blockDim = dim3(kTreeJoinThreads);
    join.stream = stream;
    join.attrs = &overlap;
    join.numAttrs = 1;
    return cudaLaunchKernelEx(&join, paged_tree_join_kernel<D>, p);
}

}  // namespace

cudaError_t tree_clusters(int head_dim, int cs, int *clusters)
{
    return head_dim == 64    ? tree_clusters_dim<64>(cs, clusters)
           : head_dim == 128 ? tree_clusters_dim<128>(cs, clusters)
                             : tree_clusters_dim<256>(cs, clusters);
}

cudaError_t launch_tree(int head_dim, const CUtensorMap &tq, const CUtensorMap &tk,
                        const CUtensorMap &tv, const TreeParams &p, cudaStream_t stream)
{
    return head_dim == 64    ? launch_tree_dim<64>(tq, tk, tv, p, stream)
           : head_dim == 128 ? launch_tree_dim<128>(tq, tk, tv, p, stream)
                             : launch_tree_dim<256>(tq, tk, tv, p, stream);
}

}  // namespace pgd
