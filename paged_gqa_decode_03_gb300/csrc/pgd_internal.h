// Shared host/device definitions of the GPU path: one set of constants for
// the launcher and the kernels so the two cannot drift (the pages' vllm-metal
// keeps its partition and block sizes in one constants file shared with the
// shaders, "Three Metal kernels" section).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace pgd {

// Partition sizes of the split-KV scheme ("Four speed-up tricks", 4).
constexpr int kPartitionLarge = 512;
constexpr int kPartitionSmall = 256;
// Most query heads per KV head one CTA handles (one n8 tensor-core tile).
constexpr int kMaxGroup = 8;
// Several query tokens per sequence on the decode kernel (its MQ form, for
// calls with few query rows per (sequence, KV head): decode steps, short
// verification steps): up to 8 columns (query token x head of the group,
// one n8 tile, as many as the group's heads in a decode) per unit.
constexpr int kMaxCols = 8;
// Cap on the per-call scratch ("Dispatch layer": 512 MiB).
constexpr size_t kMaxWorkspaceBytes = size_t(512) << 20;
// Bound on every internal pipeline wait before it reports a timeout.
constexpr uint64_t kWaitBudgetNs = 2000000000ull;

// Device error bits (mirror PGD_DEVERR_* of pgd.h).
constexpr unsigned kErrPageRange = 1u;
constexpr unsigned kErrSeqLen = 2u;
constexpr unsigned kErrTimeout = 4u;

// Sequence lengths the partition kernel keeps in shared memory, and the
// most pipeline stages a partial partition can have (512 / 32).
constexpr int kLensCap = 256;
constexpr int kMaxTailStages = 16;

// Kernel shape per head_dim: tokens per pipeline stage (T), consumer warps
// (NC, one 16-token tile each), stages in the shared-memory ring (NS).  The
// ring holds about 100 KB for every head_dim (two CTAs per SM).
template <int D> struct Shape;
// T8 / NC8 / NS8: the same for quantised pages, whose consumers do more work
// per byte (code conversion, the affine terms): twice the tokens per stage,
// fewer stages (one more where the page size leaves room: ring_stages); at
// head_dim 128 four consumer warps of two 16-token tiles each (the tiles
// share a warp's softmax reductions and the unit merge has half the states;
// eight warps of one tile measured 7-10 % slower), at 256 one tile each.
template <> struct Shape<64> {
    static constexpr int T = 64, NC = 4, NS = 6, T8 = 64, NC8 = 4, NS8 = 6;
};
template <> struct Shape<128> {
    static constexpr int T = 64, NC = 4, NS = 3, T8 = 128, NC8 = 4, NS8 = 2;
};
template <> struct Shape<256> {
    static constexpr int T = 32, NC = 2, NS = 3, T8 = 64, NC8 = 4, NS8 = 2;
};
template <int D, bool Q8> __host__ __device__ constexpr int stage_tokens_of() { return Q8 ? Shape<D>::T8 : Shape<D>::T; }
template <int D, bool Q8, bool MQ = false> __host__ __device__ constexpr int consumer_warps()
{
    return Q8 ? Shape<D>::NC8 : Shape<D>::NC;
}

// Quantised pages: 8-bit codes plus one (scale, bias) bf16 pair per 64
// values of a row.
constexpr int kQuantGroup = 64;

// Bytes of K (or V) codes / values of one stage, of their (scale, bias)
// pairs, and of a whole stage (K, V, their pairs, the group's queries).
template <int D, bool Q8 = false> __host__ __device__ constexpr int stage_kv_bytes()
{
    return stage_tokens_of<D, Q8>() * D * (Q8 ? 1 : 2);
}
// (scale, bias) pairs of one copied page piece, padded so every piece lands
// 128-byte aligned (a tensor-copy requirement).
__host__ __device__ constexpr int meta_slot_bytes(int rows, int D)
{
    return (rows * (D / kQuantGroup) * 4 + 127) / 128 * 128;
}
// The pairs of one stage: one slot per page piece of min(BS, T) rows.
template <int D, bool Q8, int BS> __host__ __device__ constexpr int stage_meta_bytes()
{
    constexpr int T = stage_tokens_of<D, Q8>(), BOX = BS < T ? BS : T;
    return Q8 ? (T / BOX) * meta_slot_bytes(BOX, D) : 0;
}
template <int D, bool MQ = false> __host__ __device__ constexpr int stage_q_bytes()
{
    return (MQ ? kMaxCols : kMaxGroup) * D * 2;
}
template <int D, bool Q8, int BS, bool MQ = false> __host__ __device__ constexpr int stage_bytes()
{
    return 2 * stage_kv_bytes<D, Q8>() + 2 * stage_meta_bytes<D, Q8, BS>() +
           stage_q_bytes<D, MQ>();
}
// Shared memory of one SM, and what a CTA needs beside its ring (the
// system's 1 KB, the static barriers and stage headers, the alignment slack).
constexpr int kSmemPerSM = 233472;
constexpr int kSmemPerCtaExtra = 1024 + 3072 + 1024;
// Quantised pages take a third stage where two CTAs per SM still fit (the
// consumers hold a stage longer per byte than with fp16 pages, so more
// bytes must be in flight per stage held).
template <int D, bool Q8, int BS> __host__ __device__ constexpr int ring_stages()
{
    if constexpr (!Q8)
        return Shape<D>::NS;
    return 2 * ((Shape<D>::NS8 + 1) * stage_bytes<D, Q8, BS>() + kSmemPerCtaExtra) <= kSmemPerSM
               ? Shape<D>::NS8 + 1
               : Shape<D>::NS8;
}
// Dynamic shared memory: the ring plus slack to align it to 1024 bytes
// (required by the 128-byte swizzle of the tensor copies).
template <int D, bool Q8, int BS, bool MQ = false> __host__ __device__ constexpr size_t dyn_smem_bytes()
{
    return size_t(ring_stages<D, Q8, BS>()) * stage_bytes<D, Q8, BS, MQ>() + 1024;
}

struct DecodeParams {
    float *out;                   // [S][Hq][D]
    const __half *q;              // [S][Hq][D]
    const int32_t *block_tables;  // [S][MB]
    const int32_t *seq_lens;      // [S]
    float *ws_m;                  // [S][Hq][NPmax] log2-space partition max
    float *ws_l;                  // [S][Hq][NPmax] partition exp2-sum
    float *ws_o;                  // [S][Hq][NPmax][D] normalised partition output
    int32_t *page_trace;          // [S][Hkv][MB] or null
    unsigned *counter;            // work-claim counter: 0 at launch, reset by the reduce
    unsigned *err;                // device error word
    const __half *k_new;          // [S][Hkv][D] newest token's K (fused append) or null
    const __half *v_new;          // [S][Hkv][D] newest token's V
    __half *k_cache;              // caches, written at the newest token's row (append)
    __half *v_cache;
    uint16_t *k_meta;             // quantised pages: [NB][Hkv][BS][D/64][2] bf16
    uint16_t *v_meta;             //   (scale, bias) pairs (written by the fused
                                  //   append), or null
    int q8_pair;                  // quantised pages: one tensor copy brings a page's
                                  //   K and V codes (tmap_k spans both arrays), 1: over
                                  //   (page, head) blocks, 2: over (head, slab) pairs
    int q8_meta_pair;             // one tensor copy brings a page's K and V (scale,
                                  //   bias) pairs (tmap_km spans both arrays): 1 with
                                  //   K's array the lower, 2 with V's; 0: two copies
    int q8_koff, q8_voff;         //   bytes of K / V codes within a page's pair of slots
    int q8_rows;                  //   the pairs at meta strides (any layout), copied
                                  //   1: row by row, 2: by a tensor copy of 16-byte rows
    long long meta_page_stride;   // quantised pages: the pairs of token r of page b,
    long long meta_head_stride;   //   KV head g start at bf16 element b*page + g*head
    long long meta_token_stride;  //   + r*token (head-major unless q8_rows)
    long long kv_page_stride;     // cache strides in halves (the copies use the
    long long kv_head_stride;     //   same ones through the tensor maps)
    long long kv_token_stride;
    float scale_log2;             // scale * log2(e)
    int S, Hq, Hkv, G, P, logP, MB, NB, NPmax;
    uint64_t wait_budget_ns;
    const unsigned *stall_flag;   // test knob: every CTA first waits (bounded) for
                                  //   *stall_flag != 0, or null
    // several query tokens per sequence (the MQ form; cu_q null otherwise):
    // sequence s owns query rows cu_q[s] .. cu_q[s+1]-1 of q / out [total_q][Hq][D],
    // the newest n_s of its tokens (query i at position L - n_s + i, causal);
    // the partials are indexed by (query row, head) instead of (sequence, head)
    const int32_t *cu_q;
    int max_q, total_q;
};

struct LaunchConfig {
    int grid;            // partition-kernel CTAs (persistent)
    int reduce_blocks;   // reduce-kernel CTAs
    cudaStream_t stream;
    cudaEvent_t ev_before, ev_after;  // optional timing hook (both or neither)
    bool skip_reduce = false;         // test knob: launch the partition kernel only
};

// The tensor maps of one decode launch: K and V (fp16 rows, or 8-bit codes),
// and for quantised pages the maps of their (scale, bias) pairs (otherwise
// K and V again, unused).
struct KVMaps {
    const CUtensorMap *k, *v, *km, *vm;
};

// Per-head_dim entry points (pgd_kernels_d64.cu, _d128.cu, _d256.cu); p.cu_q
// non-null selects the MQ form (head_dim 64 and 128).
cudaError_t launch_decode_d64(int block_size, bool trace, bool q8, const KVMaps &m,
                              const DecodeParams &p, const LaunchConfig &lc);
cudaError_t launch_decode_d128(int block_size, bool trace, bool q8, const KVMaps &m,
                               const DecodeParams &p, const LaunchConfig &lc);
cudaError_t launch_decode_d256(int block_size, bool trace, bool q8, const KVMaps &m,
                               const DecodeParams &p, const LaunchConfig &lc);
// Resident partition-kernel CTAs per SM for (head_dim, block_size, kind:
// 0 fp16 pages, 1 quantised pages, 2 the MQ form); 0 where no kernel is
// built (quantised pages at head_dim 64, the MQ form at 256).
cudaError_t occupancy_d64(int block_size, int kind, int *ctas_per_sm);
cudaError_t occupancy_d128(int block_size, int kind, int *ctas_per_sm);
cudaError_t occupancy_d256(int block_size, int kind, int *ctas_per_sm);

// Reduce kernel: one CTA per (sequence, query head); two warps suffice for
// head_dim 64 and 128 (whose workloads have at most 16 partitions per
// sequence) and keep every CTA resident at once, four for 256.
template <int D> __host__ __device__ constexpr int reduce_threads() { return D <= 128 ? 64 : 128; }

// ---------------------------------------------------------------- several query tokens
// Paged attention with n_s >= 1 query tokens per sequence (pgd_varlen.cu).
// A work unit is 128 rows of one (sequence, KV head): TQ = 128 / G query
// tokens x the G heads of the group, over one KV partition of PK tokens.
constexpr unsigned kErrQueryLen = 8u;  // a query count < 0, > its length or > max_q_len

// KV tokens per pipeline stage (NT) and stages (NSTG) per head_dim; the
// 128-row tiles and both score buffers live in 512 tensor-memory columns.
template <int D> struct VShape;
template <> struct VShape<64> {
    static constexpr int NT = 128, NSTG = 4;
};
template <> struct VShape<128> {
    static constexpr int NT = 128, NSTG = 2;  // a third stage would pass the 227 KB limit
};
template <> struct VShape<256> {
    static constexpr int NT = 64, NSTG = 2;
};
// head_dim 64 and 128 can run two query tiles per CTA
// (paged_varlen_pair_kernel): two score buffers and two O accumulators fit in
// tensor memory.  Calls whose sequences have at most one tile of query rows
// use the one-tile kernel.
template <int D> __host__ __device__ constexpr bool varlen_pairs() { return 2 * VShape<D>::NT + 2 * D <= 512; }
template <int D> __host__ __device__ constexpr size_t varlen_smem_bytes(bool pairs)
{
    // Q tile(s) + stages of K and V + alignment slack (P lives in tensor memory)
    return size_t(pairs ? 2 : 1) * 128 * D * 2 +
           size_t(VShape<D>::NSTG) * 2 * VShape<D>::NT * D * 2 + 1024;
}
constexpr int kVarlenThreads = 352;   // K producer, MMA, 8 softmax warps, V producer
constexpr int kVWarp = 10;            // the V producer warp
constexpr uint32_t kVarlenTmemCols = 512;

struct VarlenParams {
    float *out;                   // [total_q][Hq][D]
    const int32_t *cu_q;          // [S+1]
    const int32_t *block_tables;  // [S][MB]
    const int32_t *seq_lens;      // [S]
    float *ws_m, *ws_l, *ws_o;    // [total_q*Hq][NP] (m, l), [total_q*Hq][NP][D]
    unsigned *err;
    float scale_log2;
    int S, Hq, Hkv, G, TQ, QT, NP, PK, MB, NB, BS, log2BS, max_q;
    int QP;                       // query-tile units per (sequence, KV head): QT, or
                                  //   ceil(QT / 2) pairs (paged_varlen_pair_kernel)
    const int *order;             // [grid] unit of each block, longest first; null:
                                  //   block index order
    int blk_page, blk_head;       // (page, KV head) -> block coordinate of the K/V maps
    uint64_t wait_budget_ns;
};

// ---------------------------------------------------------------- weights of the step's attention
// Trees and packed prompts hold a weight p = 2^(score - reference) in fp16 for its
// product with V (the tensor cores take A and B of one type, V is fp16, and fp16
// has three bits more than bf16); scores, sums and outputs are fp32.  The
// reference is set kRefBelow under the row's maximum and stays while the maximum
// keeps within kRefRoom of it: p is at most 2^15, inside fp16's 65504, and is
// a normal number, rounded by 2^-11 of itself, down to 2^-21 of the largest, below
// that by 2^-32 of the largest at most.  (With the reference at the maximum those were
// 2^-14 and 2^-25: thousands of small weights behind one large one lost
// bits that the sum of the unrounded ones still held.)
constexpr float kRefBelow = 7.f;
constexpr float kRefRoom = 15.f;

// ---------------------------------------------------------------- trees of drafted tokens
// Attention of trees of drafted tokens over the paged cache (pgd_tree.cu).
constexpr unsigned kErrTree = 32u;     // a parent that is not an earlier node of its tree
constexpr int kTreeMaxNodes = 256;     // nodes of one sequence's tree

// A stage is kTreeNT tokens.  With trees of more than one tile (head_dim 128 and
// 256) two CTAs work on two tiles as a pair of the tensor cores, each copying half
// of every stage: half of K's tokens, half of V's head_dim.  KP, VP: the pieces in
// which a CTA's part of K and of V is copied and used; NK, NV: pieces in the rings
// (what 227 KB leave beside the Q tile and the trees' bits).
constexpr int kTreeNT = 128;
template <int D, bool PAIR> struct TreeShape;
template <> struct TreeShape<64, false> {
    static constexpr int KP = 1, VP = 1, NK = 4, NV = 4;
};
template <> struct TreeShape<128, false> {
    static constexpr int KP = 1, VP = 1, NK = 2, NV = 3;
};
template <> struct TreeShape<256, false> {  // K by 64-wide slabs, V by 32 tokens
    static constexpr int KP = 4, VP = 4, NK = 5, NV = 4;
};
template <> struct TreeShape<128, true> {
    static constexpr int KP = 1, VP = 1, NK = 4, NV = 6;
};
template <> struct TreeShape<256, true> {   // K by two slabs, V by 64 tokens
    static constexpr int KP = 2, VP = 2, NK = 4, NV = 5;
};
// Tokens of K and slabs of V that a CTA copies of a stage, and slabs of a K piece
// and tokens of a V piece.
template <int D, bool PAIR> struct TreePieces {
    using S = TreeShape<D, PAIR>;
    static constexpr int KKEYS = PAIR ? kTreeNT / 2 : kTreeNT, KSLABS = D / 64 / S::KP;
    static constexpr int VSLABS = PAIR ? D / 128 : D / 64, VKEYS = kTreeNT / S::VP;
    static constexpr int K_BYTES = KKEYS * KSLABS * 128, V_BYTES = VKEYS * VSLABS * 128;
};

struct TreeParams {
    void *out;                    // [total_q][Hq][D], fp16 (out_half) or fp32
    bool out_half, wide_rows;     // wide_rows: it starts on a 32-byte border
    const int32_t *cu_q;          // [S+1]
    const int32_t *parents;       // [total_q] parent node of each row, negative: none
    const int32_t *block_tables;  // [S][MB]
    const int32_t *seq_lens;      // [S]
    // scratch: the pieces of the units that are cut, two per run, each 128 rows
    // per tile of the unit, and where the cut units begin
    float *part_o;                // [2 * runs][cs][128][D] sums of p v
    float2 *part_ml;              // [2 * runs][cs][128] (reference maximum, exp-sum)
    int4 *cut;                    // [runs] {sequence or -1, KV head, tile group, last run}
    unsigned *err;
    float scale_log2;
    int S, Hq, Hkv, G, TQ, total_q, max_q, MB, NB, BS, log2BS;
    int cs, runs;                 // tiles (CTAs) that work together, 1 or 2; runs of work
    int k_rows, v_rows;           // tokens of one page copy of K and of V
    int blk_page, blk_head;       // (page, KV head) -> block coordinate of the K/V maps
    uint64_t wait_budget_ns;
};
// Runs that are resident at once on the current device, of one CTA or of a pair (0
// where no kernel is built); also the kernel's set-up there, once before its launches.
cudaError_t tree_resident(int head_dim, bool pair, int *runs);
cudaError_t launch_tree(int head_dim, const CUtensorMap &tq, const CUtensorMap &tk,
                        const CUtensorMap &tv, const TreeParams &p, cudaStream_t stream);

// ---------------------------------------------------------------- packed prompts
// Causal attention over whole packed prompts (pgd_prefill.cu).
constexpr int kPrefillOrderKeys = 1024;  // stage counts the sort tells apart

struct PrefillParams {
    float *out;                   // [total][Hq][D], or null with
    __half *out_half;             //   out_half, the output as fp16
    const int32_t *cu_seqlens;    // [S + 1]
    int4 *units;                  // scratch: [max_units], longest first
    int *num_units;               // scratch
    unsigned *err;
    float scale_log2;
    int S, total, max_len, Hq, Hkv, G;
    int TQ, span;                 // tokens of a tile, and of a unit (one tile or a pair)
    int max_units;
    bool wide_rows;               // the output starts on a 32-byte border
    uint64_t wait_budget_ns;
};
// The list of units, longest first (also the kernel in front of pgd_latent_prefill.cu's).
cudaError_t launch_prefill_order(const PrefillParams &p, cudaStream_t stream);
// On the current device, once before the launches of this head_dim.
cudaError_t prefill_set_up(int head_dim);
cudaError_t launch_prefill(int head_dim, const CUtensorMap &tq, const CUtensorMap &tk,
                           const CUtensorMap &tv, const PrefillParams &p, int grid,
                           cudaStream_t stream);

// ---------------------------------------------------------------- the step around the cache
// Page tables, slots, positions and lengths of a step, and the writes of its
// K and V rows (pgd_kv.cu).
constexpr unsigned kErrNoPage = 16u;      // a step needed more pages than the free list holds
constexpr int kSlotCountCap = 1 << 30;    // row and page counts saturate here
constexpr int kSlotMaxSeqs = 16384;       // requests of one call (their offsets sit in shared memory)
constexpr int kSlotSmemMax = (2 * kSlotMaxSeqs + 1) * 4;

struct SlotParams {
    int32_t *slots, *positions;           // [N] (positions or null)
    int32_t *cu_seqlens_q, *seq_lens;     // [S + 1], [S]
    int32_t *free_end;                    // [1]
    int32_t *block_tables;                // [S][MB]: read below, written from owned_s on
    const int32_t *context_lens, *query_lens;  // [S]
    const int32_t *free_pages;            // [num_free]
    const int32_t *free_start;            // [1] or null (0)
    unsigned *err;
    int S, N, num_free, log2BS, MB, NB;
    bool vector_slots, vector_positions;  // 16-byte aligned outputs
};
cudaError_t launch_kv_slots(const SlotParams &p, int num_sms, cudaStream_t stream);

struct WriteParams {
    uint16_t *k_cache, *v_cache;
    const uint16_t *k_new, *v_new;
    const int32_t *slots;                 // [rows]
    unsigned *err;
    int rows, Hkv, vec, log2BS, NB;       // vec: 16-byte pieces of a row (head_dim / 8)
    int rows_per_cta;                     // set by the launcher
    long long page_stride, head_stride, token_stride;   // halves
    long long k_token_stride, k_head_stride, v_token_stride, v_head_stride;
};
cudaError_t launch_kv_write(WriteParams p, cudaStream_t stream);

// ---------------------------------------------------------------- rotary positions
// The step's rows rotated and written (pgd_rope.cu): queries into q_out, keys and
// values into their pages.  A latent cache's rows are keys and "values" of one head.
struct RopeParams {
    uint16_t *k_cache, *v_cache, *q_out;
    const uint16_t *q, *k_new, *v_new;
    const int32_t *slots, *positions;     // [rows]
    const float *inv_freq;                // [rot / 2]
    unsigned *err;
    float magnitude;
    bool interleaved, in_place;           // in_place: q_out is q
    int rows, Hq, Hkv, rot, log2BS, NB;
    int log2q, log2k, log2v;              // of a head's 32-byte items (values / 16)
    int rows_per_cta;                     // set by the launcher, as
    uint32_t row_inverse, pair_inverse;   //   the reciprocals of a row's items and pairs
    long long page_stride, head_stride, token_stride;   // halves
    long long qo_token, qo_head, q_token, q_head, k_token, k_head, v_token, v_head;
};
cudaError_t launch_rope_write(RopeParams p, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- latent caches
// Attention over a latent cache by pairs of CTAs (pgd_latent.cu).  A stage is kLatentNT
// tokens; a CTA has kLatentRows rows of queries, copies half of a stage's tokens as
// keys in KP pieces of KSLABS 64-wide slabs, and half of the values of all of them in
// VP pieces of VKEYS tokens.  Every piece is kLatentPiece bytes; NK, NV pieces in the
// rings, NS score buffers.
constexpr int kLatentNT = 128, kLatentRows = 64, kLatentPiece = 16384;
// What a unit (a tile of a sequence's rows) counts in the division of the work: its
// stages and, in stages, its start and end.  (Of 2, 3, 4, 5 about the best: 64 requests of
// 128 heads 63.6, 63.3, 62.2, 63.9 us, 24 of up to 5 rows 54.0, 52.7, 54.6, 54.7, 32 long
// ones 133, 130, 131, 132.)
constexpr int kLatentUnitCost = 3;
template <int R> struct LatentShape {
    static constexpr int KSLABS = 2, KP = R / 128;
    static constexpr int VSLABS = R / 128, VKEYS = 128 / VSLABS, VP = VSLABS;
    static constexpr int NK = 4, NV = 4, NS = 2;
    static constexpr int NR = NK / KP;  // the rotary keys' places: one for every stage in K's ring
};
// Q with its rotary part, two stages' weights, the rotary keys, the rings (what 227 KB leave
// beside the static part at R 512)
template <int R> constexpr size_t latent_smem_bytes()
{
    return size_t(R / 64 + 1 + 2 + LatentShape<R>::NR) * kLatentRows * 128 +
           size_t(LatentShape<R>::NK + LatentShape<R>::NV) * kLatentPiece;
}
struct LatentParams {
    void *out;                    // [total_q][H][R], fp16 (out_half) or fp32
    bool out_half, wide_rows;     // wide_rows: it starts on a 32-byte border
    const int32_t *cu_q;          // [S + 1], or null: one row a sequence
    const int32_t *block_tables;  // [S][MB]
    const int32_t *seq_lens;      // [S]
    // scratch: the pieces of the units that are cut, two per run, of 64 rows in each
    // CTA, and where the cut units begin
    float *part_o;                // [2 * runs][2][64][R] sums of p c
    float2 *part_ml;              // [2 * runs][2][64] (reference maximum, exp-sum)
    int4 *cut;                    // [runs] {sequence or -1, tile, last run, -}
    int *allowed;                 // the sequences to run, of the check in front, or null: all
    unsigned *err;
    float scale_log2;
    int S, total_q, max_q, H, R, MB, NB, BS, log2BS;
    int hb, TQ, HB;               // a half tile: TQ tokens x hb heads; HB blocks of heads a token
    int k_rows, v_rows;           // tokens of one page copy of K and of V
    int runs;
    uint64_t wait_budget_ns;
    // half tiles of n query tokens
    __host__ __device__ int half_tiles(int n) const { return HB == 1 ? (n + TQ - 1) / TQ : n * HB; }
};
struct LatentMaps {
    CUtensorMap q, qr, k, kr, v;
};
// Pairs that are resident at once on the current device; also the kernel's set-up there.
cudaError_t latent_resident(int latent_dim, int *runs);
cudaError_t launch_latent(const LatentMaps &m, const LatentParams &p, cudaStream_t stream);

// Packed prompts with keys and values expanded from latent vectors
// (pgd_latent_prefill.cu): PrefillParams with a KV head per query head; the queries'
// and keys' own parts and their rotary parts are views of their own.
struct LatentPrefillMaps {
    CUtensorMap q, qr, k, kr, v;
};
constexpr int kLatentVKeys64 = 128, kLatentVKeys128 = 64;  // keys of a V copy, by head_dim
cudaError_t latent_prefill_set_up(int head_dim);
cudaError_t launch_latent_prefill(int head_dim, const LatentPrefillMaps &m, const PrefillParams &p,
                                  int grid, cudaStream_t stream);

// Quantiser of rows into quantised pages (pgd_quantize.cu).
cudaError_t launch_quantize(int head_dim, uint8_t *codes, uint16_t *meta, const uint16_t *src,
                            const int32_t *slots, int rows, int Hkv, int BS, int NB,
                            unsigned *err, cudaStream_t stream);

cudaError_t launch_varlen(int head_dim, bool pairs, const CUtensorMap &tq, const CUtensorMap &tk,
                          const CUtensorMap &tv, const VarlenParams &p, int grid, int reduce_rows,
                          cudaStream_t stream);
constexpr int kVarlenOrderKeys = 1024;  // stage counts the unit sort tells apart

}  // namespace pgd
