/*
 * pgd.h — paged grouped-query attention decode on GB300 (sm_103a).
 *
 * One decode step of attention for a batch of sequences whose keys and
 * values live in a paged fp16 KV cache.  For every sequence s and query
 * head h:
 *
 *     out[s][h][:] = softmax( q[s][h] . K_s^T * scale ) . V_s
 *
 * where K_s, V_s are the seq_lens[s] cached tokens of KV head
 * h / (num_q_heads / num_kv_heads), gathered page by page through the
 * sequence's row of block_tables.
 *
 * Sources (page title, section):
 *   "vllm-metal: hand-written Metal Paged Attention" (cf-1.com):
 *     - "What is Paged Attention": the KV cache is cut into fixed-size pages;
 *       the block_tables page table maps a sequence's logical page to a
 *       physical page.
 *     - "Metal parallel model": work per (partition, KV head, sequence), with
 *       all query heads of one GQA group together so each K/V page is read
 *       once per group.
 *     - "Four speed-up tricks", 1: log2-space online softmax with exp2.
 *     - "Four speed-up tricks", 4: split-KV partitions of 256 or 512 tokens,
 *       partials written as log2-space (max, exp-sum) plus the normalised
 *       partial output, merged by a separate reduce.
 *     - "Dispatch layer": supported GQA geometries (32,8,128), (24,4,256),
 *       (16,2,128), (16,2,256) with block sizes 32/16/8; partition choice
 *       from the GPU's core count; 512 MiB cap on the per-call scratch.
 *     - "Hands-on": diagnostics reporting the partition size last used.
 *   "voxtral.c" (dpshk.com), "Single-token attention kernel": GQA head
 *     mapping (32 query heads onto 8 KV heads), fp16 KV cache.
 *
 * Data layout (all row-major, contiguous; the pages leave it open):
 *   q             [num_seqs][num_q_heads][head_dim]             fp16 (IEEE binary16 bits)
 *   k_cache       [num_blocks][num_kv_heads][block_size][head_dim] fp16
 *   v_cache       [num_blocks][num_kv_heads][block_size][head_dim] fp16
 *   block_tables  [num_seqs][max_blocks_per_seq]                 int32 physical page ids
 *   seq_lens      [num_seqs]                                     int32
 *   out           [num_seqs][num_q_heads][head_dim]             fp32
 * Token t of sequence s is row t % block_size of physical page
 * block_tables[s][t / block_size].  Entries at or past
 * ceil(seq_lens[s] / block_size) are never read, nor are the rows of the
 * last page past the sequence end.  A sequence of length 0 gets an all-zero
 * output row.
 *
 * Supported: head_dim in {64, 128, 256}; block_size in {8, 16, 32, 64, 128};
 * num_q_heads % num_kv_heads == 0 with a group of 1..8 query heads per KV
 * head (this covers the four geometries of the pages, whose block sizes are
 * 8/16/32 and head sizes 128/256, and any other group of at most 8);
 * partition_size in {256, 512} or 0 to let the library choose.  Other cache
 * layouts than the one above: paged_gqa_decode_strided.
 *
 * Memory: every array is device memory owned by the caller.  q, k_cache and
 * v_cache must be 16-byte aligned; the int32 arrays and out 4-byte aligned.
 *
 * A call with num_seqs == 0 checks the sizes, does nothing else and may pass
 * null array pointers.
 *
 * Execution: every call is asynchronous on `stream` (a cudaStream_t; NULL is
 * the legacy default stream) and never synchronises the host.  The call
 * validates all host-side arguments before launching anything; on any error
 * it returns a non-zero status, launches nothing and leaves a message for
 * pgd_last_error().  It never aborts, exits or throws.
 *
 * Device-side checks: a physical page id outside [0, num_blocks) or a
 * sequence length outside [0, max_blocks_per_seq * block_size] found while
 * the kernels run is never dereferenced (the page reads as zeros, the
 * length is clamped) and sets a bit in a per-process device error word;
 * pgd_check_device_error() reports and clears it.
 */
#ifndef PGD_H
#define PGD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pgd_status {
    PGD_OK = 0,
    PGD_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misalignment          */
    PGD_ERR_UNSUPPORTED = 2,  /* valid but not built: head_dim, block size, G  */
    PGD_ERR_WORKSPACE = 3,    /* scratch above the 512 MiB cap, or too small   */
    PGD_ERR_CUDA = 4,         /* a CUDA runtime call failed                    */
    PGD_ERR_DEVICE = 5        /* the kernels flagged bad data (see below)      */
} pgd_status;

/* Bits of the device error word (pgd_check_device_error). */
#define PGD_DEVERR_PAGE_RANGE 1u   /* a page id to be read was outside [0, num_blocks) */
#define PGD_DEVERR_SEQ_LEN 2u      /* a length was < 0 or > max_blocks_per_seq*block_size */
#define PGD_DEVERR_TIMEOUT 4u      /* an internal pipeline wait gave up (never expected)  */

/* Upper bound of the per-call scratch, after the pages' 512 MiB GQA cap. */
#define PGD_MAX_WORKSPACE_BYTES ((size_t)512 << 20)

/*
 * paged_gqa_decode — the decode step described above.
 *
 * scale            multiplies q . k before the softmax (e.g. 1/sqrt(head_dim)).
 * partition_size   tokens per split-KV partition: 256, 512, or 0 for the
 *                  scheduler's choice from the SM count and the length
 *                  bound max_blocks_per_seq * block_size.
 * max_blocks_per_seq  row stride of block_tables; also bounds every length.
 * num_blocks       pages in each cache array (bounds every page id).
 * stream           cudaStream_t to run on.
 *
 * Scratch for the partition partials is taken from a stream-ordered memory
 * pool owned by the library and returned in stream order, so calls on
 * different streams do not share it.  Use paged_gqa_decode_ex to supply it.
 * The pool keeps what it has handed out for the next calls until
 * pgd_release().
 *
 * Work is handed out to the GPU's thread blocks through a 4-byte counter
 * that the library keeps per (device, stream) it has run on; the call
 * leaves it at zero for the next call on that stream.  The counters of a
 * device (1024 of them, 128 bytes apart) are allocated and
 * zeroed by the first call on that device (and by the first call after a
 * pgd_release()): make that call outside any stream capture.
 */
pgd_status paged_gqa_decode(float *out, const uint16_t *q, const uint16_t *k_cache,
                            const uint16_t *v_cache, const int32_t *block_tables,
                            const int32_t *seq_lens, float scale, int num_seqs,
                            int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                            int partition_size, int max_blocks_per_seq, int num_blocks,
                            void *stream);

/*
 * pgd_plan — the partition size a call with these sizes would use (resolving
 * partition_size == 0 on the current device) and the scratch bytes it needs
 * (0 when no sequence can span more than one partition).  Does not launch.
 */
pgd_status pgd_plan(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                    int block_size, int partition_size, int max_blocks_per_seq,
                    int *chosen_partition_size, size_t *workspace_bytes);

/*
 * pgd_workspace_size — bytes of caller scratch (paged_gqa_decode_ex,
 * paged_gqa_decode_strided, paged_gqa_decode_q8*) a decode call with these
 * sizes needs: the partition partials m, l [num_seqs][num_q_heads][NP] and
 * o [num_seqs][num_q_heads][NP][head_dim] fp32, each region 256-byte
 * aligned, NP = ceil(max_blocks_per_seq * block_size / partition_size); 0
 * when NP == 1 ("vllm-metal", "Four speed-up tricks", 4: the partials
 * contract; "Dispatch layer": the per-call scratch and its 512 MiB cap).
 * partition_size 0 (the scheduler's choice, made at call time from the SM
 * count and num_kv_heads, which this call does not take) returns the bytes
 * for 256, which covers either choice.  Pure arithmetic: needs no GPU and
 * launches nothing.  A result above PGD_MAX_WORKSPACE_BYTES means the call
 * itself will be refused with PGD_ERR_WORKSPACE.  Invalid or unsupported
 * sizes return SIZE_MAX with a message for pgd_last_error().  pgd_plan gives
 * the exact figure for a resolved partition size on the current device.
 */
size_t pgd_workspace_size(int num_seqs, int num_q_heads, int head_dim, int block_size,
                          int partition_size, int max_blocks_per_seq);

/*
 * pgd_release — gives back the device memory the library holds on the
 * current device: the scratch pool of the calls without caller scratch
 * (which keeps everything it has handed out, so that the next call does
 * not allocate again) and the claim counters.  It first waits for all work
 * on the device (cudaDeviceSynchronize), so nothing queued still uses them,
 * and clears this thread's cache of tensor-map descriptors (host memory).
 * The next call re-creates what it needs; the library stays usable.
 * Not freed: the fixed array of paged_gqa_decode_noalloc and the device
 * error word, which are part of the library's device image.
 * The caller must make sure no other thread calls the library on this
 * device meanwhile, must not call it during a stream capture, and must not
 * replay CUDA graphs captured before it (they hold the old counters'
 * addresses).  Returns PGD_ERR_CUDA if the wait or a free fails.
 */
pgd_status pgd_release(void);

/*
 * paged_gqa_decode_ex — paged_gqa_decode with caller-owned scratch and an
 * optional page trace.
 *
 * workspace        device memory of at least the bytes pgd_plan reports,
 *                  256-byte aligned; may be NULL when that is 0.  Its
 *                  contents need no initialisation; it must not be used by
 *                  anything else until the call's work on `stream` is done.
 * page_trace       NULL, or int32 device memory [num_seqs][num_kv_heads]
 *                  [max_blocks_per_seq].  For every page the kernel reads it
 *                  stores, at [s][kv_head][logical page], the physical id it
 *                  used to form the address.  Entries it does not read are
 *                  left untouched (fill with -1 beforehand to check that
 *                  nothing past a sequence's last page is read).
 */
pgd_status paged_gqa_decode_ex(float *out, const uint16_t *q, const uint16_t *k_cache,
                               const uint16_t *v_cache, const int32_t *block_tables,
                               const int32_t *seq_lens, float scale, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim,
                               int block_size, int partition_size, int max_blocks_per_seq,
                               int num_blocks, void *workspace, size_t workspace_bytes,
                               int32_t *page_trace, void *stream);

/*
 * paged_gqa_decode_append — the KV-cache append of the decode step fused
 * with the decode: for every sequence s with seq_lens[s] = L >= 1, the newest
 * token's key and value, k_new[s][kv_head][:] and v_new[s][kv_head][:], are
 * written into the cache at token L-1 (row (L-1) % block_size of physical
 * page block_tables[s][(L-1) / block_size], which the caller has allocated),
 * and the decode then attends over all L tokens, the newest one included.
 * One launch: the newest row is taken from k_new / v_new while its page is
 * staged, and written to the cache for the next steps.  (The step before the
 * decode path; "voxtral.c", "Next steps", plans a further fusion of its RoPE-K
 * and KV-cache write path.)
 *
 * k_new, v_new  [num_seqs][num_kv_heads][head_dim] fp16, device, 16-byte
 *               aligned.  Sequences of length 0 append nothing.
 * k_cache, v_cache are written (one row per sequence and KV head); all other
 * arguments as for paged_gqa_decode, whose scratch handling it shares.
 */
pgd_status paged_gqa_decode_append(float *out, const uint16_t *q, const uint16_t *k_new,
                                   const uint16_t *v_new, uint16_t *k_cache, uint16_t *v_cache,
                                   const int32_t *block_tables, const int32_t *seq_lens,
                                   float scale, int num_seqs, int num_q_heads, int num_kv_heads,
                                   int head_dim, int block_size, int partition_size,
                                   int max_blocks_per_seq, int num_blocks, void *stream);

/*
 * paged_gqa_decode_strided — the decode step over a cache in any layout whose
 * rows of head_dim halves are contiguous, with every option of the calls
 * above.  (The pages leave the cache layout open; this is the general form.)
 *
 * The row of token r of physical page b, KV head g starts at element
 *     b * page_stride + g * head_stride + r * token_stride
 * of k_cache and of v_cache (strides in halves: positive multiples of 8,
 * token_stride >= head_dim, each below 2^39).  Examples:
 *   head-major  [num_blocks][num_kv_heads][block_size][head_dim] (the layout of
 *               paged_gqa_decode): (Hkv*BS*D, BS*D, D)
 *   token-major [num_blocks][block_size][num_kv_heads][head_dim]:
 *               (BS*Hkv*D, D, Hkv*D)
 *   padded pages, or K and V interleaved in one allocation: any larger page
 *               stride, with k_cache / v_cache pointing at their first rows.
 * Every (page, head, token) row must lie in memory the caller owns.
 *
 * k_new, v_new  NULL for a plain decode, or both given for the fused append of
 *               paged_gqa_decode_append (rows written at the same strides).
 * workspace     NULL: library scratch, as paged_gqa_decode; otherwise as for
 *               paged_gqa_decode_ex, with workspace_bytes.
 * page_trace    as for paged_gqa_decode_ex (NULL for none).
 * Other arguments as for paged_gqa_decode.
 */
pgd_status paged_gqa_decode_strided(float *out, const uint16_t *q, const uint16_t *k_new,
                                    const uint16_t *v_new, uint16_t *k_cache, uint16_t *v_cache,
                                    const int32_t *block_tables, const int32_t *seq_lens,
                                    float scale, int num_seqs, int num_q_heads, int num_kv_heads,
                                    int head_dim, int block_size, int partition_size,
                                    int max_blocks_per_seq, int num_blocks, int64_t page_stride,
                                    int64_t head_stride, int64_t token_stride, void *workspace,
                                    size_t workspace_bytes, int32_t *page_trace, void *stream);

/*
 * paged_gqa_decode_noalloc — paged_gqa_decode that allocates nothing.
 * (No counterpart on the pages: this entry point exists for callers, not
 * for the method.)
 *
 * For callers that must not allocate device memory while they run: a
 * serving loop whose memory is all reserved up front by its own allocator
 * (a late cudaMalloc could fail or fragment it), code that may not block on
 * an allocation (cudaMalloc and cudaFree can synchronise the device), or
 * code that forbids dynamic allocation after start-up.  The caller still
 * passes every input and the output, exactly as for paged_gqa_decode.
 *
 * The partition partials go to a fixed array of PGD_NOALLOC_SCRATCH_BYTES
 * compiled into the library (every GPU on which the library is used holds
 * it until the process exits); its first 256 bytes hold this entry point's
 * work counter, zero at load and left at zero by every call.  The call never
 * calls cudaMalloc, cudaFree or any other allocating routine.  Sizes whose
 * partials need more than the rest of the array (pgd_plan's figure above
 * PGD_NOALLOC_SCRATCH_BYTES - 256) are rejected with PGD_ERR_WORKSPACE before
 * any launch.
 *
 * The first call on a device looks up the array's device address with that
 * device current; make that first call before any stream capture.  (A
 * failed lookup is not kept: the next call tries again.)
 * Every call shares the one array: calls whose work overlaps on the GPU
 * (other streams, other threads) race on it, so serialise them.  The array
 * keeps the last call's contents; the partials need no initial value
 * (every partial is written before it is read within a call).  The work
 * counter must read zero at launch: every call leaves it at zero, and a
 * call that fails after its partition kernel may have started makes the
 * next call zero it first, in stream order, with cudaMemsetAsync on the
 * array itself (no allocation).
 */
#define PGD_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

pgd_status paged_gqa_decode_noalloc(float *out, const uint16_t *q, const uint16_t *k_cache,
                                    const uint16_t *v_cache, const int32_t *block_tables,
                                    const int32_t *seq_lens, float scale, int num_seqs,
                                    int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int partition_size, int max_blocks_per_seq,
                                    int num_blocks, void *stream);

/*
 * paged_gqa_decode_host — the decode step for a caller whose per-step inputs
 * live in host memory: the page tables and lengths that a host-side block
 * manager and scheduler produce each step ("vllm-metal", introduction: the
 * serving framework above the attention path owns the scheduler and the
 * paged block manager), and the step's queries.  The K/V cache stays
 * resident on the device.
 *
 * q_host, block_tables_host, seq_lens_host  host memory, layouts as for
 *              paged_gqa_decode (read); out_host  host memory (written).
 *              Page-locked host memory (cudaHostAlloc / cudaHostRegister)
 *              lets the copies run as direct transfers; pageable memory also
 *              works, through the driver's bounce buffer.
 * k_cache, v_cache  device, as for paged_gqa_decode.
 * staging      device memory of at least pgd_host_staging_bytes() bytes,
 *              256-byte aligned, caller-owned: the device copies of q,
 *              block_tables, seq_lens and out.  It must not be used by
 *              anything else until the call returns.
 * The call copies the inputs to `staging` on `stream`, runs the decode there
 * (partition partials from the library's scratch pool, as paged_gqa_decode),
 * copies the output back and waits for `stream`: when it returns PGD_OK,
 * out_host holds the result.  Validation and error reporting as for
 * paged_gqa_decode; a failed copy or wait returns PGD_ERR_CUDA.
 */
pgd_status paged_gqa_decode_host(float *out_host, const uint16_t *q_host,
                                 const int32_t *block_tables_host, const int32_t *seq_lens_host,
                                 const uint16_t *k_cache, const uint16_t *v_cache, float scale,
                                 int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, int partition_size, int max_blocks_per_seq,
                                 int num_blocks, void *staging, size_t staging_bytes,
                                 void *stream);

/* Bytes of device staging paged_gqa_decode_host needs for these sizes (q,
 * block_tables, seq_lens and out, each region 256-byte aligned); SIZE_MAX
 * for invalid sizes.  Needs no GPU. */
size_t pgd_host_staging_bytes(int num_seqs, int num_q_heads, int head_dim,
                              int max_blocks_per_seq);

/*
 * paged_gqa_decode_q8 — the decode step over quantised pages: the affine
 * group format of the Kapitsa series (blog.hacking.pub, part 02, "how
 * weights are stored": a value is scale * q + bias with an unsigned integer
 * code q and one bf16 (scale, bias) pair per group of values), with 8-bit
 * codes and groups of 64 consecutive head_dim values of one token row.
 * About 53 % of the fp16 bytes at head_dim 128.
 *
 * k_codes, v_codes  [num_blocks][num_kv_heads][block_size][head_dim] uint8,
 *                   16-byte aligned
 * k_meta, v_meta    [num_blocks][num_kv_heads][block_size][head_dim / 64][2]
 *                   bf16 bit patterns (scale, bias), 16-byte aligned
 * The row of token t is dequantised as scale_g * code + bias_g for element d
 * in group g = d / 64; the decode is then that of paged_gqa_decode over the
 * dequantised rows (the affine map is applied in fp32 around exact fp16
 * tensor-core products of the codes; nothing is rounded to fp16 that the
 * fp16 path does not round).  Other arguments as for paged_gqa_decode_ex
 * (workspace NULL: library scratch).  head_dim 128 or 256 only; the fused
 * append is paged_gqa_decode_q8_append.
 */
pgd_status paged_gqa_decode_q8(float *out, const uint16_t *q, const uint8_t *k_codes,
                               const uint16_t *k_meta, const uint8_t *v_codes,
                               const uint16_t *v_meta, const int32_t *block_tables,
                               const int32_t *seq_lens, float scale, int num_seqs,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               int partition_size, int max_blocks_per_seq, int num_blocks,
                               void *workspace, size_t workspace_bytes, int32_t *page_trace,
                               void *stream);

/*
 * paged_gqa_decode_q8_strided — paged_gqa_decode_q8 (and, with k_new / v_new
 * given, paged_gqa_decode_q8_append) over quantised pages in any layout:
 * the codes of token r of page b, KV head g start at byte
 * b*code_page_stride + g*code_head_stride + r*code_token_stride (positive
 * multiples of 16 below 2^39, token stride >= head_dim), their head_dim / 64
 * (scale, bias) pairs at bf16 element b*meta_page_stride + g*meta_head_stride
 * + r*meta_token_stride (positive multiples of head_dim / 32 below 2^38).
 * k_new, v_new: both NULL (no append) or both given.  workspace NULL:
 * library scratch.  No page trace.
 */
pgd_status paged_gqa_decode_q8_strided(
    float *out, const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new, uint8_t *k_codes,
    uint16_t *k_meta, uint8_t *v_codes, uint16_t *v_meta, const int32_t *block_tables,
    const int32_t *seq_lens, float scale, int num_seqs, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, int partition_size, int max_blocks_per_seq, int num_blocks,
    int64_t code_page_stride, int64_t code_head_stride, int64_t code_token_stride,
    int64_t meta_page_stride, int64_t meta_head_stride, int64_t meta_token_stride,
    void *workspace, size_t workspace_bytes, void *stream);

/*
 * paged_kv_quantize — writes fp16 rows into quantised pages (the format of
 * paged_gqa_decode_q8).  The pages show the affine format only from the
 * reading side (Kapitsa part 02: value = scale * q + bias); the quantiser
 * here is the plainest reading for unsigned 8-bit codes, per group of 64
 * values of a row, every step one correctly rounded binary32 operation:
 *     bias  = bf16(min),  scale = bf16((max - min) / 255)   (nearest, ties even)
 *     code  = scale > 0 ? clamp(rint((x - bias) / scale), 0, 255) : 0
 * src    [num_rows][num_kv_heads][head_dim] fp16, 16-byte aligned (read)
 * slots  [num_rows] int32: cache row page * block_size + row of each source
 *        row (all KV heads); negative: the row is skipped
 * codes  [num_blocks][num_kv_heads][block_size][head_dim] uint8 (written)
 * meta   [num_blocks][num_kv_heads][block_size][head_dim / 64][2] bf16 (written)
 * Asynchronous on `stream`.  A slot whose page is at or past num_blocks is
 * skipped and sets PGD_DEVERR_PAGE_RANGE.  Call once for K, once for V.
 */
pgd_status paged_kv_quantize(uint8_t *codes, uint16_t *meta, const uint16_t *src,
                             const int32_t *slots, int num_rows, int num_kv_heads, int head_dim,
                             int block_size, int num_blocks, void *stream);

/*
 * paged_gqa_decode_q8_append — paged_gqa_decode_q8 with the step's new K/V
 * fused in: k_new / v_new [num_seqs][num_kv_heads][head_dim] fp16 (16-byte
 * aligned) are the newest token of each sequence (position seq_lens[s] - 1,
 * in page block_tables[s][(seq_lens[s] - 1) / block_size]).  The kernel
 * quantises them (paged_kv_quantize's steps), uses them in this step's
 * attention and writes their codes and (scale, bias) pairs into the caches
 * for the next steps.  Other arguments as paged_gqa_decode_q8 (library
 * scratch, no page trace).
 */
pgd_status paged_gqa_decode_q8_append(float *out, const uint16_t *q, const uint16_t *k_new,
                                      const uint16_t *v_new, uint8_t *k_codes, uint16_t *k_meta,
                                      uint8_t *v_codes, uint16_t *v_meta,
                                      const int32_t *block_tables, const int32_t *seq_lens,
                                      float scale, int num_seqs, int num_q_heads,
                                      int num_kv_heads, int head_dim, int block_size,
                                      int partition_size, int max_blocks_per_seq, int num_blocks,
                                      void *stream);

/*
 * paged_gqa_varlen — attention for several query tokens per sequence over the
 * paged cache: the unified paged variable-length form of "vllm-metal"
 * (introduction and "Three Metal kernels": prefill chunks, decode steps and
 * the verification step of speculative decoding in one call).  A decode step
 * is the case of one query token per sequence.
 *
 * Sequence s has n_s = cu_seqlens_q[s+1] - cu_seqlens_q[s] query tokens, rows
 * cu_seqlens_q[s] .. cu_seqlens_q[s+1]-1 of q; they are its newest n_s cached
 * tokens (their K and V already written to the cache), so query i sits at
 * position seq_lens[s] - n_s + i and attends every cached token t up to and
 * including that position (causal).  For every query row r and head h:
 *     out[r][h][:] = softmax( q[r][h] . K^T * scale over t <= pos ) . V
 *
 * q             [total_q][num_q_heads][head_dim] fp16, 16-byte aligned
 * cu_seqlens_q  [num_seqs + 1] int32, cu[0] = 0, non-decreasing, cu[S] = total_q
 * out           [total_q][num_q_heads][head_dim] fp32, written
 * max_q_len     bound on every n_s (sizes the launch)
 * cache arrays, strides, block_tables, seq_lens, scale: as for
 *               paged_gqa_decode_strided.
 * kv_partition  tokens per split-KV partition: 0 lets the library choose
 *               (no split when the query tiles alone fill the GPU), else a
 *               multiple of 128 (head_dim 64, 128) or 64 (head_dim 256).
 * workspace     NULL: library scratch; else at least pgd_varlen_plan's bytes,
 *               256-byte aligned.
 *
 * Supported: head_dim 64/128/256, block sizes 8..128, groups of up to 128
 * query heads per KV head.  Calls with head_dim <= 128, kv_partition 0, 256
 * or 512 and at most 8 (query token, head) rows per (sequence, KV head)
 * (max_q_len x group <= 8: decode steps, short verification steps) run on
 * the decode's persistent partition kernel, an HBM-bound scan; the rest on
 * the tcgen05 tensor cores.  Device-side
 * checks as for the decode: a sequence whose n_s is negative, above its
 * length or above max_q_len sets PGD_DEVERR_QUERY_LEN and is skipped (its
 * output rows are not written).
 */
#define PGD_DEVERR_QUERY_LEN 8u

pgd_status paged_gqa_varlen(float *out, const uint16_t *q, const int32_t *cu_seqlens_q,
                            const uint16_t *k_cache, const uint16_t *v_cache,
                            const int32_t *block_tables, const int32_t *seq_lens, float scale,
                            int num_seqs, int total_q, int max_q_len, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size,
                            int max_blocks_per_seq, int num_blocks, int64_t page_stride,
                            int64_t head_stride, int64_t token_stride, int kv_partition,
                            void *workspace, size_t workspace_bytes, void *stream);

/* The KV partition a paged_gqa_varlen call with these sizes would use and the
 * scratch bytes it needs: the split-KV partials, and when the work units are
 * pairs of query tiles (head_dim 64/128, max_q_len above one tile of
 * 128/G tokens) and outnumber the SMs, a 4-byte entry per unit for their
 * longest-first order (0: no scratch).  Does not launch. */
pgd_status pgd_varlen_plan(int num_seqs, int total_q, int max_q_len, int num_q_heads,
                           int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                           int kv_partition, int *chosen_kv_partition, size_t *workspace_bytes);

/*
 * paged_gqa_tree — attention of trees of drafted tokens over the paged cache:
 * the verification step of speculative decoding with more than one
 * continuation per sequence.  Arguments, layouts and checks are those of
 * paged_gqa_varlen without kv_partition (one row of q per drafted token, K and V
 * of all of them already in the cache as the sequence's newest n_s tokens, in
 * row order); what a row sees is not every earlier token but the tokens before
 * the tree, its ancestors and itself:
 *     out[r][h][:] = softmax( q[r][h] . K^T * scale over t < seq_lens[s] - n_s,
 *                             the ancestors of r, and r ) . V
 *
 * parents    [total_q] int32: the node of the same sequence's tree (0 .. n_s-1)
 *            that row r continues, an earlier one; any negative value: none (a
 *            continuation of the sequence itself).  A value that is not an
 *            earlier node counts as none and sets PGD_DEVERR_TREE.
 * out        [total_q][num_q_heads][head_dim], 16-byte aligned
 * out_type   PGD_OUT_F32 or PGD_OUT_F16 (the fp32 result rounded to nearest).
 *            In both, the weights are rounded to fp16 before they multiply V:
 *            by 2^-11 of themselves at most, or, below 2^-21 of the row's
 *            largest, by 2^-32 of that; sums are fp32.
 * max_q_len  bound on every n_s, at most PGD_TREE_MAX_NODES.  It sizes the launch:
 *            at head_dim 128 and 256 a bound above 128 / (num_q_heads /
 *            num_kv_heads) nodes has two SMs work on each unit, of which one
 *            has nothing to do where all trees are smaller (64 trees of 8
 *            nodes over 512 to 4096 tokens, 32 / 8 heads x 128: 101 us with 8,
 *            193 us with 256).
 * workspace  NULL: library scratch; else at least pgd_tree_plan's bytes, 256-byte
 *            aligned, not used by anything else until the call's work is done.
 *
 * parents[i] = i - 1 is paged_gqa_varlen's causal form.  A sequence whose length
 * is negative or past its table (PGD_DEVERR_SEQ_LEN) or whose query rows are
 * inconsistent (PGD_DEVERR_QUERY_LEN, also where they do not lie inside
 * total_q) is skipped, its rows are not written; rows behind the last sequence
 * (total_q above cu_seqlens_q[num_seqs], a padded batch) are left as they were.
 * A query row of NaN gives NaN.  K and V rows
 * of one sequence's tree must be finite: a weight of 0 does not hide an
 * infinity or NaN in a sibling's V.  out must not overlap an input.  Library
 * scratch, where there is any, is per call (also in a captured graph), and
 * there is no state between calls: calls on different streams and replays of
 * different graphs may overlap.
 */
#define PGD_OUT_F32 0
#define PGD_OUT_F16 1
#define PGD_TREE_MAX_NODES 256
#define PGD_DEVERR_TREE 32u

pgd_status paged_gqa_tree(void *out, int out_type, const uint16_t *q, const int32_t *cu_seqlens_q,
                          const int32_t *parents, const uint16_t *k_cache, const uint16_t *v_cache,
                          const int32_t *block_tables, const int32_t *seq_lens, float scale,
                          int num_seqs, int total_q, int max_q_len, int num_q_heads,
                          int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                          int num_blocks, int64_t page_stride, int64_t head_stride,
                          int64_t token_stride, void *workspace, size_t workspace_bytes,
                          void *stream);

/* Scratch bytes a paged_gqa_tree call with these sizes needs on the current
 * device: the pieces of the units that its even division of the work cuts (at
 * most 45 MB, whatever the batch). */
pgd_status pgd_tree_plan(int num_seqs, int total_q, int max_q_len, int num_q_heads,
                         int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                         size_t *workspace_bytes);

/*
 * packed_gqa_prefill — causal attention over whole packed prompts, before
 * their K and V are in any cache: q, k and v as the step's projections leave
 * them.  (paged_gqa_varlen is the form for chunks behind cached tokens.)
 *
 * Prompt s is the rows cu_seqlens[s] .. cu_seqlens[s+1]-1 of q, k and v alike;
 * for its row at position t and head h, which reads KV head
 * h / (num_q_heads / num_kv_heads):
 *     out[row][h][:] = softmax( q[row][h] . K^T * scale over positions <= t ) . V
 *
 * q            [total][num_q_heads][head_dim], k, v [total][num_kv_heads]
 *              [head_dim] fp16, 16-byte aligned, each with its own token and
 *              head stride (halves, positive multiples of 8): slices of one
 *              fused projection's output need no copy
 * cu_seqlens   [num_seqs + 1] int32, non-decreasing
 * out          [total][num_q_heads][head_dim] contiguous, 16-byte aligned
 * out_type     PGD_OUT_F32 or PGD_OUT_F16 (rounded to nearest).  The weights
 *              are rounded to fp16 before they multiply V, in both, as in
 *              paged_gqa_tree; sums are fp32.
 * max_len      bound on every prompt's length
 * workspace    NULL: library scratch (per call, also in a captured graph);
 *              else at least pgd_prefill_plan's bytes, 256-byte aligned, not
 *              used by anything else until the call's work is done
 *
 * head_dim 64/128/256, groups of up to 128 query heads; out must not overlap
 * an input.  Rows that belong to no prompt are left as they were (not written).  A prompt that is longer than
 * max_len, has a negative length or does not lie inside total is skipped and
 * sets PGD_DEVERR_QUERY_LEN.  Other prompts' rows may hold anything; within
 * one prompt an infinity or NaN in V is not hidden from earlier rows of the same
 * 128 keys by their weight of 0.  A query row of NaN gives NaN.
 */
pgd_status packed_gqa_prefill(void *out, int out_type, const uint16_t *q, const uint16_t *k,
                              const uint16_t *v, const int32_t *cu_seqlens, float scale,
                              int num_seqs, int total, int max_len, int num_q_heads,
                              int num_kv_heads, int head_dim, int64_t q_token_stride,
                              int64_t q_head_stride, int64_t k_token_stride,
                              int64_t k_head_stride, int64_t v_token_stride,
                              int64_t v_head_stride, void *workspace, size_t workspace_bytes,
                              void *stream);

/* Scratch bytes a packed_gqa_prefill call with these sizes needs (the list of
 * its work units, longest first).  Pure arithmetic. */
pgd_status pgd_prefill_plan(int num_seqs, int total, int num_q_heads, int num_kv_heads,
                            int head_dim, size_t *workspace_bytes);

/*
 * paged_kv_slots — a step's page tables, slots, positions and lengths from the
 * requests' token counts, on the GPU: what paged_kv_write / paged_kv_quantize
 * (slots) and paged_gqa_varlen / paged_gqa_tree (cu_seqlens_q, seq_lens,
 * block_tables) of the same step take.  ("vllm-metal", introduction: the paged
 * block manager above the attention path.)
 *
 * Request s has context_lens[s] cached tokens on the first owned_s =
 * ceil(context_lens[s] / block_size) pages of its row of block_tables, and gets
 * query_lens[s] more.  The pages it lacks are taken from the list of free
 * pages, request by request from entry *free_start on, and entered in its row:
 *     cu_seqlens_q[s]  = sum of query_lens[0 .. s-1]        (num_seqs + 1 values)
 *     seq_lens[s]      = context_lens[s] + query_lens[s]
 *     *free_end        = *free_start + the pages taken
 * and for row r = cu_seqlens_q[s] + i, which is token t = context_lens[s] + i:
 *     positions[r]     = t   (the row's place in the cache: a prompt's rows are
 *                        rotated by it, the nodes of a drafted tree are not, whose
 *                        rotary position is context_lens[s] + the node's depth)
 *     slots[r]         = block_tables[s][t / block_size] * block_size + t % block_size
 * Rows behind the last request, up to num_rows (a launch padded to a fixed row
 * count), get slot and position -1, which the writing calls skip.
 *
 * slots, positions  [num_rows] int32, written (positions may be NULL)
 * cu_seqlens_q      [num_seqs + 1], seq_lens [num_seqs], free_end [1]: written
 * block_tables      [num_seqs][max_blocks_per_seq]: entries below owned_s are
 *                   read (those of the rows' pages), the new ones written, no
 *                   other touched
 * context_lens, query_lens  [num_seqs]; free_pages [num_free]; free_start [1] or
 *                   NULL (0): read.
 * No array that is written may overlap another one (PGD_ERR_INVALID_ARG).
 * The result depends on the arguments alone (the same pages every time), so a
 * call may be repeated or replayed before its counts are advanced.
 *
 * num_seqs up to PGD_SLOTS_MAX_SEQS, num_blocks * block_size up to 2^31.
 * Device-side checks, each with what the call does instead: a negative count
 * counts as 0 (PGD_DEVERR_SEQ_LEN / PGD_DEVERR_QUERY_LEN); tokens past the
 * table's max_blocks_per_seq * block_size get slot -1 and seq_lens is clamped
 * (PGD_DEVERR_SEQ_LEN); rows that do not fit in num_rows are left out, of
 * cu_seqlens_q and seq_lens too (PGD_DEVERR_QUERY_LEN); where the list runs out
 * the entries and slots are -1 and *free_end counts what was needed
 * (PGD_DEVERR_NO_PAGE); a page id outside [0, num_blocks) gives slot -1
 * (PGD_DEVERR_PAGE_RANGE).
 */
#define PGD_DEVERR_NO_PAGE 16u
#define PGD_SLOTS_MAX_SEQS 16384

pgd_status paged_kv_slots(int32_t *slots, int32_t *positions, int32_t *cu_seqlens_q,
                          int32_t *seq_lens, int32_t *free_end, int32_t *block_tables,
                          const int32_t *context_lens, const int32_t *query_lens,
                          const int32_t *free_pages, const int32_t *free_start, int num_seqs,
                          int num_rows, int num_free, int block_size, int max_blocks_per_seq,
                          int num_blocks, void *stream);

/*
 * paged_kv_write — writes fp16 K and V rows into their pages, the fp16
 * counterpart of paged_kv_quantize (K and V in one call): prompt chunks,
 * drafted tokens, or the accepted ones of a verified tree at their final
 * places.
 *
 * k_new, v_new  the rows: head h of row n at element n * src_token_stride +
 *               h * src_head_stride (head_dim contiguous halves; strides in
 *               halves, positive multiples of 8: slices of a fused projection's
 *               output need no copy), 16-byte aligned, read
 * slots         [num_rows] int32 as paged_kv_slots gives them: page *
 *               block_size + row; negative: the row is skipped
 * k_cache, v_cache  written at the strides of paged_gqa_decode_strided; no other
 *               row of the cache is touched
 * Slots must differ from one another (of two rows with one slot, which one
 * stays, or pieces of both, is not defined), and the source must not overlap
 * the rows written.  A slot whose page is at or past num_blocks is skipped and
 * sets PGD_DEVERR_PAGE_RANGE.  Asynchronous on `stream`, no scratch.
 */
pgd_status paged_kv_write(uint16_t *k_cache, uint16_t *v_cache, const uint16_t *k_new,
                          const uint16_t *v_new, const int32_t *slots, int num_rows,
                          int num_kv_heads, int head_dim, int block_size, int num_blocks,
                          int64_t page_stride, int64_t head_stride, int64_t token_stride,
                          int64_t src_token_stride, int64_t src_head_stride, void *stream);

/* The same with strides of their own for k_new and v_new, as packed_gqa_prefill
 * takes them. */
pgd_status paged_kv_write_strided(uint16_t *k_cache, uint16_t *v_cache, const uint16_t *k_new,
                                  const uint16_t *v_new, const int32_t *slots, int num_rows,
                                  int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                  int64_t page_stride, int64_t head_stride, int64_t token_stride,
                                  int64_t k_token_stride, int64_t k_head_stride,
                                  int64_t v_token_stride, int64_t v_head_stride, void *stream);

/*
 * paged_rope_write — the rotary positions of a step's queries and keys, with the
 * write of its K and V rows into their pages (paged_kv_write), in one launch.
 *
 * For row n at position t = positions[n], the first rotary_dim values of every
 * query and key head are turned pair by pair, pair i by the angle t * inv_freq[i]:
 *     (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
 * where a, b are values i and i + rotary_dim / 2 of the head (interleaved 0) or 2i
 * and 2i + 1 (interleaved non-zero); its other values are copied as they are.  The
 * turned keys and the values go to cache row slots[n], the turned queries to q_out.
 * The angle's place on the circle is off by 1.1e-7 radians at most, whatever the
 * position, and by position * (|f| 2^-52 + 2 pi 2^-64) more (f below 0: 2^-54 in
 * 2^-64's place), which for |f| up to 1 reaches as much from positions of 3 x 10^8 on:
 * a token far out in a long context costs no accuracy.  Arithmetic is fp32, rounded once to fp16.
 *
 * Turned keys as rows, as the prompt operators and paged_kv_quantize take them: give
 * the key heads as further query heads (q over the query and key heads of one
 * projection, k_new its key heads, q_out a tensor of its own).
 *
 * q, q_out      [num_rows][num_q_heads][head_dim] fp16 at token and head strides of
 *               their own; q_out may be q itself, with the same strides (the values
 *               behind rotary_dim are then not touched).  It shares no memory with any
 *               other array of the call, keys that q reaches over among them, and its rows
 *               none with one another (PGD_ERR_INVALID_ARG).  Both NULL with num_q_heads
 *               0: keys alone.
 * k_new, v_new  [num_rows][num_kv_heads][head_dim], strides of their own (all four
 *               in halves, positive multiples of 8), 16-byte aligned, read
 * slots         [num_rows] int32 as for paged_kv_write; negative: the row is not
 *               written to the cache (its queries are turned all the same)
 * positions     [num_rows] int32, 0 .. 2^31 - 1, independent of the slot (a node of a
 *               drafted tree is turned by its depth in it); negative: a row of
 *               padding, of which nothing is read or written
 * inv_freq      [rotary_dim / 2] fp32, device, finite: radians a position of each
 *               pair (pgd_rope_frequencies makes the usual tables, long contexts'
 *               among them)
 * rotary_dim    a multiple of 16 up to head_dim
 * num_rows      below 2^30
 * k_cache, v_cache, strides, device checks: as for paged_kv_write.
 */
pgd_status paged_rope_write(uint16_t *k_cache, uint16_t *v_cache, uint16_t *q_out,
                            const uint16_t *q, const uint16_t *k_new, const uint16_t *v_new,
                            const int32_t *slots, const int32_t *positions,
                            const float *inv_freq, float magnitude, int interleaved, int num_rows,
                            int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                            int block_size, int num_blocks, int64_t page_stride,
                            int64_t head_stride, int64_t token_stride, int64_t q_out_token_stride,
                            int64_t q_out_head_stride, int64_t q_token_stride,
                            int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                            int64_t v_token_stride, int64_t v_head_stride, void *stream);

/*
 * pgd_rope_frequencies — a table of inverse frequencies (host memory, rotary_dim / 2
 * values) for paged_rope_write and paged_latent_write, and the magnitude that goes
 * with it.  base^(-2i / rotary_dim), and for contexts longer than the trained one
 * by `factor` (>= 1):
 *   PGD_ROPE_PLAIN     as it is
 *   PGD_ROPE_LINEAR    positions shrunk: every frequency divided by factor
 *   PGD_ROPE_BASE      the base raised to base * factor^(rotary_dim / (rotary_dim - 2)):
 *                      the highest frequency stays, the lowest shrinks by factor
 *   PGD_ROPE_BY_PARTS  pairs that turn more than beta_fast times in original_len tokens
 *                      stay, those that turn less than beta_slow times shrink by factor,
 *                      those between in proportion to their index; magnitude 0.1 ln(factor) + 1
 *                      ("YaRN", Peng et al. 2023, section 3)
 * original_len, beta_fast > beta_slow > 0 matter to BY_PARTS alone.  Arithmetic in
 * 64 bits, rounded once.  rotary_dim is even, 4 to 65536, base above 1.  *magnitude (if
 * not NULL) is 1 but for BY_PARTS.  Needs no GPU.
 */
#define PGD_ROPE_PLAIN 0
#define PGD_ROPE_LINEAR 1
#define PGD_ROPE_BASE 2
#define PGD_ROPE_BY_PARTS 3

pgd_status pgd_rope_frequencies(float *inv_freq, float *magnitude, int rotary_dim, double base,
                                int scaling, double factor, double original_len, double beta_fast,
                                double beta_slow);

/*
 * A latent cache holds one row a token for all heads: latent_dim values, from which
 * every head's key and value follow by a projection, and behind them rope_dim values
 * of one rotated key that all heads share.
 *   cache   [num_blocks][block_size][latent_dim + rope_dim] fp16, page and token
 *           strides in halves (positive multiples of 8 below 2^39, token_stride >=
 *           latent_dim + rope_dim), 16-byte aligned
 * Page tables, slots and lengths are those of the other caches (paged_kv_slots).
 * latent_dim 128, 256 or 512, rope_dim 32 or 64, block sizes 8 to 128.
 *
 * paged_latent_write — a step's rows into a latent cache: row n's latent vector as
 * it is and its key turned by its position, to cache row slots[n]; the queries'
 * rotary parts turned into q_out.  The rotation, slots, positions, inv_freq (rope_dim
 * / 2 values) and q_out's rules are those of paged_rope_write, with all of rope_dim
 * turned.  The turned key as rows (packed_latent_prefill): a second call with k_rope
 * as the one query head and negative slots, which writes nothing else.
 *
 * latent        [num_rows][latent_dim], k_rope [num_rows][rope_dim] fp16, each with
 *               its own token stride: slices of one projection's output need no copy
 * q_rope, q_out [num_rows][num_heads][rope_dim] fp16 at strides of their own, or both
 *               NULL with num_heads 0
 */
pgd_status paged_latent_write(uint16_t *cache, uint16_t *q_out, const uint16_t *q_rope,
                              const uint16_t *latent, const uint16_t *k_rope,
                              const int32_t *slots, const int32_t *positions,
                              const float *inv_freq, float magnitude, int interleaved,
                              int num_rows, int num_heads, int latent_dim, int rope_dim,
                              int block_size, int num_blocks, int64_t page_stride,
                              int64_t token_stride, int64_t q_out_token_stride,
                              int64_t q_out_head_stride, int64_t q_token_stride,
                              int64_t q_head_stride, int64_t latent_token_stride,
                              int64_t k_rope_token_stride, void *stream);

/*
 * paged_latent_attention — attention over a latent cache with the queries taken
 * through the keys' projection beforehand (the absorbed form): every head reads the
 * same rows, and a row's latent part is its key and its value.  With c_t the latent
 * part and k_t the rotated key of cached token t, for query row r and head h:
 *     out[r][h][:] = sum_t w_t c_t,
 *     w = softmax( (q[r][h] . c_t + q_rope[r][h] . k_t) * scale )
 * The caller takes out through the values' projection.
 *
 * Sequence s has the query rows cu_seqlens_q[s] .. cu_seqlens_q[s+1]-1, its newest
 * tokens, already in the cache, causal among themselves (as in paged_gqa_varlen).
 * cu_seqlens_q NULL: a decode step, one row a sequence (total_q == num_seqs), which
 * sees all of seq_lens[s] tokens; a sequence of length 0 gets zeros.  Every tile of a
 * sequence's rows runs over all of its tokens, also those that its rows do not see: a
 * chunk of n rows behind c tokens takes (c + n) / (c + n / 2) times the work it needs
 * (4096 rows: twice with nothing before them, 1.2 times behind 8192).
 *
 * out        [total_q][num_heads][latent_dim], contiguous, 16-byte aligned;
 *            out_type PGD_OUT_F32 or PGD_OUT_F16 (rounded to nearest).  The weights
 *            are rounded to fp16 before they multiply the rows, in both, as in
 *            paged_gqa_tree; sums are fp32.
 * q          [total_q][num_heads][latent_dim], q_rope [total_q][num_heads][rope_dim]
 *            fp16, 16-byte aligned, each with its own token and head strides (halves,
 *            positive multiples of 8 below 2^39): parts of one tensor, or a batched
 *            product's output [num_heads][total_q][latent_dim], need no copy
 * max_q_len  bound on every sequence's query rows (1 with cu_seqlens_q NULL)
 * total_q    the sequences' rows do not overlap.  What they come to in tiles of 128 rows
 *            (of queries x heads; one begun in each sequence), times the table's stages
 *            of 128 tokens, is to stay below 2^29 (PGD_ERR_UNSUPPORTED).  Where offsets
 *            that decrease ask for more all the same, nothing is written
 *            (PGD_DEVERR_QUERY_LEN)
 * workspace  NULL: library scratch (per call, also in a captured graph); else at
 *            least pgd_latent_plan's bytes, 256-byte aligned, not used by anything
 *            else until the call's work is done
 *
 * A sequence whose length is negative or past its table (PGD_DEVERR_SEQ_LEN) or
 * whose query rows are inconsistent (PGD_DEVERR_QUERY_LEN) is skipped, its rows are
 * not written; rows behind the last sequence are left as they were.  A page id
 * outside [0, num_blocks) reads as zeros (PGD_DEVERR_PAGE_RANGE).  A query row of NaN
 * gives NaN, and so does a score of +infinity; scores that are all -infinity give
 * zeros.  The cached rows of one sequence's own query tokens must be finite: a
 * weight of 0 does not hide an infinity or NaN in a later one.  out must not overlap
 * an input.
 */
pgd_status paged_latent_attention(void *out, int out_type, const uint16_t *q,
                                  const uint16_t *q_rope, const int32_t *cu_seqlens_q,
                                  const uint16_t *cache, const int32_t *block_tables,
                                  const int32_t *seq_lens, float scale, int num_seqs, int total_q,
                                  int max_q_len, int num_heads, int latent_dim, int rope_dim,
                                  int block_size, int max_blocks_per_seq, int num_blocks,
                                  int64_t page_stride, int64_t token_stride,
                                  int64_t q_token_stride, int64_t q_head_stride,
                                  int64_t q_rope_token_stride, int64_t q_rope_head_stride,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Scratch bytes a paged_latent_attention call with these sizes needs on the current
 * device: the pieces of the units that its even division of the work cuts. */
pgd_status pgd_latent_plan(int num_seqs, int total_q, int max_q_len, int num_heads,
                           int latent_dim, int rope_dim, int block_size, int max_blocks_per_seq,
                           size_t *workspace_bytes);

/*
 * packed_latent_prefill — causal attention over whole packed prompts whose keys and
 * values have been expanded from their latent vectors (the expanded form), before or
 * beside the latent cache's write: each head has keys of its own and, behind them,
 * the one rotated key of the token that all heads share.
 *     out[row][h][:] = softmax( (q[row][h] . [k[t][h] | k_rope[t]]) * scale
 *                               over positions t up to the row's ) . v[t][h]
 *
 * q        [total][num_heads][head_dim + rope_dim], k, v [total][num_heads][head_dim],
 *          k_rope [total][rope_dim] fp16, 16-byte aligned, strides of their own
 *          (halves, positive multiples of 8 below 2^39): halves of the up projection's
 *          output and a slice of the down projection's need no copy
 * out      [total][num_heads][head_dim] contiguous, 16-byte aligned
 * head_dim 64 or 128, rope_dim 32 or 64.  cu_seqlens, max_len, out_type, workspace
 * (pgd_latent_prefill_plan) and the rules on other rows, lengths, NaN and overlaps are
 * those of packed_gqa_prefill.
 */
pgd_status packed_latent_prefill(void *out, int out_type, const uint16_t *q, const uint16_t *k,
                                 const uint16_t *k_rope, const uint16_t *v,
                                 const int32_t *cu_seqlens, float scale, int num_seqs, int total,
                                 int max_len, int num_heads, int head_dim, int rope_dim,
                                 int64_t q_token_stride, int64_t q_head_stride,
                                 int64_t k_token_stride, int64_t k_head_stride,
                                 int64_t k_rope_token_stride, int64_t v_token_stride,
                                 int64_t v_head_stride, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* Scratch bytes a packed_latent_prefill call with these sizes needs.  Pure arithmetic. */
pgd_status pgd_latent_prefill_plan(int num_seqs, int total, int num_heads, int head_dim,
                                   int rope_dim, size_t *workspace_bytes);

/* Partition size used by this thread's last successful call (0 if none);
 * the diagnostic of the pages' "Hands-on" section. */
int pgd_last_partition_size(void);

/* Message for this thread's last failed call ("" if none). */
const char *pgd_last_error(void);

/*
 * pgd_check_device_error — waits for `stream`, then reads and clears the
 * device error word of the current device.  *bits (if not NULL) receives the
 * PGD_DEVERR_* bits set since the last check.  Returns PGD_ERR_DEVICE if any
 * bit was set, PGD_ERR_CUDA if the wait itself failed, PGD_OK otherwise.
 */
pgd_status pgd_check_device_error(void *stream, unsigned *bits);

/*
 * pgd_test_stall_next_decode — failure-detection test knob.  The next decode
 * call on this thread that passes argument validation (paged_gqa_decode*, any
 * entry point with one query token per sequence; a call rejected before
 * launching leaves the request pending) makes every CTA of its partition
 * kernel first wait for the 32-bit word at `device_flag` (device memory,
 * 4-byte aligned, read only) to become non-zero, bounded by the pipeline's
 * wait budget (2 s).  If it
 * does not, the kernel sets PGD_DEVERR_TIMEOUT in the device error word and
 * its CTAs leave before issuing any copy (the call's output is then
 * undefined); the context stays usable.  NULL cancels a pending request.
 * Returns PGD_ERR_INVALID_ARG for a misaligned pointer.  Tests only.
 */
pgd_status pgd_test_stall_next_decode(const void *device_flag);

/*
 * pgd_test_fail_next_reduce — failure-injection test knob, on the host.  When
 * enable is non-zero, the next decode call on this thread that passes
 * argument validation (paged_gqa_decode*, one query token per sequence)
 * launches its partition kernel and then, instead of launching the reduce
 * kernel, returns PGD_ERR_CUDA as if that launch had failed: its output is
 * undefined and its work counter is left as the partition kernel left it.
 * The library's recovery (the next call on that stream, or the next
 * paged_gqa_decode_noalloc call, zeroes the counter first) is what a test
 * then checks.  enable = 0 cancels a pending request.  Tests only.
 */
pgd_status pgd_test_fail_next_reduce(int enable);

/*
 * pgd_test_fail_next_set_up — failure-injection test knob, on the host.  The
 * kernels of paged_gqa_tree, packed_gqa_prefill, paged_latent_attention and
 * packed_latent_prefill are set up on a device by the first call that needs them.  When enable is non-zero, the next such set-up on
 * this thread fails: its call returns PGD_ERR_CUDA, calls that need none are not
 * affected, and the next call tries again.  enable = 0 cancels a pending
 * request.  Tests only.
 */
pgd_status pgd_test_fail_next_set_up(int enable);

/*
 * pgd_set_timing_events — measurement hook.  When both are non-NULL, every
 * later call on this thread records `before` (a cudaEvent_t) on its stream
 * just before the partition kernel and `after` just after it, so the kernel's
 * own duration can be read with cudaEventElapsedTime.  NULLs turn it off.
 */
pgd_status pgd_set_timing_events(void *before, void *after);

/* Number of SMs and resident partition-kernel CTAs per SM the scheduler
 * assumes for (head_dim, block_size) on the current device. */
pgd_status pgd_device_info(int head_dim, int block_size, int *num_sms, int *ctas_per_sm);

/* Library version, major * 10000 + minor * 100 + patch (1.1.0: strided caches,
 * head_dim 64, block sizes 64 and 128; 1.2.0: several query tokens per
 * sequence; 1.3.0: quantised pages; 1.4.0: pgd_workspace_size, pgd_release,
 * paged_gqa_decode_host; 1.5.0: paged_gqa_tree, packed_gqa_prefill,
 * paged_kv_slots, paged_kv_write; 1.5.1: paged_kv_write_strided,
 * pgd_test_fail_next_set_up; 1.6.0: paged_rope_write, pgd_rope_frequencies,
 * paged_latent_write, paged_latent_attention, packed_latent_prefill). */
int pgd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PGD_H */
