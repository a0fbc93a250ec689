/*
 * pagedattn.h -- C ABI of the GB300 (sm_103a) paged decode-attention library
 * (libpagedattn.so).
 *
 * Sources (web pages on LLM inference, cited by short tag):
 *   [QA]    "LLM推理与服务：面试问题与推荐回答" (LLM inference & serving interview Q&A)
 *   [SB11]  "Scaling Book 入门第 11 章：推理优化 — KV Cache / Continuous Batching / 量化"
 *   [H100]  "09-inference-optimization.md" (LLM-Code-Hot-100, "⚡ 推理优化")
 *   [ANIM]  "推理机制动态图解（进阶）：并行、投机解码、PD、FlashAttention、调度"
 *   [PANO]  "LLM 推理优化全景实战：从 PagedAttention 到投机解码"
 *
 * The KV cache of one attention layer is a pool of fixed-size physical blocks
 * ([QA] Q2; [PANO] §2.2-2.3).  Each sequence owns a block table mapping its
 * logical blocks to physical ones, like an operating-system page table.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Pointers are DEVICE pointers on the current CUDA device; `stream` is a
 *    cudaStream_t passed as void* (NULL = legacy default stream).  Every call is
 *    asynchronous on `stream` and returns after the launch.
 *  - The caller owns every buffer.  The library allocates no device memory and
 *    keeps no per-call state; its device-resident state is one 32-bit error
 *    word per device (see pa_device_error) and the fixed workspace array of
 *    pa_decode_split_noalloc.
 *  - 16-bit floating point (fp16 or bf16, chosen by `dtype`) for q, K, V and the
 *    output; fp32 arithmetic inside.
 *  - Layouts (dense, row-major):
 *      k_cache, v_cache  [num_blocks][num_kv_heads][block_size][head_dim]
 *                        (per page and head, block_size consecutive token rows:
 *                        the [H100] PagedKVCache page shape
 *                        [layers, heads, page_size, head_dim] for one layer)
 *      q, out            [num_seqs][q_len][num_q_heads][head_dim]
 *      k_new, v_new      [n_tokens][num_kv_heads][head_dim]
 *      block_tables      int32 [num_seqs][max_blocks_per_seq]
 *      context_lens      int32 [num_seqs]
 *      slot_mapping      int64 [n_tokens]
 *  - Token position pos of sequence i lives in slot
 *      block_tables[i][pos / block_size] * block_size + pos % block_size
 *    ([PANO] §2.3 write_kv), i.e. block slot / block_size, row slot % block_size.
 *  - context_lens count this step's new tokens: append runs first, then
 *    attention, and a new token attends to itself ([H100] "KV Cache":
 *    AttentionWithKVCache.forward updates the cache before computing scores).
 *  - GQA: query head h reads KV head h / (num_q_heads / num_kv_heads)
 *    (contiguous groups; [QA] Q7, [ANIM] §1 figure).
 *  - Supported now: block_size 8, 16 or 32 (the kernels walk 16-token tiles: a
 *    32-token block is two tiles, a tile of an 8-token pool spans two blocks);
 *    head_dim 64 or 128; q_len 1..4096 with a
 *    16-bit cache (up to 16 query rows per sequence go to the decode kernel, more
 *    to a tensor-core kernel that shares each K/V chunk among 128 query rows of a
 *    KV head: chunked prefill,
 *    [QA] Q14, [SB11] §11.3 "Continuous Batching"); q_len 1..4096 with an FP8
 *    cache too, split between the same two kernels (the many-row kernel widens
 *    each chunk of codes to fp16 in shared memory).
 *  - Alignment: every pointer 16-byte aligned.
 *
 * Errors: argument checks run on the host before any launch and return
 * PA_ERR_INVALID_ARG (null pointer, non-positive size, num_q_heads not a
 * multiple of num_kv_heads, misaligned pointer, workspace too small, sizes whose
 * indices overflow 32 bits) or PA_ERR_UNSUPPORTED (head_dim, block_size, q_len or
 * dtype outside the supported set).  A failed launch returns PA_ERR_CUDA.
 * Kernels never trap or assert: a block id outside [0, num_blocks) or a slot
 * outside the pool is skipped (attention reads zeros in its place) and sets
 * PA_ERR_DEVICE_CHECK in the device error word; a device-side wait that exceeds
 * about two seconds gives up and sets PA_ERR_DEVICE_TIMEOUT.
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = -1,
    PA_ERR_UNSUPPORTED = -2,
    PA_ERR_CUDA = -3,
    PA_ERR_DEVICE_CHECK = -4,
    PA_ERR_DEVICE_TIMEOUT = -5
} pa_status;

/* PA_FP32: the logits of pa_adjust_logits alone */
typedef enum { PA_FP16 = 0, PA_BF16 = 1, PA_FP32 = 2 } pa_dtype;

/* Human-readable name of a status code (static string, never NULL). */
PA_API const char *pa_status_string(pa_status status);

/* Library ABI version (major * 100 + minor). */
PA_API int pa_version(void);

/*
 * pa_slot_mapping -- slots of this step's new tokens ([PANO] §2.3 write_kv:
 * logical_block = pos // block_size, block_offset = pos % block_size).
 * For sequence i the new tokens are its last q_len positions
 * pos = context_lens[i] - q_len + u (u = 0..q_len-1), written to
 * slot_mapping[i*q_len + u]; a position < 0 gives -1 (skipped by pa_append_kv).
 * A position whose logical block is >= max_blocks_per_seq gives -1 and sets
 * PA_ERR_DEVICE_CHECK.  slot_mapping: int64 [num_seqs*q_len], written.
 */
PA_API pa_status pa_slot_mapping(int64_t *slot_mapping, const int32_t *block_tables,
                                 const int32_t *context_lens, int num_seqs,
                                 int max_blocks_per_seq, int block_size, int q_len,
                                 void *stream);

/*
 * pa_append_kv -- scatter this step's new K/V rows into the pool
 * ([PANO] §2.3 write_kv; [H100] PagedKVCache.append_token).
 * Row t of k_new/v_new (all heads) is copied bit for bit to slot
 * slot_mapping[t]: block slot / block_size, row slot % block_size.  Slots < 0
 * are skipped; slots >= num_blocks*block_size are skipped and set
 * PA_ERR_DEVICE_CHECK.  Two tokens with the same slot: undefined which wins.
 * k_cache, v_cache: read-write.  n_tokens == 0 is a no-op.
 */
PA_API pa_status pa_append_kv(void *k_cache, void *v_cache, const void *k_new,
                              const void *v_new, const int64_t *slot_mapping, int n_tokens,
                              int num_kv_heads, int head_dim, int block_size, int num_blocks,
                              pa_dtype dtype, void *stream);

/*
 * pa_copy_blocks -- copy-on-write support: sequences that share physical blocks
 * (parallel sampling, beam search, a cached prefix; [QA] Q2) keep sharing them
 * until one of them writes; before that write it needs a private copy.  For each
 * pair i, block src_blocks[i] (every head, every row, K and V) is copied bit for
 * bit to block dst_blocks[i].  Pairs with an id outside [0, num_blocks) are skipped
 * and set PA_ERR_DEVICE_CHECK.  A destination that is also a source or another
 * pair's destination in the same call: undefined result.  src_blocks, dst_blocks:
 * int32 [n_pairs] device arrays.  n_pairs == 0 is a no-op.
 */
PA_API pa_status pa_copy_blocks(void *k_cache, void *v_cache, const int32_t *src_blocks,
                                const int32_t *dst_blocks, int n_pairs, int num_kv_heads,
                                int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                                void *stream);

/*
 * pa_decode -- attention of every query row over its sequence's paged K/V, in
 * one pass with online softmax ([ANIM] §5: running max m, running sum l,
 * unnormalised output rescaled by exp(m_old - m_new), output O / l at the end;
 * [PANO] §2.4 for what is computed: softmax(q K^T * scale) V over the gathered
 * blocks).  Only positions t < context_lens[i] are used ([H100]
 * PagedKVCache.get_kv keeps used_slots rows of the last page).  With q_len > 1,
 * query u of sequence i sees positions t <= context_lens[i] - q_len + u (the
 * [H100] causal mask triu(diagonal = Lk - Lq + 1)).  A row that sees no
 * position (context length 0) is written as zeros.
 * out: [num_seqs][q_len][num_q_heads][head_dim], written (round to nearest even).
 * The query heads of one GQA group share every K/V read.
 */
PA_API pa_status pa_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_tables, const int32_t *context_lens,
                           int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                           int block_size, float scale, void *stream,
                           int max_blocks_per_seq, int num_blocks, int q_len, pa_dtype dtype);

/*
 * Split-KV (flash-decoding, [SB11] §11.8): one sequence's blocks are cut into
 * num_splits partitions processed by different thread blocks, then merged.
 *
 * Workspace layout (fp32, caller-allocated, pa_decode_workspace_size bytes),
 * with R = q_len * num_q_heads rows per sequence (row u*num_q_heads + h):
 *   acc [num_seqs][num_splits][R][head_dim]   unnormalised sum_t 2^(s_t - m) V_t
 *   m   [num_seqs][num_splits][R]             max_t s_t  (-inf if empty)
 *   l   [num_seqs][num_splits][R]             sum_t 2^(s_t - m)  (0 if empty)
 * where s_t = scale * log2(e) * q.k_t (base-2 units).  Section m starts at
 * byte offset align256(sizeof acc), section l at align256 after m.
 * Partition p of sequence i covers blocks [p*C, (p+1)*C) with
 * C = ceil(ceil(context_lens[i] / block_size) / num_splits); partitions past
 * the end are empty.  With 8-token blocks the partitions are counted in 16-token
 * tiles instead (C = ceil(ceil(context_lens[i] / 16) / num_splits) tiles).
 */
PA_API size_t pa_decode_workspace_size(int num_seqs, int num_q_heads, int q_len, int head_dim,
                                       int num_splits);

/* Partial pass: writes every (sequence, partition, row) entry of the workspace. */
PA_API pa_status pa_decode_partial(void *workspace, size_t workspace_bytes, const void *q,
                                   const void *k_cache, const void *v_cache,
                                   const int32_t *block_tables, const int32_t *context_lens,
                                   int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                   int block_size, float scale, int num_splits,
                                   int max_blocks_per_seq, int num_blocks, int q_len,
                                   pa_dtype dtype, void *stream);

/*
 * Combine pass (the online-softmax rescale of [ANIM] §5 applied across
 * partitions): M = max_p m_p; out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p
 * over non-empty partitions; zeros if all are empty.  Reads the workspace,
 * writes out [num_seqs][q_len][num_q_heads][head_dim].
 */
PA_API pa_status pa_decode_combine(void *out, const void *workspace, size_t workspace_bytes,
                                   int num_seqs, int num_q_heads, int head_dim, int q_len,
                                   int num_splits, pa_dtype dtype, void *stream);

/*
 * pa_append_decode -- one decode step fused: slot mapping, append of the new K/V
 * rows and attention in one launch (a second launch, the combine, when
 * num_splits > 1).  Kernel fusion of consecutive memory-bound steps follows
 * [SB11] §11.8 ("Kernel Fusion").  Equivalent to pa_slot_mapping, then
 * pa_append_kv of k_new/v_new (rows [num_seqs*q_len][num_kv_heads][head_dim], the
 * last q_len positions of each sequence), then pa_decode (num_splits == 1;
 * workspace may be NULL) or pa_decode_partial + pa_decode_combine (num_splits > 1;
 * workspace as for pa_decode_partial).  The cache ends up bit-identical to the
 * unfused sequence and out within the same tolerance.  New positions < 0 are
 * skipped; new positions beyond the block table or the pool are skipped and set
 * PA_ERR_DEVICE_CHECK.  With q_len > 16 the append is a launch of its own before
 * the attention (a CTA's rows then depend on rows other CTAs would write).
 */
PA_API pa_status pa_append_decode(void *out, const void *q, const void *k_new, const void *v_new,
                                  void *k_cache, void *v_cache, const int32_t *block_tables,
                                  const int32_t *context_lens, int num_seqs, int num_q_heads,
                                  int num_kv_heads, int head_dim, int block_size, float scale,
                                  int max_blocks_per_seq, int num_blocks, int q_len,
                                  pa_dtype dtype, int num_splits, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * pa_decode_cascade -- attention of a batch whose sequences all begin with the
 * same prefix_blocks physical blocks (a shared prompt: [QA] Q2 copy-on-write page
 * sharing and Q3 prefix caching; [SB11] §11.4 "Prefix Caching": the shared
 * prefix's KV is stored once).  Same result as pa_append_decode, computed in
 * three launches over a workspace of 1 + tail_splits partitions
 * (pa_decode_workspace_size(num_seqs, num_q_heads, q_len, head_dim,
 * 1 + tail_splits) bytes, 256-byte aligned, layout as for pa_decode_partial):
 *   partition 0      every query row of every sequence against the prefix blocks,
 *                    read once per KV head for all num_seqs * q_len * group rows;
 *                    the prefix is the first prefix_blocks entries of block-table
 *                    row 0;
 *   partitions 1..   each sequence's blocks from prefix_blocks on (with this
 *                    step's append when k_new/v_new are given), cut into
 *                    tail_splits equal parts;
 * then the combine.  With tail_splits == 1 and q_len <= 16 the tail pass is a
 * single pass that merges partition 0 into its result (no combine launch).  It
 * runs alongside the prefix pass and waits for it only before that merge.  The
 * causal limit applies in both passes.
 * Caller's contract: for every sequence, table entries [0, prefix_blocks) equal
 * those of row 0, and this step's new tokens lie at or past position
 * prefix_blocks * block_size (so the append never writes a shared block).
 * prefix_blocks * block_size must be a multiple of 16 (PA_ERR_UNSUPPORTED
 * otherwise: the two passes split at a 16-token tile).
 * k_new and v_new are both NULL (no append) or both given.  16-bit caches only.
 */
PA_API pa_status pa_decode_cascade(void *out, const void *q, const void *k_new, const void *v_new,
                                   void *k_cache, void *v_cache, const int32_t *block_tables,
                                   const int32_t *context_lens, int num_seqs, int num_q_heads,
                                   int num_kv_heads, int head_dim, int block_size, float scale,
                                   int max_blocks_per_seq, int num_blocks, int q_len,
                                   pa_dtype dtype, int prefix_blocks, int tail_splits,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * FP8 (e4m3) KV cache.  The pool holds one byte per element, same layout
 * [num_blocks][num_kv_heads][block_size][head_dim]; an element stands for
 * e4m3_value * scale[kv_head], with separate fp32 scales for K and V
 * (k_scale, v_scale: device arrays [num_kv_heads]).  Quantisation ([QA] Q4: KV
 * quantisation relieves KV memory; fewer bytes per token on a bandwidth-bound path)
 * is code = e4m3(x / scale): fp32 division, round to nearest even, magnitudes above
 * 448 saturate to 448.  head_dim 128 only.
 *
 * pa_append_kv_fp8 -- pa_append_kv for an FP8 cache: k_new/v_new are 16-bit rows of
 * type new_dtype, quantised as above into their slots.
 */
PA_API pa_status pa_append_kv_fp8(void *k_cache, void *v_cache, const void *k_new,
                                  const void *v_new, const int64_t *slot_mapping, int n_tokens,
                                  int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                  pa_dtype new_dtype, const float *k_scale, const float *v_scale,
                                  void *stream);

/*
 * pa_decode_fp8 -- attention over an FP8 cache (q and out of type dtype; fp32
 * arithmetic on the dequantised K, V).  With k_new/v_new (both non-NULL) the step's
 * new rows are first quantised into the cache as pa_append_kv_fp8 would (slots of
 * the last q_len positions, as pa_slot_mapping), in the same launch.  num_splits == 1:
 * single pass, workspace may be NULL; num_splits > 1: split-KV partial pass into the
 * workspace (layout of pa_decode_partial) and the combine.  With more than 16
 * query rows per sequence (chunked prefill over an FP8 cache, [QA] Q4 and Q14) the
 * fused append is a launch of its own before the attention, as in pa_append_decode.
 */
PA_API pa_status pa_decode_fp8(void *out, const void *q, const void *k_new, const void *v_new,
                               void *k_cache, void *v_cache, const float *k_scale,
                               const float *v_scale, const int32_t *block_tables,
                               const int32_t *context_lens, int num_seqs, int num_q_heads,
                               int num_kv_heads, int head_dim, int block_size, float scale,
                               int max_blocks_per_seq, int num_blocks, int q_len, pa_dtype dtype,
                               int num_splits, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * pa_device_error -- synchronise `stream`, then return PA_OK or the first error
 * recorded by a kernel on the current device since the last clear
 * (PA_ERR_DEVICE_TIMEOUT takes precedence over PA_ERR_DEVICE_CHECK).  With
 * clear != 0 the word is reset to zero.  Returns PA_ERR_CUDA if the
 * synchronisation itself fails.
 */
PA_API pa_status pa_device_error(void *stream, int clear);

/*
 * pa_selftest_wait_timeout -- diagnostic: launches one thread that waits, with the
 * same bounded wait the attention kernels use for their TMA stages, on a
 * shared-memory barrier that nothing ever completes.  After about two seconds the
 * wait gives up and records PA_ERR_DEVICE_TIMEOUT in the device error word
 * (read it with pa_device_error); the CUDA context stays usable.  Lets a caller
 * check the failure path without faulting or hanging the GPU.
 */
PA_API pa_status pa_selftest_wait_timeout(void *stream);

/*
 * pa_decode_split_noalloc -- the split-KV pair (pa_decode_partial, then
 * pa_decode_combine) with its workspace in a fixed device array that the library
 * owns, for callers that cannot allocate device memory where they run attention:
 * a plug-in whose host runtime owns every device allocation, or a serving loop
 * that must not allocate (nor risk the implicit device synchronisation of
 * cudaMalloc/cudaFree) once it is running.  The pages have no counterpart; this
 * is an allocation-free convenience of this library, not a step of the method.
 *
 * Arguments are those of pa_decode_partial without the workspace; out is written
 * as by pa_decode_combine.  The array holds PA_NOALLOC_SCRATCH_BYTES on every
 * device that loads the library, until the process exits.  If
 * pa_decode_workspace_size(num_seqs, num_q_heads, q_len, head_dim, num_splits)
 * exceeds it, the call returns PA_ERR_INVALID_ARG and launches nothing.  No
 * device memory is allocated or freed.  All calls on a device share the array:
 * calls that can overlap on the GPU (unordered streams) race.  The first call on
 * a device looks up the array's device address with that device current; make
 * it before any stream capture.  The address is kept for the life of the
 * process: do not use the library across a cudaDeviceReset of that device (the
 * same holds for the error word of pa_device_error).
 */
#define PA_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
PA_API pa_status pa_decode_split_noalloc(void *out, const void *q, const void *k_cache,
                                         const void *v_cache, const int32_t *block_tables,
                                         const int32_t *context_lens, int num_seqs,
                                         int num_q_heads, int num_kv_heads, int head_dim,
                                         int block_size, float scale, int num_splits,
                                         int max_blocks_per_seq, int num_blocks, int q_len,
                                         pa_dtype dtype, void *stream);

/*
 * pa_rope_append -- rotary positions of one or several axes on q and on the new K
 * rows, which go (with V, unrotated) straight into their cache slots.  With
 *   theta(i, t) = positions[pair_axis[i]][t] * f_i
 * pair i of every q and K head of token t becomes (a cos - b sin, b cos + a sin): its
 * elements a, b are i and i + rotary_dim/2, or 2i and 2i + 1 when interleaved != 0.
 * Elements from rotary_dim on are copied.  fp32 arithmetic, one rounding to the 16-bit
 * type, or (k_scale and v_scale both non-NULL: FP8 cache, head_dim 128) to
 * e4m3(x / scale[kv_head]) for the cache.  After pa_evict a token's cache row is no
 * longer its position, so positions are always explicit.
 *   positions     int32 [num_axes][n_tokens]  (e.g. time, height, width; at most 32 axes)
 *   slot_mapping  int64 [n_tokens], as for pa_append_kv; a token with a negative slot,
 *                 or one past the pool (PA_ERR_DEVICE_CHECK), has its q rotated only
 *   turns         int64 [rotary_dim/2]: f_i in turns per position, units of 2^-64
 *                 (round(2^64 f_i / (2 pi)) mod 2^64): the angle's fraction of a turn is
 *                 then exact in integers at any position
 *   pair_axis     int32 [rotary_dim/2], values in [0, num_axes) (others:
 *                 PA_ERR_DEVICE_CHECK, axis 0)
 *   q, q_out      [n_tokens][num_q_heads][head_dim], tokens q_stride / q_out_stride
 *                 elements apart; q_out may be q itself (same stride)
 *   k, v          [n_tokens][num_kv_heads][head_dim], tokens k_stride / v_stride apart
 *                 (all strides multiples of 8, at least a token's width: slices of one
 *                 fused projection need no copy)
 * rotary_dim: a multiple of 16, at most head_dim.  Two tokens with the same slot:
 * undefined which wins.  n_tokens == 0 is a no-op.
 */
PA_API pa_status pa_rope_append(void *q_out, const void *q, const void *k, const void *v,
                                void *k_cache, void *v_cache, const int32_t *positions,
                                const int64_t *slot_mapping, const int64_t *turns,
                                const int32_t *pair_axis, int n_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int rotary_dim, int num_axes,
                                int interleaved, int64_t q_out_stride, int64_t q_stride,
                                int64_t k_stride, int64_t v_stride, int block_size, int num_blocks,
                                pa_dtype dtype, const float *k_scale, const float *v_scale,
                                void *stream);

/*
 * pa_decode_scored -- pa_decode (16-bit cache) or pa_decode_fp8 (k_scale and v_scale
 * both non-NULL), q_len 1..4096, that also keeps the ledger of accumulated attention
 * weight that pa_evict goes by ([QA] Q4: the tokens that draw little attention).
 * For cached row t of KV head h
 *   share(t) = sum over the head's group and query tokens u that see t of the softmax
 *              weight of (u, head) on t
 *   scores[i][h][t] = scores[i][h][t] + share(t)   for rows that were there before
 *                   = share(t)                     for this step's rows (the last q_len)
 * and, with row_pos, row_pos[i][h][t] = seq_lens[i] - (context_lens[i] - t) for this
 * step's rows: the token's position in its sequence.  seq_lens count the sequence's
 * tokens, evicted ones included (equal to context_lens before any eviction).
 * Rows t >= context_lens[i] of both ledgers are left as they were.
 *   scores   fp32  [num_seqs][num_kv_heads][max_blocks_per_seq * block_size]
 *   row_pos  int32, the same shape; NULL (with seq_lens NULL): no positions kept
 * out, bad blocks and non-finite values are as in pa_decode; with several query tokens an
 * infinite or NaN V row of this step therefore also reaches the step's earlier tokens
 * (their weight on it is 0, and 0 times it is NaN).  The ledger is free of that: a row
 * gains nothing from query tokens that do not see it.
 * The sums have one order: results do not change from run to run.  num_splits as for
 * pa_append_decode up to 16 query tokens; above, the call takes no partitions, and out
 * must not overlap q (the ledger's pass reads q after out is written).
 * Workspace: pa_decode_scored_workspace_size bytes, 256-byte aligned (up to 16 query
 * tokens it holds 4 bytes per query row and table position); nothing in it has to
 * start at zero.  Two calls that can overlap need workspaces of their own.
 */
PA_API size_t pa_decode_scored_workspace_size(int num_seqs, int num_q_heads, int q_len,
                                              int head_dim, int num_splits,
                                              int max_blocks_per_seq, int block_size);
PA_API pa_status pa_decode_scored(void *out, float *scores, int32_t *row_pos, const void *q,
                                  const void *k_cache, const void *v_cache, const float *k_scale,
                                  const float *v_scale, const int32_t *block_tables,
                                  const int32_t *context_lens, const int32_t *seq_lens,
                                  int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                  int block_size, float scale, int max_blocks_per_seq,
                                  int num_blocks, int q_len, pa_dtype dtype, int num_splits,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * pa_evict -- eviction by accumulated attention weight ([QA] Q4).  A sequence with
 * context_lens[i] > budget keeps exactly `budget` rows, each KV head its own choice:
 * rows of the first `sinks` positions (row_pos < sinks) and of the last `recent`
 * (row_pos >= seq_lens[i] - recent), then by descending score; ties go to the lowest
 * row; NaN ranks below every number.  (If more than `budget` rows are protected, the
 * lowest rows of them stay.)  Kept rows below `budget` stay where they are; the i-th
 * kept row at or past it is copied (K, V, score, position) into the i-th evicted row
 * below it.  Attention over the shortened context needs nothing else: K rows carry
 * their rotation, and the causal limit concerns only rows appended later.
 * new_lens[i] = min(context_lens[i], budget).  The caller's allocator may take back
 * the blocks past ceil(new_lens[i] / block_size).
 * scores_out / row_pos_out: the ledgers themselves, updated in place, or both other
 * arrays (not overlapping), rows below new_lens[i] written; rows from there on are
 * left as they were.  With other arrays the call may be repeated with the same result.
 * Blocks of a sequence longer than the budget must be its own (copy shared ones with
 * pa_copy_blocks first).  A block id outside the pool, of the hole or of the row that would
 * fill it: the hole keeps its row, score and position, PA_ERR_DEVICE_CHECK.
 *   element_bytes  2 (16-bit cache) or 1 (FP8, head_dim 128): rows are moved bit for bit
 *   new_lens       int32 [num_seqs], overlapping neither context_lens nor seq_lens
 *   workspace      pa_evict_workspace_size bytes; two calls that can overlap need
 *                  workspaces of their own
 * budget >= sinks + recent, budget >= 1.
 */
PA_API size_t pa_evict_workspace_size(int num_seqs, int num_kv_heads, int budget);
PA_API pa_status pa_evict(void *k_cache, void *v_cache, float *scores_out, int32_t *row_pos_out,
                          int32_t *new_lens, const float *scores, const int32_t *row_pos,
                          const int32_t *block_tables, const int32_t *context_lens,
                          const int32_t *seq_lens, int num_seqs, int num_kv_heads, int head_dim,
                          int block_size, int max_blocks_per_seq, int num_blocks, int budget,
                          int sinks, int recent, int element_bytes, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * pa_verify_drafts -- which drafted tokens stand, and the token after them ([ANIM] §3,
 * [SB11] §11.7: accept with min(1, p/q), else resample from (p - q)+), from random
 * numbers in [0, 1) that the caller gives.  For sequence i with m = draft_lens[i]
 * drafts x_j, target rows p_j (j = 0..m) and draft rows q_j (j < m):
 *   draft j stands while accept_u[i][j] * q_j(x_j) < p_j(x_j) and all before it stand;
 *   a = num_accepted[i];
 *   weights w(v) = max(p_a(v) - q_a(v), 0) if a < m, else p_m(v); if they sum to zero
 *   (the two rows agree), w = p_a;
 *   token = the first v with w(0) + .. + w(v) > sample_u[i] * sum w.
 * out_tokens[i] = the a standing drafts, the token, then -1.  Which drafts stand is exact:
 * u q < p is compared with the exact product.  The sums w are good to about 2^-46 of the
 * row's total (pairs of fp32; the total within fp32's range and not below 2^-100, as a row
 * of probabilities is): a sample_u that falls so near a border may take either of the
 * tokens beside it.  Weights that are negative, NaN or infinite count as zero.
 * draft_probs NULL: drafts that were certain (q_j(x_j) = 1, 0 elsewhere).
 * new_lens (may be NULL, or context_lens itself): context_lens[i] - (max_draft - a), the
 * cache length after a
 * step that appended 1 + max_draft rows per sequence (the last committed token, then
 * the drafts, padded to max_draft); the next append overwrites the rejected rows.
 *   target_probs  fp32 [num_seqs][max_draft + 1][target_stride], vocab used
 *   draft_probs   fp32 [num_seqs][max_draft][draft_stride]
 *   draft_tokens  int32 [num_seqs][max_draft]; draft_lens int32 [num_seqs] or NULL (all
 *                 max_draft); accept_u fp32 [num_seqs][max_draft]; sample_u fp32 [num_seqs]
 *   out_tokens    int32 [num_seqs][max_draft + 1]; num_accepted int32 [num_seqs]
 * A draft id outside [0, vocab) is rejected, a draft_lens outside [0, max_draft] is
 * clamped, a target row without any positive entry gives token -1: each sets
 * PA_ERR_DEVICE_CHECK.  Pointers 4-byte aligned; outputs overlap neither one another nor
 * the int32 inputs (new_lens apart, as said; and new_lens or num_accepted may be
 * draft_lens itself).
 */
PA_API pa_status pa_verify_drafts(int32_t *out_tokens, int32_t *num_accepted, int32_t *new_lens,
                                  const int32_t *context_lens, const float *target_probs,
                                  const float *draft_probs, const int32_t *draft_tokens,
                                  const int32_t *draft_lens, const float *accept_u,
                                  const float *sample_u, int num_seqs, int max_draft, int vocab,
                                  int64_t target_stride, int64_t draft_stride, void *stream);

/*
 * Block-scaled FP8 cache ([QA] Q4).  A pool of e4m3 codes as for pa_append_kv_fp8, with one
 * scale for K and one for V of every block and KV head:
 *   kv_scales  fp32 [num_blocks][num_kv_heads][2]  (K, V), 16-byte aligned
 * An element stands for code * scale.  The scales come from the data: no calibration, and a
 * token of large values costs the rows of its own block their small ones, not a head's.
 * Scales count as clamped to [2^-40, 2^40] (NaN as 2^-40).  head_dim 128 only.  pa_evict moves
 * rows between blocks and is not for such a pool; pa_copy_pages copies its blocks.
 *
 * pa_append_kv_block_scaled -- the last q_len positions of every sequence, rows of k_new and
 * v_new [num_seqs * q_len][num_kv_heads][head_dim] (16-bit of type new_dtype; tokens k_stride /
 * v_stride elements apart, multiples of 8, at least a token's width), into their blocks.
 * For a block that the step writes, one KV head, and K or V:
 *   need = the least power of two with max |x| <= 448 need over the step's finite x in it,
 *          clamped as above
 *   s    = need where the block's first row is one of the step's, else max(scale, need)
 *   code = e4m3(x / s) (nearest even; magnitudes above 448, infinities among them, to 448) for the
 *          step's rows; rows before them, if s grew: code = e4m3(code * scale / s)
 * and s becomes the scale.  Rows past the step's are left as they were: they stand for nothing.  A
 * power of two moves only exponents: an older row is rounded again only where it becomes
 * subnormal.  After a rejection the next step overwrites the rejected rows; the scale keeps
 * what they needed.  Positions < 0 are skipped; positions beyond the table or the pool are
 * skipped and set PA_ERR_DEVICE_CHECK.  A block that is written must belong to one sequence
 * (pa_fork_blocks sees to it, unless a length is taken back into a block that was shared).  Caches and scales overlap nothing else.  num_seqs == 0 is a
 * no-op.
 */
PA_API pa_status pa_append_kv_block_scaled(void *k_cache, void *v_cache, float *kv_scales,
                                           const void *k_new, const void *v_new,
                                           const int32_t *block_tables, const int32_t *context_lens,
                                           int num_seqs, int num_kv_heads, int head_dim,
                                           int block_size, int max_blocks_per_seq, int num_blocks,
                                           int q_len, pa_dtype new_dtype, int64_t k_stride,
                                           int64_t v_stride, void *stream);

/*
 * pa_decode_block_scaled -- pa_decode (q_len 1..4096, GQA, causal limit, rows that see
 * nothing) over a block-scaled cache; q and out of type dtype, fp32 arithmetic on
 * code * scale.  num_splits == 1: one pass, workspace may be NULL; num_splits > 1: split-KV,
 * workspace of pa_decode_workspace_size bytes, 256-byte aligned, and the combine.  (Its
 * sections hold what pa_decode_partial writes, with m the running maximum of s_t plus the
 * base-2 logarithm of V's scale.)  Two calls that can overlap need workspaces of their own.
 * Weights are rounded to 16 bits, times their V scale relative to the largest such product.
 */
PA_API pa_status pa_decode_block_scaled(void *out, const void *q, const void *k_cache,
                                        const void *v_cache, const float *kv_scales,
                                        const int32_t *block_tables, const int32_t *context_lens,
                                        int num_seqs, int num_q_heads, int num_kv_heads,
                                        int head_dim, int block_size, float scale,
                                        int max_blocks_per_seq, int num_blocks, int q_len,
                                        pa_dtype dtype, int num_splits, void *workspace,
                                        size_t workspace_bytes, void *stream);

/*
 * The pool's blocks by reference counts, on the device ([QA] Q2: sequences share blocks until
 * one of them writes).
 *   ref_counts    int32 [num_blocks]: table entries that hold the block; 0: the block is free
 *   block_tables  an entry < 0 holds no block
 * The calls keep the counts in step with the tables; at the start every entry is -1 and every
 * count 0, or the counts are the entries' number.  Each call has one result, whatever the order
 * of its threads.  An entry outside the pool that a call gives up, shares, copies or
 * renames sets PA_ERR_DEVICE_CHECK and counts as none; so does one whose block has a count of
 * 0 that is given up (pa_free_blocks) or stands past the pool's new front
 * (pa_compact_blocks).  None of them touches a cache: with several layers over one table
 * they run once, and pa_copy_pages once a layer.  A batch has at least one sequence.  Arrays
 * are 4-byte aligned, block_tables (pa_fork_blocks apart), ref_counts and the workspace 16-byte aligned;
 * outputs overlap nothing else but where said.
 * Workspace: pa_pages_workspace_size(num_blocks, num_forks) bytes (num_forks 0 for the others);
 * two calls that can overlap need workspaces of their own.
 *
 * pa_free_blocks -- entries of sequence i at or past ceil(keep_lens[i] / block_size) give
 * their block up (its count falls by one) and become -1.  keep_lens 0: all of them; the
 * new lengths of pa_verify_drafts or pa_evict: what these no longer use.
 *
 * pa_reserve_blocks -- entries of sequence i before ceil(lens[i] / block_size) that are < 0
 * take the free blocks in ascending order, in the order of sequences and entries; their counts
 * become 1.  missing[0] = how many found none; they stay < 0.  lens past the table's width:
 * the width (PA_ERR_DEVICE_CHECK).
 *
 * pa_fork_blocks -- for fork f, sequence dst_seqs[f] becomes a copy of src_seqs[f]: the full
 * blocks are shared (their counts rise by one), a partial last block is to be copied into a
 * free one (ascending, in the order of forks), and context_lens[dst] = context_lens[src].  The
 * copies to make are listed, src_blocks[p] -> dst_blocks[p] for p < counts[0]; entries from
 * there on are left as they were.  counts[1] = forks that found no free block: these get
 * their parent's full blocks and that length.  What dst's row held before is overwritten,
 * not freed.  Every dst_seqs[f] is another sequence, and none of src_seqs (else the result is
 * undefined); ids outside the batch, or src == dst, set PA_ERR_DEVICE_CHECK and are skipped.  A
 * parent's length past its table sets it too and counts as the table's.
 *   src_seqs, dst_seqs, src_blocks, dst_blocks  int32 [num_forks <= num_seqs] (num_forks 0:
 *   counts alone are written); counts int32 [2]
 *
 * pa_compact_blocks -- the pool's blocks to its front: with live = blocks of a count other than
 * 0, the k-th of them at or past `live` gets the id of the k-th free one before it, in
 * tables and counts; counts[0] = how many, listed as above, counts[1] = live.  After the
 * copies the blocks from `live` on are free.  tables and counts are updated in place, or
 * (the _out arrays being others) the inputs are left as they were.
 *   src_blocks, dst_blocks  int32 [num_blocks / 2]
 *
 * pa_copy_pages -- whole blocks src_blocks[p] -> dst_blocks[p], p < min(counts[0], max_pairs),
 * K, V and (kv_scales non-NULL) their scales, bit for bit; element_bytes 2 (16-bit pools) or 1
 * (head_dim 128).  Caches and scales overlap nothing else.  Ids outside the pool are skipped
 * and set PA_ERR_DEVICE_CHECK.  A destination that is also a source or another pair's
 * destination: undefined result.
 */
PA_API size_t pa_pages_workspace_size(int num_blocks, int num_forks);
PA_API pa_status pa_free_blocks(int32_t *block_tables, int32_t *ref_counts, const int32_t *keep_lens,
                                int num_seqs, int max_blocks_per_seq, int num_blocks, int block_size,
                                void *stream);
PA_API pa_status pa_reserve_blocks(int32_t *block_tables, int32_t *ref_counts, const int32_t *lens,
                                   int32_t *missing, int num_seqs, int max_blocks_per_seq,
                                   int num_blocks, int block_size, void *workspace,
                                   size_t workspace_bytes, void *stream);
PA_API pa_status pa_fork_blocks(int32_t *block_tables, int32_t *context_lens, int32_t *ref_counts,
                                const int32_t *src_seqs, const int32_t *dst_seqs, int32_t *src_blocks,
                                int32_t *dst_blocks, int32_t *counts, int num_forks, int num_seqs,
                                int max_blocks_per_seq, int num_blocks, int block_size,
                                void *workspace, size_t workspace_bytes, void *stream);
PA_API pa_status pa_compact_blocks(int32_t *block_tables_out, int32_t *ref_counts_out,
                                   const int32_t *block_tables, const int32_t *ref_counts,
                                   int32_t *src_blocks, int32_t *dst_blocks, int32_t *counts,
                                   int num_seqs, int max_blocks_per_seq, int num_blocks,
                                   void *workspace, size_t workspace_bytes, void *stream);
PA_API pa_status pa_copy_pages(void *k_cache, void *v_cache, float *kv_scales,
                               const int32_t *src_blocks, const int32_t *dst_blocks,
                               const int32_t *counts, int max_pairs, int num_kv_heads, int head_dim,
                               int block_size, int num_blocks, int element_bytes, void *stream);

/*
 * pa_adjust_logits -- penalties, biases and grammar masks on a step's logits, and the
 * probabilities that pa_verify_drafts takes.  Row j of sequence i is the one behind its
 * drafts 0 .. j-1.  Its outputs are history[i][prompt_lens[i] .. history_lens[i]) and
 * those drafts; count = how often entry v stands there, seen = it stands there or in the
 * prompt, history[i][0 .. prompt_lens[i]).  Of its logit x:
 *   y = x > 0 ? x / repetition[i] : x * repetition[i]   if seen, else x
 *   y = (y - count * frequency[i]) - presence[i]        if count > 0
 *   y = y + bias_values[i][b]  for every b with bias_ids[i][b] == v, in their order
 *   y = -inf                   if bit v % 32 of the mask's word v / 32 is 0
 * each operation rounded to fp32.  probs == 0: out = y, of the logits' type.  probs != 0:
 * out fp32, softmax(y / temperature[i]); temperature <= 0 (or NaN): 1 at the largest y (the
 * lowest entry of equals), 0 elsewhere.  There a NaN counts as -inf, infinite entries share
 * the whole, and a row that its mask leaves empty is all zeros (pa_verify_drafts answers
 * -1 to it).
 *   logits       [num_seqs][rows][logits_stride], vocab used; fp16, bf16 or fp32 (dtype)
 *   out          [num_seqs][rows][out_stride]; may be logits itself where type and stride
 *                are the same, and overlaps nothing else.  (Fastest with equal strides: a row
 *                whose start in out, modulo the elements of 16 bytes there, is another than
 *                that of its logits is stored element by element.)
 *   history      int32 [num_seqs][max_history], history_lens, prompt_lens int32 [num_seqs]
 *                (prompt_lens NULL: no prompt; max_history 0: none of the three is read)
 *   drafts       int32 [num_seqs][rows - 1]
 *   repetition, presence, frequency, temperature  fp32 [num_seqs] (NULL: 1, 0, 0, 1)
 *   bias_ids, bias_values  int32, fp32 [num_seqs][num_bias], num_bias <= 1024
 *   mask         32-bit words; sequences mask_seq_stride and rows mask_row_stride words
 *                apart (0: shared)
 * All but out and logits may be NULL.  Negative ids (padding) are ignored, ids >= vocab too,
 * which set PA_ERR_DEVICE_CHECK, as a history_lens outside [0, max_history] (clamped) does.
 * vocab <= 2^18.  num_seqs == 0 is a no-op.
 */
PA_API pa_status pa_adjust_logits(void *out, const void *logits, const int32_t *history,
                                  const int32_t *history_lens, const int32_t *prompt_lens,
                                  const int32_t *drafts, const float *repetition,
                                  const float *presence, const float *frequency,
                                  const int32_t *bias_ids, const float *bias_values,
                                  const int32_t *mask, const float *temperature, int num_seqs,
                                  int rows, int vocab, int max_history, int num_bias, pa_dtype dtype,
                                  int probs, int64_t out_stride, int64_t logits_stride,
                                  int64_t mask_seq_stride, int64_t mask_row_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
