/*
 * fd_attention.h -- C ABI of the GB300 (sm_103a) flash-decoding library.
 *
 * One decode step of attention: every sequence b of a batch contributes one
 * query token per query head, which attends over that sequence's cached
 * keys and values.  The cache is token-major and either contiguous (a
 * sequence owns a run of rows starting at kv_start_idx[b]) or paged (a block
 * table maps the sequence's logical pages to physical pages of a pool).
 * K and V are fp16, bf16 or FP8-e4m3 with one fp32 scale per tensor.
 *
 * The computation is split-KV partial attention with an online softmax
 * (running max, running sum, rescaled accumulator) followed by a
 * log-sum-exp merge of the partial states, for MHA, GQA and MQA head layouts.
 *
 * Passages that define the operation:
 *  - "From SGLang kernel source to GPU trace: DeepSeek V4.1 Flash-Decode",
 *    section 3.1: the decode kernel's arguments (q, FP8 k_cache/v_cache,
 *    output, kv_start_idx and seq_len per sequence, head count, head
 *    dimension, softmax scale, batch); section 2.2: FP8 KV converted inside
 *    the load stage, not by a separate pass;
 *  - "SGLang Prefill optimisation: dissecting FlashAttention kernel
 *    bottlenecks with GPU Trace", section 2.2: the online softmax loop
 *    (scores = dot(q, k) * scale, running max, rescale factor
 *    exp(m_old - m_new), running sum, accumulator update);
 *  - "Learn CUDA from scratch, chapter 15: GPU profiling and LLM inference",
 *    section 15.26: paged addressing (physical page from the block table,
 *    row = page * page_size + offset in a [page, offset, head, dim] pool);
 *    section 15.12: one pass over a KV head serves its group of
 *    QH / KVH query heads; section 15.13: a ragged batch scans each
 *    sequence's real length only.
 *
 * Conventions (readings where the pages are silent):
 *  - q and out are dense [batch, num_q_heads, head_dim]; lse is dense fp32
 *    [batch, num_q_heads];
 *  - contiguous K/V: [kv_rows, num_kv_heads, head_dim], kv_start_idx in rows;
 *    paged K/V: [num_pages, page_size, num_kv_heads, head_dim],
 *    block_table row-major [batch, block_table_stride] of int32 page ids;
 *  - query head qh reads KV head qh / (num_q_heads / num_kv_heads);
 *  - k = k_scale * stored(k), v = v_scale * stored(v) (pass 1.0 for 16-bit
 *    caches); score = softmax_scale * dot(q, k);
 *  - lse = natural log of sum_t exp(score_t); a sequence with seq_len 0
 *    gets out = 0 and lse = -inf;
 *  - out is rounded once, to nearest even, into q's dtype.
 *
 * Ownership and synchronisation: every pointer argument is device memory
 * owned by the caller (except where a function says "host").  The library
 * allocates, frees and synchronises nothing inside fd_decode_attention; all
 * of its work is enqueued on `stream`.  The workspace is caller-owned scratch
 * memory of at least fd_workspace_bytes(...) bytes; it holds no state that
 * the caller must keep between calls except the sticky device-error word
 * read by fd_check_device_error.  Calls that share one workspace must be
 * ordered on one stream.
 *
 * Devices and host threads: calls run on the CUDA device current in the
 * calling thread, and several devices may be used from one process.  The
 * library keeps, per device, the SM count and whether each kernel's
 * shared-memory limit has been raised, and per process a small cache of TMA
 * descriptors keyed by cache pointer and shape; all of these are guarded for
 * concurrent calls from several host threads.  They are kept for the life of
 * the process: do not use the library on a device after cudaDeviceReset.
 */
#ifndef FD_ATTENTION_H_
#define FD_ATTENTION_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as a cudaStream_t / CUstream (NULL = the legacy default stream). */
typedef struct CUstream_st *fd_stream_t;
/* Same object as a cudaEvent_t / CUevent. */
typedef struct CUevent_st *fd_event_t;

typedef enum {
  FD_OK = 0,
  FD_ERR_INVALID_ARG = 1,          /* bad pointer, size or layout; nothing launched */
  FD_ERR_UNSUPPORTED = 2,          /* valid but not implemented (head_dim, dtype pair, ...) */
  FD_ERR_WORKSPACE_TOO_SMALL = 3,  /* workspace_bytes < fd_workspace_bytes(...) */
  FD_ERR_CUDA = 4,                 /* a CUDA runtime call or launch failed */
  FD_ERR_DEVICE_BOUNDS = 5,        /* a kernel met a cache row / page id out of range */
  FD_ERR_DEVICE_TIMEOUT = 6        /* a kernel's bounded wait expired */
} fd_status;

/* Element formats.  FD_I8 is a symmetric signed 8-bit code: the element's
 * value is the two's-complement integer (-128 .. 127) times its scales, no
 * zero point ("Learn CUDA from scratch, chapter 15", section 15.11: INT8 K/V
 * payloads with fp32 scales). */
typedef enum { FD_F16 = 0, FD_BF16 = 1, FD_E4M3 = 2, FD_I8 = 3 } fd_dtype;

/* Kernel selection for the split (partial attention) phase. */
typedef enum {
  FD_KERNEL_AUTO = 0,  /* FD_KERNEL_TC for one KV head with at least 64 query rows (query
                          heads times q_len), else FD_KERNEL_MMA where supported, else the
                          CUDA-core kernel */
  FD_KERNEL_SIMT = 1,  /* CUDA-core FMA kernel (every supported shape) */
  FD_KERNEL_MMA = 2,   /* tensor-core kernel with warp-level mma.sync products, operands
                          widened in registers; FD_ERR_UNSUPPORTED where it does not apply */
  FD_KERNEL_TC = 3,    /* tensor-core kernel with tcgen05 products (accumulators in tensor
                          memory, FP8 widened once per tile into shared memory): e4m3
                          caches, fp16 queries, head_dim 128, 17..128 query rows per KV
                          head (query heads per KV head times q_len), no per-token scales,
                          page sizes 8..256; FD_ERR_UNSUPPORTED elsewhere */
  FD_KERNEL_FMA = 4    /* the mma.sync kernel's TMA pipeline, plan and shapes with CUDA-core
                          FMA arithmetic instead of tensor cores (the comparison arm): e4m3
                          caches, head_dim 128, at most 8 query rows per KV head, KV heads a
                          multiple of 8, no per-token scales, page sizes of at least 8;
                          FD_ERR_UNSUPPORTED elsewhere; never chosen by FD_KERNEL_AUTO */
} fd_kernel;

/*
 * Scratch bytes fd_decode_attention needs for these sizes on the current
 * device (host function, no device work).  Returns 0 for invalid sizes.
 * The figure covers the partial (m, l, acc) states of the split phase, the
 * per-stream tile prefix of the split plan and a 256-byte header; it grows
 * with the device's SM count, not with sequence lengths.  For
 * fd_decode_attention_multi pass num_q_heads * q_len as num_q_heads.
 */
size_t fd_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int head_dim);

/*
 * One decode step of attention (see the file comment for the definition).
 *
 * q            [batch, num_q_heads, head_dim] of q_dtype (FD_F16 or FD_BF16).
 * k_cache, v_cache
 *              contiguous: [kv_rows, num_kv_heads, head_dim] of kv_dtype;
 *              paged: [kv_rows / page_size, page_size, num_kv_heads, head_dim].
 *              Base addresses 16-byte aligned.
 * kv_start_idx int32 [batch] first row of each sequence (contiguous mode), or NULL.
 * block_table  int32 [batch, block_table_stride] page ids (paged mode), or NULL.
 *              Exactly one of kv_start_idx / block_table is non-NULL.  Entries
 *              past ceil(seq_len[b] / page_size) are never read.
 * seq_len      int32 [batch] tokens per sequence (0 allowed; negative = 0).
 * kv_rows      number of token rows K and V hold (paged: pages * page_size).
 *              Rows outside [0, kv_rows) are never read: the kernel records
 *              FD_ERR_DEVICE_BOUNDS in the workspace and treats the token as
 *              absent.
 * num_q_heads, num_kv_heads
 *              num_q_heads % num_kv_heads == 0; group = num_q_heads / num_kv_heads <= 128.
 * head_dim     64 or 128.
 * page_size    paged mode: power of two in [1, 256]; contiguous mode: ignored.
 * softmax_scale, k_scale, v_scale
 *              finite fp32 factors (scores use softmax_scale * k_scale).
 * kv_dtype     FD_F16 (with q FD_F16), FD_BF16 (with q FD_BF16), FD_E4M3
 *              (OCP e4m3fn, with either q dtype) or FD_I8 (signed 8-bit
 *              codes, with either q dtype).
 * out          [batch, num_q_heads, head_dim] of q_dtype.
 * lse          fp32 [batch, num_q_heads], or NULL if not wanted.
 * workspace    device scratch of workspace_bytes >= fd_workspace_bytes(...),
 *              256-byte aligned.
 *
 * Returns FD_OK once the work is enqueued; argument errors return before any
 * launch.  Device-side index errors surface through fd_check_device_error.
 */
fd_status fd_decode_attention(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *kv_start_idx, const int32_t *block_table,
                              int block_table_stride, const int32_t *seq_len, int64_t kv_rows,
                              int batch, int num_q_heads, int num_kv_heads, int head_dim,
                              int page_size, float softmax_scale, float k_scale, float v_scale,
                              fd_dtype q_dtype, fd_dtype kv_dtype, void *out, float *lse,
                              void *workspace, size_t workspace_bytes, fd_stream_t stream);

/* Granularity of the finer K/V scales of fd_decode_attention_scaled. */
typedef enum {
  FD_SCALE_TENSOR = 0, /* none: k_scale / v_scale only                           */
  FD_SCALE_HEAD = 1,   /* one fp32 per KV head: k_scales[kvh]                     */
  FD_SCALE_TOKEN = 2   /* one fp32 per cache row and KV head: k_scales[row * KVH + kvh] */
} fd_scale_kind;

/*
 * fd_decode_attention with finer FP8 / INT8 scales ("Learn CUDA from scratch,
 * chapter 15", section 15.11: KV quantisation with a scale per tensor, per
 * head or per token).  The K and V elements of cache row `row` and KV head
 * `kvh` are decoded as
 *     k = k_scale * ks * dec(code),   v = v_scale * vs * dec(code),
 * with ks = k_scales[kvh], vs = v_scales[kvh] (FD_SCALE_HEAD) or
 * ks = k_scales[row * num_kv_heads + kvh], vs likewise (FD_SCALE_TOKEN; `row`
 * is the cache row of the token, contiguous or paged, the same index the
 * caches use).  FD_SCALE_TENSOR ignores both arrays and equals
 * fd_decode_attention.
 *
 * k_scales, v_scales  device fp32 arrays, 4-byte aligned: [num_kv_heads]
 *                     (FD_SCALE_HEAD) or [kv_rows * num_kv_heads]
 *                     (FD_SCALE_TOKEN); NULL only with FD_SCALE_TENSOR.
 * Finer scales need kv_dtype FD_E4M3 or FD_I8 (else FD_ERR_UNSUPPORTED).  Every other
 * argument, the workspace contract and the errors are those of
 * fd_decode_attention.
 */
fd_status fd_decode_attention_scaled(const void *q, const void *k_cache, const void *v_cache,
                                     const int32_t *kv_start_idx, const int32_t *block_table,
                                     int block_table_stride, const int32_t *seq_len,
                                     int64_t kv_rows, int batch, int num_q_heads,
                                     int num_kv_heads, int head_dim, int page_size,
                                     float softmax_scale, float k_scale, float v_scale,
                                     fd_scale_kind scale_kind, const float *k_scales,
                                     const float *v_scales, fd_dtype q_dtype, fd_dtype kv_dtype,
                                     void *out, float *lse, void *workspace,
                                     size_t workspace_bytes, fd_stream_t stream);

/*
 * Decode attention for q_len query tokens per sequence (a speculative-decoding
 * verify batch, "Learn CUDA from scratch, chapter 15", section 15.21: the
 * target model checks q_len drafted tokens in one pass).  The last q_len
 * tokens of each sequence are the new ones and are already in the cache
 * (seq_len counts them): query token j (0 <= j < q_len) sits at position
 * seq_len[b] - q_len + j and attends to keys 0 .. seq_len[b] - q_len + j, its
 * own and every earlier one (causal among the new tokens), with the
 * definition of fd_decode_attention.  A query with no key (seq_len[b] <
 * q_len - j) gets out = 0 and lse = -inf.
 *
 * q, out  [batch, num_q_heads, q_len, head_dim] of q_dtype (head-major: the
 *         q_len tokens of one head are adjacent rows).
 * lse     fp32 [batch, num_q_heads, q_len], or NULL.
 * q_len   1 .. 16, with (num_q_heads / num_kv_heads) * q_len <= 128 (else
 *         FD_ERR_UNSUPPORTED); q_len = 1 equals fd_decode_attention_scaled.
 * workspace_bytes >= fd_workspace_bytes(batch, num_q_heads * q_len, ...).
 * Every other argument as for fd_decode_attention_scaled.
 */
fd_status fd_decode_attention_multi(const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *kv_start_idx, const int32_t *block_table,
                                    int block_table_stride, const int32_t *seq_len,
                                    int64_t kv_rows, int batch, int q_len, int num_q_heads,
                                    int num_kv_heads, int head_dim, int page_size,
                                    float softmax_scale, float k_scale, float v_scale,
                                    fd_scale_kind scale_kind, const float *k_scales,
                                    const float *v_scales, fd_dtype q_dtype, fd_dtype kv_dtype,
                                    void *out, float *lse, void *workspace,
                                    size_t workspace_bytes, fd_stream_t stream);

/*
 * KV-cache append of one new token per sequence ("Learn CUDA from scratch,
 * chapter 15", section 15.9: cache write layouts, contiguous and paged, and
 * the single-token decode append; quantisation with the scales of section
 * 15.11; n_new > 1: the drafted tokens of a speculative verify step,
 * section 15.21).  For every sequence b with positions[b] >= 0, every new
 * token i < n_new and every KV head h, with t = positions[b] + i, the row
 * r = kv_start_idx[b] + t (contiguous) or
 * block_table[b][t / page_size] * page_size + t % page_size (paged) of K
 * receives k_new[b][i][h][0 .. head_dim), and V likewise:
 *   16-bit cache (kv_dtype == new_dtype): the elements as they are;
 *   8-bit cache (FD_E4M3 or FD_I8), QMAX = 448 or 127, s the element's scale:
 *     s = k_scale                                  FD_SCALE_TENSOR
 *       = k_scale * k_scales[h]                    FD_SCALE_HEAD
 *       = k_scale * ks,  ks = amax / (QMAX * k_scale), stored to
 *         k_scales[r * num_kv_heads + h], amax = max_d |k_new[b][i][h][d]|
 *         (ks = 1 when amax = 0)                   FD_SCALE_TOKEN
 *     code = e4m3: nearest to x / s, ties to even, |x / s| > 448 -> 448;
 *            int8: nearest integer to x / s, ties to even, clamped to +-127.
 *   Each product and quotient above is one IEEE fp32 operation.
 *
 * k_new, v_new  [batch, n_new, num_kv_heads, head_dim] of new_dtype (FD_F16
 *               or FD_BF16), 16-byte aligned, device.
 * n_new         new tokens per sequence, 1 .. 16.
 * k_cache, v_cache, kv_start_idx, block_table, block_table_stride, kv_rows,
 * page_size     as for fd_decode_attention; the caches are written.
 * positions     int32 [batch] device: the first new token's index in its
 *               sequence; < 0 leaves the sequence alone.  The block table
 *               must cover positions[b] + n_new - 1.  Rows outside [0, kv_rows) or
 *               negative page ids are not written and are recorded as
 *               FD_ERR_DEVICE_BOUNDS (fd_check_device_error).
 * k_scale, v_scale  finite; > 0 for 8-bit caches.
 * scale_kind, k_scales, v_scales  as for fd_decode_attention_scaled; with
 *               FD_SCALE_TOKEN the arrays are written at the appended rows.
 * workspace     >= 256 bytes, 256-byte aligned (the device error word); the
 *               attention's workspace serves.
 * Writes nothing but the appended rows (and their per-token scales).  Two
 * sequences whose new rows coincide race; callers give distinct rows.
 */
fd_status fd_append_kv(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                       const int32_t *kv_start_idx, const int32_t *block_table,
                       int block_table_stride, const int32_t *positions, int64_t kv_rows,
                       int batch, int n_new, int num_kv_heads, int head_dim, int page_size,
                       float k_scale, float v_scale, fd_scale_kind scale_kind, float *k_scales,
                       float *v_scales, fd_dtype new_dtype, fd_dtype kv_dtype, void *workspace,
                       size_t workspace_bytes, fd_stream_t stream);

/*
 * One decode (q_len = 1) or verify (q_len > 1) step with its KV append:
 * fd_append_kv of the step's q_len new tokens (k_new, v_new
 * [batch, q_len, num_kv_heads, head_dim] of q_dtype, the first at
 * `positions`), then fd_decode_attention_multi over the caches that now hold
 * them, in one call.  seq_len counts the new tokens (typically
 * positions[b] + q_len).  The split kernel of the attention is
 * launched as a programmatic dependent of the append: its plan overlaps the
 * append, and it waits for the append's writes before reading K/V.
 * Arguments and errors are those of the two functions; nothing is launched
 * when any argument is invalid.
 */
fd_status fd_decode_attention_append(const void *q, const void *k_new, const void *v_new,
                                     void *k_cache, void *v_cache, const int32_t *kv_start_idx,
                                     const int32_t *block_table, int block_table_stride,
                                     const int32_t *positions, const int32_t *seq_len,
                                     int64_t kv_rows, int batch, int q_len, int num_q_heads,
                                     int num_kv_heads, int head_dim, int page_size,
                                     float softmax_scale, float k_scale, float v_scale,
                                     fd_scale_kind scale_kind, float *k_scales, float *v_scales,
                                     fd_dtype q_dtype, fd_dtype kv_dtype, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, fd_stream_t stream);

/*
 * One decode step whose queries see a sliding window and the first tokens: the
 * query of sequence b, at position seq_len[b] - 1, attends to the tokens t with
 *     t >= seq_len[b] - window   or   t < sinks,
 * with the definition of fd_decode_attention over these.  With k_new the step's
 * new token is appended first, as by fd_decode_attention_append (q_len = 1);
 * without (k_new, v_new and positions NULL) the caches hold it and are only
 * read.
 *
 * A sequence longer than its row of the block table is recorded as
 * FD_ERR_DEVICE_BOUNDS, and the tiles past the row's end are absent.
 * Block-table entries of pages none of whose tokens the query sees are not
 * used, so such pages may have been given away (fd_assign_pages does that; see
 * there for sequences that it refuses) and their entries may hold anything.
 * Rows of hidden tokens have no effect, whatever bits they hold; in a contiguous
 * cache they must lie inside it (they share tiles with visible ones).
 *
 * window     >= 1 (1: the query's own token); longer than a sequence: all of it.
 * sinks      >= 0.
 * FD_KERNEL_AUTO and FD_KERNEL_MMA only (the mma.sync kernel runs), else
 * FD_ERR_UNSUPPORTED.  Workspace, other arguments and errors are those of
 * fd_decode_attention_append.
 */
fd_status fd_decode_attention_window(const void *q, const void *k_new, const void *v_new,
                                     void *k_cache, void *v_cache, const int32_t *kv_start_idx,
                                     const int32_t *block_table, int block_table_stride,
                                     const int32_t *positions, const int32_t *seq_len,
                                     int64_t kv_rows, int batch, int num_q_heads,
                                     int num_kv_heads, int head_dim, int page_size, int window,
                                     int sinks, float softmax_scale, float k_scale, float v_scale,
                                     fd_scale_kind scale_kind, float *k_scales, float *v_scales,
                                     fd_dtype q_dtype, fd_dtype kv_dtype, void *out, float *lse,
                                     void *workspace, size_t workspace_bytes, fd_stream_t stream);

/*
 * Same computation as fd_decode_attention, for callers that cannot allocate
 * device memory (for example code running inside a framework that does not
 * expose its allocator, or under a fixed memory budget).  The pages have no
 * counterpart of this function; it exists only for those callers.
 *
 * Arguments are those of fd_decode_attention without the workspace: the
 * scratch memory is a 16 MiB array compiled into the library, which every
 * GPU that loads the library holds until the process exits.  Sizes whose
 * fd_workspace_bytes(...) exceeds 16 MiB return FD_ERR_WORKSPACE_TOO_SMALL
 * before any launch.  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) with that device current; make that first
 * call before any stream capture.  Each call first clears the array's
 * device-error word, so device-side bounds errors of this entry point are not
 * reported; use fd_decode_attention when they must be.  All calls share the
 * one array: calls that can overlap on the GPU (different streams, or
 * different host threads) race on it and must be serialised by the caller.
 * Nothing is allocated or freed.  Invalid or unsupported arguments get the
 * same status as from fd_decode_attention.  The array's address is kept for
 * the life of the process: do not call this entry point after
 * cudaDeviceReset.
 */
fd_status fd_decode_attention_noalloc(const void *q, const void *k_cache, const void *v_cache,
                                      const int32_t *kv_start_idx, const int32_t *block_table,
                                      int block_table_stride, const int32_t *seq_len,
                                      int64_t kv_rows, int batch, int num_q_heads,
                                      int num_kv_heads, int head_dim, int page_size,
                                      float softmax_scale, float k_scale, float v_scale,
                                      fd_dtype q_dtype, fd_dtype kv_dtype, void *out, float *lse,
                                      fd_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The prompt path: everything between a prompt and its first decode step.
 *
 * Packed tokens.  The new tokens of a batch lie behind one another without
 * padding: q_start is a device int32 array [batch + 1], ascending, and
 * sequence b owns tokens q_start[b] .. q_start[b + 1] - 1 of every packed
 * array (none, one or many; a decode step's single tokens and a prompt's
 * thousands may share one call).  Tokens outside [q_start[0],
 * q_start[batch]) belong to no sequence: nothing is read for them and their
 * rows of every output are left as they were.  A sequence whose entries
 * descend or lie outside the packed arrays is skipped and recorded as
 * FD_ERR_DEVICE_BOUNDS (info: the offending entry); where entries descend,
 * tokens outside that range, or claimed by two of the other sequences, are
 * served for one of them or not at all.  A call of no packed rows has nothing
 * to do; its packed arrays may then be NULL.
 *
 * Caches, block tables, scales, dtypes, workspaces, streams and errors are
 * those of the decode entry points above, and so are the addressing rules:
 * rows outside [0, kv_rows), negative page ids and pages past
 * block_table_stride are never touched and are recorded as
 * FD_ERR_DEVICE_BOUNDS.
 * ---------------------------------------------------------------------------
 */

/* How rotary frequencies are scaled for contexts longer than the trained one. */
typedef enum {
  FD_ROTARY_PLAIN = 0,   /* f_i */
  FD_ROTARY_LINEAR = 1,  /* f_i / factor (positions compressed by factor) */
  FD_ROTARY_BY_PARTS = 2 /* by the turns r_i = original_positions * f_i / (2 pi) that a pair makes
                            over the trained context: g f_i + (1 - g) f_i / factor,
                            g = clamp((r_i - low_turns) / (high_turns - low_turns), 0, 1) */
} fd_rotary_scaling;

/*
 * Table of rotary positions: row p (0 <= p < positions) of `table` holds
 * amplitude * cos(p g_i) for i = 0 .. rot_dim / 2 - 1, then
 * amplitude * sin(p g_i), with g_i the scaled frequency of
 * f_i = theta^(-2 i / rot_dim).  Angles are exact to about 2^-53 of a turn per
 * position (fixed-point turns), so far positions keep fp32 accuracy.
 *
 * table      device fp32 [positions, rot_dim], 16-byte aligned.
 * positions  1 .. 2^31 - 1.
 * rot_dim    multiple of 16, 16 .. 128.
 * theta      finite, > 1.   factor  finite, >= 1 (ignored by FD_ROTARY_PLAIN).
 * original_positions > 0 and 0 <= low_turns < high_turns, finite
 *            (FD_ROTARY_BY_PARTS only).
 * amplitude  finite.
 */
fd_status fd_rotary_table(float *table, int64_t positions, int rot_dim, double theta,
                          fd_rotary_scaling scaling, double factor, double original_positions,
                          double low_turns, double high_turns, float amplitude,
                          fd_stream_t stream);

/*
 * Writes packed new tokens into the caches, any number per sequence, with
 * optional rotary positions.  Token i of sequence b (packed index
 * q_start[b] + i) stands at position t = positions[b] + i and goes to that
 * token's cache row, as in fd_append_kv (16-bit caches: the elements rounded
 * once to the cache's type; 8-bit caches: the codes and scales of
 * fd_append_kv).  With a rotary table, pair (x1, x2) i of the first rot_dim
 * dims of every query and key head becomes
 *     y1 = x1 cos_i - x2 sin_i,   y2 = x2 cos_i + x1 sin_i
 * (row t of the table) before that; values are not rotated.  A pair is dims
 * (i, i + rot_dim / 2), or with `interleaved` non-zero dims (2 i, 2 i + 1).
 * Each product, sum and quotient is one IEEE fp32 operation; keys enter the
 * 8-bit quantisation unrounded.
 *
 * q          [num_tokens, num_q_heads, head_dim] of new_dtype, tokens
 *            q_stride elements apart, or NULL (only k and v are written).
 * q_out      dense [num_tokens, num_q_heads, head_dim]; may equal q when q is
 *            dense, and must not overlap q (otherwise), k_new or v_new.
 *            Required with q.
 * k_new, v_new  [num_tokens, num_kv_heads, head_dim] of new_dtype, tokens
 *            kv_stride elements apart.
 * q_stride, kv_stride  multiples of 8 elements, at least one token's heads
 *            (so q, k and v may be slices of one projection's output).
 * positions  int32 [batch]: position of each sequence's first new token;
 *            < 0 leaves the sequence alone (its q_out rows too).
 * num_tokens rows of the packed arrays (0: nothing to do); < 2^31.
 * rotary     table of fd_rotary_table, [rotary_positions, rot_dim] fp32,
 *            16-byte aligned, or NULL (no rotation).  A token at or past
 *            rotary_positions is skipped and recorded as FD_ERR_DEVICE_BOUNDS.
 * rot_dim    multiple of 16, 16 .. head_dim (ignored without a table).
 * The other arguments are those of fd_append_kv.  Two tokens that share a
 * cache row race; callers give distinct rows.
 */
fd_status fd_append_kv_packed(const void *q, int64_t q_stride, void *q_out, const void *k_new,
                              const void *v_new, int64_t kv_stride, void *k_cache, void *v_cache,
                              const int32_t *kv_start_idx, const int32_t *block_table,
                              int block_table_stride, const int32_t *q_start,
                              const int32_t *positions, int64_t num_tokens, int64_t kv_rows,
                              int batch, int num_q_heads, int num_kv_heads, int head_dim,
                              int page_size, const float *rotary, int64_t rotary_positions,
                              int rot_dim, int interleaved, float k_scale, float v_scale,
                              fd_scale_kind scale_kind, float *k_scales, float *v_scales,
                              fd_dtype new_dtype, fd_dtype kv_dtype, void *workspace,
                              size_t workspace_bytes, fd_stream_t stream);

/*
 * fd_append_kv_packed with norms of query and key heads, and with rotary
 * positions on several axes.  In the same pass, before the rotation, a head x
 * of q becomes
 *     x_d / sqrt(sum_d x_d^2 / head_dim + norm_eps) * q_norm[d],
 * a head of k_new the same with k_norm; either may be NULL (that tensor is not
 * normed).  Values are not normed.  The sum of squares is known to 2^-40 of
 * itself and then rounded to fp32 once: it is the exact sum rounded, unless that
 * lies so near the middle of two fp32 numbers, where it may be either of them
 * (and depend on the elements' places).  The products, the quotient 1 / sqrt and
 * the rotation are single fp32 operations, and nothing is rounded to 16 bits in
 * between.  (A sum of squares beyond fp32's range is infinite: finite elements
 * become zero.  Squares below 2^-149 are rounded to a multiple of it.)
 *
 * q_norm, k_norm  device arrays [head_dim] of new_dtype, or of fp32 with
 *             norm_f32 non-zero, aligned to their elements; q_norm needs q.
 * norm_eps    finite, > 0 (ignored without q_norm and k_norm).
 * axis_positions  device int32 [num_axes], axis_stride apart: entry i of axis a
 *             is packed token i's position on it.  Pair i of the rotation takes
 *             row axis_positions[pair_axis[i]] of the table instead of the
 *             token's place in its sequence, which still decides its cache row.
 *             A token with an entry outside [0, rotary_positions) is skipped and
 *             recorded as FD_ERR_DEVICE_BOUNDS.
 * num_axes    0 (no axes: as fd_append_kv_packed) .. 4.
 * axis_stride at least num_tokens, < 2^31.
 * pair_axis   HOST array of rot_dim / 2 axes, each < num_axes; read during the
 *             call.  Runs of pairs for one axis and pairs taking turns are both
 *             ways to fill it.
 */
fd_status fd_append_kv_normed(const void *q, int64_t q_stride, void *q_out,
                              const void *k_new, const void *v_new, int64_t kv_stride,
                              void *k_cache, void *v_cache, const int32_t *kv_start_idx,
                              const int32_t *block_table, int block_table_stride,
                              const int32_t *q_start, const int32_t *positions,
                              int64_t num_tokens, int64_t kv_rows, int batch,
                              int num_q_heads, int num_kv_heads, int head_dim,
                              int page_size, const float *rotary, int64_t rotary_positions,
                              int rot_dim, int interleaved, const void *q_norm,
                              const void *k_norm, int norm_f32, float norm_eps,
                              const int32_t *axis_positions, int num_axes,
                              int64_t axis_stride, const uint8_t *pair_axis, float k_scale,
                              float v_scale, fd_scale_kind scale_kind, float *k_scales,
                              float *v_scales, fd_dtype new_dtype, fd_dtype kv_dtype,
                              void *workspace, size_t workspace_bytes, fd_stream_t stream);

/*
 * Reads cached tokens back as packed 16-bit rows: packed row i of sequence b
 * (out_start[b] <= i < out_start[b + 1]) receives token
 * first[b] + i - out_start[b] of that sequence,
 *     k = round(k_scale * ks * dec(code)),   v likewise,
 * the decode entry points' values, rounded once to out_dtype (the products of
 * scales and of scale and element are single fp32 operations).
 *
 * out_start  int32 [batch + 1], packed as q_start above.
 * first      int32 [batch] first token of each sequence, or NULL for 0; < 0
 *            leaves the sequence's rows as they were.
 * num_rows   rows of k_out and v_out (0: nothing to do); < 2^31.
 * k_out, v_out  dense [num_rows, num_kv_heads, head_dim] of out_dtype (FD_F16
 *            or FD_BF16; that of a 16-bit cache), 16-byte aligned.
 * Rows of tokens outside the cache receive zeros and are recorded.
 */
fd_status fd_read_kv(const void *k_cache, const void *v_cache, const int32_t *kv_start_idx,
                     const int32_t *block_table, int block_table_stride,
                     const int32_t *out_start, const int32_t *first, int64_t num_rows,
                     int64_t kv_rows, int batch, int num_kv_heads, int head_dim, int page_size,
                     float k_scale, float v_scale, fd_scale_kind scale_kind,
                     const float *k_scales, const float *v_scales, fd_dtype kv_dtype,
                     fd_dtype out_dtype, void *k_out, void *v_out, void *workspace,
                     size_t workspace_bytes, fd_stream_t stream);

/* Scratch bytes fd_assign_pages needs (host function); 0 for an invalid batch. */
size_t fd_assign_pages_workspace_bytes(int batch);

/*
 * Pages of one step's requests: grows and shrinks the block tables of a batch by
 * its requests' new tokens, on the device, and says where the packed new tokens
 * go.  In the words of the packed calls above: it makes q_start, positions and
 * seq_len for them.
 *
 * Sequence b has L = seq_len[b] tokens cached (negative: 0) in the first
 * ceil(L / page_size) columns of its row of the table, and gets
 * n = new_tokens[b] new ones; n < 0 says that it has ended.  Free pages are a
 * stack, free_pages[0 .. free_count[0]).
 *
 * Pages that go back:
 *   an ended sequence's pages;
 *   with a window (> 0), of a sequence that goes on the pages that neither its
 *   new tokens nor later ones see: columns c with c * page_size >= sinks and
 *   (c + 1) * page_size <= L - window + 1.
 *   released[b] is the first column that has not gone back so far (0 for a new
 *   sequence; columns below ceil(sinks / page_size) only go when the sequence
 *   ends), released_out[b] the one after this call.  The attention entry points
 *   with this window and these sinks do not use the entries of pages that are
 *   gone for tokens at L and later, nor does this one; they are left in the
 *   table.  Earlier tokens see further back: a refused sequence's n tokens,
 *   which an attention call given seq_len_out takes for those at L - n .. L - 1,
 *   and a decode query of a sequence without new tokens, at L - 1.  With a window
 *   the step's attention is therefore given fd_assign_pages_attended's attend_len
 *   as its seq_len wherever a sequence may be refused or has no new tokens.
 * They are put on the stack in order of sequences, then columns.  A page must
 * belong to one sequence alone (prefix pages that several rows name are not for
 * this call).  Ids are moved as they are.
 *
 * Pages handed out, from the top of the stack with those on it: in order of
 * sequences, then columns, ceil((L + n) / page_size) - ceil(L / page_size) for
 * each sequence, as long as they last.  A sequence is served when it needs no
 * page, or when the pages wanted up to and with it do not pass those there are
 * (so behind the first that is refused, only such as need none).  A served
 * sequence has positions[b] = L and seq_len_out[b] = L + n; an ended one -1 and
 * 0; a refused one -1 and L: the packed append leaves its tokens alone, and it
 * may ask again.  A sequence whose pages do not fit its row of the table, or
 * whose tokens do not fit the slots (or end beyond 2^31 - 1, where q_start
 * stays), is refused and recorded as FD_ERR_DEVICE_BOUNDS, as is a stack that
 * overflows (its last pages are lost).
 *
 * block_table  int32 [batch, block_table_stride], updated: only the columns of
 *              pages handed out are written. Fewer than 2^31 entries.
 * free_pages   int32 [free_capacity], updated: entries from free_count on are
 *              written by pages that go back, others never (a page handed out
 *              stays where it was, behind the new count).
 * page_size    power of two in [1, 256].
 * window, sinks  0, 0: no window; then released and released_out are NULL.
 * seq_len_out, free_count_out [1], released_out  the state after the call; each
 *              may be the same array as the one before it.
 * q_start      int32 [batch + 1]: running sum of max(new_tokens, 0), refused
 *              sequences' tokens included.
 * slots        int64 [num_slots], or NULL with 0: entry i is the cache row of
 *              packed token i, -1 if it is not served, and -1 behind the last.
 * workspace    >= fd_assign_pages_workspace_bytes(batch), 256-byte aligned.
 * No array may overlap another, other than the pairs named (FD_ERR_INVALID_ARG).
 */
fd_status fd_assign_pages(int32_t *block_table, int block_table_stride, const int32_t *seq_len,
                          const int32_t *new_tokens, int32_t *free_pages, int64_t free_capacity,
                          const int32_t *free_count, int batch, int page_size, int window,
                          int sinks, const int32_t *released, int32_t *seq_len_out,
                          int32_t *free_count_out, int32_t *released_out, int32_t *q_start,
                          int32_t *positions, int64_t *slots, int64_t num_slots,
                          void *workspace, size_t workspace_bytes, fd_stream_t stream);

/*
 * fd_assign_pages that also says how many tokens of each sequence this step's
 * attention looks at:
 *
 * attend_len   int32 [batch], or NULL: L + n of a served sequence with n > 0 new
 *              tokens, 0 of every other.  As seq_len of the attention calls it
 *              leaves refused, ended and idle sequences without a key: their
 *              output rows are zero with lse = -inf, and none of their entries
 *              of the block table is used.
 */
fd_status fd_assign_pages_attended(int32_t *block_table, int block_table_stride,
                                   const int32_t *seq_len, const int32_t *new_tokens,
                                   int32_t *free_pages, int64_t free_capacity,
                                   const int32_t *free_count, int batch, int page_size,
                                   int window, int sinks, const int32_t *released,
                                   int32_t *seq_len_out, int32_t *free_count_out,
                                   int32_t *released_out, int32_t *q_start, int32_t *positions,
                                   int64_t *slots, int64_t num_slots, int32_t *attend_len,
                                   void *workspace, size_t workspace_bytes, fd_stream_t stream);

/* Scratch bytes fd_prefill_attention needs on the current device (host
 * function), for any batch, lengths and head counts; 0 for an invalid
 * head_dim. */
size_t fd_prefill_workspace_bytes(int head_dim);

/*
 * Attention of packed new tokens over the caches, which already hold them:
 * the prompt (or a chunk of it, or single tokens) of every sequence.  The
 * last n = q_start[b + 1] - q_start[b] tokens of sequence b's seq_len[b] are
 * the new ones; new token j sits at position seq_len[b] - n + j and attends
 * to its own and every earlier key, with the definition of
 * fd_decode_attention.  A token with no key (seq_len[b] < n - j) gets out = 0
 * and lse = -inf.  Cached rows past a token's position, rows of other
 * sequences and unused pages have no effect, whatever bits they hold.
 * Probabilities are rounded to q_dtype before they multiply V (with
 * FD_SCALE_TOKEN: times their V scale).  With f16 queries a probability below
 * about 2^-20 keeps an absolute error of 2^-31, with FD_SCALE_TOKEN 2^-31 of
 * the largest |V scale| that the token sees: a seen scale above about 2^10
 * times the others (the scale 1 of an appended row of zeros among them, where
 * v_scale leaves the others far below 1) costs those precision, even where its
 * own probability is small.  bf16 queries have no such floor.
 *
 * q          [num_tokens, num_q_heads, head_dim] of q_dtype, tokens q_stride
 *            elements apart (a multiple of 8, at least one token's heads).
 * out        dense [num_tokens, num_q_heads, head_dim] of q_dtype; must not
 *            overlap q, whose rows are read by more than one thread block.
 * lse        fp32 [num_tokens, num_q_heads], or NULL.
 * num_tokens rows of q, out and lse (0: nothing to do); < 2^31.
 * workspace  >= fd_prefill_workspace_bytes(head_dim), 256-byte aligned.
 * A 128-key tile that holds a row outside the cache is treated as absent and
 * recorded.  kv_rows < 2^31.  Every other argument as for
 * fd_decode_attention_scaled.
 */
fd_status fd_prefill_attention(const void *q, int64_t q_stride, const void *k_cache,
                               const void *v_cache, const int32_t *kv_start_idx,
                               const int32_t *block_table, int block_table_stride,
                               const int32_t *q_start, const int32_t *seq_len,
                               int64_t num_tokens, int64_t kv_rows, int batch, int num_q_heads,
                               int num_kv_heads, int head_dim, int page_size,
                               float softmax_scale, float k_scale, float v_scale,
                               fd_scale_kind scale_kind, const float *k_scales,
                               const float *v_scales, fd_dtype q_dtype, fd_dtype kv_dtype,
                               void *out, float *lse, void *workspace, size_t workspace_bytes,
                               fd_stream_t stream);

/*
 * fd_prefill_attention with a sliding window and first tokens: the new token at
 * position p attends to the tokens t <= p with t > p - window or t < sinks.
 * window and sinks, and what is said of hidden tokens' pages and rows, as for
 * fd_decode_attention_window (a page is hidden when no new token of its
 * sequence sees any of its tokens); every other argument, the workspace and the
 * errors as for fd_prefill_attention.
 */
fd_status fd_prefill_attention_window(const void *q, int64_t q_stride, const void *k_cache,
                                      const void *v_cache, const int32_t *kv_start_idx,
                                      const int32_t *block_table, int block_table_stride,
                                      const int32_t *q_start, const int32_t *seq_len,
                                      int64_t num_tokens, int64_t kv_rows, int batch,
                                      int num_q_heads, int num_kv_heads, int head_dim,
                                      int page_size, int window, int sinks, float softmax_scale,
                                      float k_scale, float v_scale, fd_scale_kind scale_kind,
                                      const float *k_scales, const float *v_scales,
                                      fd_dtype q_dtype, fd_dtype kv_dtype, void *out, float *lse,
                                      void *workspace, size_t workspace_bytes,
                                      fd_stream_t stream);

/*
 * Synchronises `stream`, reads and clears the workspace's sticky device-error
 * word.  Returns FD_OK, FD_ERR_DEVICE_BOUNDS, FD_ERR_DEVICE_TIMEOUT or
 * FD_ERR_CUDA.  If info is not NULL it receives the first offending value
 * (a row or page id) or 0.
 */
fd_status fd_check_device_error(void *workspace, fd_stream_t stream, int64_t *info);

/* Static English text for a status code. */
const char *fd_status_string(fd_status status);

/* Process-wide choice of the split kernel (default FD_KERNEL_AUTO). */
fd_status fd_set_kernel(fd_kernel kernel);

/*
 * Kernel that fd_decode_attention would run for these sizes under the
 * current fd_set_kernel choice: FD_KERNEL_SIMT, FD_KERNEL_MMA, FD_KERNEL_TC or FD_KERNEL_FMA,
 * or -1 if the sizes are unsupported (num_q_heads counts every query token:
 * query heads times q_len).  The answer is for per-tensor or per-KV-head
 * scales; fd_selected_kernel_scaled answers for per-token scales too.  Host
 * function.
 */
int fd_selected_kernel(int num_q_heads, int num_kv_heads, int head_dim, fd_dtype q_dtype,
                       fd_dtype kv_dtype, int paged, int page_size);

/*
 * As fd_selected_kernel, for a call with finer K/V scales of `scale_kind`
 * (FD_SCALE_TENSOR gives the same answer as fd_selected_kernel): the kernel
 * that fd_decode_attention_scaled (or _multi, _append) would run, or -1 when
 * the call would return FD_ERR_UNSUPPORTED (for instance a forced
 * FD_KERNEL_TC or FD_KERNEL_FMA with FD_SCALE_TOKEN).  Host function.
 */
int fd_selected_kernel_scaled(int num_q_heads, int num_kv_heads, int head_dim, fd_dtype q_dtype,
                              fd_dtype kv_dtype, int paged, int page_size,
                              fd_scale_kind scale_kind);

/*
 * Profiling hook: when both events are non-NULL, fd_decode_attention records
 * `before` immediately before and `after` immediately after the split
 * kernel's launch on its stream, so that the split kernel can be timed by
 * itself.  NULL, NULL switches it off.  The setting is per host thread.
 */
fd_status fd_set_split_events(fd_event_t before, fd_event_t after);

/*
 * Test hook: copies the split plan of the last fd_decode_attention call that
 * used this workspace into host memory (synchronises `stream`).
 * plan[0..7] = {num_streams, streams_per_sequence, tile_tokens, grid,
 * total_units, units_per_cta, kernel, start_units}; stream j of sequence b
 * serves query heads [j * h, (j + 1) * h) with h = num_q_heads /
 * streams_per_sequence.  A stream with n > 0 tiles costs start_units + n
 * plan units (the start cost first), an empty stream none; CTA c takes units
 * [c * units_per_cta, (c + 1) * units_per_cta).
 * plan[8 .. 8 + num_streams] = exclusive prefix of units per stream
 * (num_streams + 1 values).  capacity = number of int32 that fit in plan.
 */
fd_status fd_debug_read_plan(const void *workspace, fd_stream_t stream, int32_t *plan,
                             int capacity);

/*
 * Test hook: gathers, with the kernels' own addressing, the stored K (or V)
 * row slice of every token of every sequence into dst, a dense device array
 * [sum_b seq_len[b], num_kv_heads, head_dim] of the cache element type,
 * sequences in order.  Rows out of range are written as zero bytes and
 * recorded like in fd_decode_attention.  Same layout arguments as
 * fd_decode_attention; workspace needs only the 256-byte header.
 */
fd_status fd_debug_gather_kv(const void *cache, const int32_t *kv_start_idx,
                             const int32_t *block_table, int block_table_stride,
                             const int32_t *seq_len, int64_t kv_rows, int batch,
                             int num_kv_heads, int head_dim, int page_size, fd_dtype kv_dtype,
                             void *dst, void *workspace, fd_stream_t stream);

/*
 * Test hook for the bounded waits of the tensor-core split kernel.  Every
 * wait of that kernel on its copy pipeline gives up after `wait_ns`
 * nanoseconds (0: the default of one second), records
 * FD_ERR_DEVICE_TIMEOUT in the workspace's error word and ends the CTA's
 * work; the asynchronous-error reporting this follows is the one of
 * "SGLang Prefill optimisation: dissecting FlashAttention kernel bottlenecks
 * with GPU Trace", section 4.2 (a device error is found by a later host
 * check, not at the launch).  With `starve_first_stage` non-zero the
 * producer of every CTA issues no copy, so the consumers' first wait runs out
 * with nothing in flight: the call itself returns FD_OK, its outputs are
 * undefined, and fd_check_device_error reports FD_ERR_DEVICE_TIMEOUT.  The
 * wait that drains copies already issued before a CTA exits keeps its own
 * one-second bound and reports FD_ERR_DEVICE_TIMEOUT too when it gives up.
 * Process-wide, from the next call on; wait_ns outside [0, 1e10] is
 * FD_ERR_INVALID_ARG.  The CUDA-core split kernel has no such waits.
 * fd_prefill_attention's waits keep the same limit, and its producer the same
 * switch.
 */
fd_status fd_debug_set_wait_limit(int64_t wait_ns, int starve_first_stage);

/*
 * Test hook: the segments of the split plan that each CTA of the split
 * kernel takes for these sizes, computed on the device by the split kernels'
 * own plan and segment walk (the plan of "Learn CUDA from scratch, chapter
 * 15", section 15.13: ragged batches scan their real lengths).  Arguments as
 * in fd_decode_attention_multi (paged: a block table is used, page_size its
 * page size; kv_start_idx, which the plan reads ahead for the first
 * segment of every CTA, may be NULL).  dst is a device int32 array of dst_len values, of which the
 * first grid * (1 + 5 * capacity_per_cta) are written: row c holds the
 * number of segments of CTA c, then (stream, t_begin, t_end, complete, slot)
 * for each of its first capacity_per_cta segments.  *grid_out (host) always
 * receives the grid; a dst_len too small for it returns FD_ERR_INVALID_ARG
 * before any launch.  A workspace of fd_workspace_bytes for these sizes is
 * needed (its plan words are written as by a decode call).  Asynchronous on
 * `stream`.
 */
fd_status fd_debug_plan_segments(const int32_t *seq_len, const int32_t *kv_start_idx, int batch,
                                 int q_len, int num_q_heads,
                                 int num_kv_heads, int head_dim, int paged, int page_size,
                                 fd_dtype q_dtype, fd_dtype kv_dtype, int32_t *dst,
                                 int64_t dst_len, int capacity_per_cta, int *grid_out,
                                 void *workspace,
                                 size_t workspace_bytes, fd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FD_ATTENTION_H_ */
