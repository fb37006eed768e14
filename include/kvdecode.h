/*
 * kvdecode.h -- C ABI of libkvdecode.so: single-token decode attention over a
 * long KV cache that reads only part of it (Quest-style block selection), and
 * what a server needs around it (positions and norms, a cache in pages, chunks
 * of new tokens, latent rows, eviction), for NVIDIA GB300 (sm_103a), one GPU.
 *
 * Sources, by page title and section:
 *  [QUEST]  "Sparse Attention -- Quest-style block-selector for long-context
 *           decode (#551)": "Method: Quest-style min/max block bounds",
 *           "S2/S3 engineering design" (fill op, selector op, FA-VEC block
 *           skip), "Knobs", "Gate ladder", "All-KV-types composition
 *           (bug-747)".
 *  [CPUATT] "cpu-attn" (Hugging Face kernels card): "Usage", "Method",
 *           "Correctness", "Requirements and limits".
 *  [SCSA]   "SCSA: Self-Calibrating Subquadratic Attention": "2. Mechanism"
 *           (the moment tail of the key groups not read exactly).
 *  [CERT]   "Certified Sparse Attention via Perturbed Retrieval": Appendix
 *           Table 4 (GQA-shared scan against one scan per query head).
 *
 * Conventions for every entry point
 *  - All device memory is allocated and owned by the caller.  The library
 *    never allocates or frees device memory and never synchronizes: every
 *    call enqueues its kernels on `stream` (a cudaStream_t passed as void*;
 *    NULL means the legacy default stream) and returns.
 *  - Arguments are checked on the host before anything is enqueued.  A call
 *    that returns anything but KVD_OK has enqueued nothing (the one
 *    exception, KVD_ERR_CUDA from a failed launch, is documented there).
 *  - Device pointers must be 16-byte aligned.  Layouts are dense row-major
 *    with the shapes given; no strides (kvd_heads, below, has one a token).
 *  - Faults found on the device (a bounded wait that ran out) are written to
 *    the cache's optional `dev_status` word (0 = fine); the kernels never
 *    trap.  Read the word after the stream has finished.
 *  - No call is thread-safe on the same cache or workspace; calls on one
 *    stream are ordered by the stream.  The library's own host state (per
 *    device: the SM count, the kernels' shared-memory attributes and
 *    occupancy, the workspace-free decode's array address) is filled once
 *    per device under a lock, so host threads driving different devices, or
 *    different caches on one device, may call at the same time.
 */
#ifndef KVDECODE_H
#define KVDECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVD_ABI_VERSION 5

/* Exported symbols (the library is built with hidden default visibility). */
#if defined(__GNUC__)
#define KVD_API __attribute__((visibility("default")))
#else
#define KVD_API
#endif

typedef enum {
    KVD_OK = 0,
    KVD_ERR_INVALID = 1,      /* bad argument: NULL/misaligned pointer, bad size */
    KVD_ERR_UNSUPPORTED = 2,  /* legal but not built: block != 64, a head_dim that is not
                                 a multiple of 16 in [16, 1024], ... */
    KVD_ERR_CAPACITY = 3,     /* append would pass max_seq */
    KVD_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
    KVD_ERR_TIMEOUT = 5,      /* device only: a bounded wait ran out (dev_status) */
    KVD_ERR_WORKSPACE = 6     /* workspace NULL, misaligned or too small */
} kvd_status;

/* KVD_BF16: paged caches only. */
typedef enum {
    KVD_F16 = 0,
    KVD_INT8 = 1,
    KVD_Q8_0 = 2,
    KVD_Q4_0 = 3,
    KVD_BF16 = 4
} kvd_kv_dtype;

/*
 * The cache: a plain descriptor of caller-owned device memory.
 *
 * Layout is head-major, so one block of `block` tokens of one (sequence,
 * KV head) is one contiguous run of memory:
 *   k, v        [batch, n_kv_heads, max_seq, head_dim]   f16 or int8 codes,
 *               or [.., head_dim / 2] bytes of 4-bit codes (q4_0)
 *   k_scale,    int8: [batch, n_kv_heads, max_seq] f32;
 *   v_scale     q8_0, q4_0: [batch, n_kv_heads, max_seq, head_dim / 32] f16
 *               (NULL for f16)
 *   kbounds     [batch, n_kv_heads, max_seq / block, head_dim, 2]  f16
 * kbounds holds the per-(KV head, block) channel-wise key envelope (QUEST,
 * Method: one minimum and one maximum per channel for every block) as interleaved
 * pairs: kbounds[..., d, 0] = kmin[d], kbounds[..., d, 1] = kmax[d] (one
 * contiguous 512-byte row per block).  It is always taken from the f16 keys
 * before quantization [QUEST All-KV-types composition].
 * int8 rows hold per-token per-head absmax codes [CPUATT Method]: scale =
 * absmax/127 (f32), code = round-half-even(x / scale) clamped to +-127, and
 * a row whose scale is 0 holds zero codes.
 * q8_0 rows hold the same codes per group of 32 channels (the llama.cpp
 * cache type of [QUEST] "All-KV-types composition"), each group with its
 * own f16 scale d = fl16(fl32(absmax_group / 127)); code = round-half-even
 * of the f32 quotient x / d, clamped to +-127 (zero codes when d is 0).
 * q4_0 rows hold 4-bit codes per group of 32 channels: m is the group's
 * value of largest magnitude (the first in channel order), the f16 scale is
 * d = fl16(fl32(m / -8)), code = clamp(round-half-even(fl32(x / d)) + 8,
 * 0, 15) (all 8 when d is 0), and the value is d * (code - 8); byte i of a
 * group holds channels 2i (low nibble) and 2i+1 (high nibble).
 * The bounds come from the f16 keys on every cache type.
 *
 * `len` (tokens cached; the same for every sequence) is host state, advanced
 * by kvd_kv_append.  Rows at or beyond `len` are never read by a decode
 * call's arithmetic (they may hold anything).
 * `dev_status` may be NULL; if set it is one device int32 that kernels set
 * to a kvd_status code when a bounded device wait runs out.
 * `moments` may be NULL; if set, [batch, n_kv_heads, max_seq / block, 2,
 * head_dim] f16: per block the mean of its stored keys, then of its stored
 * values (dequantized: code * scale for int8, code * d for q8_0, (code - 8)
 * * d for q4_0), over the block's tokens below len, each channel's f32 sum
 * in token order divided by the count and rounded to f16.  kvd_kv_append
 * and kvd_decode_step keep them for every block they write; they feed the
 * moment tail of kvd_decode_attn_tail.  Rewinding len inside a block and
 * appending again recomputes that block's means from its rows.
 * `seq_lens` may be NULL (every sequence holds len tokens); if set, a device
 * int32 [batch] with sequence b's own length, 0 <= seq_lens[b] <= len, and
 * `len` is the batch's maximum (it sizes the grids).  Every call then works
 * per sequence: kvd_kv_append writes sequence b's new rows from position
 * seq_lens[b] (the caller adds n_new to seq_lens afterwards; the library
 * never writes it), the selection ranks blocks below ceil(seq_lens[b] / block)
 * with the recent window ending at seq_lens[b], and the decode calls attend
 * tokens below seq_lens[b] (a sequence of length 0 gets a zero output).
 * kvd_decode_step appends sequence b's token at seq_lens[b] and then selects
 * and attends over its seq_lens[b] + 1 tokens (the caller adds 1 to seq_lens
 * after the step).  kvd_debug_scores does not take it (UNSUPPORTED).
 */
typedef struct kvd_cache {
    int32_t dtype;        /* kvd_kv_dtype */
    int32_t batch;        /* independent sequences, >= 1 */
    int32_t n_kv_heads;   /* Hkv >= 1 */
    int32_t head_dim;     /* D: 128 (every cache type and call), or any other multiple
                             of 16 up to 1024 ("cpu-attn", Requirements and limits)
                             for f16 and int8 caches without moments or seq_lens,
                             through kvd_kv_append(_f32), kvd_select_blocks,
                             kvd_decode_attn(_dense), kvd_decode_step(_host) and
                             kvd_workspace_bytes; other calls return UNSUPPORTED */
    int32_t max_seq;      /* capacity in tokens, a multiple of `block` */
    int32_t block;        /* B_SEL; only 64 is built [QUEST Knobs: default 64] */
    int32_t len;          /* tokens currently cached, 0 <= len <= max_seq */
    int32_t reserved;     /* must be 0 */
    void *k;
    void *v;
    void *k_scale;        /* f32 (int8) or f16 (q8_0, q4_0) scales, see above */
    void *v_scale;
    void *kbounds;
    int32_t *dev_status;
    void *moments;        /* optional block means (moment tail), see above */
    const int32_t *seq_lens;  /* optional per-sequence lengths, see above */
} kvd_cache;

/* ---------------------------------------------------------------------- */
/* Append n_new tokens to every sequence  [QUEST S2/S3 "Fill op" and       */
/* All-KV-types composition; CPUATT Method "quantize at append time"].     */
/*   k_new, v_new: device, [batch, n_new, n_kv_heads, head_dim] f16.        */
/* Writes rows len .. len+n_new-1 (f16 verbatim, or int8 codes + scales)   */
/* and the bounds of every block those rows touch: a block that already   */
/* held tokens is min/max-merged, a block that starts in the new range is  */
/* overwritten.  With cache->moments set, the key and value means of every */
/* touched block are recomputed over its rows below the new len.          */
/* On KVD_OK, cache->len += n_new (host side; the kernels                  */
/* are only enqueued).  n_new == 0 is a no-op.                             */
/* Errors: INVALID, UNSUPPORTED, CAPACITY (len + n_new > max_seq), CUDA.   */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_kv_append(kvd_cache *cache, const void *k_new, const void *v_new,
                         int32_t n_new, void *stream);

/* ---------------------------------------------------------------------- */
/* kvd_kv_append from f32 input  [CPUATT Usage: the cache takes each       */
/* token's K and V as f32; QUEST All-KV-types composition: the bounds come */
/* from the keys before quantization].                                      */
/*   k_new, v_new: device, [batch, n_new, n_kv_heads, head_dim] f32.         */
/*   f16 cache: stores each value's nearest f16 (ties to even), exactly as  */
/*   kvd_kv_append of those f16 values would.                               */
/*   int8 / q8_0 / q4_0: the rows are quantized from the f32 values; a       */
/*   block's bounds are the f32 keys' channel envelope rounded outward to   */
/*   f16 (kmin toward -inf, kmax toward +inf), merged as usual, so they     */
/*   hold every key.  Block means (when kept) come from the stored rows.    */
/* Errors and len: as kvd_kv_append.                                        */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_kv_append_f32(kvd_cache *cache, const float *k_new, const float *v_new,
                             int32_t n_new, void *stream);

/* ---------------------------------------------------------------------- */
/* Quest block selection for one query token per sequence  [QUEST Method   */
/* "Per-query upper bound", "Top-K block selection"; S2/S3 selector op:    */
/* "GQA -> max UB over the query group per KV-head"].                      */
/*   q: device [batch, n_heads, head_dim] f32; query head h belongs to KV   */
/*      head h / (n_heads / n_kv_heads) [CPUATT Usage].                    */
/*   For each (sequence, KV head) and block j < NB = ceil(len / block):    */
/*     UB(j) = max over the group's heads h of                             */
/*             sum_d max(q_h[d] * kmin_j[d], q_h[d] * kmax_j[d])            */
/*   Forced blocks: those meeting [0, sink_tokens) (sink) and those        */
/*   meeting [len - recent_tokens, len) (recent window).  Of the other     */
/*   blocks the k_sel with the largest UB are taken (all of them if fewer),*/
/*   equal bounds going to the lower block index.                          */
/*   sel_idx: device [batch, n_kv_heads, max_seq / block] int32; row r     */
/*            receives its selected block ids ascending in its first        */
/*            sel_cnt[r] entries (the rest is left untouched).             */
/*   sel_cnt: device [batch, n_kv_heads] int32; every row gets the same     */
/*            count, kvd_selected_count(len, block, k_sel, sink, recent).  */
/*   workspace: device scratch of kvd_workspace_bytes(...) bytes.          */
/* Errors: INVALID (len == 0, k_sel/sink/recent < 0, n_heads not a         */
/* multiple of n_kv_heads), UNSUPPORTED (group size not 1, 2, 4, 8 or 16;  */
/* more than 49152 blocks), WORKSPACE, CUDA.                               */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_select_blocks(const kvd_cache *cache, const float *q, int32_t n_heads,
                             int32_t k_sel, int32_t sink_tokens, int32_t recent_tokens,
                             int32_t *sel_idx, int32_t *sel_cnt,
                             void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Per-query-head selection: the ablation of the GQA-shared one  [CERT      */
/* Appendix Table 4: one scan per query head against the GQA-shared scan;   */
/* QUEST "GQA": the shared block set avoids per-head divergence].           */
/*   As kvd_select_blocks, except that query head h ranks the blocks by its  */
/*   own bound UB_h(j) (no maximum over the group), and its list is row      */
/*   (b, h) of sel_idx [batch, n_heads, max_seq / block] int32, its count    */
/*   sel_cnt[b, h] ([batch, n_heads] int32).  Forced blocks and ties as      */
/*   there.  One launch per head of a group.                                  */
/* Errors: as kvd_select_blocks.                                              */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_select_blocks_per_head(const kvd_cache *cache, const float *q,
                                      int32_t n_heads, int32_t k_sel, int32_t sink_tokens,
                                      int32_t recent_tokens, int32_t *sel_idx,
                                      int32_t *sel_cnt, void *workspace,
                                      size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Decode attention over lists per query head (kvd_select_blocks_per_head's  */
/* rows): as kvd_decode_attn, with query head h attending the blocks of row  */
/* (b, h) of sel_idx [batch, n_heads, max_seq / block] (sel_cnt [batch,      */
/* n_heads]).  Each CTA serves one query head, so a block listed for several */
/* heads of a group is read once per head.                                    */
/* Errors: as kvd_decode_attn.                                                */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_decode_attn_per_head(const kvd_cache *cache, const float *q,
                                    int32_t n_heads, float softmax_scale,
                                    const int32_t *sel_idx, const int32_t *sel_cnt,
                                    int32_t max_sel, float *out, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Split-KV decode attention over selected blocks only  [QUEST S3 FA-VEC   */
/* block skip: unselected blocks are not read; CPUATT Method].             */
/*   For query head h of KV head g, over the tokens t < len of the blocks  */
/*   listed in sel_idx[b, g, :sel_cnt[b, g]] (ascending or not; each block */
/*   once):                                                                 */
/*     f16:  logit_t = softmax_scale * sum_d q[d] * k_t[d]                  */
/*     int8: q is quantized once per head like a cache row; logit_t =      */
/*           dot_int32(q_code, k_code_t) * q_scale * k_scale_t * softmax_scale */
/*           and v_t = v_scale_t * v_code_t                                 */
/*     q8_0: q as for int8; logit_t = q_scale * softmax_scale *             */
/*           sum_g d_g(k_t) * dot_int32 over group g (32 channels), and     */
/*           v_t[c] = d_g(v_t) * v_code_t[c] with g = c / 32                */
/*     q4_0: as q8_0 with (code - 8) in place of the code                   */
/*     out_h = sum_t softmax(logit)_t * v_t       (f32 accumulation)       */
/*   An empty selection gives a zero output row.                           */
/*   out: device [batch, n_heads, head_dim] f32.                            */
/*   max_sel: an upper bound of every sel_cnt row (it only sizes the split  */
/*   grid; sel_cnt values above max_sel are still attended in full), e.g.  */
/*   kvd_selected_count(...).                                              */
/*   workspace: as for kvd_select_blocks; holds split partials and the      */
/*   per-problem arrival counters.  The workspace must be zero-filled      */
/*   before its first use; every call that completes leaves the counters   */
/*   at zero again.  After a call that reported a device fault, zero it.  */
/* Errors: INVALID, UNSUPPORTED, WORKSPACE, CUDA.                          */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_decode_attn(const kvd_cache *cache, const float *q, int32_t n_heads,
                           float softmax_scale, const int32_t *sel_idx,
                           const int32_t *sel_cnt, int32_t max_sel, float *out,
                           void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Dense decode attention over all len tokens (no bounds, no selection):  */
/* the no-skip reference arm  [QUEST Gate ladder "select-all ... sparse    */
/* must equal dense"; CPUATT Method].  Same arithmetic and arguments as    */
/* kvd_decode_attn with every block selected.                              */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_decode_attn_dense(const kvd_cache *cache, const float *q, int32_t n_heads,
                                 float softmax_scale, float *out,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Decode attention with sparse-V in eps mode  [QUEST "Adaptive tau (the   */
/* eps mode)", "Compose" item 3: inside the attended blocks, skip the V    */
/* work of positions whose weight is negligible, so that the dropped share */
/* of the softmax mass stays below eps].                                    */
/*   As kvd_decode_attn (sel_idx/sel_cnt/max_sel as there), or over every  */
/*   block when sel_idx is NULL (then sel_cnt and max_sel are ignored),     */
/*   except that, for each query head, the V term of position t is left out */
/*   of the numerator when                                                  */
/*     p_t < sparse_v_eps * mean_{u in c} p_u,   p_u = exp(s_u - max_c s)   */
/*   where c is t's chunk: the attended positions u with u / 16 == t / 16   */
/*   (a 16-token quarter of a 64-token block).  Every position stays in the */
/*   softmax denominator, so out_h = sum_{kept t} w_t v_t / sum_{all t} w_t */
/*   and the dropped share of sum_t w_t is below sparse_v_eps.              */
/*   sparse_v_eps = 0 gives kvd_decode_attn's (or the dense call's) output  */
/*   bit for bit; values above 16 drop every V term (out = 0).               */
/*   The comparison runs in f32 on the GPU: a position whose p_t lies within */
/*   rounding of the threshold may fall on either side.                     */
/* Errors: as kvd_decode_attn; INVALID also for a negative, NaN or infinite */
/* sparse_v_eps.                                                            */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_decode_attn_sv(const kvd_cache *cache, const float *q, int32_t n_heads,
                              float softmax_scale, const int32_t *sel_idx,
                              const int32_t *sel_cnt, int32_t max_sel, float sparse_v_eps,
                              float *out, void *workspace, size_t workspace_bytes,
                              void *stream);

/* ---------------------------------------------------------------------- */
/* Decode attention over the selected blocks plus the moment tail of every */
/* other block  [SCSA "2. Mechanism": a group that is not read exactly     */
/* contributes its count m times exp(a), a = softmax_scale * q . c_K, at   */
/* its value mean c_V, inside the shared normalizer; here the groups are   */
/* the Quest blocks the selection leaves out].                              */
/*   As kvd_decode_attn (same arguments), plus, for each query head h and   */
/*   each block j < NB = ceil(len / block) not listed in its row:           */
/*     term weight m_j * exp(softmax_scale * q_h . c_K(j)), value c_V(j)    */
/*   with m_j = min(block, len - j * block), c_K/c_V the f16 block means of */
/*   cache->moments, and q_h the f32 query (unquantized on every cache      */
/*   type).  out_h = (sum over listed tokens w_t v_t + sum over the other   */
/*   blocks of their terms) / (the same sum of weights).                    */
/*   Every listed row must be strictly ascending (as kvd_select_blocks      */
/*   writes it); otherwise a block may be counted both ways or not at all  */
/*   (wrong output, no fault).  Every row listing all NB blocks gives        */
/*   kvd_decode_attn's output bit for bit.                                   */
/*   Each launch reads all NB moment rows (512 bytes per block and KV head) */
/*   besides the listed blocks.                                              */
/* Errors: as kvd_decode_attn; INVALID also when cache->moments is NULL or  */
/* misaligned, or sel_idx/sel_cnt is NULL.                                  */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_decode_attn_tail(const kvd_cache *cache, const float *q,
                                int32_t n_heads, float softmax_scale,
                                const int32_t *sel_idx, const int32_t *sel_cnt,
                                int32_t max_sel, float *out, void *workspace,
                                size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* kvd_decode_attn without a workspace: the paper has no counterpart; this  */
/* is a convenience of this library.  Same arguments, arithmetic and output */
/* as kvd_decode_attn, minus workspace/workspace_bytes, for head_dim 128    */
/* only (the tuned kernels; other head dims return UNSUPPORTED).            */
/*   For callers that cannot allocate device memory when they decode: a    */
/*   plugin that an engine hands only its input and output buffers, or     */
/*   code whose device memory is owned by another allocator.  The split     */
/*   partials and arrival counters live in one array of                     */
/*   KVD_STATIC_SCRATCH_BYTES compiled into the library; every GPU that     */
/*   loads the library holds that array until the process exits.  The call */
/*   allocates nothing (no cudaMalloc/cudaFree, no library allocator).      */
/*   The first call on a device looks up the array's device address (once  */
/*   per device, with that device current); make that first call before    */
/*   any stream capture.  cudaDeviceReset drops that address: after a reset */
/*   of a device, do not call this entry point on it again in the same      */
/*   process.  Each call zeroes the counters on `stream` before             */
/*   its kernel.  All calls on a device share the array: two calls that    */
/*   may overlap on the GPU (different streams, no ordering) race and give  */
/*   wrong outputs; order them on one stream or with events.                */
/* Errors: as kvd_decode_attn (the same cache and head checks);             */
/* UNSUPPORTED for a head_dim other than 128; WORKSPACE when this call's     */
/* partials and counters would pass KVD_STATIC_SCRATCH_BYTES (on a 152-SM   */
/* GPU every accepted shape needs under 0.7 MiB, so WORKSPACE does not      */
/* occur there).                                                            */
/* ---------------------------------------------------------------------- */
#define KVD_STATIC_SCRATCH_BYTES (1u << 20)
KVD_API kvd_status kvd_decode_attn_static(const kvd_cache *cache, const float *q,
                                  int32_t n_heads, float softmax_scale,
                                  const int32_t *sel_idx, const int32_t *sel_cnt,
                                  int32_t max_sel, float *out, void *stream);

/* ---------------------------------------------------------------------- */
/* One whole decode step on device buffers: append one token per sequence */
/* (k_new, v_new: [batch, 1, n_kv_heads, head_dim] f16), then select and   */
/* attend over the len+1 cached tokens.  Equivalent to kvd_kv_append,      */
/* kvd_select_blocks and kvd_decode_attn in that order on `stream`; with   */
/* k_sel < 0 the attention is dense.  sel_idx/sel_cnt may be NULL, and then */
/* the selection lives in the workspace.  On KVD_OK cache->len has grown by */
/* one (also when a later launch failed with KVD_ERR_CUDA after the append */
/* was enqueued).                                                           */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_decode_step(kvd_cache *cache, const float *q, const void *k_new,
                           const void *v_new, int32_t n_heads, float softmax_scale,
                           int32_t k_sel, int32_t sink_tokens, int32_t recent_tokens,
                           int32_t *sel_idx, int32_t *sel_cnt, float *out,
                           void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* kvd_decode_step with HOST inputs and output: q_host ([batch, n_heads,   */
/* head_dim] f32), k_new_host/v_new_host ([batch, 1, n_kv_heads, head_dim] */
/* f16) in, out_host ([batch, n_heads, head_dim] f32) out, all enqueued on */
/* `stream`.  A buffer in page-locked host memory that CUDA maps into the  */
/* device's address space (16-byte aligned) is read or written in place by */
/* the kernels, over the host link; any other buffer is staged through    */
/* the workspace with cudaMemcpyAsync (pageable memory makes those copies   */
/* synchronous).  out_host is valid once the stream has finished, and the  */
/* host must not change the inputs before then.                             */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_decode_step_host(kvd_cache *cache, const float *q_host,
                                const void *k_new_host, const void *v_new_host,
                                int32_t n_heads, float softmax_scale, int32_t k_sel,
                                int32_t sink_tokens, int32_t recent_tokens,
                                int32_t *sel_idx, int32_t *sel_cnt, float *out_host,
                                void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/* Workspace bytes that every call above needs for this cache geometry    */
/* (batch, n_kv_heads, max_seq, dtype) and n_heads query heads, for any   */
/* len <= max_seq and any selection.  One zero-filled workspace of this    */
/* size serves all the calls (they use disjoint regions: split partials,   */
/* per-problem arrival counters, selection keys, a selection for           */
/* kvd_decode_step when the caller passes none, and the host-step staging  */
/* buffers).  The split grid follows the current device's SM count, so    */
/* query it with the device that will run the calls current.  0 on        */
/* invalid arguments.                                                       */
/* ---------------------------------------------------------------------- */
KVD_API size_t kvd_workspace_bytes(const kvd_cache *cache, int32_t n_heads);

/* Blocks selected per (sequence, KV head) for a cache of len tokens:      */
/* forced sink and recent blocks plus min(k_sel, other blocks).  -1 on     */
/* invalid arguments.  Host only.                                          */
KVD_API int32_t kvd_selected_count(int32_t len, int32_t block, int32_t k_sel,
                           int32_t sink_tokens, int32_t recent_tokens);

/* ====================================================================== */
/* Around the decode: positions, per-head norms, a cache in pages, and     */
/* attention of a chunk of new tokens.  The pages have no counterpart:     */
/* they start from queries and keys that are normed and rotated already,   */
/* and their caches are contiguous.                                        */
/* ====================================================================== */

/* Element type of activations (the cache has kvd_kv_dtype). */
typedef enum { KVD_X_F16 = 0, KVD_X_BF16 = 1, KVD_X_F32 = 2 } kvd_x_dtype;

/*
 * Rows of heads: [n_tokens, n_heads, head_dim] with the heads of one token
 * dense and `stride` elements from one token to the next, so that the query,
 * key and value parts of one fused projection can be passed as they lie.
 * x is 16-byte aligned, stride >= n_heads * head_dim, and stride times the
 * element size a multiple of 16.
 */
typedef struct kvd_heads {
    void *x;
    int64_t stride;
    int32_t dtype;        /* kvd_x_dtype */
    int32_t n_heads;
} kvd_heads;

/* How the angles per position are stretched for contexts longer than the
 * one a model was trained on; f_i = base^(-2i / rot_dim), i < rot_dim / 2. */
typedef enum {
    KVD_ROPE_NONE = 0,
    KVD_ROPE_LINEAR = 1,  /* f_i / factor */
    KVD_ROPE_NTK = 2,     /* base * factor^(rot_dim / (rot_dim - 2)) for base */
    KVD_ROPE_YARN = 3,    /* f_i for channels that turn more than `high` times in orig_len
                             positions, f_i / factor below `low` turns, a linear ramp over
                             the channels between (their whole numbers, as floor and ceil
                             give them); the rotated channels times 0.1 ln(factor) + 1 */
    KVD_ROPE_BANDS = 4    /* the same two ends, the ramp linear in the number of turns */
} kvd_rope_scaling;

/*
 * Position rotation of the first rot_dim channels of a head.  Pair i is
 * channels (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved; at position
 * p it turns by p * f_i, and both channels are scaled by mscale.
 * freqs: device, [rot_dim / 2] words: f_i / (2 pi) turns per position, times
 * 2^64 (kvd_rope_freqs).  A position times such a word, modulo 2^64, is the
 * angle's fraction of a turn to 2^-33 at any int32 position; an f32 angle has
 * lost it after some thousand positions.
 */
typedef struct kvd_rope {
    const uint64_t *freqs;
    int32_t rot_dim;      /* a multiple of 16 in [16, head_dim] */
    int32_t interleaved;  /* 0 or 1 */
    float mscale;
    int32_t reserved;     /* must be 0 */
} kvd_rope;

/* The words of kvd_rope.freqs for a host to copy to the device, and mscale.
 * factor >= 1 (ignored by NONE); orig_len, low < high: YARN (1 and 32 turns
 * where both are 0) and BANDS (1 and 4).  Host only.
 * Errors: INVALID (NULL, rot_dim not a positive multiple of 16 up to 1024,
 * base <= 1 or not finite, factor < 1, orig_len < 1, low < 0, low >= high,
 * and with YARN, which takes its logarithm, low == 0 beside a high that is not). */
KVD_API kvd_status kvd_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                                  double orig_len, double low, double high, uint64_t *freqs,
                                  float *mscale);

/* ---------------------------------------------------------------------- */
/* Per-head RMS norm and position rotation of queries and keys, one pass.  */
/*   y = R(p) (x * w / sqrt(mean(x^2) + eps)), rounded once to the output    */
/*   type; w is q_weight or k_weight ([head_dim] f32, device), and without  */
/*   one there is no norm; rope NULL leaves the rotation out.               */
/*   q, q_out, k, k_out: [n_tokens, .., head_dim]; k and k_out may be NULL.  */
/*   An output may be its own input (same address, stride and type), and    */
/*   must not overlap the inputs otherwise.                                  */
/*   positions: device int32 [n_tokens] (NULL when rope is NULL).            */
/* The outputs feed kvd_decode_attn and kvd_select_blocks (f32 queries) and */
/* kvd_kv_append (f16 or f32 keys).  n_tokens == 0 is a no-op.               */
/* Errors: INVALID; UNSUPPORTED (head_dim not a multiple of 16 in           */
/* [16, 1024], rot_dim not a multiple of 16); CUDA.                          */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_qk_norm_rope(const kvd_heads *q, const kvd_heads *q_out,
                                    const kvd_heads *k, const kvd_heads *k_out, int32_t n_tokens,
                                    int32_t head_dim, const int32_t *positions,
                                    const kvd_rope *rope, const float *q_weight,
                                    const float *k_weight, float eps, void *stream);

/*
 * A cache in pages: page j of every sequence is a page of one pool, found by
 * the sequence's row of page_table.
 *   k, v        [n_pages, n_kv_heads, page_size, head_dim]  f16, bf16 or int8 codes
 *   k_scale,    [n_pages, n_kv_heads, page_size] f32 (int8: absmax / 127 of the
 *   v_scale     token's row, as in kvd_cache; NULL otherwise)
 *   page_table  device int32 [batch, max_pages]: the page of tokens
 *               [j * page_size, (j + 1) * page_size).  Entries of pages that no
 *               token below the sequence's length needs are not read.
 *   seq_lens    device int32 [batch]: the tokens of each sequence, the new ones
 *               of the current call counted (both calls below take the same)
 *   len         host: at least the largest of seq_lens; it sizes the grids
 * An f16 or int8 kvd_cache is such a cache with one page a sequence: page_size =
 * max_seq, n_pages = batch, page_table[b][0] = b.
 * Rows at or beyond a sequence's length may hold anything, NaN too.
 * The calls below refuse (UNSUPPORTED) len above 2^30, and more than 2^31 - 1 key
 * tiles (batch * n_kv_heads * (len / 128 + 1)) or rows of the pool (n_pages *
 * n_kv_heads * page_size).
 * The int32s on the device must not change while a call runs, and are checked there: a page outside [0, n_pages), a
 * length outside [0, len], or starts that fall or leave [0, n_tokens] write
 * KVD_ERR_INVALID to dev_status.  Such a page is neither read nor written (its
 * keys are left out), and a length or a start is moved into its range.  So does
 * a sequence with more new tokens than its length: those before position 0 are
 * not appended, and see no key.
 */
typedef struct kvd_paged_cache {
    int32_t dtype;        /* KVD_F16, KVD_BF16 or KVD_INT8 */
    int32_t batch;        /* sequences >= 1 */
    int32_t n_kv_heads;
    int32_t head_dim;     /* 64 or 128 */
    int32_t n_pages;      /* pages of the pool */
    int32_t page_size;    /* tokens, a multiple of 16 */
    int32_t max_pages;    /* columns of page_table */
    int32_t len;          /* at least the largest of seq_lens, <= max_pages * page_size */
    void *k;
    void *v;
    void *k_scale;
    void *v_scale;
    const int32_t *page_table;
    const int32_t *seq_lens;
    int32_t *dev_status;  /* may be NULL */
} kvd_paged_cache;

/* ---------------------------------------------------------------------- */
/* Append new tokens of a ragged batch to their pages, with the norm and    */
/* the rotation of kvd_qk_norm_rope on the way.                              */
/*   starts: device int32 [batch + 1]: sequence b's new tokens are rows      */
/*   [starts[b], starts[b + 1]) of k, v and q, and stand at positions        */
/*   seq_lens[b] - n_b .. seq_lens[b] - 1.  Rows before starts[0] and at or  */
/*   behind starts[batch] (a padded batch) count for nothing, and their       */
/*   q_out is not written.                                                    */
/*   k, v: [n_tokens, n_kv_heads, head_dim] of one type.  Keys are normed    */
/*   (k_weight) and rotated (rope) in f32; then keys and values are rounded  */
/*   to the cache's type, or quantized as by kvd_kv_append.  Only the rows   */
/*   of new tokens are written.                                               */
/*   q, q_out (both NULL, or both given): normed and rotated as the keys are. */
/* No bounds are kept: the selection works on kvd_cache.                     */
/* Two sequences must not share a page that this call writes.                */
/* n_tokens == 0 is a no-op.                                                  */
/* Errors: INVALID; UNSUPPORTED (head_dim, page_size, rot_dim, the cache's     */
/* counts); CUDA.                                                              */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_paged_append(const kvd_paged_cache *cache, const kvd_heads *k,
                                    const kvd_heads *v, int32_t n_tokens, const int32_t *starts,
                                    const kvd_rope *rope, const float *k_weight,
                                    const kvd_heads *q, const kvd_heads *q_out,
                                    const float *q_weight, float eps, void *stream);

/* ---------------------------------------------------------------------- */
/* Attention of a ragged batch's new tokens over their sequences' pages:    */
/* a prefill chunk, single decode tokens, or both in one batch.              */
/*   starts as for kvd_paged_append (the new tokens are in the cache).       */
/*   For token i of sequence b's n_b and query head h of KV head             */
/*   h / (n_heads / n_kv_heads), with p = seq_lens[b] - n_b + i:              */
/*     out = sum_t softmax(softmax_scale * q . k_t)_t v_t  over the cached    */
/*     tokens t <= p, and p - window < t when window > 0                      */
/*   (int8: k_t = scale_t * code_t, and q stays as it is).  Logits, maxima,   */
/*   weights and their sum are f32.  For the product with the values weights   */
/*   are rounded: over bf16 to 2^-8 of each; over f16 to 2^-11 of each, but    */
/*   not below 2^-31 of the row's largest; over int8, times the value's scale, */
/*   to 2^-11 of each, but not below 2^-24 of the row's largest weight times   */
/*   the largest value scale among the 128 keys around (or 2^-60 of the        */
/*   largest of all, where that is more).                                      */
/*   A token that sees no key gets a zero row.  Rows of no sequence (before    */
/*   starts[0], at or behind starts[batch]) are not written.                   */
/*   A non-finite value row spoils the outputs of its own sequence's tokens   */
/*   in this call, those before it included.                                   */
/*   q, out: [n_tokens, n_heads, head_dim] of one type: the cache's, or f16 or */
/*   bf16 over an int8 cache.  out must not overlap q.  softmax_scale > 0.      */
/*   max_new: at least the largest n_b (it sizes the grid; the tokens of a     */
/*   larger n_b are left out, and INVALID is reported to dev_status).  With    */
/*   max_new == 0 no sequence has new tokens: a no-op, starts are not read.     */
/*   workspace: kvd_paged_workspace_bytes, zero-filled before its first use;   */
/*   every call that completes leaves its counters at zero again (after a       */
/*   KVD_ERR_TIMEOUT in dev_status, zero it).  Calls that may overlap on the    */
/*   GPU need a workspace each.                                                  */
/* n_tokens == 0 is a no-op.                                                    */
/* Errors: INVALID; UNSUPPORTED (head_dim, page_size, the cache's counts, more   */
/* than 16 query heads a KV head); WORKSPACE; CUDA.                              */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_paged_attn(const kvd_paged_cache *cache, const kvd_heads *q,
                                  int32_t n_tokens, const int32_t *starts, int32_t max_new,
                                  float softmax_scale, int32_t window, const kvd_heads *out,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of kvd_paged_attn for n_heads query heads, up to n_tokens new
 * tokens with up to max_new in one sequence, and any len the page table can hold
 * (the kernels as they are need the same for any n_tokens >= 1).  Asked with the
 * device current that will run the call.  0 on invalid arguments. */
KVD_API size_t kvd_paged_workspace_bytes(const kvd_paged_cache *cache, int32_t n_heads,
                                         int32_t n_tokens, int32_t max_new);

/* ---------------------------------------------------------------------- */
/* kvd_paged_attn that also gives each row's softmax statistic, for */
/* kvd_paged_mass or to join attention over several caches: */
/*   lse[t, h] = ln sum_s exp(softmax_scale * q . k_s)   over the keys the */
/*   row sees, -infinity where it sees none; device f32 [n_tokens, n_heads]. */
/*   Rows of no sequence are not written.  out is kvd_paged_attn's, bit for */
/*   bit.  n_tokens == 0 or max_new == 0 is a no-op, whatever lse is. */
/* Errors: as kvd_paged_attn; INVALID also for lse NULL or misaligned. */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_paged_attn_lse(const kvd_paged_cache *cache, const kvd_heads *q,
                                      int32_t n_tokens, const int32_t *starts, int32_t max_new,
                                      float softmax_scale, int32_t window, const kvd_heads *out,
                                      float *lse, void *workspace, size_t workspace_bytes,
                                      void *stream);

/* ====================================================================== */
/* Smaller caches: rows that all heads share (latent attention), and fewer */
/* rows (eviction by accumulated weight).  They have no counterpart on the */
/* pages. */
/* ====================================================================== */

/*
 * A cache of latent rows in pages: one row a token, shared by all query heads.
 * Its first `rank` channels are the token's latent vector, normed, which is the
 * value and the larger part of the key; the other rope_dim are the key's rotated
 * part.  A model with per-head projections W_k (latent to key) and W_v (latent to
 * value) asks for it with q W_k in place of q, and applies W_v to the output
 * (the absorbed form).
 *   rows        [n_pages, page_size, rank + rope_dim]  f16 or bf16
 * Pages, lengths, limits and what is checked on the device: as kvd_paged_cache with
 * one KV head.
 */
typedef struct kvd_latent_cache {
    int32_t dtype;        /* KVD_F16 or KVD_BF16 */
    int32_t batch;        /* sequences >= 1 */
    int32_t rank;         /* 128, 256, 384 or 512 */
    int32_t rope_dim;     /* 16, 32, 48 or 64 */
    int32_t n_pages;      /* pages of the pool */
    int32_t page_size;    /* tokens, a multiple of 16 */
    int32_t max_pages;    /* columns of page_table */
    int32_t len;          /* at least the largest of seq_lens, <= max_pages * page_size */
    void *rows;
    const int32_t *page_table;
    const int32_t *seq_lens;
    int32_t *dev_status;  /* may be NULL */
} kvd_latent_cache;

/* Parts of heads: kvd_heads whose heads lie head_stride elements apart, so that
 * some channels of each head can be passed as they lie.  x is 16-byte aligned, both
 * strides times the element size are multiples of 16, head_stride >= the part's
 * channels, and stride >= (n_heads - 1) * head_stride + the part's channels. */
typedef struct kvd_head_parts {
    void *x;
    int64_t stride;
    int64_t head_stride;
    int32_t dtype;        /* kvd_x_dtype */
    int32_t n_heads;
} kvd_head_parts;

/* ---------------------------------------------------------------------- */
/* Append new tokens of a ragged batch to their latent pages. */
/*   row = (c * c_weight / sqrt(mean(c^2) + eps), R(p) k_pe), each rounded */
/*   once to the cache's type; without c_weight no norm, without rope no */
/*   rotation (rot_dim <= rope_dim). */
/*   c, k_pe: [n_tokens, 1, rank] and [n_tokens, 1, rope_dim] of one type. */
/*   starts, positions and padding rows as for kvd_paged_append. */
/*   q, q_out (both NULL, or both given): the queries' rotated parts */
/*   [n_tokens, n_heads, rope_dim], turned as the keys' are; q_out may be q */
/*   itself (same address, strides and type) and must not overlap it otherwise. */
/* n_tokens == 0 is a no-op. */
/* Errors: INVALID; UNSUPPORTED (rank, rope_dim, page_size, rot_dim, the cache's */
/* counts); CUDA. */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_latent_append(const kvd_latent_cache *cache, const kvd_heads *c,
                                     const kvd_heads *k_pe, int32_t n_tokens,
                                     const int32_t *starts, const kvd_rope *rope,
                                     const float *c_weight, const kvd_head_parts *q,
                                     const kvd_head_parts *q_out, float eps, void *stream);

/* ---------------------------------------------------------------------- */
/* Attention of a ragged batch's new tokens over their latent pages. */
/*   For token i of sequence b's n_b and query head h, p = seq_lens[b] - n_b + i: */
/*     z_t = softmax_scale * q . row_t  (all rank + rope_dim channels) */
/*     out = sum_t softmax(z)_t row_t[:rank]    over the cached tokens t <= p, */
/*     and p - window < t when window > 0; lse = ln sum_t exp(z_t). */
/*   Logits, maxima, weights and their sum are f32.  For the product with the */
/*   rows weights are rounded: over bf16 to 2^-8 of each; over f16 to 2^-11 of */
/*   each, but not below 2^-31 of the row's largest. */
/*   A token that sees no key gets a zero row and an lse of -infinity.  Rows of no */
/*   sequence are not written.  A non-finite row of the cache spoils the outputs */
/*   of its own sequence's tokens in this call, those before it included. */
/*   q: [n_tokens, n_heads, rank + rope_dim], out: [n_tokens, n_heads, rank], of the */
/*   cache's type; out must not overlap q.  n_heads <= 1024.  softmax_scale > 0. */
/*   lse: device f32 [n_tokens, n_heads], or NULL. */
/*   starts, max_new, window, workspace (kvd_latent_workspace_bytes): as for */
/*   kvd_paged_attn; this workspace needs no zeros. */
/* n_tokens == 0 or max_new == 0 is a no-op. */
/* Errors: INVALID; UNSUPPORTED (rank, rope_dim, page_size, the cache's counts, n_heads); */
/* WORKSPACE; CUDA. */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_latent_attn(const kvd_latent_cache *cache, const kvd_heads *q,
                                   int32_t n_tokens, const int32_t *starts, int32_t max_new,
                                   float softmax_scale, int32_t window, const kvd_heads *out,
                                   float *lse, void *workspace, size_t workspace_bytes,
                                   void *stream);

/* Workspace bytes of kvd_latent_attn, as kvd_paged_workspace_bytes.  0 on invalid
 * arguments. */
KVD_API size_t kvd_latent_workspace_bytes(const kvd_latent_cache *cache, int32_t n_heads,
                                          int32_t n_tokens, int32_t max_new);

/* ---------------------------------------------------------------------- */
/* Accumulated attention weight of each cached token, for an eviction. */
/*   For sequence b, KV head g and cached token t < seq_lens[b]: */
/*     out[b, g, t] = (t < seq_lens[b] - n_b ? decay * mass[b, g, t] : 0) */
/*                    + sum over the new tokens that see t and g's query heads */
/*                      of exp(softmax_scale * q . k_t - lse) */
/*   that is, the weights of the attention call with the same q, starts, */
/*   max_new, softmax_scale and window, whose lse it is; the new tokens begin at 0. */
/*   What stands at or behind seq_lens[b], and a row whose lse is -infinity, count */
/*   for nothing; the former is not written.  Keys on a bad page get no weight. */
/*   A row whose lse is NaN spoils the weights that it adds to. */
/*   Logits, weights and sums are f32, added in a fixed order: repeated calls give */
/*   the same bits.  Beside its logit's error a weight is off by 2^-19 + |lse| 2^-22 of */
/*   itself, as lse is a number of 24 bits: 2^-15 at |lse| = 100, 2^-12 at 1000; one */
/*   below 2^-126 may count as 0. */
/*   q: [n_tokens, n_heads, head_dim] (latent: rank + rope_dim), the type that the */
/*   attention call takes; lse: f32 [n_tokens, n_heads]. */
/*   mass, out: f32 [batch, n_kv_heads, ..], mass_stride and out_stride elements */
/*   from one (sequence, head) to the next, both >= len; out may be mass itself (same */
/*   stride) and must not overlap it otherwise.  decay is finite and >= 0 (0: mass is */
/*   not read, and may be NULL). */
/*   n_tokens == 0 or max_new == 0: only the decay. */
/* Errors: INVALID; UNSUPPORTED (as the attention calls); CUDA. */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_paged_mass(const kvd_paged_cache *cache, const kvd_heads *q,
                                  const float *lse, int32_t n_tokens, const int32_t *starts,
                                  int32_t max_new, float softmax_scale, int32_t window, const float *mass,
                                  int64_t mass_stride, float decay, float *out, int64_t out_stride,
                                  void *stream);
KVD_API kvd_status kvd_latent_mass(const kvd_latent_cache *cache, const kvd_heads *q,
                                   const float *lse, int32_t n_tokens, const int32_t *starts,
                                   int32_t max_new, float softmax_scale, int32_t window,
                                   const float *mass, int64_t mass_stride, float decay, float *out,
                                   int64_t out_stride, void *stream);

/* ---------------------------------------------------------------------- */
/* Eviction: of each (sequence, KV head) the tokens that stay, in order, to */
/* the pages of another table. */
/*   A sequence of more than `keep` tokens keeps its first `sink`, its last */
/*   `recent`, and of those between the ones with the largest mass, `keep` in */
/*   all; equal masses (-0 is 0) go to the lower index, and NaN is below every */
/*   number.  A shorter one keeps all. */
/*   mass: f32 [batch, n_kv_heads, ..], mass_stride >= len elements apart. */
/*   kept: device int32 [batch, n_kv_heads, keep]: the kept tokens' old indices, */
/*   ascending, min(keep, seq_lens[b]) of them (the rest of a row is left as it was). */
/*   Row r of the kept, codes and scales as they are, goes to token r of the */
/*   sequence in page_table_out (device int32 [batch, max_pages_out], pages of the */
/*   same pool).  mass_out (may be NULL), f32 [batch, n_kv_heads, ..] mass_out_stride */
/*   >= keep elements apart, gets their masses; it must not overlap mass. */
/*   seq_lens_out: device int32 [batch], min(keep, seq_lens[b]).  It must not be */
/*   seq_lens itself. */
/*   No page of page_table_out may be one that this call reads, or stand in it twice, */
/*   among the entries that the kept rows need (wrong rows, no fault).  A caller goes */
/*   on with the new table and lengths, and may then give the old pages back. */
/*   The keys keep the rotation of their old positions: later tokens' positions are no */
/*   longer their places in the cache.  So norm and rotate them with kvd_qk_norm_rope, at */
/*   positions that the caller counts, and append without rope and key or query weights. */
/*   Latent: k_pe so (one head), and the queries' rotated parts as n_tokens * n_heads rows */
/*   of one head each, their heads' stride as the rows' and each token's position once a */
/*   head (tokens have to lie n_heads such strides apart); c and c_weight as always. */
/*   A window of the attention and mass calls counts places in the cache, not positions: */
/*   after an eviction it is the last `window` tokens that stayed. */
/*   Bad pages of either table are reported as INVALID to dev_status, and their rows are */
/*   not moved. */
/* Errors: INVALID (keep < 1, sink or recent < 0, sink + recent > keep, strides, too few */
/* columns in page_table_out for min(keep, len)); UNSUPPORTED (as kvd_paged_append); CUDA. */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_paged_evict(const kvd_paged_cache *cache, const float *mass,
                                   int64_t mass_stride, int32_t keep, int32_t sink, int32_t recent,
                                   const int32_t *page_table_out, int32_t max_pages_out,
                                   int32_t *kept, int32_t *seq_lens_out, float *mass_out,
                                   int64_t mass_out_stride, void *stream);
KVD_API kvd_status kvd_latent_evict(const kvd_latent_cache *cache, const float *mass,
                                    int64_t mass_stride, int32_t keep, int32_t sink, int32_t recent,
                                    const int32_t *page_table_out, int32_t max_pages_out,
                                    int32_t *kept, int32_t *seq_lens_out, float *mass_out,
                                    int64_t mass_out_stride, void *stream);

/* Static description of a status code.  Host only. */
KVD_API const char *kvd_status_string(kvd_status status);

/* KVD_ABI_VERSION of the built library.  Host only. */
KVD_API int32_t kvd_abi_version(void);

/* ---------------------------------------------------------------------- */
/* Test exports: the exact integer q.k dots and the block bounds, computed */
/* by the same device routines the decode and select kernels use.         */
/*   kvd_debug_qk_int8: dots [batch, n_heads, len] int32, q_codes [batch,   */
/*   n_heads, head_dim] int8, q_scales [batch, n_heads] f32 (int8 cache     */
/*   only)  [CPUATT Method: integer logit dots, exact].                      */
/*   kvd_debug_scores: ub [batch, n_kv_heads, NB] f32, the group bound UB(j)*/
/*   of every block j < NB = ceil(len / block)  [QUEST Method].             */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_debug_qk_int8(const kvd_cache *cache, const float *q, int32_t n_heads,
                             int32_t *dots, int8_t *q_codes, float *q_scales, void *stream);
KVD_API kvd_status kvd_debug_scores(const kvd_cache *cache, const float *q, int32_t n_heads,
                            float *ub, void *stream);

/* ---------------------------------------------------------------------- */
/* Test export of the bounded-wait paths: one kernel waits on an mbarrier   */
/* phase that nothing completes, in each of the forms that kernels wait in, */
/* gives up after limit_us microseconds of wall time in each (the kernels   */
/* themselves after 2 s), and writes KVD_ERR_TIMEOUT to *dev_status (a      */
/* device int32) unless it holds a code already; KVD_ERR_CUDA if one did    */
/* not give up.  The kernel then returns normally: the context stays        */
/* usable.  Errors: INVALID (dev_status NULL or misaligned, limit_us 0 or   */
/* above 1,000,000), CUDA.                                                  */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_debug_wait_timeout(int32_t *dev_status, int32_t limit_us, void *stream);

/* ---------------------------------------------------------------------- */
/* Profiling export (no counterpart on the pages): stage marks.  In a      */
/* library built with KVD_MARKS (build.py: environment KVD_MARKS=1) the    */
/* kernels write the GPU's global nanosecond timer at numbered points of   */
/* their work into `marks`, a caller-owned device buffer of at least       */
/* 3 * 4096 * 16 * 8 bytes (16-byte aligned): region k (0 selection,       */
/* 1 decode, 2 other kernels) holds 16 slots per CTA for up to 4096 CTAs,  */
/* numbered x-fastest.  Later launches write into it until it is replaced; */
/* marks = NULL turns recording off.  Host only; nothing is launched.      */
/* Errors: UNSUPPORTED in every build without marks (the default);         */
/* INVALID when the buffer is too small or misaligned.                     */
/* ---------------------------------------------------------------------- */
KVD_API kvd_status kvd_debug_stage_marks(void *marks, size_t bytes);

#ifdef __cplusplus
}
#endif
#endif /* KVDECODE_H */
