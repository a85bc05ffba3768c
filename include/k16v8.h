/*
 * k16v8.h -- C ABI of libk16v8.so: paged grouped-query attention over an
 * asymmetric KV cache that keeps keys in FP16 and values in E4M3 FP8 with one
 * FP32 scale per (layer, KV head) -- the "K16/V8" route of
 * "Phi-4: quality transfer and interrupted throughput studies" (knlp.io).
 *
 * What the page fixes (intro section): the candidate stores FP16 keys and
 * E4M3 FP8 values with the model's own scales, in a per-layer token-slot pool
 * of a 32 GiB budget; the geometry is 40 layers, 40 query heads, 10 KV heads,
 * head dimension 128.  Section "Matched diagnostic profiles" names the work
 * this library implements: the attention kernels, the merge kernels, and the
 * value gather that writes the compressed cache.
 *
 * Conventions shared by every call
 *  - Pointers named as device pointers must point to device memory of the
 *    current device; the caller owns all memory.  The library allocates
 *    nothing and keeps no state between calls, apart from the built-in
 *    scratch array of k16v8_paged_decode_attention_static.
 *  - Every launching call is asynchronous on `stream` (a cudaStream_t passed
 *    as void*; NULL is the legacy default stream).  Only
 *    k16v8_read_device_error synchronises.
 *  - Arguments are validated on the host before anything is launched; a
 *    non-OK status means nothing was launched.
 *  - Cache layout (pages of K16V8_PAGE_SIZE tokens), element (page, kv head,
 *    offset, d) at ((page*num_kv_heads + head)*16 + offset)*head_dim + d:
 *      k_cache  fp16  [num_pages][num_kv_heads][16][head_dim]
 *      v_cache  E4M3  [num_pages][num_kv_heads][16][head_dim]  (one byte)
 *      v_scale  fp32  [num_kv_heads]   value = v_scale[h] * e4m3(code)
 *  - A slot is page*16 + offset.  block_table[b][i] holds the page of
 *    positions 16i..16i+15 of sequence b.
 *  - Supported shapes: head_dim == 128; attention calls need
 *    num_qo_heads == 4*num_kv_heads (query head h reads KV head h/4).  Other
 *    shapes return K16V8_ERR_UNSUPPORTED_SHAPE.
 *  - Out-of-range slots, page ids or sequence lengths met on the device are
 *    never dereferenced: the kernel skips or masks them and ORs a
 *    K16V8_DEVERR_* bit into the caller's int32 error word (if non-NULL),
 *    which k16v8_read_device_error returns.
 */
#ifndef K16V8_H
#define K16V8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define K16V8_PAGE_SIZE 16
#define K16V8_HEAD_DIM 128
#define K16V8_GQA_GROUP 4
#define K16V8_MAX_SPLIT_CHUNK 8192
#define K16V8_MAX_TREE_NODES 64   /* nodes of one sequence's drafted tree */
#define K16V8_MAX_VOCAB (1 << 19) /* probabilities per row of tree_verify */
#define K16V8_MAX_ROPE_AXES 4      /* axes of a position (time, height, width, ...) */
#define K16V8_E4M3_MAX 448         /* the largest E4M3 value */

typedef enum {
    K16V8_OK = 0,
    K16V8_ERR_INVALID_ARG = 1,        /* null pointer, negative size, misalignment */
    K16V8_ERR_UNSUPPORTED_SHAPE = 2,  /* head_dim / GQA group not supported */
    K16V8_ERR_WORKSPACE_TOO_SMALL = 3,
    K16V8_ERR_CUDA = 4,               /* a CUDA runtime call or launch failed */
    K16V8_ERR_DEVICE_BOUNDS = 5,      /* returned by k16v8_read_device_error */
    K16V8_ERR_STATIC_SCRATCH_LIMIT = 6 /* problem too large for the built-in scratch */
} k16v8_status;

typedef enum { K16V8_F16 = 0, K16V8_F32 = 1, K16V8_BF16 = 2 } k16v8_dtype;

/* Bits of the device error word. */
#define K16V8_DEVERR_SLOT 0x1    /* kv_append: slot >= num_pages*16 */
#define K16V8_DEVERR_PAGE 0x2    /* block_table entry outside [0, num_pages) */
#define K16V8_DEVERR_SEQLEN 0x4  /* seq_len < 0, > max_seq_len, or > 16*max_pages_per_seq */
#define K16V8_DEVERR_TIMEOUT 0x8 /* a bounded wait on an async copy gave up */
#define K16V8_DEVERR_INTERNAL 0x10 /* a kernel's own layout check failed; nothing was written */
#define K16V8_DEVERR_POSITION 0x20 /* rope_kv_append: position < 0 or >= 2^24 */
#define K16V8_DEVERR_TREE 0x40   /* a parent, token or path entry that is none of its tree */
#define K16V8_DEVERR_PROBS 0x80  /* tree_verify: sums far above 1 */

/*
 * kv_append -- "the candidate also gathers values and writes the compressed
 * cache" ("Matched diagnostic profiles"); storage format from the intro.
 *
 * For every token t with slot s = slot_mapping[t] >= 0 and every KV head h:
 *   k_cache[s/16][h][s%16][:] = k[t][h][:]                      (fp16 copy)
 *   v_cache[s/16][h][s%16][:] = E4M3_rn_satfinite(fl32(v[t][h][:]) / v_scale[h])
 * The division is IEEE fp32 round-to-nearest; the E4M3 rounding is
 * round-to-nearest-even with finite overflow and +-inf saturating to +-448
 * (NaN stays NaN).  Negative slots are skipped (padding).  Slots at or above
 * num_pages*16 are skipped and flag K16V8_DEVERR_SLOT.  Duplicate slots in
 * one call leave an unspecified one of the writers.
 *
 *   k              device, fp16 [num_tokens][num_kv_heads][head_dim], token
 *                  stride k_token_stride elements (0 = num_kv_heads*head_dim)
 *   v              device, fp16 or fp32 (v_dtype) likewise, v_token_stride
 *   slot_mapping   device, int64 [num_tokens]
 *   v_scale        device, fp32 [num_kv_heads]
 *   k_cache/v_cache device, the layer's pool (written in place)
 *   dev_error      device int32 word or NULL
 * k, v, caches: 16-byte aligned; token strides multiples of 8 elements.
 */
int32_t k16v8_kv_append(const void *k, int64_t k_token_stride, const void *v,
                        int32_t v_dtype, int64_t v_token_stride,
                        const int64_t *slot_mapping, int32_t num_tokens,
                        const float *v_scale, void *k_cache, uint8_t *v_cache,
                        int32_t num_pages, int32_t num_kv_heads, int32_t head_dim,
                        int32_t *dev_error, void *stream);

/*
 * Workspace for split-KV decode: partial outputs fp32
 * [batch][num_qo_heads][max_chunks][head_dim] followed by partial LSEs fp32
 * [batch][num_qo_heads][max_chunks], max_chunks = ceil(max_seq_len /
 * split_chunk) (at least 1), each region 256-byte aligned.  Returns 0 for
 * invalid arguments.
 */
size_t k16v8_decode_workspace_size(int32_t batch, int32_t num_qo_heads,
                                   int32_t head_dim, int32_t max_seq_len,
                                   int32_t split_chunk);

/* Byte offsets of the two workspace regions and max_chunks (host only). */
int32_t k16v8_decode_workspace_layout(int32_t batch, int32_t num_qo_heads,
                                      int32_t head_dim, int32_t max_seq_len,
                                      int32_t split_chunk,
                                      size_t *partial_o_offset,
                                      size_t *partial_lse_offset,
                                      int32_t *max_chunks);

/*
 * paged_decode_split -- the attention kernels of "Matched diagnostic
 * profiles", split over the KV sequence.
 *
 * One decode query per sequence.  For sequence b, query head h (KV head
 * g = h/4) and chunk c covering positions [c*split_chunk,
 * min((c+1)*split_chunk, L_b)), with s_j = sm_scale * q[b][h].k_j and
 * v_j = v_scale[g] * e4m3(v8_j):
 *   m_c = max_j s_j,  l_c = sum_j exp(s_j - m_c),
 *   partial_o[b][h][c][:] = sum_j exp(s_j - m_c) v_j / l_c
 *   partial_lse[b][h][c]  = m_c + ln l_c           (natural log)
 * Chunks at or beyond ceil(L_b / split_chunk) are not written.
 *
 *   q            device, fp16 [batch][num_qo_heads][head_dim], 16-B aligned
 *   block_table  device, int32 [batch][max_pages_per_seq]
 *   seq_lens     device, int32 [batch]; each <= max_seq_len (host hint that
 *                sizes the grid without a device->host copy)
 *   split_chunk  tokens per chunk: a multiple of 16 in [16, 8192]
 *   workspace    device, >= k16v8_decode_workspace_size(...) bytes, 256-B
 *                aligned; receives the partials
 *   sm_scale     softmax scale (1/sqrt(head_dim) for plain attention)
 */
int32_t k16v8_paged_decode_split(const void *q, const void *k_cache,
                                 const uint8_t *v_cache, const float *v_scale,
                                 const int32_t *block_table,
                                 int32_t max_pages_per_seq,
                                 const int32_t *seq_lens, int32_t max_seq_len,
                                 int32_t batch, int32_t num_qo_heads,
                                 int32_t num_kv_heads, int32_t head_dim,
                                 int32_t num_pages, float sm_scale,
                                 int32_t split_chunk, void *workspace,
                                 size_t workspace_bytes, int32_t *dev_error,
                                 void *stream);

/*
 * merge_states -- the merge kernels of "Matched diagnostic profiles": the
 * log-sum-exp combination of split-KV partials.  For each (b, h), over the
 * n_b = ceil(min(L_b, max_chunks*split_chunk) / split_chunk) live chunks:
 *   lse = M + ln sum_c exp(lse_c - M)   (M = max_c lse_c)
 *   out = sum_c exp(lse_c - lse) * o_c       -> fp16, lse -> fp32
 * n_b == 0 (an empty sequence) gives out = 0, lse = -inf.
 *
 *   partial_o    device, fp32 [batch][num_qo_heads][max_chunks][head_dim]
 *   partial_lse  device, fp32 [batch][num_qo_heads][max_chunks]
 *   seq_lens     device, int32 [batch]
 *   out          device, fp16 [batch][num_qo_heads][head_dim], 8-B aligned
 *   lse          device, fp32 [batch][num_qo_heads] or NULL
 */
int32_t k16v8_merge_states(const float *partial_o, const float *partial_lse,
                           int32_t batch, int32_t num_qo_heads,
                           int32_t max_chunks, int32_t head_dim,
                           const int32_t *seq_lens, int32_t split_chunk,
                           void *out, float *lse, void *stream);

/*
 * paged_decode_attention -- k16v8_paged_decode_split followed by
 * k16v8_merge_states on the same stream, writing fp16 out
 * [batch][num_qo_heads][head_dim] and fp32 lse [batch][num_qo_heads] (lse may
 * be NULL).  Arguments as for the two calls.  When max_seq_len <= split_chunk
 * (one chunk per sequence) only the split kernel is launched: each CTA
 * writes its rows of out / lse directly (zero rows and -inf for an empty
 * sequence), bit-equal to the merge of the single partial, and the
 * workspace is not written (it must still be given and large enough).
 * out must be 8-byte aligned.
 */
int32_t k16v8_paged_decode_attention(const void *q, const void *k_cache,
                                     const uint8_t *v_cache, const float *v_scale,
                                     const int32_t *block_table,
                                     int32_t max_pages_per_seq,
                                     const int32_t *seq_lens, int32_t max_seq_len,
                                     int32_t batch, int32_t num_qo_heads,
                                     int32_t num_kv_heads, int32_t head_dim,
                                     int32_t num_pages, float sm_scale,
                                     int32_t split_chunk, void *workspace,
                                     size_t workspace_bytes, void *out, float *lse,
                                     int32_t *dev_error, void *stream);

/*
 * paged_decode_attention_balanced -- the same result as
 * k16v8_paged_decode_attention (split-KV attention, then the log-sum-exp
 * merge, "Matched diagnostic profiles"), with the split chosen by the device
 * instead of a fixed split_chunk: all (sequence, KV head, page) tiles are
 * cut into one full wave of equal CTA ranges (SMs x 4 CTAs), so ragged
 * batches leave no tail wave.  Two launches (attention, merge) on `stream`.
 *
 *   batch        0 .. 8192 (0: nothing is launched)
 *   workspace    device, 256-B aligned, at least
 *                k16v8_decode_balanced_workspace_size(batch, num_qo_heads,
 *                head_dim) bytes, sized for the CURRENT device's SM count;
 *                contents need no initialisation and are overwritten
 *   seq_lens     device int32 [batch]; no max_seq_len is needed
 *   flags        0, or K16V8_DECODE_METADATA_READY: the caller guarantees
 *                that block_table and seq_lens are not written by the kernel
 *                launched immediately before this call on `stream` (host
 *                copies and earlier kernels are fine).  The attention kernel
 *                then reads them, plans its work and asks L2 to prefetch
 *                each warp's first cache pages before it waits for that
 *                kernel to finish (programmatic dependent launch); nothing
 *                of the cache reaches the SMs, and q, the workspace and the
 *                outputs are not touched, until after the wait.  Without
 *                the flag nothing is read before the wait.
 * Other arguments, outputs and device errors as for
 * k16v8_paged_decode_attention.  batch * max_pages_per_seq * num_kv_heads
 * and num_pages * num_kv_heads must stay below 2^31 - 1
 * (K16V8_ERR_INVALID_ARG otherwise).
 */
#define K16V8_DECODE_METADATA_READY 0x1

size_t k16v8_decode_balanced_workspace_size(int32_t batch, int32_t num_qo_heads,
                                            int32_t head_dim);

/*
 * The two launches of paged_decode_attention_balanced, for callers that
 * schedule them separately (same arguments; the workspace carries the work
 * plan and the partials from the first to the second).
 * paged_decode_balanced_split already writes the rows of every (sequence,
 * KV head) segment that one CTA held whole; merge_balanced writes the rest
 * (cut segments, and empty sequences: zeros and LSE -inf).
 */
int32_t k16v8_paged_decode_balanced_split(
    const void *q, const void *k_cache, const uint8_t *v_cache, const float *v_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes, void *out,
    float *lse, int32_t flags, int32_t *dev_error, void *stream);

int32_t k16v8_merge_balanced(const void *workspace, size_t workspace_bytes, int32_t batch,
                             int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                             void *out, float *lse, void *stream);

int32_t k16v8_paged_decode_attention_balanced(
    const void *q, const void *k_cache, const uint8_t *v_cache, const float *v_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes, void *out,
    float *lse, int32_t flags, int32_t *dev_error, void *stream);

/*
 * paged_decode_append_balanced_split / paged_decode_append_attention_balanced
 * -- the load-balanced decode with the step's cache write folded in:
 * equivalent to k16v8_kv_append of each sequence's new token at position
 * seq_lens[b] - 1 (slot block_table[b][(L-1)/16]*16 + (L-1)%16) followed by
 * k16v8_paged_decode_balanced_split (and, for _attention_balanced,
 * k16v8_merge_balanced), one kernel fewer per step ("Matched diagnostic
 * profiles": the candidate writes the compressed cache during decode).
 *   k_new, v_new  device fp16 [batch][num_kv_heads][head_dim], contiguous,
 *                 16-B aligned: the K and V of each sequence's new token
 *                 (read after the dependency wait)
 *   seq_lens      lengths INCLUDING the new token (L = 0: nothing appended)
 * Other arguments, flags, outputs and errors as for
 * k16v8_paged_decode_balanced_split / _attention_balanced; the cache row is
 * written with the rounding of k16v8_kv_append.  A row whose page id is
 * rejected is neither written nor attended (K16V8_DEVERR_PAGE).
 */
int32_t k16v8_paged_decode_append_balanced_split(
    const void *q, const void *k_new, const void *v_new, void *k_cache, uint8_t *v_cache,
    const float *v_scale, const int32_t *block_table, int32_t max_pages_per_seq,
    const int32_t *seq_lens, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t flags, int32_t *dev_error, void *stream);

int32_t k16v8_paged_decode_append_attention_balanced(
    const void *q, const void *k_new, const void *v_new, void *k_cache, uint8_t *v_cache,
    const float *v_scale, const int32_t *block_table, int32_t max_pages_per_seq,
    const int32_t *seq_lens, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t flags, int32_t *dev_error, void *stream);

/*
 * paged_decode_append_split / paged_decode_append_attention -- one decode
 * step's cache write fused into the attention kernel: equivalent to
 * k16v8_kv_append of each sequence's new token at position seq_lens[b] - 1
 * (slot block_table[b][(L-1)/16]*16 + (L-1)%16) followed by
 * k16v8_paged_decode_split (and, for _attention, k16v8_merge_states), in one
 * kernel instead of two.  "The candidate also gathers values and writes the
 * compressed cache" ("Matched diagnostic profiles") is the step folded in.
 *
 *   k_new, v_new  device fp16 [batch][num_kv_heads][head_dim], contiguous,
 *                 16-B aligned: the K and V of each sequence's new token
 *   seq_lens      lengths INCLUDING the new token (a sequence with L = 0 has
 *                 no new token and is skipped)
 * Other arguments as for k16v8_paged_decode_split / _attention (including
 * the one-chunk case of _attention: a single launch that writes out / lse).
 * The cache row is written with the same rounding as k16v8_kv_append.
 */
int32_t k16v8_paged_decode_append_split(const void *q, const void *k_new, const void *v_new,
                                        void *k_cache, uint8_t *v_cache, const float *v_scale,
                                        const int32_t *block_table, int32_t max_pages_per_seq,
                                        const int32_t *seq_lens, int32_t max_seq_len,
                                        int32_t batch, int32_t num_qo_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t num_pages, float sm_scale, int32_t split_chunk,
                                        void *workspace, size_t workspace_bytes,
                                        int32_t *dev_error, void *stream);

int32_t k16v8_paged_decode_append_attention(
    const void *q, const void *k_new, const void *v_new, void *k_cache, uint8_t *v_cache,
    const float *v_scale, const int32_t *block_table, int32_t max_pages_per_seq,
    const int32_t *seq_lens, int32_t max_seq_len, int32_t batch, int32_t num_qo_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t num_pages, float sm_scale,
    int32_t split_chunk, void *workspace, size_t workspace_bytes, void *out, float *lse,
    int32_t *dev_error, void *stream);

/*
 * FP16-KV control: the same cache write and split-KV decode for a pool that
 * stores values as fp16 ([num_pages][num_kv_heads][16][head_dim], 2 bytes,
 * no scale) -- the native controls of the subject page store FP16 keys and
 * values (intro), 5,120 B per token per layer instead of 3,840.  Kept to
 * measure the asymmetric format against it on the same kernels.
 *   k16v8_kv_append_v16: k, v fp16 [num_tokens][num_kv_heads][head_dim]
 *     (token strides as for k16v8_kv_append) copied to the caches.
 *   k16v8_paged_decode_split_v16 / _attention_v16: as the K16/V8 calls,
 *     with v_cache16 in place of (v_cache, v_scale).  Within a 16-token page
 *     the P.V products are summed in fp16, so |v| must stay below 4,094.
 */
int32_t k16v8_kv_append_v16(const void *k, int64_t k_token_stride, const void *v,
                            int64_t v_token_stride, const int64_t *slot_mapping,
                            int32_t num_tokens, void *k_cache, void *v_cache16,
                            int32_t num_pages, int32_t num_kv_heads, int32_t head_dim,
                            int32_t *dev_error, void *stream);

int32_t k16v8_paged_decode_split_v16(const void *q, const void *k_cache, const void *v_cache16,
                                     const int32_t *block_table, int32_t max_pages_per_seq,
                                     const int32_t *seq_lens, int32_t max_seq_len, int32_t batch,
                                     int32_t num_qo_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t num_pages, float sm_scale,
                                     int32_t split_chunk, void *workspace,
                                     size_t workspace_bytes, int32_t *dev_error, void *stream);

int32_t k16v8_paged_decode_attention_v16(const void *q, const void *k_cache,
                                         const void *v_cache16, const int32_t *block_table,
                                         int32_t max_pages_per_seq, const int32_t *seq_lens,
                                         int32_t max_seq_len, int32_t batch,
                                         int32_t num_qo_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t num_pages, float sm_scale,
                                         int32_t split_chunk, void *workspace,
                                         size_t workspace_bytes, void *out, float *lse,
                                         int32_t *dev_error, void *stream);

/*
 * paged_prefill_attention -- causal attention of a chunk of new prompt tokens
 * against the paged cache, on tensor cores.  The page's throughput metric
 * includes prefill ("Fixed throughput studies"); its 8K profile admits fresh
 * prompts before batch-16 decode ("Matched diagnostic profiles").  The
 * cache must already hold the chunk (call k16v8_kv_append first).
 *
 * Sequence b has qlen_b = qo_indptr[b+1] - qo_indptr[b] new tokens: the last
 * qlen_b of its seq_lens[b] cached positions.  Query row i of that sequence
 * sits at position p = seq_lens[b] - qlen_b + (i - qo_indptr[b]) and attends
 * to positions 0..p (causal).  With s_j = sm_scale * q[i][h].k_j and
 * v_j = v_scale[h/4] * e4m3(v8_j):
 *   out[i][h][:] = sum_{j<=p} exp(s_j - lse) v_j,   lse[i][h] = ln sum_{j<=p} exp(s_j)
 *
 *   q           device fp16 [total_q][num_qo_heads][head_dim], 16-B aligned
 *   qo_indptr   device int32 [batch+1], non-decreasing, qo_indptr[0] = 0,
 *               qo_indptr[batch] = total_q
 *   max_qlen    host hint: the largest qlen_b (sizes the grid)
 *   block_table, seq_lens, caches, v_scale: as for decode
 *   out         device fp16 [total_q][num_qo_heads][head_dim], 16-B aligned
 *   lse         device fp32 [total_q][num_qo_heads] or NULL
 * A sequence with qlen_b > seq_lens[b], seq_lens[b] > 16*max_pages_per_seq
 * or rows outside [0, total_q) flags K16V8_DEVERR_SEQLEN and is skipped; page ids outside [0, num_pages)
 * flag K16V8_DEVERR_PAGE and are not read.  No workspace is needed.
 */
int32_t k16v8_paged_prefill_attention(const void *q, const int32_t *qo_indptr,
                                      int32_t total_q, int32_t max_qlen,
                                      const void *k_cache, const uint8_t *v_cache,
                                      const float *v_scale, const int32_t *block_table,
                                      int32_t max_pages_per_seq, const int32_t *seq_lens,
                                      int32_t batch, int32_t num_qo_heads,
                                      int32_t num_kv_heads, int32_t head_dim,
                                      int32_t num_pages, float sm_scale, void *out,
                                      float *lse, int32_t *dev_error, void *stream);

/*
 * paged_prefill_attention_split -- the same causal prefill with the KV range
 * of each work item (a pair of 32-token query tiles of one sequence and KV
 * head) cut into up to 4 parts that run as separate CTAs, for calls whose
 * items would not fill the GPU in whole waves (e.g. one 1,024-token chunk of
 * one prompt: 16 pairs x 10 KV heads = 160 items on 152 SMs leaves a
 * near-empty second wave).  Every part writes its rows normalised by its own
 * softmax sum (fp16) and their LSE to the workspace; the part that finishes
 * last (an atomic counter per item, no waiting) combines them,
 * o = sum_p e^(lse_p - lse) o_p with lse = log sum_p e^lse_p, and writes out
 * and lse.  The fp16 rounding of the parts adds at most one fp16 ulp of each
 * part's share to the fp16 output.
 *   kv_splits   0: chosen from max_qlen, batch, num_kv_heads and the SM
 *               count (1 unless the items make less than two waves, then
 *               the count of 1..4 that best fills whole waves); 1..4 forced.
 *               A part holds at least 8 KV tiles (1,024 positions), so items
 *               with fewer than 16 tiles are not split whatever the count.
 *   max_seq_len an upper bound on this call's seq_lens, or 0 if unknown: with
 *               kv_splits = 0 it caps the parts at what the longest pair can
 *               use (one per 8 KV tiles), so calls over short prefixes
 *               launch no CTAs that would find nothing to do.  Only a hint:
 *               longer sequences are still computed correctly.
 *   workspace   device, k16v8_prefill_workspace_size(max_qlen, batch,
 *               num_qo_heads, num_kv_heads, head_dim, kv_splits,
 *               max_seq_len) bytes
 *               (0: no split, NULL allowed), 256-B aligned, zero-filled
 *               before its first use; a call that raises no device error
 *               leaves it ready for the next call (its counters back at 0).
 *               Calls that overlap on the GPU must not share one.
 * Other arguments, outputs and errors as for k16v8_paged_prefill_attention;
 * K16V8_ERR_WORKSPACE_TOO_SMALL if workspace_bytes is short,
 * K16V8_ERR_INVALID_ARG for kv_splits < 0, max_seq_len < 0 or a NULL /
 * unaligned workspace that is needed.
 */
size_t k16v8_prefill_workspace_size(int32_t max_qlen, int32_t batch, int32_t num_qo_heads,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t kv_splits,
                                    int32_t max_seq_len);

int32_t k16v8_paged_prefill_attention_split(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const void *k_cache, const uint8_t *v_cache, const float *v_scale, const int32_t *block_table,
    int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t batch, int32_t num_qo_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t num_pages, float sm_scale, int32_t kv_splits,
    int32_t max_seq_len, void *workspace, size_t workspace_bytes, void *out, float *lse,
    int32_t *dev_error, void *stream);

/*
 * paged_decode_attention_static -- the same computation as
 * k16v8_paged_decode_attention, for callers that cannot allocate device
 * memory: a host that runs inside an engine whose memory manager owns every
 * byte of the device, or code that must not call the CUDA allocator at all
 * (hard real-time paths, plug-ins loaded into a process that forbids it).
 * There is no counterpart in the paper; this is a packaging variant only.
 *
 * The split-KV partials go to a scratch array built into the library
 * (K16V8_STATIC_SCRATCH_BYTES bytes of device memory that every GPU which
 * loads the library keeps until the process exits) instead of a caller
 * workspace.  The call allocates nothing.
 *  - Needs k16v8_decode_workspace_size(batch, num_qo_heads, head_dim,
 *    max_seq_len, split_chunk) <= K16V8_STATIC_SCRATCH_BYTES, else returns
 *    K16V8_ERR_STATIC_SCRATCH_LIMIT and launches nothing.
 *  - The first call on a device looks up that device's address of the
 *    array (with the device current); make that first call before any
 *    stream capture.
 *  - Every call on a device shares the one array, and nothing in it needs to
 *    start at zero (each call writes every partial it reads).  Calls whose
 *    kernels overlap on the GPU (different streams, or concurrent host
 *    threads) race on it: serialise them.
 * Other arguments, layouts and errors as for k16v8_paged_decode_attention.
 */
#define K16V8_STATIC_SCRATCH_BYTES (32u << 20)
int32_t k16v8_paged_decode_attention_static(
    const void *q, const void *k_cache, const uint8_t *v_cache, const float *v_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, int32_t split_chunk, void *out,
    float *lse, int32_t *dev_error, void *stream);

/*
 * Test hooks of the bounded waits.  Every wait of a k16v8 kernel on an
 * asynchronous copy or a hand-off between warp roles gives up after a
 * bounded number of polls, sets K16V8_DEVERR_TIMEOUT in the error word,
 * lets the copies and tensor-core operations it did issue complete, and
 * returns, so a lost hand-off never hangs the GPU and the stream stays
 * usable.  The page records failures rather than hiding them ("Fixed
 * throughput studies"); these two calls let a test reach that path without
 * any fault: each runs the named call with the same arguments, except that
 * the first CTA of the grid withholds one copy (issues nothing and arrives
 * nowhere for it) and waits for it with a short limit.
 *   k16v8_paged_decode_split_wait_test: as k16v8_paged_decode_split; warp
 *     0 of CTA (chunk 0, KV head 0, sequence 0) withholds its first page.
 *   k16v8_paged_prefill_attention_wait_test: as
 *     k16v8_paged_prefill_attention; CTA (0, 0, 0) (the last query-tile
 *     pair of sequence 0, KV head 0) withholds its first KV tile.
 * The withholding CTA's results are incomplete (its partial, or its output
 * rows, are not valid); every other CTA computes normally.  After the call
 * the error word holds K16V8_DEVERR_TIMEOUT (if that CTA had work) and
 * later calls on the stream run normally.  Not for production use.
 */
int32_t k16v8_paged_decode_split_wait_test(const void *q, const void *k_cache,
                                           const uint8_t *v_cache, const float *v_scale,
                                           const int32_t *block_table,
                                           int32_t max_pages_per_seq,
                                           const int32_t *seq_lens, int32_t max_seq_len,
                                           int32_t batch, int32_t num_qo_heads,
                                           int32_t num_kv_heads, int32_t head_dim,
                                           int32_t num_pages, float sm_scale,
                                           int32_t split_chunk, void *workspace,
                                           size_t workspace_bytes, int32_t *dev_error,
                                           void *stream);

int32_t k16v8_paged_prefill_attention_wait_test(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const void *k_cache, const uint8_t *v_cache, const float *v_scale, const int32_t *block_table,
    int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t batch, int32_t num_qo_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t num_pages, float sm_scale, void *out,
    float *lse, int32_t *dev_error, void *stream);

/*
 * Speculative step.  A sequence's drafted tree has n nodes: node 0 is its
 * last committed token, node i > 0 hangs on node parents[i] < i.  The nodes
 * take the last n cached positions (base = seq_len - n, node i at base + i)
 * and rows qo_indptr[b] .. qo_indptr[b+1] - 1 of every ragged array; rows
 * beyond qo_indptr[batch] are neither read nor written.  A step:
 * k16v8_rope_kv_append writes the nodes (positions base + depth, slots of
 * base + i), k16v8_paged_tree_attention attends, k16v8_tree_verify picks the
 * accepted path and the next token, k16v8_kv_compact moves the accepted rows
 * to base, base + 1, ....  No counterpart on the page; the cache format and
 * the geometry are its intro's.
 */

/*
 * rope_kv_append -- rotary positions fused with k16v8_kv_append.
 *
 * Pair i (0 <= i < rotary_dim/2) of a head x at position p is turned by the
 * angle p * inv_freq[i] (formed beyond fp32, so far positions keep their
 * angle); with c = attn_factor * cos, s = attn_factor * sin:
 *   a' = a c - b s,  b' = b c + a s
 *   interleaved = 0: a = x[i], b = x[i + rotary_dim/2]   (half layout)
 *   interleaved = 1: a = x[2i], b = x[2i + 1]
 * Dims rotary_dim .. head_dim - 1 pass through.  For every token t with slot
 * s = slot_mapping[t] >= 0:
 *   q_out[t][h][:] = fp16(rotated q[t][h])          every query head
 *   k_cache[s/16][h][s%16][:] = fp16(rotated k[t][h])
 *   v_cache[s/16][h][s%16][:] = E4M3_rn_satfinite(fl32(v[t][h][:]) / v_scale[h])
 * (one rounding from fp32 each; a value beyond fp16's range becomes inf).  A
 * token with a negative slot is padding: nothing is written for it.  A slot
 * at or above num_pages*16 flags K16V8_DEVERR_SLOT, a position outside
 * [0, 2^24) K16V8_DEVERR_POSITION, and the token is skipped.  Duplicate slots
 * in one call leave an unspecified one of the writers.
 *
 *   q, k, v       device, [num_tokens][heads][head_dim] of x_dtype (fp16,
 *                 fp32 or bf16), token strides in elements (0 = dense), e.g.
 *                 slices of one fused projection
 *   positions     device int32 [num_tokens]
 *   inv_freq      device fp32 [rotary_dim/2], already scaled for long contexts
 *   rotary_dim    a multiple of 16 in [16, head_dim]
 *   attn_factor   finite; 1 without scaling
 *   q_out         device fp16 [num_tokens][num_qo_heads][head_dim]; may be q
 *                 itself when q is dense fp16.  num_qo_heads = 0: keys and
 *                 values only (q, q_out NULL)
 * q, k, v, q_out, caches: 16-byte aligned; token strides multiples of 16 bytes.
 */
int32_t k16v8_rope_kv_append(const void *q, int64_t q_token_stride, const void *k,
                             int64_t k_token_stride, const void *v, int64_t v_token_stride,
                             int32_t x_dtype, const int32_t *positions, const float *inv_freq,
                             int32_t rotary_dim, int32_t interleaved, float attn_factor,
                             const int64_t *slot_mapping, int32_t num_tokens,
                             const float *v_scale, void *q_out, void *k_cache, uint8_t *v_cache,
                             int32_t num_pages, int32_t num_qo_heads, int32_t num_kv_heads,
                             int32_t head_dim, int32_t *dev_error, void *stream);

/*
 * paged_tree_attention -- attention of every node of every tree over the
 * paged cache, which must already hold the nodes.  Node i of sequence b sees
 * the positions below base and position base + j exactly when bit j of
 * tree_mask[qo_indptr[b] + i] is set (bits >= n are ignored; set a node's own
 * bit for it to see itself, an ancestor's for each of its ancestors).  Over
 * what it sees, with s_j = sm_scale * q.k_j and v_j = v_scale[h/4] * e4m3(v8_j):
 *   lse = ln sum exp(s_j),  out = sum exp(s_j - lse) v_j
 * A row that sees nothing gives out = 0, lse = -inf.  What is stored at a
 * position that a row does not see (NaN, inf) does not reach that row.  The
 * weights are rounded to fp16 before they meet the values: 2^-11 relative, or
 * 2^-32 of the row's largest weight where that is more.
 *
 *   q            device fp16 [total_q][num_qo_heads][head_dim], 16-B aligned
 *   qo_indptr    device int32 [batch+1]
 *   max_nodes    host hint: the largest tree, <= K16V8_MAX_TREE_NODES
 *   tree_mask    device uint64 [total_q]
 *   seq_lens     device int32 [batch], the nodes included, <= max_seq_len
 *   max_seq_len  at most 2^30; batch at most 8192, num_kv_heads at most 4095,
 *                num_pages * num_kv_heads * 16 below 2^31
 *   sm_scale     finite, >= 0
 *   workspace    device, 256-B aligned, k16v8_tree_workspace_size(...) bytes
 *                for the same arguments on the same device (0 only where they
 *                are refused); needs no initialisation.  Calls that overlap on
 *                the GPU, replays of captured ones too, must not share one.
 *   out, lse     as for k16v8_paged_prefill_attention (lse may be NULL)
 * A sequence with rows outside [0, total_q), n > max_nodes, n > seq_len or
 * seq_len > max_seq_len flags K16V8_DEVERR_SEQLEN and is skipped; a page id
 * outside the pool flags K16V8_DEVERR_PAGE and its positions are seen by no
 * row.
 */
size_t k16v8_tree_workspace_size(int32_t total_q, int32_t batch, int32_t max_nodes,
                                 int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t max_seq_len);

int32_t k16v8_paged_tree_attention(const void *q, const int32_t *qo_indptr, int32_t total_q,
                                   int32_t max_nodes, const uint64_t *tree_mask,
                                   const void *k_cache, const uint8_t *v_cache,
                                   const float *v_scale, const int32_t *block_table,
                                   int32_t max_pages_per_seq, const int32_t *seq_lens,
                                   int32_t max_seq_len, int32_t batch, int32_t num_qo_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
                                   float sm_scale, void *workspace, size_t workspace_bytes,
                                   void *out, float *lse, int32_t *dev_error, void *stream);

/*
 * Test hook of its bounded waits, as the two above: CTA 0 (the first tiles of
 * the first sequence's KV head 0) withholds the keys of its first tile, so its
 * rows, and those joined with them, are not valid.
 */
int32_t k16v8_paged_tree_attention_wait_test(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_nodes,
    const uint64_t *tree_mask, const void *k_cache, const uint8_t *v_cache, const float *v_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream);

/*
 * tree_verify -- which nodes the target accepts (rejection sampling that
 * leaves the target's distribution unchanged) and the token after them.
 *
 * Row i of target_probs is the target's distribution of the token after node
 * i, row i of draft_probs the distribution from which node i's children were
 * drawn independently (NULL: children that were not sampled).  The walk starts
 * at node 0 with weights r = target_probs[0], Z = 1.  The children c of the
 * current node are tried in index order, x = tokens[c]:
 *   draft_probs given: accepted when u[c] * q[x] * Z < r[x]; else
 *                      r <- max(r - Z q, 0), Z <- sum r
 *   draft_probs NULL:  accepted when u[c] * Z < r[x]; else r[x] <- 0, Z <- sum r
 * An accepted child becomes the current node (r its row, Z = 1).  Where no
 * child is left, next_token is the smallest j with r_0 + ... + r_j > u[0] * sum r.
 * Should r have no weight left, the node's own row is used; a row without any
 * weight gives -1.  Weights are rounded to units of 2^-44 and summed exactly, so
 * the results do not depend on how the work is split.
 *
 *   target_probs, draft_probs  device fp32 [total_q][vocab_size], row strides
 *                 in elements (0 = vocab_size); values in [0, 1] (others are
 *                 clamped, NaN counts as 0), rows that sum to about 1 (the
 *                 formulas hold for others, up to the sums below)
 *   tokens        device int32 [total_q] (node 0's is not read)
 *   parents       device int32 [total_q], indices within the tree (node 0's is
 *                 not read)
 *   uniforms      device fp32 [total_q] in [0, 1): u above
 *   path          device int32 [batch][max_nodes]: the accepted nodes, 0 first,
 *                 then -1
 *   path_len      device int32 [batch] (0: no tree)
 *   next_token    device int32 [batch] (-1: no tree)
 * A node whose parent is not an earlier node of its tree, or whose token is
 * outside [0, vocab_size), flags K16V8_DEVERR_TREE and is never reached; rows
 * outside [0, total_q) or n > max_nodes flag K16V8_DEVERR_SEQLEN and give
 * path_len 0, a path of -1 and next_token -1.  So does, with
 * K16V8_DEVERR_PROBS, a tree at one of whose nodes the Z of the rejected
 * children add up to 64 or a row sums to 2^19 (rows that sum to at most 1.01
 * never do).
 */
int32_t k16v8_tree_verify(const float *target_probs, int64_t target_row_stride,
                          const float *draft_probs, int64_t draft_row_stride,
                          const int32_t *tokens, const int32_t *parents,
                          const int32_t *qo_indptr, int32_t total_q, int32_t max_nodes,
                          const float *uniforms, int32_t vocab_size, int32_t batch,
                          int32_t *path, int32_t *path_len, int32_t *next_token,
                          int32_t *dev_error, void *stream);

/*
 * kv_compact -- after verification: cache row base + path[b][j] moves to
 * base + j for every j < path_len[b], every KV head and every layer, in one
 * launch; new_seq_lens[b] = base + path_len[b].  Other rows keep their bytes
 * (those of rejected nodes among them).
 *
 *   k_caches, v_caches  device arrays of num_layers device addresses, the
 *                 layers' caches (distinct buffers of num_pages pages that
 *                 share the block table; NULL or not 16-byte aligned: flags
 *                 K16V8_DEVERR_PAGE, and nothing of the layer moves)
 *   seq_lens      device int32 [batch], the nodes included
 *   qo_indptr     device int32 [batch+1]: n = qo_indptr[b+1] - qo_indptr[b]
 *   path          device int32 [batch][max_nodes], strictly increasing
 *   new_seq_lens  device int32 [batch] or NULL; overlaps no input (refused
 *                 for the int32 arrays)
 * A path that does not increase strictly within its tree flags
 * K16V8_DEVERR_TREE, a sequence with n > seq_len, n > max_nodes or
 * seq_len > 16*max_pages_per_seq K16V8_DEVERR_SEQLEN: nothing of it moves and
 * its length stays.  A row whose page id is outside the pool is not moved
 * (K16V8_DEVERR_PAGE).  num_layers = 0 or batch = 0: nothing is launched.
 */
int32_t k16v8_kv_compact(const uint64_t *k_caches, const uint64_t *v_caches, int32_t num_layers,
                         const int32_t *block_table, int32_t max_pages_per_seq,
                         const int32_t *seq_lens, const int32_t *qo_indptr, const int32_t *path,
                         int32_t max_nodes, const int32_t *path_len, int32_t batch,
                         int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
                         int32_t *new_seq_lens, int32_t *dev_error, void *stream);

/*
 * rope_axes_kv_append -- k16v8_rope_kv_append for positions with several axes
 * (time, height and width of images and video): pair i is turned by the
 * position on axis pair_axis[i], angle positions[pair_axis[i]][t] * inv_freq[i].
 * Everything else is as there; a token with a position outside [0, 2^24) on
 * any axis is skipped and flags K16V8_DEVERR_POSITION.
 *
 *   positions  device int32 [num_axes][num_tokens]
 *   num_axes   1 .. K16V8_MAX_ROPE_AXES
 *   pair_axis  HOST int8 [rotary_dim/2], each in [0, num_axes); read during the
 *              call
 */
int32_t k16v8_rope_axes_kv_append(
    const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride, const void *v,
    int64_t v_token_stride, int32_t x_dtype, const int32_t *positions, int32_t num_axes,
    const int8_t *pair_axis, const float *inv_freq, int32_t rotary_dim, int32_t interleaved,
    float attn_factor, const int64_t *slot_mapping, int32_t num_tokens, const float *v_scale,
    void *q_out, void *k_cache, uint8_t *v_cache, int32_t num_pages, int32_t num_qo_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t *dev_error, void *stream);

/*
 * The K8/V8 cache: keys and values both in E4M3, with a scale for every page
 * and KV head of either.  No counterpart on the page (whose keys are FP16); the
 * geometry, the pages and the block tables are the same.
 *   k_cache   E4M3 [num_pages][num_kv_heads][16][head_dim]   (one byte)
 *   v_cache   E4M3 likewise
 *   kv_scale  fp32 [num_pages][num_kv_heads][2]: of the keys, of the values
 *   key = kv_scale[page][h][0] * e4m3(code),  value = kv_scale[page][h][1] * e4m3(code)
 * A scale is a power of two in [2^-15, 2^7]; the product is then an fp16 number.
 * The attention calls need num_pages * num_kv_heads * 16 below 2^31 and a batch
 * of at most 8192 (decode: batch * max_pages_per_seq * num_kv_heads below 2^31 -
 * 8192, too), the write a batch of at most 65535; K16V8_ERR_INVALID_ARG otherwise.
 */

/*
 * rope_kv_append_k8v8 -- the cache write of the K8/V8 cache, with rotary
 * positions as in k16v8_rope_axes_kv_append (rotary_dim = 0: without).
 * Sequence b has n = qo_indptr[b+1] - qo_indptr[b] new tokens, rows
 * qo_indptr[b] .. of q, k and v, which take its last n positions:
 * seq_lens[b] - n .. seq_lens[b] - 1.  Rows outside every sequence are neither
 * read nor written.  Of every page that gets rows, and every KV head, for K
 * (turned) and V alike, with x the new rows in fp32:
 *   s = the smallest power of two in [2^-15, 2^7] with max |x| <= 448 s
 *       (infinities and NaN left out); where the page holds earlier rows (a
 *       position of it is below the first new one), not below its scale
 *   scale = s, code = E4M3_rn_satfinite(x / s)
 *   earlier rows of the page, where the scale has grown:
 *   code' = E4M3_rn_satfinite(code * old scale / s)
 * Rows behind the last position stay as they are.  q_out = fp16(turned q).
 *
 *   q, k, v, q_out, positions, pair_axis, inv_freq, interleaved, attn_factor
 *                as in k16v8_rope_axes_kv_append (num_qo_heads = 0: K and V only)
 *   rotary_dim   0 or a multiple of 16 up to head_dim; 0: positions, pair_axis
 *                and inv_freq are not read
 *   qo_indptr    device int32 [batch+1], not decreasing (where it does, the
 *                sequence flags K16V8_DEVERR_SEQLEN and rows of others may be
 *                left out)
 *   seq_lens     device int32 [batch], the new tokens included
 *   block_table  device int32 [batch][max_pages_per_seq]; only entries of pages
 *                that get rows are read.  A page that gets rows belongs to one
 *                sequence (a shared one is copied first)
 *   kv_scale     8-byte aligned, written in place
 * A sequence with rows outside [0, num_tokens), n > seq_len or a length beyond
 * its table flags K16V8_DEVERR_SEQLEN and is skipped; a page id outside the pool
 * flags K16V8_DEVERR_PAGE and its tokens are skipped; a token with a position
 * outside [0, 2^24) flags K16V8_DEVERR_POSITION and is skipped.
 */
int32_t k16v8_rope_kv_append_k8v8(
    const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride, const void *v,
    int64_t v_token_stride, int32_t x_dtype, const int32_t *qo_indptr, int32_t num_tokens,
    const int32_t *positions, int32_t num_axes, const int8_t *pair_axis, const float *inv_freq,
    int32_t rotary_dim, int32_t interleaved, float attn_factor, const int32_t *block_table,
    int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t batch, void *q_out,
    uint8_t *k_cache, uint8_t *v_cache, float *kv_scale, int32_t num_pages, int32_t num_qo_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t *dev_error, void *stream);

/*
 * paged_decode_attention_k8v8 -- k16v8_paged_decode_attention_balanced over the
 * K8/V8 cache: one query row per sequence, every position of it seen.
 *   sm_scale   finite, >= 0
 *   block_table  device int32 [batch][max_pages_per_seq] (may be NULL where that
 *              is 0)
 *   workspace  k16v8_decode_workspace_size_k8v8(...) bytes (0 only where the sizes
 *              are refused), 256-B aligned, needs no initialisation; calls that
 *              overlap on the GPU, replays of captured ones too, must not share one
 *   q, out     device fp16 [batch][num_qo_heads][head_dim], 16-B aligned; out may
 *              be q
 *   lse        device fp32 [batch][num_qo_heads] or NULL
 * A sequence of length 0 gives out = 0, lse = -inf.  Lengths outside [0, 16 *
 * max_pages_per_seq] flag K16V8_DEVERR_SEQLEN and are clamped; a page id outside
 * the pool flags K16V8_DEVERR_PAGE and its positions are left out.  The weights are
 * rounded to fp16 before they meet the values, as in the prefill call: 2^-11
 * relative, or 2^-32 of the row's largest weight where that is more, whatever the
 * pages' scales.
 */
size_t k16v8_decode_workspace_size_k8v8(int32_t batch, int32_t num_qo_heads, int32_t head_dim);

int32_t k16v8_paged_decode_attention_k8v8(
    const void *q, const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens, int32_t batch,
    int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
    float sm_scale, void *workspace, size_t workspace_bytes, void *out, float *lse,
    int32_t *dev_error, void *stream);

/*
 * paged_prefill_attention_k8v8, paged_cross_attention_k8v8 -- attention of
 * several query rows per sequence over the K8/V8 cache, on the tensor cores.
 * Sequence b has rows qo_indptr[b] .. qo_indptr[b+1] - 1 of q, n of them, and
 * L = seq_lens[b] cached positions.
 *   prefill: causal; its rows are the last n positions (already in the cache),
 *            row i sees positions 0 .. L - n + i
 *   cross:   every row sees all L positions (an encoder's states, written with
 *            k16v8_rope_kv_append_k8v8 and num_qo_heads = 0); n and L are
 *            unrelated, L may be 0
 * One row per sequence is better served by k16v8_paged_decode_attention_k8v8,
 * which sees all positions too (1,024 sequences of 50 to 100: 54 against 261 us).
 * Over what a row sees: lse = ln sum exp(s_j), out = sum exp(s_j - lse) v_j, s_j
 * = sm_scale * q.k_j.  A row that sees nothing gives out = 0, lse = -inf.  What
 * is stored at a position that a row does not see (NaN, inf) does not reach it.
 * The weights are rounded to fp16 before they meet the values: 2^-11 relative,
 * or 2^-32 of the row's largest weight where that is more.
 *
 *   q            device fp16 [total_q][num_qo_heads][head_dim], 16-B aligned
 *   qo_indptr    device int32 [batch+1]
 *   max_qlen     host: no sequence has more rows
 *   max_seq_len  host: no sequence is longer; at most 2^30 and 16 *
 *                max_pages_per_seq.  num_kv_heads at most 4095
 *   sm_scale     finite, >= 0
 *   workspace    device, 256-B aligned, k16v8_attention_workspace_size_k8v8(...)
 *                bytes for the same arguments on the same device (0 only where
 *                they are refused); needs no initialisation.  Calls that overlap
 *                on the GPU, replays of captured ones too, must not share one.
 *   out          device fp16 like q, or q itself; lse device fp32 [total_q][num_qo_heads] or
 *                NULL.  Rows of no sequence are left as they are
 * A sequence with rows outside [0, total_q), n > max_qlen, a length outside [0,
 * max_seq_len] or (prefill) n > L flags K16V8_DEVERR_SEQLEN and is skipped; a
 * page id outside the pool flags K16V8_DEVERR_PAGE and its positions are seen by
 * no row.
 */
size_t k16v8_attention_workspace_size_k8v8(int32_t max_qlen, int32_t num_qo_heads,
                                           int32_t num_kv_heads, int32_t head_dim);

int32_t k16v8_paged_prefill_attention_k8v8(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream);

int32_t k16v8_paged_cross_attention_k8v8(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream);

/*
 * Test hook of its bounded waits, as k16v8_paged_tree_attention_wait_test: CTA 0
 * (the first tiles of the first sequence's KV head 0) withholds the keys of its
 * first tile, so its rows, and those joined with them, are not valid.
 */
int32_t k16v8_paged_prefill_attention_k8v8_wait_test(
    const void *q, const int32_t *qo_indptr, int32_t total_q, int32_t max_qlen,
    const uint8_t *k_cache, const uint8_t *v_cache, const float *kv_scale,
    const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
    int32_t max_seq_len, int32_t batch, int32_t num_qo_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t num_pages, float sm_scale, void *workspace, size_t workspace_bytes,
    void *out, float *lse, int32_t *dev_error, void *stream);

/*
 * Wait for `stream`, then copy the device error word to *host_value and
 * return K16V8_OK when it is zero, K16V8_ERR_DEVICE_BOUNDS otherwise
 * (K16V8_ERR_CUDA if the synchronisation or copy fails).
 */
int32_t k16v8_read_device_error(const int32_t *dev_error, void *stream,
                                int32_t *host_value);

/* Static, human-readable name of a status code. */
const char *k16v8_status_string(int32_t status);

#ifdef __cplusplus
}
#endif

#endif /* K16V8_H */
