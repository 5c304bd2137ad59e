/*
 * kda_layers.h -- C ABI of the operators around the KDA layers of a hybrid
 * stack: the projections before and after a mixer, linear attention with one
 * decay per head (a sequence mixer of the same state layout as KDA, without
 * the delta rule), and the full-attention layers' paged key-value cache.
 *
 *     linear          out = act(x w^T + bias) + residual
 *     decay prefill   S_t = lambda S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
 *     decay decode    the same for one new token per sequence
 *     paged append    keys and values of new tokens into the pages of a cache
 *     paged decode    softmax attention of one new token over that cache
 *
 * The conventions of kda.h hold: device pointers owned by the caller, calls
 * asynchronous on `stream`, argument errors found on the host before anything
 * is launched, no device memory allocated, no call traps.  Four more:
 *   - Per-token tensors [T, H, d] that are read (q, k, v, x) take a row stride
 *     (ld*, in elements, at least H d; a row is dense), so slices of one fused
 *     projection are passed as they are.  Rows past 2^31 elements are fine.
 *     What is written is dense, and overlaps nothing that the call reads
 *     unless stated.
 *   - `status` is a device uint32 or NULL.  The call never clears it; the
 *     first condition found on the device (a malformed offset, length, slot or
 *     page, KDA_ERR_INVALID_ARG; an expired bounded wait,
 *     KDA_ERR_DEVICE_TIMEOUT) is recorded in it, and kda_check_device_status
 *     reads it.  What is malformed is treated as absent: it is never read or
 *     written.
 *   - Every pointer is aligned to its elements (status to 4 bytes), and further
 *     where stated; KDA_ERR_INVALID_ARG otherwise.
 *   - A row's result depends on that row's inputs alone: infinities and NaN in
 *     other sequences, in later tokens, or in cache slots that no token was
 *     written to do not reach it.  (Its own infinities may give NaN where the
 *     formula has an infinity.)
 */
#ifndef KDA_GB300_LAYERS_H
#define KDA_GB300_LAYERS_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_ACT_NONE = 0,
    KDA_ACT_RELU = 1,
    KDA_ACT_GELU = 2,     /* y Phi(y), with the error function */
    KDA_ACT_SILU = 3,     /* y sigmoid(y) */
    KDA_ACT_SIGMOID = 4   /* e.g. KDA's beta from its projection */
} kda_act_t;

/*
 * kda_linear -- out = act(x w^T + bias) + residual, in one pass over out.
 *   x         [M, K] bf16, row stride ldx >= K
 *   w         [N, K] bf16, dense (a weight as trained: one row per output)
 *   bias      [N] float32, or NULL
 *   residual  [M, N] of out_dtype, dense, or NULL; it may be the same buffer
 *             as out
 *   out       [M, N] of out_dtype (KDA_BF16 or KDA_F32), dense (written)
 * Products are summed in float32 and rounded once, after the residual.  The
 * tensor cores' own sums lose up to an ulp, 2^-23, at each step of 16 products:
 * a float32 output is summed there in parts of 512 products, which are added in
 * float32, a bf16 output in parts of up to 65536 (2^-11 of the result at most,
 * where its rounding takes 2^-9).
 * Any M, N >= 0 and K >= 1 below 2^31, any row stride and alignment of elements.
 * K a multiple of 8 with 16-byte aligned rows is loaded by TMA, anything else by
 * way of registers: three times slower for few rows, ten times for thousands.
 * Out and residual with 16-byte aligned rows are stored and loaded by TMA for
 * many rows, others take about twice the time.
 */
kda_status_t kda_linear(const void *x, int64_t ldx, const void *w, const float *bias,
                        const void *residual, void *out, int64_t M, int64_t N, int64_t K,
                        kda_act_t act, kda_dtype_t out_dtype, uint32_t *status,
                        kda_stream_t stream);

/*
 * kda_decay_prefill_workspace_size -- bytes of workspace with which
 * kda_decay_prefill splits batches of few long chains over the GPU; 0 where
 * these sizes have no use for one.
 */
size_t kda_decay_prefill_workspace_size(int64_t total_tokens, int num_seqs, int H, int dk, int dv,
                                        kda_dtype_t dtype);

/*
 * kda_decay_prefill -- linear attention with one decay per head over a packed
 * batch of sequences, per (sequence, head):
 *     S_t = exp(log_decay) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
 *   q, k           [total_tokens, H, dk], v [total_tokens, H, dv], of dtype, row
 *                  strides ldq, ldk, ldv
 *   log_decay      [H] float32, device; <= 0 for a decay, -inf for no memory, NaN
 *                  for NaN from the first token on
 *   cu_seqlens     [num_seqs + 1] int32, device, as for kda_chunk_prefill
 *   initial_state  [num_seqs, H, dk, dv] float32, or NULL for zeros
 *   final_state    [num_seqs, H, dk, dv] float32 (written), or NULL; it may be
 *                  the same buffer as initial_state
 *   out            [total_tokens, H, dv] of dtype (written)
 *   workspace      16-byte aligned, or NULL; with fewer bytes than the size
 *                  above the call runs every chain in one piece
 * dk, dv in {32, 64, 128}.  States, and what is added to them, are float32
 * throughout.  Of a bf16 call's outputs the weights lambda^(i-j) q_i . k_j within
 * a chunk of 64 tokens, and the copy of the state that multiplies q, are rounded
 * to bf16 (2^-9 of each, as the output's own rounding) for the tensor cores;
 * rows that no 16-byte copy can start on are worked on in float32.
 */
kda_status_t kda_decay_prefill(const void *q, int64_t ldq, const void *k, int64_t ldk,
                               const void *v, int64_t ldv, const float *log_decay,
                               const int32_t *cu_seqlens, int num_seqs, int64_t total_tokens,
                               int H, int dk, int dv, kda_dtype_t dtype, float scale,
                               const float *initial_state, float *final_state, void *out,
                               void *workspace, size_t workspace_bytes, uint32_t *status,
                               kda_stream_t stream);

/*
 * kda_decay_decode -- one new token for each of N sequences, states in a pool
 * and updated in place (slots as for kda_decode_tokens: negative = padding
 * row, zero outputs; >= pool_size = recorded, padded; NULL = slot i).
 *   q, k        [N, H, dk], v [N, H, dv], of dtype, row strides ldq, ldk, ldv
 *   state_pool  [pool_size, H, dk, dv] float32, 16-byte aligned
 *   out         [N, H, dv] of dtype (written)
 */
kda_status_t kda_decay_decode(const void *q, int64_t ldq, const void *k, int64_t ldk,
                              const void *v, int64_t ldv, const float *log_decay,
                              float *state_pool, int pool_size, const int32_t *slot_ids, void *out,
                              int N, int H, int dk, int dv, kda_dtype_t dtype, float scale,
                              uint32_t *status, kda_stream_t stream);

/*
 * kda_paged_append -- writes new tokens' keys and values into a paged cache.
 *   k, v             [total_tokens, Hkv, d] of dtype, row strides ldk, ldv
 *   k_cache, v_cache [num_pages, Hkv, page_size, d] of dtype, 16-byte aligned: a
 *                    page of one head is one contiguous block
 *   page_table       [num_seqs, max_pages] int32, device: token p of a sequence
 *                    lives in page page_table[seq][p / page_size]
 *   start_pos        [num_seqs] int32, device: tokens already cached
 *   cu_seqlens       [num_seqs + 1] int32, device, or NULL for one token per
 *                    sequence (total_tokens = num_seqs)
 * Token t of sequence i goes to position start_pos[i] + t - cu_seqlens[i].
 * page_size is a power of two up to 1024, d in {32, 64, 128}.  A position past
 * the table, or a page id outside the cache, is recorded in *status and skipped.
 */
kda_status_t kda_paged_append(const void *k, int64_t ldk, const void *v, int64_t ldv, void *k_cache,
                              void *v_cache, int num_pages, int page_size,
                              const int32_t *page_table, int max_pages, const int32_t *start_pos,
                              const int32_t *cu_seqlens, int num_seqs, int64_t total_tokens, int Hkv,
                              int d, kda_dtype_t dtype, uint32_t *status, kda_stream_t stream);

/* Workspace of kda_paged_decode (its partial results) for sequences of up to
 * max_tokens = max_pages page_size tokens. */
size_t kda_paged_decode_workspace_size(int num_seqs, int64_t max_tokens, int Hq, int Hkv, int d,
                                       kda_dtype_t dtype);

/*
 * kda_paged_decode -- softmax attention of one token per sequence over the
 * first seq_lens[i] tokens of its cache (the new token's own key and value
 * appended before):
 *     out = softmax(scale q K^T) V,   lse = log sum exp(scale q K^T)
 *   q            [num_seqs, Hq, d] of dtype, row stride ldq; query head h reads
 *                key-value head h / (Hq / Hkv); Hq is a multiple of Hkv
 *   k_cache, v_cache, page_table: as for kda_paged_append; the caches may be
 *                NULL where num_pages is 0, the table where max_pages is
 *   seq_lens     [num_seqs] int32, device; 0 gives zero outputs and lse -inf.  A
 *                negative length counts as 0 and one past the table as the
 *                table's end, both recorded in *status
 *   out          [num_seqs, Hq, d] of dtype (written)
 *   lse          [num_seqs, Hq] float32 (written), or NULL
 *   workspace    16-byte aligned, kda_paged_decode_workspace_size() bytes
 * Scores, maxima and sums are float32.  With bf16 caches of 64 or 128 channels and
 * pages of at least eight tokens the softmax weights are rounded to bf16 (2^-9 of
 * each, as the output's own rounding) for their product with V, though not for
 * their sum.
 * Tokens on a page whose id lies outside the cache are recorded and left out.
 * A table covers at most 2^30 tokens per sequence.
 */
kda_status_t kda_paged_decode(const void *q, int64_t ldq, const void *k_cache, const void *v_cache,
                              int num_pages, int page_size, const int32_t *page_table,
                              int max_pages, const int32_t *seq_lens, int num_seqs, int Hq, int Hkv,
                              int d, kda_dtype_t dtype, float scale, void *out, float *lse,
                              void *workspace, size_t workspace_bytes, uint32_t *status,
                              kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_LAYERS_H */
