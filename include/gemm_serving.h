/*
 * gemm_serving.h - the operators of a serving step around the GEMMs and the attention of
 * gemm.h: rotary positions with per-head norms, the same written into a paged key/value cache,
 * and attention that reads such a cache, whose batch may share a long prefix.
 *
 * All calls take a context of gemm.h, are asynchronous on `stream` (a cudaStream_t; NULL = the
 * legacy default stream), allocate nothing, may be captured into a CUDA graph (the contents of
 * device arrays, lengths and page tables among them, may change between replays), and return a
 * gemm_status before anything is enqueued if an argument is refused. Forward only.
 *
 * Paged cache. Keys and values of all sequences live in num_pages pages of page_size rows per
 * key head. A sequence's own keys 0, 1, 2, ... are in row (k mod page_size) of page
 * page_table[s][k / page_size]. The table's entries past the sequence's last page are not read.
 *
 * Ragged batch. Sequence s has the new tokens q_start[s] .. q_start[s + 1] - 1 of the flat token
 * dimension (any number, zero included) and, with them, kv_lens[s] own keys. If the batch has a
 * shared prefix of P keys (whole pages: prefix_pages), these come before every sequence's own
 * keys. New token i of n stands at position P + kv_lens[s] - n + i and sees the keys at
 * positions up to its own (if that is negative: none). Tokens from q_start[num_seqs] on belong
 * to no sequence: nothing of theirs is written.
 *
 * Lengths and page numbers are read on the device. A value out of range (q_start decreasing or
 * past num_tokens, kv_lens negative, more keys than the table has pages for, a new token before
 * the sequence's first own key in gemm_kv_append, a page number outside [0, num_pages)) makes no
 * access out of range: it is limited to the range (a bad page: reads as zeros, is not written),
 * and gemm_last_device_error returns GEMM_ERR_INDEX.
 */
#ifndef GB300_GEMM_SERVING_H
#define GB300_GEMM_SERVING_H

#include <stdint.h>

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of queries, keys, values, norm weights and outputs. */
enum gemm_dtype { GEMM_F16 = 0, GEMM_BF16 = 1 };

/* Vectors of head_dim values for tokens x heads, head_dim contiguous: the vector of (token t,
 * head h) starts at data + t * token_stride + h * head_stride (elements; both multiples of 8 and
 * not negative, data 16-byte aligned). A slice of a packed projection and a head-major tensor
 * are both of this form. heads = 0 (data may be NULL) leaves the operand out. */
typedef struct gemm_heads {
    void *data;
    int64_t heads, token_stride, head_stride;
} gemm_heads;

/* The paged cache: key (or value) vector of (page, head, row) at k (or v) + page * page_stride +
 * head * head_stride + row * row_stride (elements, multiples of 8, positive). head_dim 64 or
 * 128; page_size a power of two from 16 to 1024; num_pages up to 2^31 - 2. */
typedef struct gemm_kv_cache {
    void *k, *v;
    int64_t num_pages, page_size, kv_heads, head_dim;
    int64_t page_stride, head_stride, row_stride;
    int32_t dtype; /* gemm_dtype */
} gemm_kv_cache;

/* The ragged batch. Device arrays of int32 (4-byte aligned): q_start[num_seqs + 1],
 * kv_lens[num_seqs], page_table[num_seqs] rows of table_width entries table_stride apart,
 * prefix_pages[num_prefix_pages] (NULL without a prefix). num_tokens: the size of the flat token
 * dimension. max_q: the largest number of new tokens of a sequence, as far as the caller knows
 * (0: unknown); results do not depend on it, the choice of kernels does.
 * num_seqs is at most 2^24, num_tokens at most 2^31 - 1024, (table_width + num_prefix_pages) * page_size at most 2^31 - 1024. */
typedef struct gemm_kv_batch {
    int64_t num_seqs, num_tokens, max_q;
    const int32_t *q_start, *kv_lens, *page_table;
    int64_t table_width, table_stride;
    const int32_t *prefix_pages;
    int64_t num_prefix_pages;
} gemm_kv_batch;

/* Norm and rotation of query and key heads.
 *   q_norm, k_norm: head_dim weights (device, 16-byte aligned) of an RMS norm over each head,
 *     y = x / sqrt(mean(x^2) + eps) * w, done first, the mean in FP32 (magnitudes up to 1e18);
 *     NULL: no norm.
 *   rotary_dim: the first rotary_dim values of a head are rotated (a multiple of 16, 0 for none,
 *     up to head_dim), in pairs (i, i + rotary_dim / 2), or (2i, 2i + 1) if interleaved. Pair i
 *     at position p turns by p * table[i] * 2^-64 of a full turn, computed modulo one turn in
 *     64-bit integers, so that far positions add no error but the table's own, p times; the
 *     sine takes the angle to 2^-26 of a turn:
 *       (a, b) -> scale * (a cos - b sin, b cos + a sin).
 *   table: rotary_dim / 2 words (device, 8-byte aligned), see gemm_rope_table. */
typedef struct gemm_rope {
    const uint64_t *table;
    int64_t rotary_dim;
    const void *q_norm, *k_norm;
    float eps, scale;
    int32_t interleaved;
} gemm_rope;

/* How gemm_rope_table stretches the frequencies f_i = base^(-2i / rotary_dim) for contexts
 * `factor` times as long as the model was trained on (factor >= 1). */
enum gemm_rope_scaling {
    GEMM_ROPE_PLAIN = 0,  /* f_i                                                          */
    GEMM_ROPE_LINEAR = 1, /* f_i / factor (positions interpolated)                        */
    GEMM_ROPE_NTK = 2,    /* base replaced by base * factor^(rotary_dim / (rotary_dim - 2)) */
    GEMM_ROPE_YARN = 3    /* "YaRN" by parts (Peng et al., 2023): f_i / factor where fewer than 1
                             turn fits the original length, f_i where more than 32 do, between
                             them a mix linear in the number of turns, as in the paper (code
                             that mixes linearly in the pair's index has other frequencies
                             there: for its checkpoints fill a table of your own);
                             *scale = 0.1 ln(factor) + 1, else 1                           */
};

/* Fills `table` (HOST memory, rotary_dim / 2 words) with the turns per position of each pair in
 * units of 2^-64 (f_i / 2 pi times 2^64, rounded; computed in FP64, so within 2^-55 of a turn), and
 * *scale (may be NULL) with the factor for gemm_rope.scale. `original`: the trained length in
 * positions (read for GEMM_ROPE_YARN only). Computes on the host; needs no context. GEMM_ERR_ARG if
 * rotary_dim is not a positive multiple of 16 up to 128, base <= 1, factor < 1 or not finite, or
 * original <= 0 where it is read. */
int gemm_rope_table(int64_t rotary_dim, double base, int scaling, double factor, double original,
                    uint64_t *table, float *scale);

/* q_out, k_out = norm and rotation of q and k (FP32 arithmetic, one rounding), token t at
 * position positions[t] (device, int32, any value). head_dim 64 or 128. The outputs have their
 * inputs' head counts and strides of their own (head-major outputs feed gemm_attention_fwd). An
 * output may be its own input (same data and strides); otherwise no two of the four overlap.
 * tokens = 0 is a no-op. One kernel launch. */
int gemm_qk_rope(gemm_ctx *ctx, int dtype, int64_t tokens, int64_t head_dim, const gemm_heads *q,
                 const gemm_heads *k, const int32_t *positions, const gemm_rope *rope, const gemm_heads *q_out,
                 const gemm_heads *k_out, void *stream);

/* The same for the new tokens of a batch at the positions given above: q_out = norm and rotation
 * of q (q->heads = 0: left out), and each token's key (norm and rotation of k) and value (v as it
 * is) written to its row of the cache. k->heads = v->heads = cache->kv_heads. q_out may be q;
 * the cache may not overlap q, k, v or q_out. No two tokens of a call may have the same row of
 * the same page (their writes would race). Of the prefix only num_prefix_pages is used.
 * num_tokens = 0 or num_seqs = 0 is a no-op. One kernel launch. */
int gemm_kv_append(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_heads *q,
                   const gemm_heads *k, const gemm_heads *v, const gemm_rope *rope, const gemm_heads *q_out,
                   void *stream);

/* out[t][h][:] = sum_j softmax_j(scale * q[t][h][:] . K[j][h'][:]) V[j][h'][:] over the keys j
 * that token t sees (scale: any sign, |scale| up to 2.35e38; 0 for the mean, of which
 * scores of -inf are no part), h' = h / (q->heads / kv_heads); q->heads is a multiple of kv_heads, at most
 * 128 times it, and num_tokens * q->heads at most 2^33. lse (may be NULL): FP32,
 * lse[t * lse_stride + h] = ln sum_j exp(scale * q . K_j). A token that sees no key gets out = 0 and
 * lse = -inf; one that sees keys, all of scores -inf, lse = -inf and out = NaN (0/0).
 * FP32 scores, statistics and sums; probabilities are rounded to the element type for the
 * product with V (FP16: with 11 bits down to 2^-25 of the row's largest, with fewer down to 2^-36). Keys and values that a token does not see are ignored whatever they are (NaN
 * too).
 * out has q's heads and strides of its own and may not overlap q, the cache or the workspace.
 * workspace: 256-byte aligned device memory of at least gemm_paged_attention_workspace bytes,
 * used from this call until the stream has passed it and by no other call meanwhile (captured
 * graphs that may run at the same time need one each); its contents on entry do not matter.
 * At most four kernel launches. In-kernel waits report through gemm_last_device_error. */
int gemm_paged_attention(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_heads *q,
                         float scale, const gemm_heads *out, float *lse, int64_t lse_stride, void *workspace,
                         int64_t workspace_bytes, void *stream);

/* Workspace bytes of gemm_paged_attention for these arguments (sizes and counts are read, device
 * arrays are not), 0 when the call has nothing to do, or a negative gemm_status. */
int64_t gemm_paged_attention_workspace(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch,
                                       int64_t q_heads);

#ifdef __cplusplus
}
#endif

#endif /* GB300_GEMM_SERVING_H */
