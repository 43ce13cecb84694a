/*
 * gemm_decode.h - operators of decoding a few tokens at a time, beside those of gemm_serving.h on
 * the same paged cache: attention for trees of drafted tokens (and the masks and positions of
 * such trees), a cache held to a bounded size by the attention weight that its keys have drawn,
 * rows of a cache moved up (what an eviction or an accepted path keeps), and products with 4-bit
 * weights for few rows.
 *
 * As in gemm_serving.h: all calls are asynchronous on `stream`, allocate nothing, may be captured
 * into a CUDA graph (the contents of device arrays may change between replays), and return a
 * gemm_status before anything is enqueued if an argument is refused. Lengths, indexes and page
 * numbers are read on the device; a value out of range makes no access out of range, and
 * gemm_last_device_error returns GEMM_ERR_INDEX. Forward only.
 *
 * A step that verifies drafts: gemm_tree_mask (positions and mask from the parents), gemm_qk_rope
 * at those positions, gemm_kv_append without table and norms (a drafted token's key goes to the
 * row of its index, not of its depth), gemm_tree_attention, and, once it is known which nodes
 * were right, gemm_kv_compact with their indexes. After an eviction a sequence has fewer keys
 * than positions: its new tokens' positions, too, are the caller's to give (gemm_qk_rope, then
 * gemm_kv_append without table).
 */
#ifndef GB300_GEMM_DECODE_H
#define GB300_GEMM_DECODE_H

#include <stdint.h>

#include "gemm_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- trees of drafted tokens --------------------------------------------------------------
 *
 * The new tokens of a sequence (gemm_kv_batch) are the nodes of a tree, or of several: token i's
 * key is at row kv_lens[s] - n + i of the sequence's own keys. Bit j (bit j mod 32 of word j / 32)
 * of a token's row of the mask says whether it sees the key of the sequence's new token j; every
 * key before the new tokens' is seen. Bits from n on do not matter. Any mask will do, rows without a
 * bit and bits that are no tree among them. A sequence may have up to 32 * mask_words new tokens
 * (more: GEMM_ERR_INDEX, keys without a bit are not seen), and as many as it has own keys (more
 * of them: GEMM_ERR_INDEX, key j is then new token j's).
 */
#define GEMM_TREE_MAX_WORDS 64

/* mask: mask_words words for token t at mask + t * mask_stride (device, 4-byte aligned). */
typedef struct gemm_tree {
    const uint32_t *mask;
    int64_t mask_words, mask_stride;
} gemm_tree;

/* Masks and positions of trees given by parents[t] (device, int32, one per token): the index,
 * among its sequence's new tokens, of the node before it, which is lower than its own, or -1 for
 * a node that follows the sequence's last key before the new ones. A node sees itself and the
 * nodes on its way up; its position (positions[t], int32; NULL: not wanted) is
 * prefix_len + kv_lens[s] - n + the number of nodes above it (with fewer own keys than new tokens
 * prefix_len + that number, and GEMM_ERR_INDEX). A parent out of range counts as -1
 * (GEMM_ERR_INDEX); a node past the 32 * mask_words-th (GEMM_ERR_INDEX) gets no bits and the position
 * of a node without a parent. Of the batch, q_start, kv_lens and the counts are read. Rows of tokens
 * that belong to no sequence are not written. One kernel launch. */
int gemm_tree_mask(gemm_ctx *ctx, const gemm_kv_batch *batch, int64_t prefix_len, const int32_t *parents, uint32_t *mask,
                   int64_t mask_words, int64_t mask_stride, int32_t *positions, void *stream);

/* gemm_paged_attention with the mask in the place of the order of the new tokens: token t sees
 * the whole prefix, the sequence's own keys before the new tokens', and those of the new ones
 * that its bits name. All else (arguments, limits, precision, rows that see nothing, workspace)
 * is as there. mask_words from 1 to GEMM_TREE_MAX_WORDS. */
int gemm_tree_attention(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_tree *tree,
                        const gemm_heads *q, float scale, const gemm_heads *out, float *lse, int64_t lse_stride,
                        void *workspace, int64_t workspace_bytes, void *stream);

/* Workspace bytes of gemm_tree_attention (as gemm_paged_attention_workspace). */
int64_t gemm_tree_attention_workspace(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch,
                                      int64_t q_heads);

/* ---- eviction by attention weight ------------------------------------------------------------ */

/* The lengths and pages of num_seqs sequences, as in gemm_kv_batch. */
typedef struct gemm_kv_seqs {
    int64_t num_seqs;
    const int32_t *kv_lens, *page_table;
    int64_t table_width, table_stride;
} gemm_kv_seqs;

/* One FP32 weight for each key and key head of a paged cache: that of (page, head, row) at
 * data + page * page_stride + head * head_stride + row (4-byte aligned, strides positive). */
typedef struct gemm_kv_weights {
    float *data;
    int64_t page_stride, head_stride;
} gemm_kv_weights;

/* Adds the attention weight that the batch's new tokens give to each of their sequence's own keys:
 *   w[j][h'] = decay * w[j][h'] + sum over tokens t, query heads h of h' of exp(scale * q[t][h] . K[j][h'] - lse[t][h])
 * over the last `window` new tokens (0: all) that see key j (the order of gemm_serving.h); a sequence
 * without new tokens keeps its weights. lse is
 * what gemm_paged_attention left for the same q and scale. The rows of the new tokens' own keys start
 * from 0, whatever they held; with decay 0 all do. FP32 scores and sums, in a fixed order (the same
 * bits each time). A token whose lse is -inf gives nothing. decay from 0 to 1. cache->v is not
 * read and may be NULL; the keys of a prefix get no weights, and num_prefix_pages is not read. Rows past a sequence's
 * last key are left as they are. No two sequences may share a page. One kernel launch. */
int gemm_kv_weigh(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_batch *batch, const gemm_heads *q, float scale,
                  const float *lse, int64_t lse_stride, int64_t window, float decay, const gemm_kv_weights *weights,
                  void *stream);

/* Chooses, for each sequence and key head, the min(kv_lens[s], keep) keys to keep: the first `first`,
 * the last `recent`, and of those between the ones of largest weight (of equal weights the lower
 * index; NaN is below all others). index[s * seq_stride + h * head_stride + i], i < keep (device,
 * int32), gets their indexes in ascending order, -1 past the last; counts[s] their number. first +
 * recent <= keep. kv_heads, page_size (a power of two from 16 to 1024) and num_pages are the weights'. Weights of a bad page
 * number count as 0. keep = 0 gives counts of 0. One kernel launch. */
int gemm_kv_select(gemm_ctx *ctx, const gemm_kv_seqs *seqs, int64_t num_pages, int64_t page_size, int64_t kv_heads,
                   const gemm_kv_weights *weights, int64_t keep, int64_t first, int64_t recent, int32_t *index,
                   int64_t seq_stride, int64_t head_stride, int32_t *counts, void *stream);

/* Moves rows of the cache up, in place: for each sequence and key head the key and value (and, if
 * weights is not NULL, the weight) of row start[s] + index[s][h][j] go to row start[s] + j, for
 * j < counts[s]. index as above (seq_stride and head_stride in elements; head_stride 0: one list for
 * all heads) with room for `most` entries each; start NULL: 0. Indexes are relative to start, and
 * index[j] >= j, which every ascending list meets (an entry that does not, or that leads to kv_lens[s] or past it:
 * GEMM_ERR_INDEX, not moved). counts[s] outside [0, most] is limited to it (GEMM_ERR_INDEX).
 * new_lens[s] (may be NULL; may be neither kv_lens nor another array that is read) gets start[s] + counts[s]. Rows from
 * there on are left as they are. No two sequences may share a page that is written. One kernel launch. */
int gemm_kv_compact(gemm_ctx *ctx, const gemm_kv_cache *cache, const gemm_kv_seqs *seqs, const gemm_kv_weights *weights,
                    const int32_t *index, int64_t seq_stride, int64_t head_stride, int64_t most, const int32_t *start,
                    const int32_t *counts, int32_t *new_lens, void *stream);

/* ---- products with 4-bit weights ------------------------------------------------------------ */

/* The weights W of a layer with N outputs and K inputs, in groups of `group` (32, 64 or 128)
 * consecutive inputs of one output:
 *   W[n][k] = (code[n][k] - zero[n][k / group]) * scale[n][k / group]
 *   codes: N rows of K / 2 bytes, input k in byte k / 2, even k in the low half (16-byte aligned);
 *   scales: N rows of K / group values of the call's type (2-byte aligned);
 *   zeros: N rows of K / group bytes, of which the low four bits count; NULL: 8 everywhere. */
typedef struct gemm_w4 {
    const uint8_t *codes;
    const void *scales;
    const uint8_t *zeros;
    int64_t group;
} gemm_w4;

/* C[M][N] = act(A[M][K] W^T + bias[N]): gemm_run's product and epilogues (GEMM_EPI_SOFTMAX excepted)
 * for few rows, which its time is the reading of W for. Any M up to 2^18 (0: nothing to do); it is
 * made for M up to 64. N a multiple of 8, K of the group, both up to 2^24 (K = 0: act(bias)). A and C have rows of lda and
 * ldc elements (multiples of 8, at least K and N), all pointers 16-byte aligned (scales 2, zeros 1). dtype: type of A, scales,
 * bias and C. No weight is rounded: codes enter the products exactly, each group is summed in FP32 before its scale is
 * applied, and the result is rounded once. (Up to eight rows, code A and zero A are summed apart where the |A| are below 2^113, so
 * that FP32's errors are relative to 15 scale |A| - BF16: 143 - not to |W| |A|.) C may not overlap any other operand. One
 * kernel launch. Finite A and scales of any size: what leaves FP32's range is a scaled group's sum, or a sum of these, that does. (FP32's
 * smallest step, 2^-149, may be one of 2^-137 for each group in BF16.) */
int gemm_w4_run(gemm_ctx *ctx, int dtype, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const gemm_w4 *w,
                const void *bias, void *C, int64_t ldc, int epilogue, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_GEMM_DECODE_H */
