/*
 * moe_speculate.h -- C ABI of the operators that turn logits into tokens and move the
 * paged 8-bit cache of moe_layer.h between sequences, for GB300 (sm_103a), in the same
 * library: speculative decoding with trees of drafted tokens, and several samples or
 * beams of a prompt.
 *
 *   moe_kv_append_tree  the append of a tree of new tokens to each sequence
 *   moe_kv_attend_tree  the attention of such tokens: each sees the tokens before the
 *                       tree, the way to its root, and itself
 *   moe_kv_compact      keeps the accepted ones of a sequence's newest tokens
 *   moe_kv_fork         makes sequences that go on from others
 *   moe_sample          samples a token from each row of logits, by given random numbers
 *
 * The conventions are those of moe_layer.h.
 */
#ifndef MOE_SPECULATE_H
#define MOE_SPECULATE_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------- trees of new tokens
 * In these two calls the new tokens of each sequence of the batch are a tree (or
 * several): parent_dev[q_off[b] + i], an int32 for each of the step's N, is the token
 * before new token i, counted inside the sequence's new tokens, or -1 where i follows
 * the tokens before the tree.  A parent comes before its children: one outside
 * [-1, i) counts as -1 and is flagged for moe_kv_check where it is met.  New token i is
 * stored at position kv_len[b] - n + i as in moe_kv_append, whatever its parent.
 * A sequence has at most MOE_KV_MAX_TREE new tokens: batch->max_q above that is
 * refused, a longer sequence is flagged and treated as one whose length is out of
 * range.  A chain (parent i - 1) gives what moe_kv_append and moe_kv_attend give. */
#define MOE_KV_MAX_TREE 256

/* moe_kv_append, but a token turns by the angle of position kv_len[b] - n + its
 * depth (0 at a root).  The position that it is stored at has to be inside the table
 * too. */
moe_status_t moe_kv_append_tree(moe_kv_t kv, const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                                const void *v_dev, int64_t v_stride, void *q_out_dev, const moe_kv_batch *batch,
                                const int32_t *parent_dev, void *ws_dev, void *stream);

/* moe_kv_attend, but token i sees the kv_len[b] - n tokens before the tree and, of the
 * tree, itself, its parent, that one's parent and so on. */
moe_status_t moe_kv_attend_tree(moe_kv_t kv, const void *q_dev, int64_t q_stride, float scale, void *o_dev,
                                const moe_kv_batch *batch, const int32_t *parent_dev, void *ws_dev, void *stream);

/* Keep n_keep[b] of the n newest tokens of each sequence: of the tokens at
 * kv_len[b] - n + i, those with i = keep[b, 0] < keep[b, 1] < ..., which move to
 * kv_len[b] - n, kv_len[b] - n + 1, ...; kv_len_out[b] = kv_len[b] - n + n_keep[b].
 *   keep_dev       int32 [B, max_keep], entries behind n_keep[b] are not read
 *   n_keep_dev     int32 [B], 0 .. min(n, max_keep)
 *   kv_len_out_dev int32 [B], apart from batch->kv_len_dev
 * n = q_off[b + 1] - q_off[b] as in the step that appended them (batch->N only bounds
 * the offsets, batch->max_q is not used), at most MOE_KV_MAX_TREE.  The codes stay what
 * they are where the scale does: a page that receives tokens gets the largest of
 * its own scale (if it keeps tokens of its own) and theirs; codes whose scale was
 * smaller are requantised (nearest, ties to even; exact for scales that are powers of
 * two as far as E4M3's exponent reaches), the page's other codes as well.  Slots behind the kept tokens
 * hold anything (no NaN code in v that was not there).  A sequence whose entries are
 * out of range or not ascending, whose length is out of range, or where the id of a page is that a
 * kept token comes from or goes to, is left as it is, kv_len_out[b] = kv_len[b], and flagged for moe_kv_check. */
moe_status_t moe_kv_compact(moe_kv_t kv, const int32_t *keep_dev, const int32_t *n_keep_dev, int max_keep,
                            int32_t *kv_len_out_dev, const moe_kv_batch *batch, void *ws_dev, void *stream);

/* C sequences that go on from some of B: child c has sequence src[c]'s tokens,
 *   pages_out[c, :] = pages[src[c], :],  kv_len_out[c] = kv_len[src[c]],
 * and where fresh[c] >= 0 that page in the place of the one that the next token
 * goes to (page kv_len / MOE_KV_PAGE of the sequence), with a copy of its codes and scales
 * if it holds tokens; fresh[c] < 0 leaves the sequence's own page there, for one
 * child at most (another that is left a partly filled one is flagged; a next page that holds no
 * tokens yet is the caller's to give before they append).  The full pages are shared.
 *   src_dev, fresh_dev int32 [C]; kv_len_dev int32 [B]; pages_dev int32 [B, max_pages]
 *   kv_len_out_dev int32 [C], pages_out_dev int32 [C, max_pages], apart from the inputs
 * B and C 0 .. MOE_KV_MAX_SEQS (C = 0: a no-op).  A fresh page is in no sequence's table; it is not
 * used where the sequence fills its table.  A child whose src or length is out of
 * range, whose fresh page is not a page or an earlier child's too, that is left a partly filled page
 * as an earlier child is, or whose page to copy is out of range, gets -1 in all of pages_out[c, :] and
 * length 0, and is flagged for moe_kv_check. */
moe_status_t moe_kv_fork(moe_kv_t kv, const int32_t *src_dev, const int32_t *fresh_dev, int C, const int32_t *kv_len_dev,
                         const int32_t *pages_dev, int max_pages, int B, int32_t *kv_len_out_dev, int32_t *pages_out_dev,
                         void *ws_dev, void *stream);

/* --------------------------------------------------------------- moe_sample
 * A token for each of T rows of V logits.  The tokens of a row are ranked by their
 * logits, the largest first, equal ones by index; with w_i = exp((l_i - max) / t),
 *   - min-p leaves the tokens with w_i >= min_p,
 *   - top-k the first k of them,
 *   - top-p of these the fewest first ones whose weights add up to top_p of all of
 *     theirs or more (one at least),
 * and the token is the first one, in rank, at which the weights add up to more than
 * u times the sum of all that are left.  prob is its weight over that sum.
 *   logits_dev float [T, V] (bf16 = 0) or bf16 (1), rows `stride` elements apart
 *   u_dev      float [T], random numbers in [0, 1)
 *   each setting: an array of T values on the device, or, where that is NULL, one for
 *   all rows.  temperature 1e-6 or less (or NaN): the token of rank 0; top_k <= 0: no
 *   limit; top_p >= 1 (or NaN): no limit, <= 0: rank 0 alone; min_p <= 0 (or NaN): no
 *   limit, >= 1: the tokens whose logit is the largest.
 *   token_dev  int32 [T]; prob_dev float [T] or NULL; apart from the inputs and each other
 * NaN counts as -infinity, and so as a token of weight 0, which is never given.  Where
 * the largest logit is +infinity the tokens at +infinity weigh 1, all others 0; a token whose
 * distance to the largest overflows fp32 weighs 0 (at temperatures above 1e36 too).  A row
 * of nothing but -infinity gives token -1 and prob 0.  u below 0 or NaN counts as 0, u of 1 and
 * above gives the last token that is left and weighs half of 2^-45 or more.
 * Weights are whole numbers of units of 2^-45 (the largest weighs 1), which are summed the
 * same in any order.  A weight is off by half a unit and 2^-36 of itself, one of less than
 * 2^-16 by a unit at most; a sum over n tokens so by n units and 2^-36 of itself: 2^-27 at the
 * worst, far less where errors of both signs meet.  What is decided on a border (min-p's, top-p's, the
 * token's) differs from the formula's only where the sums come nearer to it than that.  A
 * token of less than half a unit is never given, but counts in the sums that borders are
 * parts of (from 2^-63.5 down it weighs nothing).
 * T >= 0 (0: a no-op), 1 <= V <= MOE_SAMPLE_MAX_VOCAB, stride >= V; pointers to their
 * elements' alignment. */
#define MOE_SAMPLE_MAX_VOCAB 262144

typedef struct {
    const void *logits_dev;
    int64_t stride;
    int bf16;
    int T, V;
    const float *u_dev;
    const float *temperature_dev;
    float temperature;
    const int32_t *top_k_dev;
    int top_k;
    const float *top_p_dev;
    float top_p;
    const float *min_p_dev;
    float min_p;
    int32_t *token_dev;
    float *prob_dev;
} moe_sample_desc;

moe_status_t moe_sample(const moe_sample_desc *desc, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_SPECULATE_H */
