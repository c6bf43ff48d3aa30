/*
 * moe_layer.h -- C ABI of the operators around the routed experts in a decoder
 * layer, for GB300 (sm_103a), in the same library as moe_nvfp4.h:
 *
 *   moe_norm        residual addition and root-mean-square norm, output in
 *                   bf16 and / or in 8 bits with block scales
 *   moe_linear      matrix-vector products with NVFP4 weights (the experts'
 *                   format): dense projections and router logits
 *   moe_kv_append   rotation of queries and keys, and the append of keys and
 *                   values to a paged cache held in 8 bits
 *   moe_kv_attend   causal attention over that cache
 *
 * The conventions are those of moe_nvfp4.h: *_dev pointers are device pointers
 * on the current device that the caller owns, `stream` is a cudaStream_t (NULL:
 * the legacy default stream), work is enqueued asynchronously, a status other
 * than MOE_OK leaves nothing enqueued (moe_last_error has the message), nothing
 * is allocated on the device, and there is no other path: an argument the
 * sm_103a kernels do not take is an error.  Every kernel here waits for the
 * work queued before it on the stream before it reads or writes anything, and
 * gives the same bits from run to run.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- moe_norm
 * For each of T rows of H elements:
 *   s = x + r            (fp32; s = x without a residual)
 *   r_out = bf16(s)
 *   y = s / sqrt(mean(s^2) + eps) * w            (fp32, from the unrounded s)
 *   y_dev = bf16(y)
 *   q_dev = E4M3(y / sc), sc = the smallest power of two (at least 2^-64) with
 *           |y| <= 448 sc over the 128 columns of a block; q_scale_dev = sc
 * The power of two keeps E4M3's own rounding the only one of the 8-bit output.
 *   x_dev     bf16 [T, H] (x_f32 = 0) or float (1), rows x_stride elements apart
 *   r_dev     bf16 [T, H] contiguous, or NULL: no residual
 *   r_out_dev bf16 [T, H], may be r_dev itself, or NULL: s is not kept
 *   w_dev     bf16 [H]
 *   y_dev     bf16 [T, H] or NULL; q_dev uint8 [T, H] with q_scale_dev float
 *             [T, H/128], or both NULL; one of the two outputs at least
 *   T >= 0 (0: a no-op); H a multiple of 8 up to 16384, and of 128 with q_dev
 * All pointers 16-byte aligned (q_scale_dev 4-byte), x_stride >= H and a
 * multiple of 8 (bf16) or 4 (float).  A sum of squares past fp32's range gives
 * a row of zeros (s beyond about 1e17); a NaN or infinity in a row gives
 * NaN in it (E4M3's NaN code in q; its block scale then counts finite elements). */
moe_status_t moe_norm(const void *x_dev, int x_f32, int64_t x_stride, const void *r_dev, void *r_out_dev,
                      const void *w_dev, float eps, void *y_dev, uint8_t *q_dev, float *q_scale_dev, int T, int H,
                      void *stream);

/* -------------------------------------------------------------- moe_linear
 *   y[t, n] = ts[n] * sum_k E2M1(q[n, k]) * E4M3(s[n, k/16]) * x[t, k]
 * with NVFP4 weights laid out as an expert's projection in moe_plan_desc, and
 * a tensor scale for each row (fused projections keep theirs).  The weights
 * are used exactly; x enters as fp16 after a power-of-two prescale of its row or
 * of each 128 of it: exact for elements down to 2^-28 of the largest there, what
 * is smaller off by at most 2^-38 of that largest; sums in fp32.  Weight block scales may have
 * their sign set; a NaN code gives NaN.
 *   q_dev uint8 [N, K/2], s_dev uint8 [N, K/16], ts_dev float [N]
 *   x_dev bf16 [T, K], rows x_stride elements apart
 *   y_dev float [T, N] (y_bf16 = 0) or bf16 (1), contiguous, fully written
 *   N >= 1, K a multiple of 32 up to 2^22, T >= 0 (0: a no-op).  Meant for decode
 *   batches: up to 24 tokens read the weights once; more run in groups of 24 (of
 *   32 where the weights have many rows, K is a multiple of 256 and s_dev 16-byte
 *   aligned), each reading them again (from L2 as far as they fit).
 *   Which kernel runs, and so the order of the sums, depends on T too: the same token
 *   can have other last bits in a batch of another size.
 *   A device-side wait that ran out (bounded as in moe_nvfp4.h) leaves NaN in the
 *   outputs of its block's rows: this call has no workspace to flag it in.
 * q_dev and x_dev 16-byte aligned, s_dev 2-byte, ts_dev 4-byte, y_dev to its
 * element; x_stride >= K and a multiple of 8. */
moe_status_t moe_linear(const uint8_t *q_dev, const uint8_t *s_dev, const float *ts_dev, int N, int K,
                        const void *x_dev, int64_t x_stride, void *y_dev, int y_bf16, int T, void *stream);

/* ---------------------------------------------------- the paged 8-bit cache
 * A pool of n_pages pages of MOE_KV_PAGE tokens.  For each page and kv head:
 *   k  uint8 [MOE_KV_PAGE, head_dim]   E4M3 codes, token after token
 *   v  uint8 [head_dim, MOE_KV_PAGE]   E4M3 codes, transposed: a row of the
 *                                      attention's second product is contiguous
 *   one float scale of k and one of v: value = E4M3(code) * scale
 * Sequence b's token t lies in page pages[b, t / MOE_KV_PAGE].  moe_kv_append
 * writes scales that are powers of two, so that raising one (a later token of
 * the page is larger) shifts the codes already there without rounding them
 * again, as far as E4M3's exponent reaches.  moe_kv_attend takes any scales from
 * 2^-64 to 2^60.  v must hold no NaN code (0x7F, 0xFF) anywhere in a page that is read,
 * unused slots included: zero a new pool once; moe_kv_append writes none. */
#define MOE_KV_PAGE 64
#define MOE_KV_MAX_SEQS 512

typedef struct moe_kv *moe_kv_t;

typedef struct {
    int n_pages;         /* >= 1                                                    */
    int q_heads;         /* a multiple of kv_heads; query heads g * (q_heads /      */
    int kv_heads;        /*   kv_heads) .. share kv head g                          */
    int head_dim;        /* 64 or 128                                               */
    uint8_t *k_dev;      /* [n_pages, kv_heads, MOE_KV_PAGE, head_dim]              */
    uint8_t *v_dev;      /* [n_pages, kv_heads, head_dim, MOE_KV_PAGE]              */
    float *k_scale_dev;  /* [n_pages, kv_heads]                                     */
    float *v_scale_dev;  /* [n_pages, kv_heads]                                     */
    /* Rotation: of the first rot_dim elements of a head (even, 0 .. head_dim; 0:
     * none), pair j of rot_dim / 2 turns by the angle whose cosine and sine are
     * rope[position, 2j], rope[position, 2j + 1].  Pairs are elements (2j, 2j + 1)
     * with rot_interleaved, else (j, j + rot_dim / 2).  Any scaling for long
     * contexts (of frequencies or of magnitudes) is in the table. */
    int rot_dim, rot_interleaved, rope_positions;
    const float *rope_dev; /* [rope_positions, rot_dim], 8-byte aligned             */
    int device;          /* CUDA device of the pointers; -1: the current device     */
} moe_kv_desc;

/* The sequences of one step.  Sequence b has the new tokens q_off[b] ..
 * q_off[b + 1] - 1 of the step's N, and holds kv_len[b] tokens with them: new
 * token i of n is at position kv_len[b] - n + i. */
typedef struct {
    const int32_t *q_off_dev;  /* [B + 1], non-decreasing, q_off[0] >= 0, q_off[B] <= N */
    const int32_t *kv_len_dev; /* [B], 0 .. max_pages * MOE_KV_PAGE                     */
    const int32_t *pages_dev;  /* [B, max_pages]                                        */
    int max_pages;             /* >= 1                                                  */
    int B;                     /* 0 .. MOE_KV_MAX_SEQS                                  */
    int N;                     /* new tokens in all, >= 0                               */
    int max_q;                 /* largest number of new tokens of a sequence, 0 .. N:   */
                               /*   chooses tiles and grid (a smaller value than the   */
                               /*   true one costs time, not correctness)              */
} moe_kv_batch;

/* Check the description and keep it (host memory; no device work).  k_dev and
 * v_dev 16-byte aligned, the float arrays 4-byte (rope_dev 8). */
moe_status_t moe_kv_create(const moe_kv_desc *desc, moe_kv_t *out);
void moe_kv_destroy(moe_kv_t kv);

/* Workspace for moe_kv_append and moe_kv_attend (fixed per handle): zeroed once
 * by moe_kv_workspace_init, 256-byte aligned, one per stream that runs them
 * concurrently.  Launches on one workspace from two streams are ordered as
 * those of moe_nvfp4.h are. */
size_t moe_kv_workspace_bytes(moe_kv_t kv);
moe_status_t moe_kv_workspace_init(moe_kv_t kv, void *ws_dev, size_t bytes, void *stream);

/* Rotate and append.  q [N, q_heads, head_dim], k and v [N, kv_heads, head_dim]
 * in bf16, head_dim and heads contiguous, tokens q_stride, k_stride and
 * v_stride elements apart (slices of one projection's output): 16-byte aligned
 * pointers, strides multiples of 8 and at least a token's elements.
 *   q_out  bf16 [N, q_heads, head_dim] contiguous: the rotated queries, may be q
 *          itself where that is contiguous too (q and q_out both NULL: keys and
 *          values only)
 * Rotations are in fp32 (each product and sum rounded); keys are quantised from
 * there.  In each page and head that gets new tokens the scale is the smallest
 * power of two (2^-64 .. 2^60) with |values| <= 448 scale over the new ones,
 * and where the page's first new token is not its slot 0, no smaller than
 * the scale already there; if that grows the page's other codes are requantised
 * (nearest, ties to even).  A token whose key or value in a head holds a NaN, an
 * infinity or a magnitude above 448 * 2^60 is kept out of the scales: its key
 * codes are NaN, its value codes 0, so that outputs that attend to it are NaN
 * and others are untouched.
 * Appending the same tokens again leaves the cache as it is.
 * Tokens whose page id or position is out of range are dropped, with the other
 * new tokens of that page (their rows of q_out are 0), and flagged for
 * moe_kv_check. */
moe_status_t moe_kv_append(moe_kv_t kv, const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                           const void *v_dev, int64_t v_stride, void *q_out_dev, const moe_kv_batch *batch,
                           void *ws_dev, void *stream);

/* Attention of the step's queries over the cache:
 *   o[i, h] = softmax_t(scale * q[i, h] . k[t, g]) . v[t, g],   t = 0 .. position of i
 * q bf16 [N, q_heads, head_dim] (tokens q_stride elements apart, 16-byte
 * aligned, stride a multiple of 8); o bf16 [N, q_heads, head_dim] contiguous, 16-byte aligned.
 * A query that sees no token (kv_len[b] smaller than its new tokens) gets 0.
 * Rows of o outside every sequence are not written.  Products use the 8-bit
 * codes' exact values.  With up to 16 rows (a sequence's new tokens x query heads
 * of a kv head) q enters as fp16 (exact for elements down to 2^-28 of the row's
 * largest), with more as the sum of two E4M3 digits (exact for elements down to 2^-9
 * of it, smaller ones off by at most 2^-17 of it);
 * softmax weights are rounded to fp16 (2^-11 of each, or 2^-30 of the row's largest weight x
 * scale of v if more); sums, maxima and the softmax in fp32, where the additions of
 * the second product cut instead of rounding: values of one sign lose up to 2^-12 of
 * their sum with more than 16 rows, 2^-30 a token (of those that one block adds up)
 * with up to 16.  A page id out of range counts
 * as tokens that nothing sees and is flagged for moe_kv_check. */
moe_status_t moe_kv_attend(moe_kv_t kv, const void *q_dev, int64_t q_stride, float scale, void *o_dev,
                           const moe_kv_batch *batch, void *ws_dev, void *stream);

/* Synchronise `stream`, read and clear the workspace's error word: MOE_OK,
 * MOE_ERR_TIMEOUT (initialise the workspace again), MOE_ERR_BAD_INDEX, or
 * MOE_ERR_CUDA. */
moe_status_t moe_kv_check(moe_kv_t kv, void *ws_dev, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
