/*
 * moe_block.h -- C ABI of the operators around the Mixture-of-Experts layer of
 * moe.h: the block boundary (norms, gate and residual between one layer and
 * the next) and the log probabilities of tokens.
 *
 * Conventions as in moe.h: return MOE_OK or a negative MOE_ERR_* code with a
 * message in moe_last_error(); every buffer is the caller's; device work is
 * asynchronous on `stream` of the current device; arguments are checked on
 * the host before any launch.  Further:
 *   - Matrices are row-major; a leading dimension `ld_*` is the distance
 *     between rows in elements, at least the row's width.
 *   - Pointers are aligned to their element's size (MOE_ERR_ALIGN
 *     otherwise).  Rows that start on 16-byte boundaries are read fastest.
 *   - Output buffers overlap no input unless a call says so.
 *   - No call here allocates, synchronises or keeps anything from one call
 *     for the next, so each may be captured into a CUDA graph.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the operators' inputs and outputs. */
enum {
    MOE_BF16 = 0,
    MOE_F16 = 1,
    MOE_F32 = 2
};

/* ---- Block boundary ---------------------------------------------------------
 * Between one block and the next, per token (row) of `hidden` values:
 *     r  = y * rsqrt(mean(y^2) + eps) * (w_add + w_post)     post_norm = 1
 *     r  = y                                                 post_norm = 0
 *     h' = residual_scale * h + gate * r
 *     x  = h' * rsqrt(mean(h'^2) + eps) * (w_add + w_pre)    pre_norm = 1
 *     x  = h'                                                pre_norm = 0
 * All arithmetic is in 32 bits; h' and x are each rounded once, when they are
 * stored, so x is computed from the unrounded h'.
 *
 *   rows >= 0 (0: no work); hidden in [1, 16384].
 *   y:      the block's output, or NULL for none (r = 0, as in front of the
 *           first block: then x is the norm of residual_scale * h).
 *   h:      the residual stream, or NULL for none (h' = gate * r).  At least
 *           one of y and h is set.
 *   gate:   NULL for 1, else element (t, j) is at
 *           gate[t * ld_gate_row + j * ld_gate_col]: (0, 1) one value per
 *           channel, (1, 0) one per token, (ld, 1) one per token and channel.
 *           ld_gate_col is 0 or 1, ld_gate_row >= 0.
 *   w_post, w_pre: `hidden` weights of type w_type, or NULL for zeros (with
 *           w_add = 1: a norm without weights).
 *   w_add:  0, or 1 for weights stored as their distance from one.
 *   eps > 0.
 *   h_out:  h' in type h_type, or NULL.  May be h itself (with ld_h_out =
 *           ld_h).
 *   x_out:  x in type x_type, or NULL.  At least one of the two is set.
 *
 * Many rows are fastest, near the memory's rate, where y, h, h_out and x_out are
 * all set, with both norms, `hidden` a multiple of 8 from 264 to 8192, rows and
 * weights on 16-byte boundaries, and a gate per channel or none.  Any other form
 * takes up to about twice as long for its bytes, rows off 16-byte boundaries
 * or of a width that 8 does not divide three to four times. */
typedef struct moe_block_norm_args {
    const void *y, *h, *gate, *w_post, *w_pre;
    void *h_out, *x_out;
    int64_t ld_y, ld_h, ld_gate_row, ld_gate_col, ld_h_out, ld_x_out;
    int32_t rows, hidden;
    int32_t y_type, h_type, gate_type, w_type, x_type;
    int32_t post_norm, pre_norm;
    float w_add, eps, residual_scale;
} moe_block_norm_args;

int moe_block_norm(const moe_block_norm_args *args, void *stream);

/* ---- Log probabilities of tokens ---------------------------------------------
 * Per row of `vocab` logits l, with z = scale * l (scale = 1 / temperature):
 *     lse     = log sum_v exp(z_v)
 *     logprob = z_target - lse                     for each given token
 *     rank    = 1 + tokens before the target by (logit descending, id
 *               ascending)                         for each given token
 *     entropy = -sum_v p_v log p_v,  p = exp(z - lse), 0 log 0 = 0
 *     the top_n tokens by (logit descending, id ascending) with their
 *     log probabilities
 * in one pass over the logits, in 32 bits.  Where a row's largest z is 2^31 ln 2 or
 * more from 0, two different logits differ by 88 or more in z, and the row's
 * probability is that of its largest logits, in equal shares; such a row is read
 * a second time.
 *
 *   rows in [0, 2^27] (0: no work); vocab in [1, 2^24]; n_targets in [0, 8]; top_n in [0, 32].
 *   scale:   in [2^-64, 2^64].
 *   targets: device int32 [rows][n_targets].
 *   target_logprobs: device float [rows][n_targets]; target_ranks: device
 *            int32 [rows][n_targets]; lse, entropy: device float [rows];
 *            top_ids: device int32, top_logprobs: device float
 *            [rows][top_n].  Each may be NULL.
 *
 * A logit of -inf (or one whose z overflows to -inf) has probability 0: its
 * log probability is -inf and it is never listed among the top tokens; places
 * left over hold id -1 and -inf.  A row with no other logits gives lse -inf
 * and entropy 0.  A target outside [0, vocab) gives log probability -inf and
 * rank 0.  A row with a NaN or a z of +inf gives NaN for lse, entropy and the
 * log probabilities of its tokens; NaNs are never listed and come before no
 * target, and a target whose logit is NaN has rank 1. */
typedef struct moe_token_logprobs_args {
    const void *logits;
    const int32_t *targets;
    float *target_logprobs;
    int32_t *target_ranks;
    float *entropy, *lse;
    int32_t *top_ids;
    float *top_logprobs;
    int64_t ld_logits;
    int32_t rows, vocab;
    int32_t logits_type, n_targets, top_n;
    float scale;
} moe_token_logprobs_args;

int moe_token_logprobs(const moe_token_logprobs_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
