/*
 * moe_cache.h -- C ABI of the paged key/value cache and of the attention that
 * reads it, for the layers around the Mixture-of-Experts layer of moe.h.
 * Conventions as in moe.h and moe_block.h.
 */
#ifndef MOE_CACHE_H
#define MOE_CACHE_H

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further element type, of caches only: e4m3 codes (sign, 4 exponent bits with
 * bias 7, 3 mantissa bits; no infinities) with one float scale per token and
 * head, a power of two (or NaN) as moe_cache_write makes it. */
enum {
    MOE_E4M3 = 3
};

/* ---- The cache of one layer -----------------------------------------------------
 * Keys and values of `n_pages` pages of `page_size` slots, a slot holding one
 * token: element d of head h in slot i of page p is at
 *     k[p * page_stride + i * slot_stride + h * head_stride + d]
 * (v alike), its scale, in a cache of type MOE_E4M3, at
 *     k_scale[p * scale_page_stride + i * scale_slot_stride + h * scale_head_stride].
 *   type:      MOE_BF16, MOE_F16 or MOE_E4M3.
 *   head_dim:  a multiple of 16 in [16, 256].
 *   kv_heads:  in [1, 1024]; page_size in [1, 2^20]; n_pages in [0, 2^31 - 1].
 *   strides:   in elements, >= 0; k and v 16-byte aligned, their strides
 *              multiples of 16 bytes.  Different slots lie in different places.
 * Slots whose heads, or heads whose slots, follow each other are read alike;
 * scales are read fastest where a head's slots follow each other. */
typedef struct moe_kv_cache {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, slot_stride, head_stride;
    int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
    int32_t type, n_pages, page_size, kv_heads, head_dim;
} moe_kv_cache;

/* ---- The sequences of a call -------------------------------------------------------
 * Sequence s has the n = starts[s + 1] - starts[s] rows from starts[s] on of
 * the call's tensors: tokens at the positions kv_lens[s] - n to kv_lens[s] - 1
 * of the sequence.  Position p lies in slot p % page_size of page
 * page_table[s * ld_table + p / page_size].
 *   starts:     device int32 [n_seqs + 1], 0 <= starts[0] <= starts[1] ... <= rows.
 *   kv_lens:    device int32 [n_seqs].
 *   page_table: device int32 [n_seqs][ld_table], `table_width` of each row in use.
 *   n_seqs:     in [0, 65536].
 *   rows:       rows of the call's tensors, in [0, 2^24].  Rows of no sequence
 *               are neither read nor written.
 *   max_rows:   the most rows of one sequence, or more: a hint that chooses
 *               between kernels.  They compute the same, with the roundings and
 *               the range of float16 values that moe_attention states for each.
 * All of it is read by the kernels only, so a captured call follows what the
 * buffers hold when it is replayed.  Device values outside the contract touch no
 * other memory: starts are taken as if cut to [0, rows] and kv_lens to
 * [0, table_width * page_size] (and to 2^30), and a page outside [0, n_pages) is one that
 * is missing. A missing page, or a position below 0, is not written, is read
 * as zeros, and is seen by no token.  Where starts, cut so, fall, moe_attention
 * writes nothing and moe_attention_check reports it; moe_cache_write and
 * moe_cache_read take a row as one of the sequences that it lies in, or of none. */
typedef struct moe_sequences {
    const int32_t *starts, *kv_lens, *page_table;
    int64_t ld_table;
    int32_t n_seqs, rows, max_rows, table_width;
} moe_sequences;

/* Writes the rows' keys and values into the cache, quantising them on the way:
 *   k, v:  device [rows][kv_heads][head_dim] of type `type` (MOE_BF16, MOE_F16
 *          or MOE_F32), rows ld_k and ld_v elements apart, heads following each
 *          other.
 * A 16-bit cache gets each value rounded to nearest even.  A cache of type
 * MOE_E4M3 gets, per token and head, the smallest power of two s >= 2^-126
 * with max |x| <= 448 s (1 for zeros) and the codes x / s rounded to nearest
 * even; a head that holds a NaN or an infinity gets a NaN scale and NaN codes.
 * No two rows of a call may share a slot.
 * Calls of rows * kv_heads * t > 2^31 - 256, where t is head_dim / 16 rounded up to
 * a power of two, are MOE_ERR_ARG, here and in moe_cache_read. */
int moe_cache_write(const moe_kv_cache *cache, const moe_sequences *seqs, const void *k, int64_t ld_k, const void *v,
                    int64_t ld_v, int32_t type, void *stream);

/* The reverse: the rows' keys and values from the cache, code * scale, rounded
 * once to `type`.  With starts that are the sums of kv_lens whole sequences are
 * read.  Arguments as above. */
int moe_cache_read(const moe_kv_cache *cache, const moe_sequences *seqs, void *k, int64_t ld_k, void *v, int64_t ld_v,
                   int32_t type, void *stream);

/* ---- Attention of new tokens over the cache -----------------------------------------
 * For row t of a sequence, at position a, and query head h, whose keys and
 * values are head h / (q_heads / kv_heads) of the cache:
 *     z_j   = scale * sum_d q[t][h][d] k_j[d]
 *     lse   = log sum_j exp(z_j)
 *     out_d = sum_j exp(z_j - lse) v_j[d]
 * over the positions j < kv_len that the row sees: j <= a if causal, j > a -
 * window if window > 0.  What it does not see has no part in its result,
 * whatever the cache holds there.  A row that sees nothing, or z of -inf only,
 * has out 0 and lse -inf; a NaN or a z of +inf among what it sees gives NaN.
 * The new tokens' own keys and values must be in the cache before (moe_cache_write
 * on the same stream).
 *
 *   q:      device [rows][q_heads][head_dim], 16-byte aligned, rows ld_q apart
 *           (a multiple of 8), heads following each other.
 *   out:    device, same shape and type, rows ld_out apart (likewise).
 *   lse:    device float [rows][q_heads], or NULL.
 *   q_type: the cache's type if that is MOE_BF16 or MOE_F16, either of the two
 *           for MOE_E4M3.
 *   q_heads: a multiple of kv_heads, at most 4096, and at most 128 for each of
 *           them; rows times query heads a key head is at most 2^30.
 *   scale:  > 0 and finite.   causal: 0 or 1.   window: >= 0, 0 for none.
 * Calls that might be 2^31 places of work are MOE_ERR_UNSUPPORTED:
 *     (rows * q_heads / kv_heads / R + n_seqs) * kv_heads * (positions / B + 4)
 * with R = 256 and B = 128 for heads of up to 128, R = 128 and B = 64 for larger ones, and
 * positions = table_width * page_size (at most 2^30).
 *
 * Products run on the tensor cores with fp32 sums; z, the sums of exponentials
 * and out are kept in fp32.  The exponentials are rounded to q_type for the second
 * product (few rows of an e4m3 cache: exponentials times the values' scales, to float16),
 * at most half a step each, so that a result moves by less than half a step of the
 * mean |v|.  float16 has no steps below 2^-39 (many rows: 2^-31) of a row's largest
 * exponential or, in few rows of an e4m3 cache, 2^-33 of its largest exponential times
 * scale; exponentials below 2^-126 of the largest are 0; sums need |v| times positions
 * below 2^118.  out is rounded once, when it is stored.  The order of sums goes by the
 * sequences, max_rows (as the kernel goes by it) and the GPU's number of SMs alone.
 * Few rows (max_rows times query heads a key head up to 16) take e4m3 values as they
 * are; more of them read them in q_type: exactly for MOE_BF16 (but below 2^-126), as float16
 * for MOE_F16, which is exact if the head's largest magnitude lies in [2^-7, 57344], and
 * infinite from 65520 on.  So float16 queries over an e4m3 cache of such magnitudes get
 * other results where some sequence has many rows: bf16 ones do not.
 *
 * Keys and values in pages of a multiple of 16 slots are read fastest; pages of
 * an odd number of slots, or of 2 or 4 times one, and 16-bit caches with a stride of 0 or
 * of 2^40 bytes or more, take about twice as long where many rows attend. */
typedef struct moe_attention_args {
    const void *q;
    void *out;
    float *lse;
    int64_t ld_q, ld_out;
    int32_t q_type, q_heads;
    int32_t causal, window;
    float scale;
} moe_attention_args;

/* Bytes of device workspace for calls with these heads (0 on a bad size) on
 * the current device.  One workspace must not be used by two calls that overlap
 * on the GPU; it may serve any number of caches in turn. */
size_t moe_attention_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim);

/* Zero-fills the workspace's control words on `stream`; required once before
 * its first use. */
int moe_attention_workspace_init(void *workspace, size_t workspace_bytes, void *stream);

/* workspace: 256-byte aligned, moe_attention_workspace_bytes(...) bytes. */
int moe_attention(const moe_attention_args *args, const moe_kv_cache *cache, const moe_sequences *seqs, void *workspace,
                  size_t workspace_bytes, void *stream);

/* Synchronises `stream` and reads the error word that device code latches in
 * the workspace: MOE_OK, MOE_ERR_TIMEOUT (a bounded wait ran out; outputs of
 * the calls since the last check are undefined) or MOE_ERR_ARG (the starts of a call
 * fell; it wrote nothing).  Clears it after an error. */
int moe_attention_check(void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_CACHE_H */
