/*
 * moe_fp8.h -- C ABI of linear layers in 8-bit floating point, for the
 * projections and the output head around the Mixture-of-Experts layer of
 * moe.h.  Conventions as in moe.h and moe_block.h.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Linear layers in 8-bit floating point -------------------------------------
 * out[t][n] = sum_b xs[t][b] ws[n / 128][b] sum_{k in block b} xq[t][k] w[n][k]
 * with blocks b of 128 inputs (the last one may be short):
 *   w:   e4m3 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits; no
 *        infinities), one float scale ws per 128 outputs x 128 inputs;
 *   x:   quantised by the call: per row and block the smallest power of two
 *        xs >= 2^-126 with max |x| <= 448 xs (1 for a block of zeros), and
 *        xq = x / xs rounded to the nearest e4m3 value, ties to even.  A
 *        power of two keeps that division and the product with xs exact.
 * The products run on the tensor cores (tcgen05, 8-bit operands, fp32
 * accumulators in tensor memory over one block of 128 inputs); the blocks are
 * scaled by xs ws, one fp32 product (so that it should not leave fp32's normal
 * range, as it may for inputs below 1e-35 with weight scales below 1), and summed
 * in fp32 registers, in an order that depends on the shapes only.  A row of x that holds a NaN or an infinity gives NaN in all
 * of its outputs. */
typedef struct moe_fp8 moe_fp8;

/* Handle of one weight matrix: pointers, shapes and the tiled-load descriptor.
 *   n, k:     outputs and inputs, n in [1, 2^24], k in [1, 65536].
 *   codes:    device uint8 [n][ld_codes], 16-byte aligned, ld_codes >= k a
 *             multiple of 16; bytes past k in a row are not used.
 *   scales:   device float [ceil(n/128)][ceil(k/128)].
 * Both stay the caller's and must outlive the handle.  Requires an sm_103
 * device; no device work. */
int moe_fp8_open(int32_t n, int32_t k, const uint8_t *codes, int64_t ld_codes, const float *scales, moe_fp8 **out);

/* Frees the handle (host memory only).  NULL is accepted. */
void moe_fp8_close(moe_fp8 *w);

/* Bytes of device workspace that calls with up to max_rows rows need (0 on a
 * bad handle or size).  One workspace must not be used by two calls that
 * overlap on the GPU; it may serve several handles in turn. */
size_t moe_fp8_workspace_bytes(const moe_fp8 *w, int32_t max_rows);

/* Zero-fills the workspace's control words on `stream`; required once before
 * its first use. */
int moe_fp8_workspace_init(const moe_fp8 *w, void *workspace, size_t workspace_bytes, void *stream);

/* out = x w^T for `rows` rows (0: no work).  x: device [rows][ld_x] of type
 * x_type; out: device [rows][ld_out] of type out_type, rounded once from fp32.
 * workspace: 256-byte aligned, moe_fp8_workspace_bytes(w, rows) bytes. */
int moe_fp8_linear(moe_fp8 *w, const void *x, int32_t x_type, int64_t ld_x, int32_t rows, void *out,
                   int32_t out_type, int64_t ld_out, void *workspace, size_t workspace_bytes, void *stream);

/* Synchronises `stream` and reads the error word that device code latches in
 * the workspace: MOE_OK or MOE_ERR_TIMEOUT (a bounded wait ran out; outputs of
 * the calls since the last check are undefined).  Clears it after an error. */
int moe_fp8_check(const moe_fp8 *w, void *workspace, void *stream);

/* Quantises weights: device [n][ld_w] of type w_type to codes and scales as
 * moe_fp8_open takes them, scale = max |w| / 448 of each 128 x 128 block (1
 * for a block of zeros, or of values so small that this quotient is 0: their
 * codes are 0), rounded to nearest, ties to even.  Bytes past k in a row of
 * codes are set to 0.  NaNs and infinities are outside the contract. */
int moe_fp8_quantize_weights(const void *weights, int32_t w_type, int64_t ld_w, int32_t n, int32_t k,
                             uint8_t *codes, int64_t ld_codes, float *scales, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_H */
