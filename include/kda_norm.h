/*
 * kda_norm.h - C ABI of the norms around a block, fused with its output gate,
 * residual scale and residual add.
 *
 * Per row of D channels, with N(x) = x / sqrt(mean_j x_j^2 + eps), a block's
 * output z, its gate g and the residual stream r:
 *     r' = r + res_scale * sigmoid(g) * N(z) * w_post      (after the block)
 *     y  = N(r') * w_pre                                   (before the next one)
 * Each part can be left out: without w_post z is added unnormalized, without
 * gate the sigmoid is 1, without z r' = r (the first norm of a model), without
 * y only r' is written (the last block). Every intermediate is fp32; y is the
 * norm of the fp32 sum r', also where resid_out rounds it to bf16. The gate is
 * read and applied as kda_epilogue's is. A row's sum of squares is fp32 too: past
 * 3.4e38 (D values of 1.8e19 / sqrt(D)) N is 0 in the row, or NaN with an infinity.
 * Squares below 1.2e-38 (values below 1.1e-19) lose bits and below 1e-45 are 0,
 * which shows only where eps is no larger: with eps = 0 a row of such values gives
 * infinities and one of zeros NaN.
 */
#ifndef KDA_NORM_H
#define KDA_NORM_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* KDA_NORM_RESID_BF16: resid and resid_out hold bf16 instead of float.
 * KDA_NORM_Y_BF16: y holds bf16 instead of float. Other bits are KDA_ERR_INVALID. */
enum kda_norm_flag { KDA_NORM_RESID_BF16 = 1, KDA_NORM_Y_BF16 = 2 };

/* Widest row. */
#define KDA_NORM_MAX_D 16384

/*
 * Row i of an array starts at base + i * stride (elements; stride >= D, else
 * KDA_ERR_INVALID).
 *   resid      float or bf16, required
 *   z          bf16, or NULL; with z resid_out is required, without it
 *              resid_out, w_post and gate must be NULL (KDA_ERR_INVALID)
 *   resid_out  as resid; may be resid itself with the same stride (in place)
 *   y          float or bf16, or NULL; y and w_pre come together
 *   w_post     float [D], or NULL: no norm of z
 *   gate       bf16, or NULL
 *   w_pre      float [D]
 * At least one of z and y is needed. No other output may overlap an input or an
 * output. Pointers need their element's alignment only (KDA_ERR_ALIGN), and so
 * do strides and D. res_scale must be finite, eps finite and >= 0
 * (KDA_ERR_INVALID); D in [1, KDA_NORM_MAX_D] (KDA_ERR_UNSUPPORTED past it).
 * rows == 0 enqueues nothing. Nothing is allocated; the kernel goes on `stream`.
 */
int kda_block_norm(const void *resid, int64_t resid_stride, const uint16_t *z, int64_t z_stride,
                   void *resid_out, int64_t resid_out_stride, void *y, int64_t y_stride,
                   const float *w_post, const uint16_t *gate, int64_t gate_stride, float res_scale,
                   const float *w_pre, float eps, int32_t rows, int32_t D, int32_t flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_NORM_H */
