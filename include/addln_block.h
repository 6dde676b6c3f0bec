/*
 * addln_block.h - the boundary between two blocks of a transformer, fused:
 * the norm of a block's output, its gate and scales, the residual sum, and
 * the norm before the next block; forward and backward.  Exported by the
 * same library as addln.h, whose conventions (device pointers, contiguous
 * row-major tensors, streams, return codes, no allocation) hold here too.
 * The residual sum and norm are those of add_layernorm_fwd ("算子融合的收益量化"
 * section 1, "算子融合与Kernel合并" 4.2), widened by what later models put
 * around them; the pages have no counterpart of the rest.
 *
 * Per row i, columns j:
 *     n = post(f)                    f, normalised with post_gamma, post_beta
 *     h = residual_scale x + block_scale (gate n)
 *     y = pre(h)                     h, normalised with pre_gamma, pre_beta
 * where a norm is, of a row v,
 *     ADDLN_NORM_NONE   v itself (post), or no y at all (pre)
 *     ADDLN_NORM_RMS    v rstd gamma (+ beta),  rstd = 1 / sqrt(mean(v^2) + eps)
 *     ADDLN_NORM_LAYER  (v - mean) rstd gamma (+ beta),
 *                       rstd = 1 / sqrt(mean((v - mean)^2) + eps)
 * and the gate is
 *     ADDLN_GATE_NONE     1
 *     ADDLN_GATE_CHANNEL  fp32 [H], one value a column (a learnt layer scale)
 *     ADDLN_GATE_ROWS     rows in the I/O dtype; row i takes gate row
 *                         i / rows_per_gate (1: a gate of its own for every
 *                         row; the sequence length: one for each sequence),
 *                         gate row k starting gate_stride elements after row
 *                         k - 1
 *
 * Arithmetic is fp32; h and y are rounded to the I/O dtype to nearest-even,
 * and y is taken of the unrounded h.  gamma, beta and the statistics are
 * fp32.  H as in addln_max_hidden.
 */
#ifndef ADDLN_BLOCK_H
#define ADDLN_BLOCK_H

#include "addln.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ADDLN_NORM_NONE 0
#define ADDLN_NORM_RMS 1
#define ADDLN_NORM_LAYER 2

#define ADDLN_GATE_NONE 0
#define ADDLN_GATE_CHANNEL 1
#define ADDLN_GATE_ROWS 2

#define ADDLN_ERR_ALIGN (-12) /* a pointer is not a multiple of its element's size */
#define ADDLN_ERR_KIND (-13)  /* unknown norm or gate kind, or arguments that contradict the kind */
#define ADDLN_ERR_SCALE (-14) /* a scale or limit that is NaN, infinite or out of its range */
#define ADDLN_ERR_HOST_MEMORY (-15) /* the host's memory ran out inside the call */

/*
 * Forward.
 *   f, x        [rows, H] the block's output and the residual stream (required)
 *   post_gamma  [H] (required with a post norm); post_beta [H] or NULL
 *   gate        as gate_kind says; gate_stride >= H and rows_per_gate >= 1
 *               are read for ADDLN_GATE_ROWS alone, whose gate has
 *               ceil(rows / rows_per_gate) rows
 *   pre_gamma   [H] (required with a pre norm); pre_beta [H] or NULL
 *   h           [rows, H] the new residual stream (required)
 *   y           [rows, H] required with a pre norm, NULL without
 *   post_mean, post_rstd, pre_mean, pre_rstd
 *               [rows] statistics for the backward, each NULL-able; the means
 *               are written for layer norms alone
 *   eps         >= 0, for both norms.  With eps = 0 a row whose mean square
 *               (layer: variance) is 0 gives NaN, the 0 * inf of the formula
 * A row whose sum of squares (layer: of squared deviations) passes fp32 has
 * 1 / sqrt = 0 and so y = beta; one with infinities or NaN is NaN.
 * h and y may each be exactly f or x (in place), not the same one; any other
 * overlap of an output is ADDLN_ERR_ALIAS.  rows == 0 is a no-op.
 */
int block_norm_fwd(const void *f, const void *x, int post, const float *post_gamma,
                   const float *post_beta, const void *gate, int gate_kind, int64_t gate_stride,
                   int64_t rows_per_gate, float residual_scale, float block_scale, int pre,
                   const float *pre_gamma, const float *pre_beta, void *h, void *y,
                   float *post_mean, float *post_rstd, float *pre_mean, float *pre_rstd,
                   int64_t rows, int64_t H, float eps, int dtype, void *stream);

/*
 * Backward.  From dy (the gradient of y) and dh (what reaches h from
 * elsewhere: h is the residual stream), either of them NULL but not both:
 *     hhat = (h - pre_mean) pre_rstd,  u = dy pre_gamma
 *     D    = pre_rstd (u - mean(u) - hhat mean(u hhat)) + dh   (rms: no mean(u))
 *     dx   = residual_scale D
 *     dn   = block_scale D gate,  fhat = (f - post_mean) post_rstd
 *     v    = dn post_gamma
 *     df   = post_rstd (v - mean(v) - fhat mean(v fhat))  (none: df = dn)
 *     dpre_gamma = sum dy hhat, dpre_beta = sum dy,
 *     dpost_gamma = sum dn fhat, dpost_beta = sum dn, dgate = sum block_scale D n
 * the sums over all rows (dgate: over the rows that the gate row serves).
 *   f, h         [rows, H] f may be NULL without post norm and gate, h without dy
 *   statistics   as saved by the forward (required where they are used)
 *   df, dx       [rows, H] outputs (required); each may be dy, dh, f or h
 *                exactly, not the same one
 *   dpost_gamma, dpost_beta, dpre_gamma, dpre_beta
 *                [H] fp32 outputs, each NULL-able; NULL where the norm is none.
 *                Without dy, dpre_gamma and dpre_beta are zeros
 *   dgate        fp32 [H] (channel), or [ceil(rows / rows_per_gate), H] in the
 *                I/O dtype, contiguous (rows); NULL-able
 *   workspace    device scratch of at least block_norm_bwd_workspace_size()
 *                bytes, 16-byte aligned, the caller's; no two calls that may
 *                overlap on the GPU share one.  Its contents need no
 *                initialisation.
 * The sums run in a fixed order: the same call on the same GPU model gives
 * the same bits.  rows == 0 zero-fills the parameters' gradients.
 */
int block_norm_bwd(const void *dy, const void *dh, const void *f, const void *h, int post,
                   const float *post_gamma, const float *post_beta, const float *post_mean,
                   const float *post_rstd, const void *gate, int gate_kind, int64_t gate_stride,
                   int64_t rows_per_gate, float residual_scale, float block_scale, int pre,
                   const float *pre_gamma, const float *pre_mean, const float *pre_rstd, void *df,
                   void *dx, float *dpost_gamma, float *dpost_beta, void *dgate,
                   float *dpre_gamma, float *dpre_beta, int64_t rows, int64_t H, int dtype,
                   void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace block_norm_bwd needs on the current device for this many
 * rows or fewer, whatever the buffers' alignment (0 when rows == 0), or a
 * negative code. */
int64_t block_norm_bwd_workspace_size(int64_t rows, int64_t H, int dtype, int gate_kind,
                                      int64_t rows_per_gate);

#ifdef __cplusplus
}
#endif

#endif /* ADDLN_BLOCK_H */
