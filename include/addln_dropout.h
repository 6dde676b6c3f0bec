/*
 * addln_dropout.h - dropout with a mask that is never stored, alone and at the
 * boundary between two blocks of a transformer (bias, dropout, residual sum,
 * norm), forward and backward.  Exported by the same library as addln.h and
 * addln_block.h, whose conventions (device pointers, contiguous row-major
 * tensors, streams, return codes, norm kinds, no allocation) hold here too.
 *
 * The mask is a function of a seed, an offset and an element's index in its
 * tensor, so that the backward, or any later call, makes the same one again:
 * Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", 2011) with
 *     key      the seed (64 bits, the low half first)
 *     counter  index / 8 (64 bits), then the offset (64 bits)
 * whose 128 bits serve 8 elements with 16 bits each, the lowest first.  With
 * t = p * 65536 rounded to the nearest whole number (ties to even), an element
 * is kept where its 16 bits are at least t, and multiplied by
 * 65536 / (65536 - t); a dropped one is 0, whatever it was (NaN and infinities
 * too).  So p is used to 16 bits, and the expectation is exact for the p that
 * is used: p below 2^-17 drops nothing, p above 1 - 2^-17 everything.
 * Masks of calls with different (seed, offset) are independent: use a new
 * offset for every call, the same one for its backward.
 *
 * Seed and offset are the arguments, or, where rng is not NULL, device memory:
 * rng[0] the seed and rng[1] the offset (8-byte aligned), read by the kernel
 * when it runs.  A captured graph is given rng, and advances it between
 * replays.
 */
#ifndef ADDLN_DROPOUT_H
#define ADDLN_DROPOUT_H

#include "addln_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * y = dropout(x) over n elements; the backward is the same call on the
 * gradient.  y may be exactly x.  p in [0, 1], else ADDLN_ERR_SCALE.
 */
int dropout_fwd(const void *x, void *y, int64_t n, double p, const int64_t *rng, uint64_t seed,
                uint64_t offset, int dtype, void *stream);

/*
 * Per row i, columns j:
 *     d = dropout(f + bias),  h = x + d,  y = norm(h)
 *   f          [rows, H] the block's output (required)
 *   x          [rows, H] the residual stream, or NULL: h = d
 *   bias       fp32 [H], or NULL
 *   norm       ADDLN_NORM_NONE, _RMS or _LAYER (addln_block.h), with gamma [H]
 *              (required) and beta [H] or NULL, fp32
 *   h          [rows, H], NULL-able with a norm (post-norm models that do not train)
 *   y          [rows, H] required with a norm, NULL without
 *   mean, rstd fp32 [rows] for the backward, each NULL-able; the mean is
 *              written for layer norms alone
 * Arithmetic is fp32; h and y are rounded once, y is taken of the unrounded h.
 * h and y may each be exactly f or x, not the same one; any other overlap of
 * an output is ADDLN_ERR_ALIAS.  eps as in block_norm_fwd.  rows == 0 is a
 * no-op.
 */
int dropout_add_norm_fwd(const void *f, const void *x, const float *bias, double p,
                         const int64_t *rng, uint64_t seed, uint64_t offset, int norm,
                         const float *gamma, const float *beta, void *h, void *y, float *mean,
                         float *rstd, int64_t rows, int64_t H, float eps, int dtype, void *stream);

/*
 * Backward.  From dy (the gradient of y; NULL without a norm, or where none
 * reaches y) and dh (what reaches h from elsewhere; NULL-able), not both NULL:
 *     hhat = (h - mean) rstd,  u = dy gamma
 *     D    = rstd (u - mean(u) - hhat mean(u hhat)) + dh   (rms: no mean(u))
 *     dx   = D,  df = dropout(D)   (kept and scaled as in the forward)
 *     dbias = sum df,  dgamma = sum dy hhat,  dbeta = sum dy  (over the rows)
 *   h, mean, rstd  as the forward left them (required with dy; mean: layer
 *                  norms alone)
 *   df, dx         [rows, H]; df required, dx NULL-able; each may be exactly
 *                  dy, dh or h, not the same one
 *   dbias, dgamma, dbeta
 *                  fp32 [H], each NULL-able; dgamma and dbeta NULL without a
 *                  norm, and zeros without dy
 *   workspace      device scratch of at least
 *                  dropout_add_norm_bwd_workspace_size() bytes, 16-byte
 *                  aligned, where dbias, dgamma or dbeta is given; no two calls
 *                  that may overlap on the GPU share one
 * The sums run in a fixed order: the same call on the same GPU model gives the
 * same bits.  rows == 0 zero-fills dbias, dgamma and dbeta.
 */
int dropout_add_norm_bwd(const void *dy, const void *dh, const void *h, double p,
                         const int64_t *rng, uint64_t seed, uint64_t offset, int norm,
                         const float *gamma, const float *mean, const float *rstd, void *df,
                         void *dx, float *dbias, float *dgamma, float *dbeta, int64_t rows,
                         int64_t H, int dtype, void *workspace, int64_t workspace_bytes,
                         void *stream);

/* Bytes of workspace that dropout_add_norm_bwd needs on the current device for
 * this many rows or fewer (0 when rows == 0), or a negative code. */
int64_t dropout_add_norm_bwd_workspace_size(int64_t rows, int64_t H, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* ADDLN_DROPOUT_H */
