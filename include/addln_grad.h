/*
 * addln_grad.h - the norm over all gradients of a training step, and the
 * gradients scaled so that it is at most max_norm.  Exported by the same
 * library as addln.h, whose conventions (device pointers, streams, return
 * codes, no allocation) hold here too.  The pages have no counterpart: this
 * is what follows the backward passes of this library in a training step.
 *
 *     norm   = scale sqrt(sum over all tensors and elements of g^2)
 *     factor = scale min(1, max_norm / (norm + 1e-6))
 *     out    = g factor                         rounded once to out's dtype
 * scale is 1 / loss scale (1: none).  A NaN among the gradients makes norm
 * and every out NaN, an infinite norm a factor of 0 (and NaN where g is
 * infinite), as the formulas say.  An infinite max_norm is no limit: the
 * factor is scale whatever the norm, unless that is NaN.
 *
 * Arrays of pointers, sizes and dtypes are HOST arrays of count entries; they
 * are read before the call returns (a captured call keeps their values).
 *   grads      device pointers, NULL-able where the size is 0; their elements
 *              are contiguous
 *   sizes      elements of each, >= 0
 *   dtypes     ADDLN_FP32 / FP16 / BF16 of each
 *   outs       device pointers (NULL: in place, outs = grads and out_dtypes =
 *              dtypes); each out has its gradient's dtype or fp32, and is
 *              exactly its gradient or apart from all gradients and outs
 *   workspace  device scratch of at least grad_norm_workspace_size(count)
 *              bytes, 16-byte aligned, the caller's; no two calls that may
 *              overlap on the GPU share one; needs no initialisation
 * The squares are summed in a fixed order (fp32 within a thread's share of a
 * few dozen elements, pairs of fp32 values beyond; shares whose squares leave
 * fp32's range are summed in fp64), so the same call gives the same bits.
 * Where nothing is to be scaled in place (factor 1), nothing is written.
 */
#ifndef ADDLN_GRAD_H
#define ADDLN_GRAD_H

#include "addln_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* norm (fp32, one element) of the gradients; 0 for none. */
int grad_norm(const void *const *grads, const int64_t *sizes, const int *dtypes, int64_t count,
              float scale, float *norm, void *workspace, int64_t workspace_bytes, void *stream);

/* Scales by a norm that is already on the device (e.g. joined over several
 * GPUs).  max_norm >= 0, or infinite: no limit. */
int grad_clip(const void *const *grads, void *const *outs, const int64_t *sizes, const int *dtypes,
              const int *out_dtypes, int64_t count, float scale, float max_norm, const float *norm,
              void *stream);

/* Both: norm is written, and the gradients scaled by it. */
int grad_norm_clip(const void *const *grads, void *const *outs, const int64_t *sizes,
                   const int *dtypes, const int *out_dtypes, int64_t count, float scale,
                   float max_norm, float *norm, void *workspace, int64_t workspace_bytes,
                   void *stream);

/* Bytes of workspace for this many tensors, or ADDLN_ERR_SHAPE. */
int64_t grad_norm_workspace_size(int64_t count);

#ifdef __cplusplus
}
#endif

#endif /* ADDLN_GRAD_H */
