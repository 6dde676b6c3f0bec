/*
 * addln_quant.h - residual sum and norm with an output in 8 bits and its
 * scales, for the matrix product that follows, and reading such rows back.
 * Exported by the same library as addln.h and addln_block.h, whose conventions
 * (device pointers, contiguous row-major tensors, streams, return codes, norm
 * kinds, no allocation) hold here too.
 *
 * A value y is held as q, 8 bits, and stands for q * scale:
 *     ADDLN_Q_E4M3  4 exponent and 3 mantissa bits, no infinities; largest 448
 *     ADDLN_Q_E5M2  5 and 2; largest 57344
 *     ADDLN_Q_INT8  whole numbers from -127 to 127
 * q is y / scale rounded to nearest, ties to even, and cut at +- the largest.
 * Of the scales,
 *     ADDLN_SCALE_ROW     fp32 [rows]: the row's largest |y| / the format's
 *                         largest value
 *     ADDLN_SCALE_GROUP   fp32, the same for every `group` columns of a row
 *                         (32, 64 or 128; the row's last group may be shorter)
 *     ADDLN_SCALE_POW2    the same groups, each with the least power of two 2^e
 *                         by which no value is cut, one byte e + 127
 *     ADDLN_SCALE_TENSOR  fp32 [1], given, at least 2^-126: values beyond are cut
 * and the scales of groups lie as [rows, groups], or with group_major as
 * [groups, rows]; a tensor-core product with block scales wants those of POW2
 * in tiles of 128 rows by 4 groups, an order that is not made here.  No scale
 * that is made here is below 2^-126 (rows of zeros).
 * Where the largest |y| is NaN or infinite the scale is NaN (byte 255), and
 * so is q, in integers 0.  With a given scale NaN gives NaN (integers: 0) and
 * an infinity the largest value.
 */
#ifndef ADDLN_QUANT_H
#define ADDLN_QUANT_H

#include "addln_block.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ADDLN_Q_E4M3 0
#define ADDLN_Q_E5M2 1
#define ADDLN_Q_INT8 2

#define ADDLN_SCALE_ROW 0
#define ADDLN_SCALE_GROUP 1
#define ADDLN_SCALE_POW2 2
#define ADDLN_SCALE_TENSOR 3

/*
 * Per row:  h = x + residual,  y = norm(h),  q and scale of y as above.
 *   x           [rows, H] (required)
 *   residual    [rows, H], or NULL: h = x
 *   norm        ADDLN_NORM_NONE (y = h), _RMS or _LAYER, with gamma [H]
 *               (required) and beta [H] or NULL, fp32
 *   q           [rows, H] bytes (required)
 *   scale       written; read for ADDLN_SCALE_TENSOR (required)
 *   group, group_major
 *               read for GROUP and POW2 alone
 *   h           [rows, H] in the I/O dtype, NULL-able; may be exactly x or
 *               residual
 *   mean, rstd  fp32 [rows] statistics of h, each NULL-able, NULL without a
 *               norm; the mean is written for layer norms alone
 * Arithmetic is fp32; y and its scale are taken of the unrounded h.  eps as in
 * block_norm_fwd.  Any other overlap of an output is ADDLN_ERR_ALIAS; a format,
 * scaling or group other than these is ADDLN_ERR_KIND.  rows == 0 is a no-op.
 * block_norm_bwd is the backward with respect to the values that q stands for
 * (the rounding's derivative taken as 1): dy their gradient, h and the
 * statistics as written here.
 */
int norm_quant_fwd(const void *x, const void *residual, int norm, const float *gamma,
                   const float *beta, void *q, int format, int scaling, int64_t group,
                   int group_major, void *scale, void *h, float *mean, float *rstd, int64_t rows,
                   int64_t H, float eps, int dtype, void *stream);

/*
 * out = q * scale, in fp32 and rounded to dtype: reads back what
 * norm_quant_fwd wrote, with its format, scaling, group and group_major.
 * H up to addln_max_hidden(ADDLN_BF16) for every dtype.
 */
int dequant_rows(const void *q, int format, int scaling, int64_t group, int group_major,
                 const void *scale, void *out, int64_t rows, int64_t H, int dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ADDLN_QUANT_H */
