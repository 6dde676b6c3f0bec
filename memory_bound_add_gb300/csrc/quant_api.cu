// C-ABI entry points declared in include/addln_quant.h: the argument checks
// (all before the first CUDA call), and whether rows lie on the borders that
// the kernels' wide accesses need.
#include <math.h>

#include <cuda_runtime.h>

#include "../../include/addln_quant.h"
#include "abi.h"
#include "quant.h"

using namespace addln::abi;
using addln::LaunchCtx;
using addln::ScaleSpec;

namespace {

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// Format, scaling and group; *bytes: of the scales.
int scale_spec(const void* scale, int format, int scaling, int64_t group, int group_major, int64_t rows, int64_t H,
               ScaleSpec* s, int64_t* bytes) {
  if (format < ADDLN_Q_E4M3 || format > ADDLN_Q_INT8 || scaling < ADDLN_SCALE_ROW || scaling > ADDLN_SCALE_TENSOR)
    return ADDLN_ERR_KIND;
  const bool groups = scaling == ADDLN_SCALE_GROUP || scaling == ADDLN_SCALE_POW2;
  if (groups && group != 32 && group != 64 && group != 128) return ADDLN_ERR_KIND;
  s->scale = const_cast<void*>(scale);
  s->format = format;
  s->scaling = scaling;
  s->group_major = groups && group_major != 0;
  s->lanes_shift = !groups ? 0 : group == 32 ? 5 : group == 64 ? 6 : 7;
  s->groups = groups ? static_cast<int>((H + group - 1) / group) : 1;
  *bytes = scaling == ADDLN_SCALE_TENSOR ? 4 : rows * s->groups * (scaling == ADDLN_SCALE_POW2 ? 1 : 4);
  return ADDLN_OK;
}

}  // namespace

extern "C" {

int norm_quant_fwd(const void* x, const void* residual, int norm, const float* gamma, const float* beta, void* q,
                   int format, int scaling, int64_t group, int group_major, void* scale, void* h, float* mean,
                   float* rstd, int64_t rows, int64_t H, float eps, int dtype, void* stream) try {
  if (!valid_dtype(dtype)) return ADDLN_ERR_DTYPE;
  if (rows < 0 || H <= 0 || H > max_hidden(dtype) || rows > INT64_MAX / (H * 4)) return ADDLN_ERR_SHAPE;
  if (norm < ADDLN_NORM_NONE || norm > ADDLN_NORM_LAYER) return ADDLN_ERR_KIND;
  ScaleSpec s;
  int64_t scale_bytes;
  int rc = scale_spec(scale, format, scaling, group, group_major, rows, H, &s, &scale_bytes);
  if (rc != ADDLN_OK) return rc;
  if (!(eps >= 0.0f) || isinf(eps)) return ADDLN_ERR_EPS;
  const bool has = norm != ADDLN_NORM_NONE;
  if (!has && (gamma || beta || mean || rstd)) return ADDLN_ERR_KIND;
  if (rows == 0) return ADDLN_OK;
  if (!x || !q || !scale || (has && !gamma)) return ADDLN_ERR_NULL;
  if (norm != ADDLN_NORM_LAYER) mean = nullptr;  // only layer norms have means to write
  const int es = elem_bytes(dtype);
  const uintptr_t data = bits(x) | bits(residual) | bits(h), params = bits(gamma) | bits(beta);
  if ((data & (es - 1)) || ((params | bits(mean) | bits(rstd)) & 3) || (scaling != ADDLN_SCALE_POW2 && (bits(scale) & 3)))
    return ADDLN_ERR_ALIGN;
  // a 16-byte vector of the I/O type becomes 16 / es bytes of q
  const bool begins = (data & 15) == 0 && (bits(q) & (16 / es - 1)) == 0;
  const bool rest = ((params | static_cast<uintptr_t>(H * es)) & 15) == 0;
  const int mode = !begins ? addln::kShifted : rest ? addln::kAligned : addln::kEdged;
  const int64_t tb = rows * H * es;
  const bool given = scaling == ADDLN_SCALE_TENSOR;
  const Range sr = range_of(scale, scale_bytes), none = range_of(nullptr, 0);
  const Range outs[5] = {range_of(h, tb), range_of(q, rows * H), given ? none : sr, range_of(mean, rows * 4),
                         range_of(rstd, rows * 4)};
  const Range ins[5] = {range_of(x, tb), range_of(residual, tb), range_of(gamma, H * 4), range_of(beta, H * 4),
                        given ? sr : none};
  for (int i = 0; i < 5; ++i) {
    for (int k = 0; k < 5; ++k)
      if (bad_pair(outs[i], ins[k], i < 1 && k < 2)) return ADDLN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return ADDLN_ERR_ALIAS;
  }
  LaunchCtx c;
  rc = addln::launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  addln::QuantArgs a{x, residual, gamma, beta, q, h, mean, rstd, s, rows, static_cast<int>(H), norm, eps,
                     static_cast<float>(1.0 / static_cast<double>(H))};
  return addln::launch_norm_quant(dtype, mode, a, c);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int dequant_rows(const void* q, int format, int scaling, int64_t group, int group_major, const void* scale, void* out,
                 int64_t rows, int64_t H, int dtype, void* stream) try {
  if (!valid_dtype(dtype)) return ADDLN_ERR_DTYPE;
  if (rows < 0 || H <= 0 || H > max_hidden(ADDLN_BF16) || rows > INT64_MAX / (H * 4)) return ADDLN_ERR_SHAPE;
  ScaleSpec s;
  int64_t scale_bytes;
  int rc = scale_spec(scale, format, scaling, group, group_major, rows, H, &s, &scale_bytes);
  if (rc != ADDLN_OK || rows == 0) return rc;
  if (!q || !scale || !out) return ADDLN_ERR_NULL;
  const int es = elem_bytes(dtype);
  if ((bits(out) & (es - 1)) || (scaling != ADDLN_SCALE_POW2 && (bits(scale) & 3))) return ADDLN_ERR_ALIGN;
  const bool aligned = ((bits(out) | static_cast<uintptr_t>(H * es)) & 15) == 0 && (bits(q) & (16 / es - 1)) == 0;
  const Range o = range_of(out, rows * H * es);
  if (overlap(o, range_of(q, rows * H)) || overlap(o, range_of(scale, scale_bytes))) return ADDLN_ERR_ALIAS;
  LaunchCtx c;
  rc = addln::launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  return addln::launch_dequant(dtype, aligned, addln::DequantArgs{q, out, s, rows, static_cast<int>(H)}, c);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

}  // extern "C"
