// C-ABI entry points declared in include/addln_dropout.h: the argument checks
// (all before the first CUDA call), and whether rows lie on 16-byte borders.
#include <math.h>

#include <cuda_runtime.h>

#include "../../include/addln_dropout.h"
#include "abi.h"
#include "drop.h"

using namespace addln::abi;
using addln::DropSpec;
using addln::LaunchCtx;

namespace {

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

int check_shape(int64_t rows, int64_t H, int dtype) {
  if (!valid_dtype(dtype)) return ADDLN_ERR_DTYPE;
  if (rows < 0 || H <= 0 || H > max_hidden(dtype) || rows > INT64_MAX / (H * 4)) return ADDLN_ERR_SHAPE;
  return ADDLN_OK;
}

// The mask's numbers for p in [0, 1] and n elements.
int drop_spec(double p, const int64_t* rng, uint64_t seed, uint64_t offset, int64_t n, DropSpec* d) {
  if (!(p >= 0.0 && p <= 1.0)) return ADDLN_ERR_SCALE;
  const int64_t t = static_cast<int64_t>(nearbyint(p * 65536.0));
  d->rng = rng;
  d->seed = seed;
  d->offset = offset;
  d->above = static_cast<uint32_t>(t * 65536 - 1);
  d->on = t > 0;
  d->wide = n > (int64_t{1} << 35);
  d->scale = t < 65536 ? static_cast<float>(65536.0 / static_cast<double>(65536 - t)) : 0.f;
  return (bits(rng) & 7) ? ADDLN_ERR_ALIGN : ADDLN_OK;
}

// Outputs against inputs and each other; the first `in_place` outputs may be
// exactly one of the first `tensors` inputs.
int check_alias(const Range* outs, int n_out, int in_place, const Range* ins, int n_in, int tensors) {
  for (int i = 0; i < n_out; ++i) {
    for (int k = 0; k < n_in; ++k)
      if (bad_pair(outs[i], ins[k], i < in_place && k < tensors)) return ADDLN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return ADDLN_ERR_ALIAS;
  }
  return ADDLN_OK;
}

// How the rows of tensors at these addresses, and the vectors beside them (each
// ored), lie.
int mode_of(uintptr_t data, uintptr_t params, int64_t row_bytes) {
  if (data & 15) return addln::kShifted;
  return (params | static_cast<uintptr_t>(row_bytes)) & 15 ? addln::kEdged : addln::kAligned;
}

bool valid_norm(int k) { return k >= ADDLN_NORM_NONE && k <= ADDLN_NORM_LAYER; }

}  // namespace

extern "C" {

int dropout_fwd(const void* x, void* y, int64_t n, double p, const int64_t* rng, uint64_t seed, uint64_t offset,
                int dtype, void* stream) try {
  if (!valid_dtype(dtype)) return ADDLN_ERR_DTYPE;
  if (n < 0 || n > INT64_MAX / 4) return ADDLN_ERR_SHAPE;
  DropSpec d;
  int rc = drop_spec(p, rng, seed, offset, n, &d);
  if (rc != ADDLN_OK || n == 0) return rc;
  if (!x || !y) return ADDLN_ERR_NULL;
  const int es = elem_bytes(dtype);
  if ((bits(x) | bits(y)) & (es - 1)) return ADDLN_ERR_ALIGN;
  const Range out = range_of(y, n * es);
  if (bad_pair(out, range_of(x, n * es), true) || overlap(out, range_of(rng, 16))) return ADDLN_ERR_ALIAS;
  LaunchCtx c;
  rc = addln::launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  return addln::launch_dropout(dtype, x, y, n, d, c);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int dropout_add_norm_fwd(const void* f, const void* x, const float* bias, double p, const int64_t* rng,
                         uint64_t seed, uint64_t offset, int norm, const float* gamma, const float* beta, void* h,
                         void* y, float* mean, float* rstd, int64_t rows, int64_t H, float eps, int dtype,
                         void* stream) try {
  int rc = check_shape(rows, H, dtype);
  if (rc != ADDLN_OK) return rc;
  if (!valid_norm(norm)) return ADDLN_ERR_KIND;
  DropSpec d;
  rc = drop_spec(p, rng, seed, offset, rows * H, &d);
  if (rc != ADDLN_OK) return rc;
  if (!(eps >= 0.0f) || isinf(eps)) return ADDLN_ERR_EPS;
  const bool has = norm != ADDLN_NORM_NONE;
  if (!has && (y || gamma || beta || mean || rstd)) return ADDLN_ERR_KIND;
  if (rows == 0) return ADDLN_OK;
  if (!f || (has ? !y || !gamma : !h)) return ADDLN_ERR_NULL;
  if (norm != ADDLN_NORM_LAYER) mean = nullptr;  // only layer norms have means to write
  const int es = elem_bytes(dtype);
  const uintptr_t data = bits(f) | bits(x) | bits(h) | bits(y), params = bits(bias) | bits(gamma) | bits(beta);
  if ((data & (es - 1)) || ((params | bits(mean) | bits(rstd)) & 3)) return ADDLN_ERR_ALIGN;
  const int mode = mode_of(data, params, H * es);
  const int64_t tb = rows * H * es;
  const Range outs[4] = {range_of(h, tb), range_of(y, tb), range_of(mean, rows * 4), range_of(rstd, rows * 4)};
  const Range ins[6] = {range_of(f, tb), range_of(x, tb), range_of(bias, H * 4), range_of(gamma, H * 4),
                        range_of(beta, H * 4), range_of(rng, 16)};
  rc = check_alias(outs, 4, 2, ins, 6, 2);
  if (rc != ADDLN_OK) return rc;
  LaunchCtx c;
  rc = addln::launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  addln::DropFwdArgs a{f, x, bias, gamma, beta, h, y, mean, rstd, d, rows, static_cast<int>(H), norm, eps,
                       static_cast<float>(1.0 / static_cast<double>(H))};
  return addln::launch_drop_fwd(dtype, mode, a, c);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int64_t dropout_add_norm_bwd_workspace_size(int64_t rows, int64_t H, int dtype) try {
  int rc = check_shape(rows, H, dtype);
  if (rc != ADDLN_OK) return rc;
  if (rows == 0) return 0;
  LaunchCtx c;
  rc = addln::launch_context(nullptr, &c);
  if (rc != ADDLN_OK) return rc;
  // the most over the kernels that the call may turn out to take
  int64_t most = 0;
  for (int kind = 0; kind < 12; ++kind) {
    const int mode = kind / 4;
    if (mode == addln::kAligned && H * elem_bytes(dtype) % 16 != 0) continue;
    const int64_t n = addln::drop_bwd_workspace_bytes(dtype, mode, kind & 1, kind & 2, rows, static_cast<int>(H), c.dev);
    if (n < 0) return n;
    if (n > most) most = n;
  }
  return most;
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int dropout_add_norm_bwd(const void* dy, const void* dh, const void* h, double p, const int64_t* rng, uint64_t seed,
                         uint64_t offset, int norm, const float* gamma, const float* mean, const float* rstd, void* df,
                         void* dx, float* dbias, float* dgamma, float* dbeta, int64_t rows, int64_t H, int dtype,
                         void* workspace, int64_t workspace_bytes, void* stream) try {
  int rc = check_shape(rows, H, dtype);
  if (rc != ADDLN_OK) return rc;
  if (!valid_norm(norm)) return ADDLN_ERR_KIND;
  DropSpec d;
  rc = drop_spec(p, rng, seed, offset, rows * H, &d);
  if (rc != ADDLN_OK) return rc;
  if (norm == ADDLN_NORM_NONE && (dy || gamma || mean || rstd || dgamma || dbeta)) return ADDLN_ERR_KIND;
  if (workspace_bytes < 0) return ADDLN_ERR_WORKSPACE;
  if ((bits(dbias) | bits(dgamma) | bits(dbeta)) & 3) return ADDLN_ERR_ALIGN;
  if (rows == 0) {
    for (float* t : {dbias, dgamma, dbeta})
      if (t && cudaMemsetAsync(t, 0, H * 4, static_cast<cudaStream_t>(stream)) != cudaSuccess) return ADDLN_ERR_CUDA;
    return ADDLN_OK;
  }
  if ((!dy && !dh) || !df || (dy && (!h || !gamma || !rstd)) || (dy && norm == ADDLN_NORM_LAYER && !mean))
    return ADDLN_ERR_NULL;
  // what is not read decides nothing
  if (!dy) h = nullptr, rstd = nullptr, gamma = nullptr;
  if (!dy || norm != ADDLN_NORM_LAYER) mean = nullptr;
  const int es = elem_bytes(dtype);
  const uintptr_t data = bits(dy) | bits(dh) | bits(h) | bits(df) | bits(dx);
  if ((data & (es - 1)) || ((bits(gamma) | bits(mean) | bits(rstd)) & 3)) return ADDLN_ERR_ALIGN;
  const int mode = mode_of(data, bits(gamma), H * es);
  const int64_t tb = rows * H * es;
  const bool cols = dbias || dgamma || dbeta;
  const Range ins[7] = {range_of(dy, tb), range_of(dh, tb), range_of(h, tb), range_of(gamma, H * 4),
                        range_of(mean, rows * 4), range_of(rstd, rows * 4), range_of(rng, 16)};
  const Range outs[6] = {range_of(df, tb), range_of(dx, tb), range_of(dbias, H * 4), range_of(dgamma, H * 4),
                         range_of(dbeta, H * 4), range_of(cols ? workspace : nullptr, workspace_bytes)};
  rc = check_alias(outs, 6, 2, ins, 7, 3);
  if (rc != ADDLN_OK) return rc;
  LaunchCtx c;
  rc = addln::launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  addln::DropBwdArgs a{dy, dh, h, gamma, mean, rstd, df, dx, dbias, dgamma, dbeta, nullptr, d, rows, 0,
                       static_cast<int>(H), 0, norm, static_cast<float>(1.0 / static_cast<double>(H))};
  return addln::launch_drop_bwd(dtype, mode, a, workspace, workspace_bytes, c);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

}  // extern "C"
