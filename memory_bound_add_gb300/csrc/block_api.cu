// C-ABI entry points declared in include/addln_block.h: the argument checks
// (all before the first CUDA call), and whether rows lie on 16-byte borders.
#include <math.h>

#include <cuda_runtime.h>

#include "../../include/addln_block.h"
#include "abi.h"
#include "block.h"

using namespace addln::abi;
using addln::LaunchCtx;

namespace {

bool valid_norm(int k) { return k >= ADDLN_NORM_NONE && k <= ADDLN_NORM_LAYER; }

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// Dtype, shape, kinds and scales; *gate_rows: rows of a per-row gate.
// *rows_per_gate is cut to the rows there are, which changes no row's gate row:
// the kernels' 32-bit arithmetic of gate rows holds wherever rows fits 32 bits.
int check_spec(int post, int pre, int gate_kind, int64_t gate_stride, int64_t* rows_per_gate, float a,
               float s, int64_t rows, int64_t H, int dtype, int64_t* gate_rows) {
  if (!valid_dtype(dtype)) return ADDLN_ERR_DTYPE;
  if (rows < 0 || H <= 0 || H > max_hidden(dtype) || rows > INT64_MAX / (H * 4)) return ADDLN_ERR_SHAPE;
  if (!valid_norm(post) || !valid_norm(pre) || gate_kind < ADDLN_GATE_NONE || gate_kind > ADDLN_GATE_ROWS)
    return ADDLN_ERR_KIND;
  if (!isfinite(a) || !isfinite(s)) return ADDLN_ERR_SCALE;
  *gate_rows = 0;
  if (gate_kind == ADDLN_GATE_ROWS) {
    if (*rows_per_gate < 1 || gate_stride < H) return ADDLN_ERR_SHAPE;
    if (rows > 0 && *rows_per_gate > rows) *rows_per_gate = rows;
    *gate_rows = rows / *rows_per_gate + (rows % *rows_per_gate != 0);
    if (*gate_rows > 0 && gate_stride > INT64_MAX / 8 / *gate_rows) return ADDLN_ERR_SHAPE;
  }
  return ADDLN_OK;
}

int64_t gate_bytes(int gate_kind, int64_t gate_rows, int64_t gate_stride, int64_t H, int es) {
  if (gate_kind == ADDLN_GATE_CHANNEL) return H * 4;
  if (gate_kind == ADDLN_GATE_ROWS && gate_rows > 0) return ((gate_rows - 1) * gate_stride + H) * es;
  return 0;
}

// Whether rows of H elements at these addresses (the tensors in the I/O
// dtype, and the fp32 vectors, each ored; stride: a gate's row stride) begin
// and end on 16-byte borders.
bool rows_aligned(uintptr_t data, uintptr_t params, int64_t H, int64_t stride, int es) {
  return ((data | params | static_cast<uintptr_t>(H * es) | static_cast<uintptr_t>(stride * es)) & 15) == 0;
}

// Whether some address is not a multiple of its element.
bool misplaced(uintptr_t data, uintptr_t params, int es) { return (data & (es - 1)) || (params & 3); }

}  // namespace

extern "C" {

int block_norm_fwd(const void* f, const void* x, int post, const float* post_gamma, const float* post_beta,
                   const void* gate, int gate_kind, int64_t gate_stride, int64_t rows_per_gate,
                   float residual_scale, float block_scale, int pre, const float* pre_gamma,
                   const float* pre_beta, void* h, void* y, float* post_mean, float* post_rstd,
                   float* pre_mean, float* pre_rstd, int64_t rows, int64_t H, float eps, int dtype,
                   void* stream) try {
  int64_t gate_rows;
  int rc = check_spec(post, pre, gate_kind, gate_stride, &rows_per_gate, residual_scale, block_scale, rows, H,
                      dtype, &gate_rows);
  if (rc != ADDLN_OK) return rc;
  if (!(eps >= 0.0f) || isinf(eps)) return ADDLN_ERR_EPS;
  if ((pre == ADDLN_NORM_NONE && (y || pre_gamma || pre_beta || pre_mean || pre_rstd)) ||
      (post == ADDLN_NORM_NONE && (post_gamma || post_beta || post_mean || post_rstd)) ||
      (gate_kind == ADDLN_GATE_NONE && gate))
    return ADDLN_ERR_KIND;
  if (rows == 0) return ADDLN_OK;
  const bool has_pre = pre != ADDLN_NORM_NONE, has_post = post != ADDLN_NORM_NONE;
  if (!f || !x || !h || (has_pre && (!y || !pre_gamma)) || (has_post && !post_gamma) ||
      (gate_kind != ADDLN_GATE_NONE && !gate))
    return ADDLN_ERR_NULL;
  // only layer norms have means to write
  if (post != ADDLN_NORM_LAYER) post_mean = nullptr;
  if (pre != ADDLN_NORM_LAYER) pre_mean = nullptr;

  const int es = elem_bytes(dtype);
  const bool gr = gate_kind == ADDLN_GATE_ROWS;
  const uintptr_t data = bits(f) | bits(x) | bits(h) | bits(y) | (gr ? bits(gate) : 0);
  const uintptr_t params = bits(post_gamma) | bits(post_beta) | bits(pre_gamma) | bits(pre_beta) |
                           (gate_kind == ADDLN_GATE_CHANNEL ? bits(gate) : 0);
  if (misplaced(data, params | bits(post_mean) | bits(post_rstd) | bits(pre_mean) | bits(pre_rstd), es))
    return ADDLN_ERR_ALIGN;
  const bool aligned = rows_aligned(data, params, H, gr ? gate_stride : 0, es);

  const int64_t tb = rows * H * es;
  const Range outs[6] = {range_of(h, tb), range_of(y, tb), range_of(post_mean, rows * 4),
                         range_of(post_rstd, rows * 4), range_of(pre_mean, rows * 4), range_of(pre_rstd, rows * 4)};
  const Range ins[7] = {range_of(f, tb), range_of(x, tb), range_of(post_gamma, H * 4), range_of(post_beta, H * 4),
                        range_of(gate, gate_bytes(gate_kind, gate_rows, gate_stride, H, es)),
                        range_of(pre_gamma, H * 4), range_of(pre_beta, H * 4)};
  for (int i = 0; i < 6; ++i) {
    for (int k = 0; k < 7; ++k)
      if (bad_pair(outs[i], ins[k], i < 2 && k < 2)) return ADDLN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return ADDLN_ERR_ALIAS;
  }

  LaunchCtx c;
  rc = addln::launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  addln::BlockFwdArgs p{f, x, post_gamma, post_beta, gate, pre_gamma, pre_beta, h, y, post_mean, post_rstd,
                        pre_mean, pre_rstd, rows, gate_rows, gate_stride, rows_per_gate, static_cast<int>(H),
                        post, pre, gate_kind, residual_scale, block_scale, eps,
                        static_cast<float>(1.0 / static_cast<double>(H))};
  const bool layer_or_bias = post == ADDLN_NORM_LAYER || pre == ADDLN_NORM_LAYER || post_beta || pre_beta;
  return addln::launch_block_fwd(dtype, aligned, layer_or_bias, p, c);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int64_t block_norm_bwd_workspace_size(int64_t rows, int64_t H, int dtype, int gate_kind,
                                      int64_t rows_per_gate) try {
  int64_t gate_rows;
  int rc = check_spec(ADDLN_NORM_NONE, ADDLN_NORM_NONE, gate_kind, H, &rows_per_gate, 1.f, 1.f, rows, H, dtype,
                      &gate_rows);
  if (rc != ADDLN_OK) return rc;
  if (rows == 0) return 0;
  LaunchCtx c;
  rc = addln::launch_context(nullptr, &c);
  if (rc != ADDLN_OK) return rc;
  // the most over the kernels that the call may turn out to take
  int64_t most = 0;
  for (int kind = 0; kind < 4; ++kind) {
    const bool aligned = kind & 1, full = kind & 2;
    if (aligned && H * elem_bytes(dtype) % 16 != 0) continue;
    const int64_t n = addln::block_bwd_workspace_bytes(dtype, aligned, full, rows, static_cast<int>(H), gate_kind,
                                                       rows_per_gate, c.dev);
    if (n < 0) return n;
    if (n > most) most = n;
  }
  return most;
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int block_norm_bwd(const void* dy, const void* dh, const void* f, const void* h, int post,
                   const float* post_gamma, const float* post_beta, const float* post_mean,
                   const float* post_rstd, const void* gate, int gate_kind, int64_t gate_stride,
                   int64_t rows_per_gate, float residual_scale, float block_scale, int pre,
                   const float* pre_gamma, const float* pre_mean, const float* pre_rstd, void* df, void* dx,
                   float* dpost_gamma, float* dpost_beta, void* dgate, float* dpre_gamma, float* dpre_beta,
                   int64_t rows, int64_t H, int dtype, void* workspace, int64_t workspace_bytes,
                   void* stream) try {
  int64_t gate_rows;
  int rc = check_spec(post, pre, gate_kind, gate_stride, &rows_per_gate, residual_scale, block_scale, rows, H,
                      dtype, &gate_rows);
  if (rc != ADDLN_OK) return rc;
  const bool has_post = post != ADDLN_NORM_NONE, has_pre = pre != ADDLN_NORM_NONE;
  const bool gr = gate_kind == ADDLN_GATE_ROWS;
  if ((!has_pre && (dy || pre_gamma || pre_mean || pre_rstd || dpre_gamma || dpre_beta)) ||
      (!has_post && (post_gamma || post_beta || post_mean || post_rstd || dpost_gamma || dpost_beta)) ||
      (gate_kind == ADDLN_GATE_NONE && (gate || dgate)))
    return ADDLN_ERR_KIND;
  if (workspace_bytes < 0) return ADDLN_ERR_WORKSPACE;
  const int es = elem_bytes(dtype);
  const uintptr_t outs32 = bits(dpost_gamma) | bits(dpost_beta) | bits(dpre_gamma) | bits(dpre_beta) |
                           (gr ? 0 : bits(dgate));
  if ((outs32 & 3) || (bits(dgate) & (es - 1))) return ADDLN_ERR_ALIGN;
  if (rows == 0) {
    float* sums[5] = {dpost_gamma, dpost_beta, dpre_gamma, dpre_beta, gr ? nullptr : static_cast<float*>(dgate)};
    for (float* t : sums)
      if (t && cudaMemsetAsync(t, 0, H * 4, static_cast<cudaStream_t>(stream)) != cudaSuccess) return ADDLN_ERR_CUDA;
    return ADDLN_OK;
  }
  const bool need_f = has_post || gate_kind != ADDLN_GATE_NONE;
  if ((!dy && !dh) || !df || !dx || (need_f && !f) || (dy && (!h || !pre_gamma || !pre_rstd)) ||
      (dy && pre == ADDLN_NORM_LAYER && !pre_mean) || (has_post && (!post_gamma || !post_rstd)) ||
      (post == ADDLN_NORM_LAYER && !post_mean) || (gate_kind != ADDLN_GATE_NONE && !gate))
    return ADDLN_ERR_NULL;
  // what is not read decides nothing
  if (!need_f) f = nullptr;
  if (!dy) h = nullptr;
  if (post != ADDLN_NORM_LAYER) post_mean = nullptr;
  if (pre != ADDLN_NORM_LAYER || !dy) pre_mean = nullptr;
  if (!dy) pre_rstd = nullptr;

  const uintptr_t data = bits(dy) | bits(dh) | bits(f) | bits(h) | bits(df) | bits(dx) |
                         (gr ? bits(gate) | bits(dgate) : 0);
  const uintptr_t params = bits(post_gamma) | bits(post_beta) | bits(pre_gamma) |
                           (gate_kind == ADDLN_GATE_CHANNEL ? bits(gate) : 0);
  if (misplaced(data, params | bits(post_mean) | bits(post_rstd) | bits(pre_mean) | bits(pre_rstd), es))
    return ADDLN_ERR_ALIGN;
  const bool aligned = rows_aligned(data, params, H, gr ? gate_stride : 0, es);

  const int64_t tb = rows * H * es;
  const bool scratch = outs32 != 0 || (gr && dgate && rows_per_gate > 1);
  const Range ins[12] = {range_of(dy, tb), range_of(dh, tb), range_of(f, tb), range_of(h, tb),
                         range_of(post_gamma, H * 4), range_of(post_beta, H * 4), range_of(pre_gamma, H * 4),
                         range_of(post_mean, rows * 4), range_of(post_rstd, rows * 4),
                         range_of(pre_mean, rows * 4), range_of(pre_rstd, rows * 4),
                         range_of(gate, gate_bytes(gate_kind, gate_rows, gate_stride, H, es))};
  const Range outs[8] = {range_of(df, tb), range_of(dx, tb), range_of(dpost_gamma, H * 4),
                         range_of(dpost_beta, H * 4), range_of(dpre_gamma, H * 4), range_of(dpre_beta, H * 4),
                         range_of(dgate, gr ? gate_rows * H * es : H * 4),
                         range_of(scratch ? workspace : nullptr, workspace_bytes)};
  for (int i = 0; i < 8; ++i) {
    for (int k = 0; k < 12; ++k)
      if (bad_pair(outs[i], ins[k], i < 2 && k < 4)) return ADDLN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return ADDLN_ERR_ALIAS;
  }

  LaunchCtx c;
  rc = addln::launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  addln::BlockBwdArgs p{dy, dh, f, h, post_mean, post_rstd, pre_mean, pre_rstd, post_gamma, post_beta, gate,
                        pre_gamma, df, dx, dpost_gamma, dpost_beta, dgate, dpre_gamma, dpre_beta, nullptr,
                        nullptr, rows, 0, 0, gate_rows, gate_stride, rows_per_gate, static_cast<int>(H), 0, post,
                        pre, gate_kind, residual_scale, block_scale,
                        static_cast<float>(1.0 / static_cast<double>(H))};
  const bool full = post == ADDLN_NORM_LAYER || pre == ADDLN_NORM_LAYER || post_beta || dpost_beta || dpre_beta;
  return addln::launch_block_bwd(dtype, aligned, full, p, workspace, workspace_bytes, c);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

}  // extern "C"
