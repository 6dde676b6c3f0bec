// Internal interface between the block-boundary entry points (block_api.cu)
// and their kernels.
#pragma once

#include <stdint.h>

#include "launch.h"

namespace addln {

// How rows lie: on 16-byte borders; anywhere; anywhere, but all of a walker's rows
// of all tensors the same distance past the borders (block.cuh).
constexpr int kAligned = 0, kShifted = 1, kEdged = 2;

// How walkers (a warp, a CTA or a cluster for each row) cover the rows.
struct Walk {
  int C;             // CTAs of a row
  int slice;         // columns each of them owns
  int rows_per_cta;  // rows a CTA walks side by side, a warp for each; else 1
  int cta_warps;     // warps a row has in one CTA
  int warps;         // warps a row has
  int width;         // lanes that join the warps' sums: a power of two, at most 32
};

// Arguments of one forward launch; the meaning of each is block_norm_fwd's.
// gate_rows: rows of a per-row gate.
struct BlockFwdArgs {
  const void* f;
  const void* x;
  const float* post_gamma;
  const float* post_beta;
  const void* gate;
  const float* pre_gamma;
  const float* pre_beta;
  void* h;
  void* y;
  float* post_mean;
  float* post_rstd;
  float* pre_mean;
  float* pre_rstd;
  int64_t rows;
  int64_t gate_rows, gate_stride, rows_per_gate;
  int H;
  int post, pre, gate_kind;
  float a, s, eps, inv_h;
  int slots, ring_slots;  // rows staged ahead, 1 or 2; slots there are
  int kept_at, sums_at;   // where parameters and row sums lie in shared memory
  Walk w;
};

// Arguments of one backward launch (block_norm_bwd).  part: [parts][A][Hp]
// fp32 column partials, one for each CTA or cluster; seg: [walkers][2][Hp] fp32 sums of a per-row gate's
// gradient over the rows of a gate row that the walker shares with others
// (first and last of its range).  Hp: H rounded up to 4.
struct BlockBwdArgs {
  const void* dy;
  const void* dh;
  const void* f;
  const void* h;
  const float* post_mean;
  const float* post_rstd;
  const float* pre_mean;
  const float* pre_rstd;
  const float* post_gamma;
  const float* post_beta;
  const void* gate;
  const float* pre_gamma;
  void* df;
  void* dx;
  float* dpost_gamma;
  float* dpost_beta;
  void* dgate;
  float* dpre_gamma;
  float* dpre_beta;
  float* part;
  float* seg;
  int64_t rows, walkers, parts;
  int64_t gate_rows, gate_stride, rows_per_gate;
  int H, Hp;
  int post, pre, gate_kind;
  float a, s, inv_h;
  int kept_at, sums_at;  // where parameters and row sums lie in shared memory
  Walk w;
};

// aligned: every row of every tensor in the I/O dtype begins on a 16-byte
// border and ends on one.
int launch_block_fwd(int dtype, bool aligned, bool layer_or_bias, const BlockFwdArgs& p, const LaunchCtx& c);
// Bytes of workspace of a backward call, or a negative code.
int64_t block_bwd_workspace_bytes(int dtype, bool aligned, bool full, int64_t rows, int H, int gate_kind,
                                  int64_t rows_per_gate, const DeviceInfo& dev);
int launch_block_bwd(int dtype, bool aligned, bool full, BlockBwdArgs p, void* ws, int64_t ws_bytes,
                     const LaunchCtx& c);

int read_bounds_block_fwd(unsigned long long* word);
int read_bounds_block_bwd(unsigned long long* word);
int read_bounds_grad(unsigned long long* word);

}  // namespace addln
