// Internal interface between the dropout entry points (drop_api.cu) and their
// kernels.
#pragma once

#include <stdint.h>

#include "block.h"

namespace addln {

// A mask, as the kernels take it.  above: an element is kept where its 16
// bits, in the upper half of a word, make that word larger (t 65536 - 1).
// on: something is dropped (t > 0).  wide: the tensor has more than 2^32 blocks
// of 8 elements.  scale: of what is kept.
struct DropSpec {
  const int64_t* rng;  // seed and offset in device memory, or NULL
  uint64_t seed, offset;
  uint32_t above;
  int on, wide;
  float scale;
};

// Arguments of one forward launch; the meaning of each is
// dropout_add_norm_fwd's.
struct DropFwdArgs {
  const void* f;
  const void* x;
  const float* bias;
  const float* gamma;
  const float* beta;
  void* h;
  void* y;
  float* mean;
  float* rstd;
  DropSpec drop;
  int64_t rows;
  int H, norm;
  float eps, inv_h;
  int slots, ring_slots;  // rows staged ahead, 1 or 2; slots there are
  int kept_at, sums_at;   // where parameters and row sums lie in shared memory
  Walk w;
};

// Arguments of one backward launch.  part: [parts][A][Hp] fp32 column
// partials, one for each CTA or cluster: dgamma, then (where the kernel has
// them) dbeta, then dbias.  Hp: H rounded up to 4.
struct DropBwdArgs {
  const void* dy;
  const void* dh;
  const void* h;
  const float* gamma;
  const float* mean;
  const float* rstd;
  void* df;
  void* dx;
  float* dbias;
  float* dgamma;
  float* dbeta;
  float* part;
  DropSpec drop;
  int64_t rows, parts;
  int H, Hp, norm;
  float inv_h;
  int kept_at, sums_at;
  Walk w;
};

int launch_dropout(int dtype, const void* x, void* y, int64_t n, const DropSpec& drop, const LaunchCtx& c);
// mode: kAligned where every row of every tensor in the I/O dtype, and every vector,
// begins and ends on 16-byte borders, kEdged where every such tensor begins on one.
int launch_drop_fwd(int dtype, int mode, const DropFwdArgs& p, const LaunchCtx& c);
int64_t drop_bwd_workspace_bytes(int dtype, int mode, bool full, bool bias, int64_t rows, int H, const DeviceInfo& dev);
int launch_drop_bwd(int dtype, int mode, const DropBwdArgs& p, void* ws, int64_t ws_bytes, const LaunchCtx& c);

int read_bounds_drop(unsigned long long* word);
int read_bounds_drop_fwd(unsigned long long* word);
int read_bounds_drop_bwd(unsigned long long* word);

}  // namespace addln
