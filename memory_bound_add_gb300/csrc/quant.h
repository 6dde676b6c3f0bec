// Internal interface between the 8-bit entry points (quant_api.cu) and their
// kernels.
#pragma once

#include <stdint.h>

#include "block.h"

namespace addln {

// Where the scales of a call are: as quant_api.cu's callers give them; group a
// power of two (0: one for the row, or given), groups: of a row.
struct ScaleSpec {
  void* scale;
  int format, scaling, group_major;
  int lanes_shift;  // log2(group)
  int groups;
};

// Arguments of one norm_quant_fwd launch; the meaning of each is the entry
// point's.
struct QuantArgs {
  const void* x;
  const void* r;
  const float* gamma;
  const float* beta;
  void* q;
  void* h;
  float* mean;
  float* rstd;
  ScaleSpec s;
  int64_t rows;
  int H, norm;
  float eps, inv_h;
  int slots, ring_slots;
  int kept_at, sums_at;
  Walk w;
};

// Arguments of one dequant_rows launch.  scale_row, scale_group: scales between a
// group's and the next row's, and the next group's; scales: all of them; pieces: of
// a row, 32 16-byte vectors of out each; reciprocal: 2^32 / H, rounded up.
struct DequantArgs {
  const void* q;
  void* out;
  ScaleSpec s;
  int64_t rows;
  int H, pieces;
  uint32_t reciprocal;
  int64_t scale_row, scale_group, scales;
};

// mode: kAligned where every row of every tensor in the I/O dtype, and every vector,
// begins and ends on 16-byte borders, and every row of q on borders of 16 bytes over
// the I/O type's size; kEdged where all these tensors begin on such.
int launch_norm_quant(int dtype, int mode, const QuantArgs& p, const LaunchCtx& c);
// aligned: as kAligned, of out and q.
int launch_dequant(int dtype, bool aligned, const DequantArgs& p, const LaunchCtx& c);

int read_bounds_quant(unsigned long long* word);
int read_bounds_dequant(unsigned long long* word);

}  // namespace addln
