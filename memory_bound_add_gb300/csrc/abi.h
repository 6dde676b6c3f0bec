// Argument checks shared by the C-ABI layers: dtypes, alignment, and the
// overlap rules of outputs.
#pragma once

#include <stdint.h>

#include "../../include/addln.h"
#include "launch.h"

namespace addln {
namespace abi {

inline int elem_bytes(int dtype) { return dtype == ADDLN_FP32 ? 4 : 2; }

inline bool valid_dtype(int dtype) {
  return dtype == ADDLN_FP32 || dtype == ADDLN_FP16 || dtype == ADDLN_BF16;
}

inline int64_t max_hidden(int dtype) {
  return dtype == ADDLN_FP32 ? addln::kMaxHidden32 : addln::kMaxHidden16;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
  bool present;
};
inline Range range_of(const void* p, int64_t bytes) {
  Range r;
  r.present = p != nullptr && bytes > 0;
  r.lo = reinterpret_cast<uintptr_t>(p);
  r.hi = r.lo + static_cast<uintptr_t>(bytes);
  return r;
}
inline bool overlap(const Range& a, const Range& b) {
  return a.present && b.present && a.lo < b.hi && b.lo < a.hi;
}
// An output may coincide exactly with an input of the same size (in place).
inline bool bad_pair(const Range& out, const Range& in, bool in_place_ok) {
  if (!overlap(out, in)) return false;
  return !(in_place_ok && out.lo == in.lo && out.hi == in.hi);
}

}  // namespace abi
}  // namespace addln
