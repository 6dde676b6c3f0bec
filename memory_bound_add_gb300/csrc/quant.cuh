// Shared by the 8-bit kernels (quant.cu, dequant.cu): the formats, and rows of
// bytes that may begin anywhere.
#pragma once

#include "../../include/addln_quant.h"
#include "block.cuh"
#include "quant.h"

namespace addln {
namespace blk {

// VE neighbouring columns of a row of bytes, as one word.
template <int VE>
struct Bytes;
template <>
struct Bytes<8> {
  using W = uint64_t;
};
template <>
struct Bytes<4> {
  using W = uint32_t;
};

__device__ __forceinline__ int q_top(int format) {
  return format == ADDLN_Q_E4M3 ? 448 : format == ADDLN_Q_E5M2 ? 57344 : 127;
}

// Four values to the four bytes of a word.  The fp8 conversions and the integer
// one round to nearest, ties to even, and cut; a NaN becomes the format's NaN,
// as an integer 0.  kQWhole: integers of values that are at most 127 by their
// scale; a sum with 1.5 2^23 leaves them rounded in its low byte (2.5 instructions
// an element less).
constexpr int kQWhole = 8;
template <int FMT>
__device__ __forceinline__ uint32_t to_q(float2 a, float2 b) {
  // the low bytes of four words
  auto bytes = [](uint32_t p, uint32_t q, uint32_t r, uint32_t s) {
    return __byte_perm(__byte_perm(p, q, 0x0040), __byte_perm(r, s, 0x0040), 0x5410);
  };
  if constexpr (FMT == ADDLN_Q_E4M3 || FMT == ADDLN_Q_E5M2) {
    uint16_t lo, hi;
    if constexpr (FMT == ADDLN_Q_E4M3) {
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
    } else {
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
      asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
    }
    return lo | static_cast<uint32_t>(hi) << 16;
  } else if constexpr (FMT == kQWhole) {
    const float2 big = dup2(12582912.f);
    a = add2(a, big), b = add2(b, big);
    return bytes(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  } else {
    auto whole = [](float v) { return static_cast<uint32_t>(min(max(__float2int_rn(v), -127), 127)); };
    return bytes(whole(a.x), whole(a.y), whole(b.x), whole(b.y));
  }
}

// Four bytes of a word to what they are without their scale.  Integers: a byte
// with its sign turned becomes the low mantissa byte of 2^23, which is then taken
// off again (a conversion has a quarter of the rate).
template <int FMT>
__device__ __forceinline__ void from_q(uint32_t w, float2& a, float2& b) {
  if constexpr (FMT == ADDLN_Q_INT8) {
    w ^= 0x80808080u;
    auto at = [&](int e) { return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + e)); };
    const float2 off = dup2(-8388736.f);
    a = add2(make_float2(at(0), at(1)), off), b = add2(make_float2(at(2), at(3)), off);
  } else {
    uint32_t u, v;
    const uint16_t lo = static_cast<uint16_t>(w), hi = static_cast<uint16_t>(w >> 16);
    if constexpr (FMT == ADDLN_Q_E4M3) {
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(u) : "h"(lo));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"(hi));
    } else {
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(u) : "h"(lo));
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(v) : "h"(hi));
    }
    a = Io<kF16>::w2f(u), b = Io<kF16>::w2f(v);
  }
}

template <typename W>
__device__ __forceinline__ void st_stream_word(char* p, W v) {
  if constexpr (sizeof(W) == 8)
    asm volatile("st.global.cs.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
  else
    asm volatile("st.global.cs.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Writer (block.cuh) for rows of bytes: a row's groups of VE bytes in the order
// of k.  Rows that begin off the words' borders (shifted) are written in whole words
// too, each of a group's begin and its neighbour's end.
template <int VE, int NV, int MODE>
struct ByteWriter {
  using W = typename Bytes<VE>::W;
  W prev;  // the last group, of lane 31

  __device__ __forceinline__ void put(const Cols<VE, NV>& cs, void* base, int64_t off, int k, W v, int site, int64_t extent) {
    off += k * cs.kStep;
    char* p = static_cast<char*>(base) + off;
    if constexpr (MODE == kAligned) {
      if (cs.ok(k) && ADDLN_IN(site, off, VE, extent)) st_stream_word<W>(p, v);
    } else if constexpr (MODE == kEdged) {
      const int lo = k == 0 ? cs.low : 0, hi = cs.valid(k);
      if (lo == 0 && hi == VE) {
        if (ADDLN_IN(site, off, VE, extent)) st_stream_word<W>(p, v);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (e >= lo && e < hi && ADDLN_IN(site, off + e, 1, extent)) p[e] = static_cast<char>(v >> (8 * e));
      }
    } else {
      const int lane = threadIdx.x & 31;
      const int s = static_cast<int>(reinterpret_cast<uintptr_t>(p) & (VE - 1));  // the same for the warp
      W w = v;
      int lo = 0, hi = cs.valid(k);
      if (s != 0) {
        const W send = lane == 31 && k > 0 ? prev : v;
        const W n = __shfl_sync(0xffffffffu, send, (lane + 31) & 31);
        prev = v;
        w = (n >> (8 * (VE - s))) | (v << (8 * s));
        const bool has = k > 0 || lane > 0;
        const int before = min(max(cs.left - (k * cs.kStep - VE), 0), VE) - (VE - s);
        lo = has ? 0 : s;
        hi = hi > 0 ? s + min(hi, VE - s) : has ? max(before, 0) : 0;
        p -= s;
        off -= s;
      }
      if (lo == 0 && hi == VE) {
        if (ADDLN_IN(site, off, VE, extent)) st_stream_word<W>(p, w);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (e >= lo && e < hi && ADDLN_IN(site, off + e, 1, extent)) p[e] = static_cast<char>(w >> (8 * e));
      }
      // nobody follows the warp's last group: its own end
      if (s != 0 && k == NV - 1 && lane == 31) {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (e >= VE - s && e < cs.valid(k) && ADDLN_IN(site, off + s + e, 1, extent)) p[s + e] = static_cast<char>(v >> (8 * e));
      }
    }
  }
};

}  // namespace blk
}  // namespace addln
