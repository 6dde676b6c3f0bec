// out = q * scale, rows of 8 bits read back.  Bound by memory: 1 + S bytes an
// element.
#include "quant.cuh"

namespace addln {
namespace blk {

constexpr int kDequantThreads = 256;

// A warp's row of words from offset `at` of q on, this lane's first; n: bytes of
// the row from there on.  Rows that begin off the words' borders (SH): each lane
// reads the word that its bytes begin in and takes the rest from the next lane's;
// words that reach over the tensor's own ends are put together from their bytes.
template <int VE, bool SH>
__device__ __forceinline__ typename Bytes<VE>::W load_word(const void* q, int64_t at, int n, int64_t extent) {
  using W = typename Bytes<VE>::W;
  const char* p = static_cast<const char*>(q) + at;
  if constexpr (!SH) {
    return n > 0 && ADDLN_IN(820, at, VE, extent) ? __ldcs(reinterpret_cast<const W*>(p)) : 0;
  } else {
    const int s = static_cast<int>(reinterpret_cast<uintptr_t>(p) & (VE - 1));  // the same for the warp
    auto word = [&](int64_t o) {
      const char* a = static_cast<const char*>(q) + o;
      if (o >= 0 && o + VE <= extent) return __ldg(reinterpret_cast<const W*>(a));
      W w = 0;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (o + e >= 0 && o + e < extent) w |= static_cast<W>(__ldg(reinterpret_cast<const uint8_t*>(a) + e)) << (8 * e);
      return w;
    };
    const W lo = n + s > 0 ? word(at - s) : 0;  // of a lane past the end: its neighbour's last bytes
    if (s == 0) return lo;
    W hi = __shfl_down_sync(0xffffffffu, lo, 1);
    if ((threadIdx.x & 31) == 31) hi = n > VE - s ? word(at - s + VE) : 0;
    return (lo >> (8 * s)) | (hi << (8 * (VE - s)));
  }
}

// A scale from its bits.  2^(e - 127) as bits is e << 23, but for 2^-127 and NaN.
__device__ __forceinline__ float scale_from(uint32_t e, bool pow2) {
  return __uint_as_float(!pow2 ? e : e == 255 ? 0x7fffffffu : e == 0 ? 0x400000u : e << 23);
}
__device__ __forceinline__ uint32_t load_scale(const DequantArgs& p, int64_t i, bool pow2) {
  if (!ADDLN_IN(822, i, 1, p.scales)) return 0;
  return pow2 ? __ldg(static_cast<const uint8_t*>(p.s.scale) + i) : __ldg(static_cast<const uint32_t*>(p.s.scale) + i);
}

// Tensors that begin on such borders are one run of vectors of 32 bytes of out, one
// a thread: 32-byte stores, and 16 bytes of q a load (8 for fp32).  32768x8192 from
// e4m3 to bf16 110 us (7.3 TB/s) where warps of rows, 8 bytes a load, take 183; four
// vectors a thread are no faster there and slower below (4096x768 3.9 us, one 2.9).
//
// RAGGED: rows are not whole vectors, so that a row's or a group's end may lie in
// one.  Its elements then have up to three scales (the rest of a group, a row's
// short last one, the next row's first): those before b1, those before b2, the
// others.
template <int DT, int FMT, bool RAGGED>
__global__ void __launch_bounds__(kDequantThreads) k_dequant_run(const __grid_constant__ DequantArgs p) {
  using IO = Io<DT>;
  constexpr int S = IO::kBytes, VW = 32 / S, N = VW / 4;  // columns and words of q a vector
  pdl_trigger();
  pdl_wait();
  const uint64_t e0 = static_cast<uint64_t>(blockIdx.x) * (kDequantThreads * VW);
  const uint64_t elements = static_cast<uint64_t>(p.rows) * p.H;
  const uint64_t row0 = (e0 >> 32) ? e0 / static_cast<uint32_t>(p.H) : static_cast<uint32_t>(e0) / static_cast<uint32_t>(p.H);
  const uint64_t at = e0 + threadIdx.x * VW;
  if (at >= elements) return;
  // l is below 2^16: the product's upper half with 2^32 / H rounded up is the
  // exact quotient
  const uint32_t l = static_cast<uint32_t>(e0 - row0 * p.H) + threadIdx.x * VW;
  const uint32_t r = __umulhi(l, p.reciprocal);
  int c = static_cast<int>(l - r * p.H);
  int64_t row = static_cast<int64_t>(row0 + r);
  const bool pow2 = p.s.scaling == ADDLN_SCALE_POW2;
  const int shift = p.s.lanes_shift;
  auto scale = [&] {
    return row < p.rows ? load_scale(p, row * p.scale_row + (c >> shift) * p.scale_group, pow2) : 0;
  };
  const bool tail = RAGGED && at + VW > elements;
  const uint8_t* q = static_cast<const uint8_t*>(p.q) + at;
  uint32_t w[N] = {};
  if (tail) {
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (at + e < elements && ADDLN_IN(825, at + e, 1, elements)) w[e / 4] |= static_cast<uint32_t>(__ldg(q + e)) << (8 * (e % 4));
  } else if (ADDLN_IN(825, at, VW, elements)) {
    if constexpr (N == 4) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(q));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(q));
      w[0] = u.x, w[1] = u.y;
    }
  }
  const uint32_t s0 = scale();
  uint32_t s1 = 0, s2 = 0;
  int b1 = VW, b2 = VW;
  if constexpr (RAGGED) {
    auto left = [&] { return min(p.H - c, (((c >> shift) + 1) << shift) - c); };  // of the group
    auto next = [&](int n) {
      c += n;
      if (c == p.H) c = 0, ++row;
    };
    int n = left();
    if (n < VW) {
      b1 = n;
      next(n);
      s1 = scale();
      n = left();
      if (b1 + n < VW) {
        b2 = b1 + n;
        next(n);
        s2 = scale();
      }
    }
  }
  const float a = scale_from(s0, pow2);
  float2 f[VW / 2];
#pragma unroll
  for (int i = 0; i < N; ++i) from_q<FMT>(w[i], f[2 * i], f[2 * i + 1]);
  if (!RAGGED || b1 == VW) {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) f[i] = mul2(f[i], dup2(a));
  } else {
    const float b = scale_from(s1, pow2), d = scale_from(s2, pow2);
    auto of = [&](int e) { return e < b1 ? a : e < b2 ? b : d; };
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) f[i] = mul2(f[i], make_float2(of(2 * i), of(2 * i + 1)));
  }
  const uint4 lo = IO::from_pairs(f), hi = IO::from_pairs(f + VW / 4);
  char* out = static_cast<char*>(p.out) + at * S;
  if (tail) {
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (at + e < elements && ADDLN_IN(826, (at + e) * S, S, elements * S))
        store_element<S>(out + e * S, e < VW / 2 ? lo : hi, e % (VW / 2));
  } else if (ADDLN_IN(826, at * S, 32, elements * S)) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                 "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                 : "memory");
  }
}

// Other rows: a warp takes 32 VE columns of R rows, whose loads are all in flight.
constexpr int R = 4;

template <int DT, int FMT, bool SH>
__global__ void __launch_bounds__(kDequantThreads) k_dequant(const __grid_constant__ DequantArgs p) {
  using IO = Io<DT>;
  constexpr int S = IO::kBytes, VE = IO::kVec, Q = VE / 2;
  using W = typename Bytes<VE>::W;
  pdl_trigger();
  pdl_wait();
  const uint32_t warp = blockIdx.x * (kDequantThreads / 32) + (threadIdx.x >> 5);
  const uint32_t block = warp / static_cast<uint32_t>(p.pieces);
  const int piece = static_cast<int>(warp - block * static_cast<uint32_t>(p.pieces));
  const int64_t row0 = static_cast<int64_t>(block) * R;
  if (row0 >= p.rows) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(R), p.rows - row0));
  const int64_t elements = p.rows * static_cast<int64_t>(p.H);
  Cols<VE, 1> cs;
  cs.c0 = piece * (32 * VE) + (threadIdx.x & 31) * VE;
  cs.left = p.H - cs.c0;
  const int64_t at0 = row0 * p.H + cs.c0;
  const bool pow2 = p.s.scaling == ADDLN_SCALE_POW2;
  const int64_t s0 = row0 * p.scale_row + (cs.c0 >> p.s.lanes_shift) * p.scale_group;
  W w[R];
  uint32_t s[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    w[j] = 0, s[j] = 0;
    if (j < n) {
      w[j] = load_word<VE, SH>(p.q, at0 + static_cast<int64_t>(j) * p.H, cs.left, elements);
      if (cs.left > 0) s[j] = load_scale(p, s0 + j * p.scale_row, pow2);
    }
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (j >= n) break;
    const float2 sc = dup2(scale_from(s[j], pow2));
    float2 v[Q];
    from_q<FMT>(static_cast<uint32_t>(w[j]), v[0], v[1]);
    if constexpr (VE == 8) from_q<FMT>(static_cast<uint32_t>(w[j] >> 32), v[2], v[3]);
#pragma unroll
    for (int i = 0; i < Q; ++i) v[i] = mul2(v[i], sc);
    Writer<DT, 1, SH> out;
    out.put(cs, p.out, (at0 + static_cast<int64_t>(j) * p.H) * S, 0, IO::from_pairs(v), 824, elements * S);
  }
}

namespace {
using DequantKernel = void (*)(DequantArgs);
enum Run { kNone, kWhole, kRagged };  // of vectors
template <int DT, int FMT>
DequantKernel pick(Run run, bool aligned) {
  return run == kWhole    ? &k_dequant_run<DT, FMT, false>
         : run == kRagged ? &k_dequant_run<DT, FMT, true>
         : aligned        ? &k_dequant<DT, FMT, false>
                          : &k_dequant<DT, FMT, true>;
}
template <int DT>
DequantKernel pick(int format, Run run, bool aligned) {
  return format == ADDLN_Q_E4M3   ? pick<DT, ADDLN_Q_E4M3>(run, aligned)
         : format == ADDLN_Q_E5M2 ? pick<DT, ADDLN_Q_E5M2>(run, aligned)
                                  : pick<DT, ADDLN_Q_INT8>(run, aligned);
}
}  // namespace
}  // namespace blk

int launch_dequant(int dtype, bool aligned, const DequantArgs& args, const LaunchCtx& c) {
  using namespace blk;
  DequantArgs p = args;
  const int step = dtype == kF32 ? 128 : 256, VW = step / 16;
  p.pieces = (p.H + step - 1) / step;
  const bool group = p.s.scaling == ADDLN_SCALE_GROUP || p.s.scaling == ADDLN_SCALE_POW2;
  p.scale_row = p.s.scaling == ADDLN_SCALE_TENSOR ? 0 : p.s.group_major ? 1 : p.s.groups;
  p.scale_group = !group ? 0 : p.s.group_major ? p.rows : 1;
  p.scales = p.s.scaling == ADDLN_SCALE_TENSOR ? 1 : p.rows * p.s.groups;
  if (!group) p.s.lanes_shift = 24;  // one group, longer than any row
  const bool begins = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0 && (reinterpret_cast<uintptr_t>(p.q) & (VW - 1)) == 0;
  // (rows shorter than a group's 32 columns: more than three scales a vector)
  const Run run = !begins || p.H < 32 ? kNone : p.H % VW == 0 ? kWhole : kRagged;
  const DequantKernel k = dtype == kF32   ? pick<kF32>(p.s.format, run, aligned)
                          : dtype == kF16 ? pick<kF16>(p.s.format, run, aligned)
                                          : pick<kBF16>(p.s.format, run, aligned);
  int64_t units = (p.rows + R - 1) / R * p.pieces, per = kDequantThreads / 32;  // warps
  if (run != kNone) {
    p.reciprocal = static_cast<uint32_t>(((uint64_t{1} << 32) + p.H - 1) / p.H);
    units = (p.rows * p.H + VW - 1) / VW, per = kDequantThreads;
  }
  const int64_t ctas = (units + per - 1) / per;
  if (ctas > (run != kNone ? 0x7fffffff : 1 << 28)) return ADDLN_ERR_SHAPE;  // (a warp's number has 32 bits)
  const cudaError_t e = launch_kernel(k, dim3(static_cast<unsigned>(ctas)), dim3(kDequantThreads), 0, c.stream, c.pdl, p);
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_dequant)

}  // namespace addln
