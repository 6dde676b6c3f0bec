// out = q * scale, rows of 8 bits read back.  Bound by memory: 1 + S bytes an
// element.
#include "quant.cuh"

namespace addln {
namespace blk {

constexpr int kDequantThreads = 256;
constexpr int kPieces = 4;  // pieces of a row that a warp has in flight

// VE bytes from offset `at` of q on, which may be any; what lies past `n` of
// them is 0 and not read.
template <int VE, bool SH>
__device__ __forceinline__ typename Bytes<VE>::W load_bytes(const void* q, int64_t at, int n, int64_t extent) {
  using W = typename Bytes<VE>::W;
  const char* p = static_cast<const char*>(q) + at;
  if constexpr (!SH) {
    return n > 0 && ADDLN_IN(820, at, VE, extent) ? __ldcs(reinterpret_cast<const W*>(p)) : 0;
  } else {
    W w = 0;
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (e < n && ADDLN_IN(821, at + e, 1, extent))
        w |= static_cast<W>(__ldg(reinterpret_cast<const uint8_t*>(p) + e)) << (8 * e);
    return w;
  }
}

// A warp takes pieces of 32 VE columns of a row, kPieces at a time.
template <int DT, bool SH>
__global__ void __launch_bounds__(kDequantThreads) k_dequant(const __grid_constant__ DequantArgs p, int pieces) {
  using IO = Io<DT>;
  constexpr int S = IO::kBytes, VE = IO::kVec, Q = VE / 2;
  using W = typename Bytes<VE>::W;
  using C = Cols<VE, 1>;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * (kDequantThreads / 32) + (threadIdx.x >> 5)) * kPieces;
  const int64_t elements = p.rows * static_cast<int64_t>(p.H);
  int64_t row = u0 / pieces;
  int piece = static_cast<int>(u0 - row * pieces);
  const int format = p.s.format, scaling = p.s.scaling;
  W w[kPieces];
  float s[kPieces];
  int64_t rows[kPieces];
  int at[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    rows[j] = row, at[j] = piece * C::kStep;
    const int c = at[j] + lane * VE;
    w[j] = 0, s[j] = 0.f;
    if (row < p.rows && c < p.H) {
      w[j] = load_bytes<VE, SH>(p.q, row * p.H + c, p.H - c, elements);
      if (scaling == ADDLN_SCALE_TENSOR || scaling == ADDLN_SCALE_ROW) {
        const int64_t i = scaling == ADDLN_SCALE_ROW ? row : 0;
        if (ADDLN_IN(822, 4 * i, 4, scaling == ADDLN_SCALE_ROW ? 4 * p.rows : 4)) s[j] = __ldg(static_cast<const float*>(p.s.scale) + i);
      } else {
        const int g = c >> p.s.lanes_shift;
        const int64_t i = p.s.group_major ? g * p.rows + row : row * p.s.groups + g;
        if (ADDLN_IN(823, i, 1, p.rows * p.s.groups)) {
          if (scaling == ADDLN_SCALE_GROUP) {
            s[j] = __ldg(static_cast<const float*>(p.s.scale) + i);
          } else {
            // 2^(e - 127): as bits e << 23, but for 2^-127 and NaN
            const uint32_t e = __ldg(static_cast<const uint8_t*>(p.s.scale) + i);
            s[j] = __uint_as_float(e == 255 ? 0x7fffffffu : e == 0 ? 0x400000u : e << 23);
          }
        }
      }
    }
    if (++piece == pieces) piece = 0, ++row;
  }
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    if (rows[j] >= p.rows) break;
    C cs;
    cs.c0 = at[j] + lane * VE;
    cs.left = p.H - cs.c0;
    float2 v[Q];
    from_q(format, static_cast<uint32_t>(w[j]), v[0], v[1]);
    if constexpr (VE == 8) from_q(format, static_cast<uint32_t>(w[j] >> 32), v[2], v[3]);
#pragma unroll
    for (int i = 0; i < Q; ++i) v[i] = mul2(v[i], dup2(s[j]));
    Writer<DT, 1, SH> out;
    out.put(cs, p.out, (rows[j] * p.H + cs.c0) * S, 0, IO::from_pairs(v), 824, elements * S);
  }
}

}  // namespace blk

int launch_dequant(int dtype, bool aligned, const DequantArgs& p, const LaunchCtx& c) {
  using namespace blk;
  void (*k)(DequantArgs, int) = dtype == kF32   ? (aligned ? &k_dequant<kF32, false> : &k_dequant<kF32, true>)
                                : dtype == kF16 ? (aligned ? &k_dequant<kF16, false> : &k_dequant<kF16, true>)
                                                : (aligned ? &k_dequant<kBF16, false> : &k_dequant<kBF16, true>);
  const int step = dtype == kF32 ? 128 : 256, pieces = (p.H + step - 1) / step;
  const int64_t per = kDequantThreads / 32 * kPieces, ctas = (p.rows * pieces + per - 1) / per;
  if (ctas > 0x7fffffff) return ADDLN_ERR_SHAPE;
  const cudaError_t e = launch_kernel(k, dim3(static_cast<unsigned>(ctas)), dim3(kDequantThreads), 0, c.stream, c.pdl, p, pieces);
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_dequant)

}  // namespace addln
