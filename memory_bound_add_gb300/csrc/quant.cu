// Residual sum, norm and an output in 8 bits with its scales, in one pass:
//   h = x + r,  y = norm(h),  q = round(y / scale)
// x and r are read once, h, q and the scales written once; statistics and
// largest values are of values in registers.
#include <type_traits>

#include "quant.cuh"

namespace addln {
namespace blk {

// Largest |v|; a NaN stays one.
__device__ __forceinline__ float abs_max(float m, float2 v) {
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(v.x), "f"(v.y));
  return m;
}
// Over a warp's lanes, of numbers that are not negative: their bits have the same
// order, with infinity and then NaN above all.
__device__ __forceinline__ float warp_max(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// Largest over the walker, and with SUM the sum of q, in every thread, in one
// exchange.
template <bool SUM, bool SIDES>
__device__ __forceinline__ void walker_max(Exchange<SIDES>& ex, float& m, float& q) {
  m = warp_max(m);
  if constexpr (SUM) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
  }
  if (ex.w.warps == 1) return;
  const float4* b = ex(make_float4(m, q, 0.f, 0.f));
  const int width = ex.w.width;
  m = 0.f, q = 0.f;
  for (int i = (threadIdx.x & 31) & (width - 1); i < ex.w.warps; i += 32) m = max_nan(m, b[i].x), q += b[i].y;
  m = warp_max(m);
  if constexpr (SUM)
    for (int off = 1; off < width; off <<= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
}

// A scale and its reciprocal, of the largest |y|.
struct Scale {
  float s, inv;
};

__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The quotient amax / top is taken as a product with 1 / top, and
// y / scale later as one with the scale's reciprocal, which is good to a unit in
// the last place: y's position between two values of 8 bits moves by some 2^-22
// of itself.
__device__ __forceinline__ Scale scale_of(float amax, float inv_top) {
  // NaN for NaN and infinities
  const float s = max_nan(amax * inv_top, 0x1p-126f) + (amax - amax);
  return {s, reciprocal(s)};
}

// The least power of two 2^e with amax <= top 2^e: top = m 2^t, and amax's
// exponent goes up by one where its mantissa is above m's.
__device__ __forceinline__ Scale pow2_of(float largest, int format) {
  const float nan = __uint_as_float(0x7fffffffu);
  const uint32_t amax = __float_as_uint(largest);
  if (amax >= 0x7f800000u) return {nan, nan};
  const uint32_t mantissa = format == ADDLN_Q_INT8 ? 0x7e0000u : 0x600000u;
  const int t = format == ADDLN_Q_E4M3 ? 8 : format == ADDLN_Q_E5M2 ? 15 : 6;
  const int e = max(static_cast<int>((amax + (0x7fffffu - mantissa)) >> 23) - t, 1);  // biased
  return {__uint_as_float(static_cast<uint32_t>(e) << 23), __uint_as_float(static_cast<uint32_t>(254 - e) << 23)};
}

// Without FULL gamma is kept times this, which goes back with 1 / rms: values next to
// the type's lowest, whose 1 / rms is 0, then stay finite (and so become 0).  In return
// rows whose |x gamma| is below 2^-110 lose digits of their scale to fp32's least numbers.
constexpr float kGammaScale = 0x1p-16f;

// gamma and, with FULL, beta: in registers or in shared memory, as in
// block_fwd.cu.
__host__ __device__ constexpr bool quant_in_registers(int columns, bool full, int mode) {
  return columns <= 8 || !(full || mode == kShifted);
}

template <int VE, int NV, bool FULL, int MODE>
struct QuantParams {
  static constexpr bool kRegs = quant_in_registers(NV * VE, FULL, MODE);
  static constexpr int P = kRegs ? NV * VE / 2 : 1, N = FULL ? 2 : 1;
  float2 r[N][P];
  Kept<VE, NV> kept;

  __device__ __forceinline__ void get(int i, int k, float2 (&v)[VE / 2]) const {
    if constexpr (kRegs) {
#pragma unroll
      for (int j = 0; j < VE / 2; ++j) v[j] = r[i][k * VE / 2 + j];
    } else {
      kept.get(i, k, v);
    }
  }
  // vector i, group k; zeros past the slice, whose slots would reach the row's
  // largest value by way of the beta
  __device__ __forceinline__ void load(const QuantArgs& p, int i, const Cols<VE, NV>& cs, int k) {
    const float* from = i == 0 ? p.gamma : p.beta;
    float v[VE];
    load_params<VE, MODE>(from, cs.col(k), cs.end(), 0.f, v, 800);
    if constexpr (!FULL) {
#pragma unroll
      for (int e = 0; e < VE; ++e) v[e] *= kGammaScale;
    }
    if constexpr (kRegs) {
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) r[i][k * VE / 2 + e] = make_float2(v[2 * e], v[2 * e + 1]);
    } else {
      kept.put(i, k, v);
    }
  }
};

// FULL: a layer norm or a beta.  MODE: how rows lie.
//
// The call moves 3 S + 1 bytes an element.  32768x8192 bf16 rms to e4m3, groups of 128:
// 293 us (6.45 TB/s, 0.96 of a copy); 8192x4096 a scale a row 38.3 (0.91), 65536x768
// powers of two 54.9 (0.96); 2048x4096 fp16 10.7 (0.82: 3.4 rows a walker).  19 to 21
// instructions an element use half of the issue slots; 96 registers (five CTAs an SM)
// and half the columns a thread measured the same or slower.  Layer norms use 45% of the
// issue slots too: they are bound by latency (two passes over the registers and two
// exchanges a row) at 16 warps an SM: 8192x4096 to int8 49.3 us (0.71), 4097x1001 9.9
// (0.43); with several CTAs a row 4096x20000 to e4m3, a scale a row, 230 (0.37).  Groups
// of odd widths take shifted rows, 50 to 60 instructions an element: 8192x5001 91 us
// (0.48).
//
// (128 registers: see k_drop_fwd.)
template <int DT, int NV, bool FULL, int MODE>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__((NV > 0 ? 128 : 0))
    k_norm_quant(const __grid_constant__ QuantArgs p) {
  using IO = Io<DT>;
  constexpr bool SH = MODE == kShifted;
  constexpr int S = IO::kBytes, VE = IO::kVec, Q = VE / 2;
  constexpr int P = NV * Q;
  using R = Ring<DT, NV, 2, MODE>;
  using W = typename Bytes<VE>::W;
  extern __shared__ __align__(128) unsigned char smem[];
  if (p.w.C > 1) cluster_started();
  const int slots = p.slots;
  const int lane = threadIdx.x & 31;
  const int side = (threadIdx.x >> 5) / p.w.cta_warps, warp = (threadIdx.x >> 5) - side * p.w.cta_warps;
  const int rank = p.w.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.w.C);
  const int64_t stride = static_cast<int64_t>(gridDim.x / p.w.C) * p.w.rows_per_cta;
  int64_t row = first_row<MODE>(blockIdx.x / p.w.C, p.w.rows_per_cta, side);
  const int col0 = rank * p.w.slice;
  const int64_t elements = p.rows * static_cast<int64_t>(p.H), extent = elements * S;
  Exchange<!quant_in_registers(NV * VE, FULL, MODE)> ex{p.w, p.sums_at + side * 2 * p.w.warps * 16, 0};
  const bool leader = rank == 0 && lane == 0 && warp == 0;
  const bool has_r = p.r != nullptr, has_norm = p.norm != ADDLN_NORM_NONE;
  R ring;
  ring.base = smem_addr(smem) + (threadIdx.x >> 5) * p.ring_slots * R::kSlot + lane * 16;
  Cols<VE, NV> cs;
  if constexpr (MODE == kEdged)
    cs.init_edged(warp, col0, p.w.slice, p.H, static_cast<int>(row * p.H & (VE - 1)));
  else
    cs.init(warp, col0, min(p.w.slice, p.H - col0));
  auto fetch = [&](int slot, int64_t r) {
    if (r < p.rows) {
      const int64_t at = (r * p.H + cs.c0) * S;
      ring.template fetch<0>(cs, slot, p.x, at, 811, extent);
      if (has_r) ring.template fetch<1>(cs, slot, p.r, at, 803, extent);
    }
    ring.commit();
  };
  // where a walker has few rows
  if (p.rows <= 8 * stride)
    for (int s = 0; s < slots && row + s * stride < p.rows; ++s) {
      const int64_t at = ((row + s * stride) * p.H + cs.c0) * S;
      prefetch_row<S>(p.x, at, cs, 810, extent);
      prefetch_row<S>(p.r, at, cs, 810, extent);
    }
  pdl_trigger();
  pdl_wait();
  for (int s = 0; s < slots; ++s) fetch(s, row + s * stride);
  QuantParams<VE, NV, FULL, MODE> par;
  constexpr bool kRegs = QuantParams<VE, NV, FULL, MODE>::kRegs;
  if constexpr (!kRegs)
    par.kept.base = smem_addr(smem) + p.kept_at + warp * Kept<VE, NV>::template bytes<FULL ? 2 : 1>() + lane * 16;
  if constexpr (kRegs) {
#pragma unroll
    for (int i = 0; i < par.N; ++i)
#pragma unroll
      for (int k = 0; k < NV; ++k) par.load(p, i, cs, k);
  } else {
    // the rows side by side share the work
    for (int t = side; t < par.N * NV; t += p.w.rows_per_cta) par.load(p, t / NV, cs, t % NV);
    __syncthreads();
  }
  const int format = p.s.format, scaling = p.s.scaling;
  const float inv_top = 1.f / static_cast<float>(q_top(format));
  float given = 0.f;
  if (scaling == ADDLN_SCALE_TENSOR && ADDLN_IN(804, 0, 4, 4)) given = reciprocal(__ldg(static_cast<const float*>(p.s.scale)));
  if (p.w.C > 1) cluster_wait_started();

  for (int slot = 0; row < p.rows; row += stride, slot = slot + 1 == slots ? 0 : slot + 1) {
    if (slots == 1) ring.template wait<0>(); else ring.template wait<1>();
    ring.meet();
    const int64_t at = row * p.H + cs.c0, off = at * S;
    const int sx = SH ? low4(p.x, off) : 0, sr = SH && has_r ? low4(p.r, off) : 0;
    float2 v[P];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      IO::to_pairs(ring.take(slot, 0, k, sx), v + k * Q);
      if (has_r) {
        float2 r[Q];
        IO::to_pairs(ring.take(slot, 1, k, sr), r);
#pragma unroll
        for (int i = 0; i < Q; ++i) v[k * Q + i] = add2(v[k * Q + i], r[i]);
      }
    }
    // columns before the row have the end of another; those past it are zeros
    if constexpr (MODE == kEdged) cs.clear_low(v);
    ring.meet();
    fetch(slot, row + slots * stride);  // the slot has been read
    if (p.h != nullptr) {
      Writer<DT, NV, MODE> out;
#pragma unroll
      for (int k = 0; k < NV; ++k) out.put(cs, p.h, off, k, IO::from_pairs(v + k * Q), 805, extent);
    }
    // y = v f from here on: an rms norm's 1 / rms is left out of v, and goes
    // into the scale
    float f = 1.f, m = 0.f;
    if (has_norm) {
      RowStat st{0.f, 0.f, 0.f};
      if constexpr (FULL) {
        st = row_norm<VE, NV, FULL>(ex, v, cs, p.norm == ADDLN_NORM_LAYER, p.inv_h, p.eps);
        const float2 negm = dup2(-st.m), r2 = dup2(st.M2);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float2 g[Q], e[Q];
          par.get(0, k, g);
          par.get(1, k, e);
#pragma unroll
          for (int i = 0; i < Q; ++i) v[k * Q + i] = fma2(mul2(add2(v[k * Q + i], negm), r2), g[i], e[i]);
        }
      } else {
        float2 q[2] = {dup2(0.f), dup2(0.f)};
#pragma unroll
        for (int j = 0; j < P; ++j) q[j & 1] = fma2(v[j], v[j], q[j & 1]);
        q[0] = add2(q[0], q[1]);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float2 g[Q];
          par.get(0, k, g);
#pragma unroll
          for (int i = 0; i < Q; ++i) v[k * Q + i] = mul2(v[k * Q + i], g[i]);
        }
        float sum = q[0].x + q[0].y;
        if (scaling == ADDLN_SCALE_ROW) {
#pragma unroll
          for (int j = 0; j < P; ++j) m = abs_max(m, v[j]);
          walker_max<true>(ex, m, sum);
        } else {
          sum = walker_sum(ex, sum);
        }
        st.M2 = row_rstd(sum, p.inv_h, p.eps);
        f = st.M2 * (1.f / kGammaScale);
      }
      if (leader && ADDLN_IN(806, 4 * row, 4, 4 * p.rows)) {
        if (p.rstd) p.rstd[row] = st.M2;
        if (FULL && p.mean) p.mean[row] = st.mean;
      }
    }
    float inv[NV];  // 1 / scale of group k
    if (scaling == ADDLN_SCALE_ROW || scaling == ADDLN_SCALE_TENSOR) {
      float one = given;
      if (scaling == ADDLN_SCALE_ROW) {
        if (FULL || !has_norm) {
#pragma unroll
          for (int j = 0; j < P; ++j) m = abs_max(m, v[j]);
          float unused = 0.f;
          walker_max<false>(ex, m, unused);
        }
        const Scale sc = scale_of(m * f, inv_top);
        if (leader && ADDLN_IN(807, 4 * row, 4, 4 * p.rows)) static_cast<float*>(p.s.scale)[row] = sc.s;
        one = sc.inv;
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) inv[k] = one;
    } else {
      // A lane's NV largest values, over the 4 to 32 lanes of a group.  The first
      // two steps halve the values that a lane carries, so that lane l of four ends
      // with value k = 2 (l & 1) + (l >> 1 & 1) and makes its scale alone, and the
      // scales' reciprocals go back.
      constexpr int N = NV == 3 ? 4 : NV;
      const int lanes = (1 << p.s.lanes_shift) / VE;
      float x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        x[k] = 0.f;
        if (k < NV)
#pragma unroll
          for (int i = 0; i < Q; ++i) x[k] = abs_max(x[k], v[k * Q + i]);
      }
      int o = 1;
      if constexpr (N >= 2) {
        const bool up = lane & 1;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float keep = up ? x[i + N / 2] : x[i], give = up ? x[i] : x[i + N / 2];
          x[i] = max_nan(keep, __shfl_xor_sync(0xffffffffu, give, 1));
        }
        o = 2;
      }
      if constexpr (N == 4) {
        const bool up = lane & 2;
        const float keep = up ? x[1] : x[0], give = up ? x[0] : x[1];
        x[0] = max_nan(keep, __shfl_xor_sync(0xffffffffu, give, 2));
        o = 4;
      }
      for (; o < lanes; o <<= 1) x[0] = max_nan(x[0], __shfl_xor_sync(0xffffffffu, x[0], o));
      const bool pow2 = scaling == ADDLN_SCALE_POW2;
      const Scale sc = pow2 ? pow2_of(x[0] * f, format) : scale_of(x[0] * f, inv_top);
      const int l = lane & (lanes - 1);  // of the group
      const int k = N == 1 ? 0 : N == 2 ? l & 1 : (l & 1) * 2 + (l >> 1 & 1);
      if (l < N && k < NV && cs.left + l * VE > k * cs.kStep) {
        const int g = (cs.c0 - l * VE + k * cs.kStep) >> p.s.lanes_shift;
        const int64_t i = p.s.group_major ? g * p.rows + row : row * p.s.groups + g;
        if (ADDLN_IN(808, i, 1, p.rows * p.s.groups)) {
          if (pow2)
            static_cast<uint8_t*>(p.s.scale)[i] = static_cast<uint8_t>(min(__float_as_uint(sc.s) >> 23, 255u));
          else
            static_cast<float*>(p.s.scale)[i] = sc.s;
        }
      }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int from = N == 1 ? 0 : N == 2 ? k : (k >> 1) + (k & 1) * 2;
        inv[k] = __shfl_sync(0xffffffffu, sc.inv, (lane & -N) + from);
      }
    }
    if constexpr (!FULL) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float both = inv[k] * f;
        // beyond fp32's range (values near 0, such as a group of zeros in a row
        // that has others): one after the other
        if (isinf(both)) {
#pragma unroll
          for (int i = 0; i < Q; ++i) v[k * Q + i] = mul2(v[k * Q + i], dup2(f));
        } else {
          inv[k] = both;
        }
      }
    }
    W w[NV];
    auto round = [&](auto fmt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float2 i2 = dup2(inv[k]);
        w[k] = to_q<decltype(fmt)::value>(mul2(v[k * Q], i2), mul2(v[k * Q + 1], i2));
        if constexpr (VE == 8)
          w[k] |= static_cast<W>(to_q<decltype(fmt)::value>(mul2(v[k * Q + 2], i2), mul2(v[k * Q + 3], i2))) << 32;
        // a NaN scale's integers
        if (decltype(fmt)::value == kQWhole && isnan(inv[k])) w[k] = 0;
      }
    };
    if (format == ADDLN_Q_E4M3)
      round(std::integral_constant<int, ADDLN_Q_E4M3>());
    else if (format == ADDLN_Q_E5M2)
      round(std::integral_constant<int, ADDLN_Q_E5M2>());
    else if (scaling != ADDLN_SCALE_TENSOR)
      round(std::integral_constant<int, kQWhole>());
    else
      round(std::integral_constant<int, ADDLN_Q_INT8>());
    ByteWriter<VE, NV, MODE> out;
#pragma unroll
    for (int k = 0; k < NV; ++k) out.put(cs, p.q, at, k, w[k], 809, elements);
  }
  // a CTA's shared memory has to outlive its peers' writes into it
  if (p.w.C > 1) cooperative_groups::this_cluster().sync();
}

// ------------------------------------------------------------------ host
namespace {

struct Choice {
  void (*k)(QuantArgs) = nullptr;
  Spread s;
};

template <int DT, int NV, int MODE>
Choice make(const QuantArgs& p, bool full, int sms) {
  constexpr int VE = Io<DT>::kVec;
  Choice c;
  c.k = full ? &k_norm_quant<DT, NV, true, MODE> : &k_norm_quant<DT, NV, false, MODE>;
  const bool shared = !quant_in_registers(NV * VE, full, MODE);
  // a CTA's slice of a row holds whole groups
  c.s = spread(MODE == kEdged ? p.H + VE - 1 : p.H, VE, NV, p.rows, sms, Ring<DT, NV, 2, MODE>::kSlot,
               !shared ? 0 : full ? Kept<VE, NV>::template bytes<2>() : Kept<VE, NV>::template bytes<1>(), 128);
  return c;
}

template <int DT, int MODE>
Choice choose(const QuantArgs& p, bool full, int sms) {
  constexpr int VE = Io<DT>::kVec;
  switch (groups_a_thread(((MODE == kEdged ? p.H + VE - 1 : p.H) + VE - 1) / VE)) {
    case 1: return make<DT, 1, MODE>(p, full, sms);
    case 2: return make<DT, 2, MODE>(p, full, sms);
    case 3: return make<DT, 3, MODE>(p, full, sms);
    default: return make<DT, 4, MODE>(p, full, sms);
  }
}

template <int DT>
Choice choose(const QuantArgs& p, int mode, bool full, int sms) {
  return mode == kAligned ? choose<DT, kAligned>(p, full, sms)
         : mode == kEdged ? choose<DT, kEdged>(p, full, sms)
                          : choose<DT, kShifted>(p, full, sms);
}

}  // namespace
}  // namespace blk

int launch_norm_quant(int dtype, int mode, const QuantArgs& args, const LaunchCtx& c) {
  using namespace blk;
  const bool full = args.norm == ADDLN_NORM_LAYER || args.beta;
  const bool groups = args.s.scaling == ADDLN_SCALE_GROUP || args.s.scaling == ADDLN_SCALE_POW2;
  // a granule of an edged row may lie in two groups
  if (mode == kEdged && groups) mode = kShifted;
  const Choice ch = dtype == kF32 ? choose<kF32>(args, mode, full, c.dev.sms)
                    : dtype == kF16 ? choose<kF16>(args, mode, full, c.dev.sms)
                                    : choose<kBF16>(args, mode, full, c.dev.sms);
  QuantArgs p = args;
  p.w = walk_of(ch.s.sh);
  p.kept_at = ch.s.kept_at;
  p.sums_at = ch.s.sums_at;
  p.ring_slots = ch.s.ring_slots;
  const int fit = resident_units(reinterpret_cast<const void*>(ch.k), ch.s.sh, ch.s.smem, c.dev);
  if (fit < 0) return fit;
  if (mode == kEdged && fit < 8) return launch_norm_quant(dtype, kShifted, args, c);
  p.slots = slots_ahead(p.rows, fit, ch.s);
  const int64_t need = (p.rows + ch.s.sh.rows - 1) / ch.s.sh.rows;
  const cudaError_t e = launch_units(ch.k, units_for(need, fit, mode == kEdged), ch.s.sh, ch.s.smem, c, p);
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_quant)

}  // namespace addln
