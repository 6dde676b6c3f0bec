// Bias, dropout, residual sum and norm, forward, in one pass:
//   h = x + dropout(f + bias),  y = norm(h)
// f and x are read once, h and y written once; the statistics are of values in
// registers, the unrounded h.  The mask is made where it is used.
#include "philox.cuh"

namespace addln {
namespace blk {

// The vectors: gamma, and with FULL bias and beta.  Few columns a thread: in
// registers; else in shared memory, one copy for all rows that a CTA has side
// by side (as in block_fwd.cu).
__host__ __device__ constexpr bool drop_in_registers(int columns, bool full, int mode) {
  return columns <= 8 || !(full || mode == kShifted);
}

template <int VE, int NV, bool FULL, int MODE>
struct DropParams {
  static constexpr bool kRegs = drop_in_registers(NV * VE, FULL, MODE);
  static constexpr int P = kRegs ? NV * VE / 2 : 1, N = FULL ? 3 : 1;
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
  // statistics by way of the bias
  __device__ __forceinline__ void load(const DropFwdArgs& p, int i, const Cols<VE, NV>& cs, int k) {
    const float* from = i == 0 ? p.gamma : i == 1 ? p.bias : p.beta;
    float v[VE];
    load_params<VE, MODE>(from, cs.col(k), cs.end(), 0.f, v, 770);
    if constexpr (kRegs) {
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) r[i][k * VE / 2 + e] = make_float2(v[2 * e], v[2 * e + 1]);
    } else {
      kept.put(i, k, v);
    }
  }
};

// FULL: a layer norm, or a bias or a beta.  MODE: how rows lie.
//
// The call moves 4 rows H elements (3 without a norm) and is bound by memory where
// rows are many: 32768x8192 bf16 rms 316 us (6.8 TB/s, 1.02 of a copy), 8192x4096 43.9
// (0.92), 65536x768 layer 67.7 (0.89), odd widths too: 8192x5001 56.0 (0.87).  The
// tile (up to 32 columns a thread, 128 registers, two rows ahead) is block_fwd.cu's.
// A mask costs 8.6 instructions an element of 23, and half of the issue slots are used:
// layer norms and few rows a walker are bound by the latency of a row's chain (loads,
// mask, exchanges, stores) at 16 warps an SM: 8192x4096 layer with bias 53.5 us (0.75),
// 4097x1001 rms 9.1 (0.54), 4096x768 fp16 layer 7.9 (0.48).  Rows of several CTAs meet
// through the cluster twice: 4096x11008 fp32 rms with bias 201 us (0.54), 4096x20000 bf16
// 208 (0.47), layer 222 (0.44).  Rows of at most 128 columns leave most of a warp's lanes
// without any: 65536x128 layer with bias 32.2 (0.31).
//
// (128 registers: as block_fwd.cu's kFwdRegs, which has the sweep.  nvcc takes the number
// beside a thread count only where it depends on a template's argument.)
template <int DT, int NV, bool FULL, int MODE>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__((NV > 0 ? 128 : 0))
    k_drop_fwd(const __grid_constant__ DropFwdArgs p) {
  using IO = Io<DT>;
  constexpr bool SH = MODE == kShifted;
  constexpr int S = IO::kBytes, VE = IO::kVec, Q = VE / 2;
  constexpr int P = NV * Q;
  using R = Ring<DT, NV, 2, MODE>;
  extern __shared__ __align__(128) unsigned char smem[];
  if (p.w.C > 1) cluster_started();
  const int slots = p.slots;
  const int lane = threadIdx.x & 31;
  const int side = (threadIdx.x >> 5) / p.w.cta_warps, warp = (threadIdx.x >> 5) - side * p.w.cta_warps;
  const int rank = p.w.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.w.C);
  const int64_t stride = static_cast<int64_t>(gridDim.x / p.w.C) * p.w.rows_per_cta;
  int64_t row = first_row<MODE>(blockIdx.x / p.w.C, p.w.rows_per_cta, side);
  const int col0 = rank * p.w.slice;
  const int64_t extent = p.rows * static_cast<int64_t>(p.H) * S;
  Exchange<!drop_in_registers(NV * VE, FULL, MODE)> ex{p.w, p.sums_at + side * 2 * p.w.warps * 16, 0};
  const bool leader = rank == 0 && lane == 0 && warp == 0;
  const bool has_x = p.x != nullptr;
  R ring;
  ring.base = smem_addr(smem) + (threadIdx.x >> 5) * p.ring_slots * R::kSlot + lane * 16;
  Cols<VE, NV> cs;
  if constexpr (MODE == kEdged)
    cs.init_edged(warp, col0, p.w.slice, p.H, static_cast<int>(row * p.H & (VE - 1)));
  else
    cs.init(warp, col0, min(p.w.slice, p.H - col0));
  auto offset = [&](int64_t r) { return (r * p.H + cs.c0) * S; };
  auto fetch = [&](int slot, int64_t r) {
    if (r < p.rows) {
      const int64_t at = offset(r);
      ring.template fetch<0>(cs, slot, p.f, at, 773, extent);
      if (has_x) ring.template fetch<1>(cs, slot, p.x, at, 774, extent);
    }
    ring.commit();
  };
  // where a walker has few rows
  if (p.rows <= 8 * stride)
    for (int s = 0; s < slots && row + s * stride < p.rows; ++s) {
      const int64_t at = ((row + s * stride) * p.H + cs.c0) * S;
      prefetch_row<S>(p.f, at, cs, 778, extent);
      prefetch_row<S>(p.x, at, cs, 778, extent);
    }
  pdl_trigger();
  pdl_wait();
  for (int s = 0; s < slots; ++s) fetch(s, row + s * stride);
  Philox<true> rng;
  rng.init(p.drop);
  DropParams<VE, NV, FULL, MODE> par;
  constexpr bool kRegs = DropParams<VE, NV, FULL, MODE>::kRegs;
  if constexpr (!kRegs)
    par.kept.base = smem_addr(smem) + p.kept_at + warp * Kept<VE, NV>::template bytes<FULL ? 3 : 1>() + lane * 16;
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
  if (p.w.C > 1) cluster_wait_started();
  const float2 scale = dup2(p.drop.scale);

  for (int slot = 0; row < p.rows; row += stride, slot = slot + 1 == slots ? 0 : slot + 1) {
    const int64_t off = offset(row);
    const uint64_t at = static_cast<uint64_t>(row * p.H + cs.c0);
    Mask<VE, NV, MODE> mask;
    if (p.drop.on) mask.row(rng, at, p.drop.above, p.drop.wide);
    if (slots == 1) ring.template wait<0>(); else ring.template wait<1>();
    ring.meet();
    const int sf = SH ? low4(p.f, off) : 0, sx = SH && has_x ? low4(p.x, off) : 0;
    float2 v[P];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 z[Q], x[Q], b[Q];
      IO::to_pairs(ring.take(slot, 0, k, sf), z);
      if constexpr (FULL) {
        par.get(1, k, b);
#pragma unroll
        for (int i = 0; i < Q; ++i) z[i] = add2(z[i], b[i]);
      }
      if (p.drop.on) mask.apply(rng, at, k, p.drop.above, p.drop.wide, scale, z);
      if (has_x) {
        IO::to_pairs(ring.take(slot, 1, k, sx), x);
#pragma unroll
        for (int i = 0; i < Q; ++i) z[i] = add2(z[i], x[i]);
      }
#pragma unroll
      for (int i = 0; i < Q; ++i) v[k * Q + i] = z[i];
    }
    // columns before the row have the end of another; those past it are zeros
    if constexpr (MODE == kEdged) cs.clear_low(v);
    ring.meet();
    fetch(slot, row + slots * stride);  // the slot has been read
    if (p.h != nullptr) {
      Writer<DT, NV, MODE> out;
#pragma unroll
      for (int k = 0; k < NV; ++k) out.put(cs, p.h, off, k, IO::from_pairs(v + k * Q), 775, extent);
    }
    if (p.norm == ADDLN_NORM_NONE) continue;
    const RowStat st = row_norm<VE, NV, FULL>(ex, v, cs, p.norm == ADDLN_NORM_LAYER, p.inv_h, p.eps);
    if (leader && ADDLN_IN(776, 4 * row, 4, 4 * p.rows)) {
      if (p.rstd) p.rstd[row] = st.M2;
      if (FULL && p.mean) p.mean[row] = st.mean;
    }
    const float2 negm = dup2(-st.m), r2 = dup2(st.M2);
    Writer<DT, NV, MODE> out;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 g[Q], e[Q];
      par.get(0, k, g);
      if constexpr (FULL) par.get(2, k, e);
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int j = k * Q + i;
        if constexpr (FULL)
          v[j] = fma2(mul2(add2(v[j], negm), r2), g[i], e[i]);
        else
          v[j] = mul2(mul2(v[j], r2), g[i]);
      }
      out.put(cs, p.y, off, k, IO::from_pairs(v + k * Q), 777, extent);
    }
  }
  // a CTA's shared memory has to outlive its peers' writes into it
  if (p.w.C > 1) cooperative_groups::this_cluster().sync();
}

// ------------------------------------------------------------------ host
namespace {

struct Choice {
  void (*k)(DropFwdArgs) = nullptr;
  Spread s;
};

template <int DT, int NV, int MODE>
Choice make(const DropFwdArgs& p, bool full, int sms) {
  constexpr int VE = Io<DT>::kVec;
  Choice c;
  c.k = full ? &k_drop_fwd<DT, NV, true, MODE> : &k_drop_fwd<DT, NV, false, MODE>;
  const bool shared = !drop_in_registers(NV * VE, full, MODE);
  c.s = spread(MODE == kEdged ? p.H + VE - 1 : p.H, VE, NV, p.rows, sms, Ring<DT, NV, 2, MODE>::kSlot,
               !shared ? 0 : full ? Kept<VE, NV>::template bytes<3>() : Kept<VE, NV>::template bytes<1>(), 16);
  return c;
}

template <int DT, int MODE>
Choice choose(const DropFwdArgs& p, bool full, int sms) {
  constexpr int VE = Io<DT>::kVec;
  switch (groups_a_thread(((MODE == kEdged ? p.H + VE - 1 : p.H) + VE - 1) / VE)) {
    case 1: return make<DT, 1, MODE>(p, full, sms);
    case 2: return make<DT, 2, MODE>(p, full, sms);
    case 3: return make<DT, 3, MODE>(p, full, sms);
    default: return make<DT, 4, MODE>(p, full, sms);
  }
}

template <int DT>
Choice choose(const DropFwdArgs& p, int mode, bool full, int sms) {
  return mode == kAligned ? choose<DT, kAligned>(p, full, sms)
         : mode == kEdged ? choose<DT, kEdged>(p, full, sms)
                          : choose<DT, kShifted>(p, full, sms);
}

}  // namespace
}  // namespace blk

int launch_drop_fwd(int dtype, int mode, const DropFwdArgs& args, const LaunchCtx& c) {
  using namespace blk;
  const bool full = args.norm == ADDLN_NORM_LAYER || args.bias || args.beta;
  const Choice ch = dtype == kF32 ? choose<kF32>(args, mode, full, c.dev.sms)
                    : dtype == kF16 ? choose<kF16>(args, mode, full, c.dev.sms)
                                    : choose<kBF16>(args, mode, full, c.dev.sms);
  DropFwdArgs p = args;
  p.w = walk_of(ch.s.sh);
  p.kept_at = ch.s.kept_at;
  p.sums_at = ch.s.sums_at;
  p.ring_slots = ch.s.ring_slots;
  const int fit = resident_units(reinterpret_cast<const void*>(ch.k), ch.s.sh, ch.s.smem, c.dev);
  if (fit < 0) return fit;
  if (mode == kEdged && fit < 8) return launch_drop_fwd(dtype, kShifted, args, c);
  p.slots = slots_ahead(p.rows, fit, ch.s);
  const int64_t need = (p.rows + ch.s.sh.rows - 1) / ch.s.sh.rows;
  const cudaError_t e = launch_units(ch.k, units_for(need, fit, mode == kEdged), ch.s.sh, ch.s.smem, c, p);
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_drop_fwd)

}  // namespace addln
