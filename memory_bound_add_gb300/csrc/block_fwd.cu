// The boundary between two blocks of a transformer, forward, in one pass:
//   n = post(f)           norm of the block's output (none, rms or layer)
//   h = a x + s (gate n)  the residual stream
//   y = pre(h)            norm before the next block (none, rms or layer)
// read f and x (and gate rows) once, write h and y once.  Both statistics of
// a row are taken of values in registers: of f, and of the unrounded h.
#include "block.cuh"

#include <mutex>
#include <unordered_map>

#include "block.h"

namespace addln {
namespace blk {

// Byte extents of a forward launch's buffers (for ADDLN_IN).
__device__ __forceinline__ int64_t f_rows_bytes(const BlockFwdArgs& p, int S) {
  return p.rows * static_cast<int64_t>(p.H) * S;
}
__device__ __forceinline__ int64_t f_gate_bytes(const BlockFwdArgs& p, int S) {
  return ((p.gate_rows - 1) * p.gate_stride + p.H) * S;
}

// The parameters as the row's arithmetic uses them: w = s gate gamma and
// b = s gate beta of the post norm (gate: a per-channel one; without a post
// norm w = s gate, b = 0), and gamma and beta of the pre norm.  Loading them
// again for every row costs more of L1's bandwidth than the row itself: two
// vectors (no layer norm, no bias) stay in registers, and four of at most
// eight columns a thread; four of more, and two of more of shifted rows, lie
// in shared memory, one copy for all rows that the CTA has side by side.  us,
// all in registers / as here / all in shared memory: 2048x4096 fp16 rms 12.1,
// 12.0, 15.1; one row of 4096 2.8, 2.8, 3.2; 65536x768 bf16 layer 80.8, 68.8,
// 68.9; 8192x5001 bf16 rms 121, 100, 100.
__host__ __device__ constexpr bool in_registers(int columns, bool ln, bool sh) { return columns <= 8 || !(ln || sh); }

template <int VE, int NV, bool LN, bool SH>
struct Params {
  static constexpr bool kRegs = in_registers(NV * VE, LN, SH);
  static constexpr int P = kRegs ? NV * VE / 2 : 1;
  float2 r[LN ? 4 : 2][P];  // w, gamma, and with LN b, beta
  Kept<VE, NV> kept;        // the same vectors

  // vector i of group k
  __device__ __forceinline__ void get(int i, int k, float2 (&v)[VE / 2]) const {
    if constexpr (kRegs) {
#pragma unroll
      for (int j = 0; j < VE / 2; ++j) v[j] = r[i][k * VE / 2 + j];
    } else {
      kept.get(i, k, v);
    }
  }

  // group k, at column c, from the call's arguments
  __device__ __forceinline__ void load(const BlockFwdArgs& p, int c, int k) {
    float v[4][VE], gt[VE];
    load_params<VE, SH>(p.gate_kind == ADDLN_GATE_CHANNEL ? static_cast<const float*>(p.gate) : nullptr, c, p.H, 1.f, gt, 702);
    load_params<VE, SH>(p.post_gamma, c, p.H, 1.f, v[0], 704);
    load_params<VE, SH>(p.pre_gamma, c, p.H, 0.f, v[1], 711);
    load_params<VE, SH>(LN ? p.post_beta : nullptr, c, p.H, 0.f, v[2], 708);
    load_params<VE, SH>(LN ? p.pre_beta : nullptr, c, p.H, 0.f, v[3], 712);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float f = p.s * gt[e];
      v[0][e] *= f;
      v[2][e] *= f;
    }
#pragma unroll
    for (int i = 0; i < (LN ? 4 : 2); ++i) {
      if constexpr (kRegs) {
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) r[i][k * VE / 2 + e] = make_float2(v[i][2 * e], v[i][2 * e + 1]);
      } else {
        kept.put(i, k, v[i]);
      }
    }
  }
};

// Registers a thread: with the parameters kept, 128-thread CTAs four to an SM.
// Caps of 96, 80 and 64 (5, 6 and 8 CTAs) spill or reload and measured slower:
// 2048x4096 fp16 rms/rms 13.3 us a pass at 128, 20.0 at 80, 22.7 at 64;
// 32768x8192 bf16 335, 471, 575.  Left to the thread count alone (which allows
// as many), the compiler goes for 64 where it can, and spills.  A template, since
// nvcc takes this beside a thread count only where it depends on one.
template <int DT>
constexpr int kFwdRegs = 128;

// The gate row of a row.
__device__ __forceinline__ int64_t gate_row_of(int64_t row, int64_t rpg, bool small) {
  return small ? static_cast<uint32_t>(row) / static_cast<uint32_t>(rpg) : row / rpg;
}

// LN: some norm of the call is a layer norm, or has a bias.  GR: a gate with
// rows.  SH: some rows do not begin on 16-byte borders.
//
// Every walker takes rows at a stride of all walkers, so that the memory that
// is in use at a time is one piece.  The call moves 4 rows H elements and
// should be bound by memory: 32768x8192 bf16 rms/rms with gate rows takes 330
// us (6.5 TB/s, 0.96 of a copy).  Shorter calls have 2 to 14 rows a walker and
// pay for the first loads and the last stores of each: 2048x4096 fp16 12.0 us
// (0.82); a layer norm adds a second pass over its registers and 512 threads
// meet twice a row: 8192x4096 bf16 layer/layer 59 us (0.67), 4096x768 fp16 8.5
// (0.44); shifted rows add shuffles and halved stores: 8192x5001 bf16 100 us
// (0.48).  One row of 4096 takes 2.8 us, a launch.
template <int DT, int NV, bool LN, bool GR, bool SH>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__((kFwdRegs<DT>))
    k_block_fwd(const __grid_constant__ BlockFwdArgs p) {
  using IO = Io<DT>;
  constexpr int S = IO::kBytes, VE = IO::kVec, Q = VE / 2;
  constexpr int P = NV * Q;
  constexpr int NT = GR ? 3 : 2;
  constexpr int kStepBytes = Cols<VE, NV>::kStep * S;
  using R = Ring<DT, NV, NT, SH>;
  extern __shared__ __align__(128) unsigned char smem[];
  if (p.w.C > 1) cluster_started();
  const int slots = p.slots;
  const int lane = threadIdx.x & 31;
  const int side = (threadIdx.x >> 5) / p.w.cta_warps, warp = (threadIdx.x >> 5) - side * p.w.cta_warps;
  const int rank = p.w.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.w.C);
  const int64_t stride = static_cast<int64_t>(gridDim.x / p.w.C) * p.w.rows_per_cta;
  int64_t row = static_cast<int64_t>(blockIdx.x / p.w.C) * p.w.rows_per_cta + side;
  const int col0 = rank * p.w.slice;
  Exchange<!in_registers(NV * VE, LN, SH)> ex{p.w, p.sums_at + side * 2 * p.w.warps * 16, 0};
  const bool leader = rank == 0 && lane == 0 && warp == 0;
  R ring;
  ring.base = smem_addr(smem) + (threadIdx.x >> 5) * p.ring_slots * R::kSlot + lane * 16;
  Cols<VE, NV> cs;
  cs.init(warp, col0, min(p.w.slice, p.H - col0));
  // byte offset of this thread's group 0 in a row, and in its gate row
  auto offset = [&](int64_t r) { return (r * p.H + cs.c0) * S; };
  auto gate_offset = [&](int64_t r) {
    return (gate_row_of(r, p.rows_per_gate, p.rows <= 0x7fffffff) * p.gate_stride + cs.c0) * S;
  };

  auto fetch = [&](int slot, int64_t r) {
    if (r < p.rows) {
      const int64_t at = offset(r);
      ring.template fetch<0>(cs, slot, p.f, at, 701, f_rows_bytes(p, S));
      ring.template fetch<1>(cs, slot, p.x, at, 701, f_rows_bytes(p, S));
      if constexpr (GR) ring.template fetch<2>(cs, slot, p.gate, gate_offset(r), 705, f_gate_bytes(p, S));
    }
    ring.commit();
  };
  // While the previous kernel of the stream may still be finishing, ask L2
  // for the first rows (a hint: nothing is read before the wait below, and
  // every SM's writes land in L2), where a walker has few of them.
  if (p.rows <= 8 * stride) {
    const int chunk0 = cs.c0 * S - lane * 16;  // the warp's chunk of a row
    const int bytes = min(NV * kStepBytes, (col0 + min(p.w.slice, p.H - col0)) * S - chunk0);
    for (int s = 0; s < slots; ++s) {
      const int64_t at = (row + s * stride) * p.H * S + chunk0 + lane * 128;
      if (row + s * stride < p.rows && lane * 128 < bytes && ADDLN_IN(710, at, 1, f_rows_bytes(p, S))) {
        prefetch_line(static_cast<const char*>(p.f) + at);
        prefetch_line(static_cast<const char*>(p.x) + at);
      }
    }
  }
  pdl_trigger();
  pdl_wait();
  for (int s = 0; s < slots; ++s) fetch(s, row + s * stride);
  Params<VE, NV, LN, SH> par;
  constexpr bool kRegs = Params<VE, NV, LN, SH>::kRegs;
  if constexpr (!kRegs)
    par.kept.base = smem_addr(smem) + p.kept_at + warp * Kept<VE, NV>::template bytes<LN ? 4 : 2>() + lane * 16;
  if (kRegs || side == 0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) par.load(p, cs.col(k), k);
  }
  if constexpr (!kRegs) __syncthreads();
  if (p.w.C > 1) cluster_wait_started();

  for (int slot = 0; row < p.rows; row += stride, slot = slot + 1 == slots ? 0 : slot + 1) {
    if (slots == 1) ring.template wait<0>(); else ring.template wait<1>();
    ring.meet();
    const int64_t off = offset(row);
    float2 v[P];
    {
      const int s = SH ? low4(p.f, off) : 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) IO::to_pairs(ring.take(slot, 0, k, s), v + k * Q);
      if constexpr (SH) cs.clear(v);
    }
    RowStat st{0.f, 0.f, 1.f};
    if (p.post != ADDLN_NORM_NONE) {
      st = row_norm<VE, NV, LN>(ex, v, cs, p.post == ADDLN_NORM_LAYER, p.inv_h, p.eps);
      if (leader && ADDLN_IN(703, 4 * row, 4, 4 * p.rows)) {
        if (p.post_rstd) p.post_rstd[row] = st.M2;
        if (LN && p.post_mean) p.post_mean[row] = st.mean;
      }
    }
    // v = ((v - m) rstd) w + b, times the row's gate, plus a x
    {
      const float2 negm = dup2(-st.m), r2 = dup2(st.M2), a2 = dup2(p.a);
      const int sx = SH ? low4(p.x, off) : 0, sg = SH && GR ? low4(p.gate, gate_offset(row)) : 0;
      auto affine = [&](float2 u, float2 w, float2 b, float2 gt, float2 x) {
        if constexpr (LN) u = add2(u, negm);
        u = mul2(u, r2);
        const float2 ax = mul2(a2, x);
        if constexpr (GR) return fma2(LN ? fma2(u, w, b) : mul2(u, w), gt, ax);
        return fma2(u, w, LN ? add2(b, ax) : ax);
      };
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float2 gt[Q], x[Q], w[Q], b[Q];
        IO::to_pairs(ring.take(slot, 1, k, sx), x);
        if constexpr (GR) IO::to_pairs(ring.take(slot, 2, k, sg), gt);
        par.get(0, k, w);
        if constexpr (LN) par.get(2, k, b);
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          if constexpr (!LN) b[i] = dup2(0.f);
          v[k * Q + i] = affine(v[k * Q + i], w[i], b[i], GR ? gt[i] : dup2(1.f), x[i]);
        }
      }
    }
    cs.clear(v);
    ring.meet();
    fetch(slot, row + slots * stride);  // the slot has been read
    {
      Writer<DT, NV, SH> out;
#pragma unroll
      for (int k = 0; k < NV; ++k) out.put(cs, p.h, off, k, IO::from_pairs(v + k * Q), 706, f_rows_bytes(p, S));
    }
    if (p.pre == ADDLN_NORM_NONE) continue;
    st = row_norm<VE, NV, LN>(ex, v, cs, p.pre == ADDLN_NORM_LAYER, p.inv_h, p.eps);
    if (leader && ADDLN_IN(707, 4 * row, 4, 4 * p.rows)) {
      if (p.pre_rstd) p.pre_rstd[row] = st.M2;
      if (LN && p.pre_mean) p.pre_mean[row] = st.mean;
    }
    const float2 negm = dup2(-st.m), r2 = dup2(st.M2);
    Writer<DT, NV, SH> out;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 g[Q], e[Q];
      par.get(1, k, g);
      if constexpr (LN) par.get(3, k, e);
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int j = k * Q + i;
        if constexpr (LN)
          v[j] = fma2(mul2(add2(v[j], negm), r2), g[i], e[i]);
        else
          v[j] = mul2(mul2(v[j], r2), g[i]);
      }
      out.put(cs, p.y, off, k, IO::from_pairs(v + k * Q), 709, f_rows_bytes(p, S));
    }
  }
  // a CTA's shared memory has to outlive its peers' writes into it
  if (p.w.C > 1) cooperative_groups::this_cluster().sync();
}

// ------------------------------------------------------------------ host
namespace {

struct Key {
  const void* f;
  int device, threads, C, smem;
  bool operator==(const Key& o) const {
    return f == o.f && device == o.device && threads == o.threads && C == o.C && smem == o.smem;
  }
};
struct KeyHash {
  size_t operator()(const Key& k) const {
    return std::hash<const void*>()(k.f) ^ (static_cast<size_t>(k.device) << 20) ^
           (static_cast<size_t>(k.threads) << 28) ^ (static_cast<size_t>(k.C) << 44) ^
           (static_cast<size_t>(k.smem) << 48);
  }
};
std::mutex g_mu;
std::unordered_map<Key, int, KeyHash> g_occ;

struct Choice {
  void (*k)(BlockFwdArgs) = nullptr;
  Shape sh{};
  int smem = 0, kept_at = 0, sums_at = 0, ring_slots = 0;
};

// NV groups of VE columns a thread.  With the parameters in registers: a warp
// for a row where 32 threads hold it, four rows to a CTA (one: 32768x256 bf16
// 12.4 us instead of 11.4); else a CTA of up to kMaxThreads; else a cluster.
// With parameters in shared memory: rows side by side in a CTA of up to
// kMaxThreads, as many as leave the ring two slots, or one; a cluster where one
// row's parameters and ring do not fit (us of a cluster of two / of one CTA:
// 4096x10240 bf16 layer 202 / 99).
template <int DT, int NV, bool SH>
Choice make(const BlockFwdArgs& p, bool ln, int sms) {
  constexpr int VE = Io<DT>::kVec;
  Choice c;
  const bool gr = p.gate_kind == ADDLN_GATE_ROWS;
  c.k = gr ? (ln ? &k_block_fwd<DT, NV, true, true, SH> : &k_block_fwd<DT, NV, false, true, SH>)
           : (ln ? &k_block_fwd<DT, NV, true, false, SH> : &k_block_fwd<DT, NV, false, false, SH>);
  const int groups = (p.H + VE - 1) / VE;
  const bool shared = !in_registers(NV * VE, ln, SH);
  int threads, slot, kept, sums;
  auto bytes = [&] { return c.sh.rows * (c.ring_slots * slot + sums) + kept; };
  for (c.sh.C = (groups + NV * kMaxThreads - 1) / (NV * kMaxThreads);; ++c.sh.C) {
    c.sh.slice = c.sh.C == 1 ? p.H : ((p.H + c.sh.C - 1) / c.sh.C + 15) / 16 * 16;
    threads = ((c.sh.slice + VE - 1) / VE + 32 * NV - 1) / (32 * NV) * 32;
    slot = threads / 32 * static_cast<int>(gr ? Ring<DT, NV, 3, SH>::kSlot : Ring<DT, NV, 2, SH>::kSlot);
    kept = shared ? threads / 32 * static_cast<int>(ln ? Kept<VE, NV>::template bytes<4>() : Kept<VE, NV>::template bytes<2>()) : 0;
    sums = 2 * (threads / 32) * c.sh.C * 16;
    c.sh.rows = c.ring_slots = 1;
    if (bytes() <= kMaxSmem || c.sh.C == kMaxCluster) break;
  }
  c.sh.rows = c.sh.C > 1 ? 1 : rows_side_by_side(shared ? kMaxThreads / threads : threads == 32 ? 4 : 1, p.rows, sms);
  c.ring_slots = kMaxSlots;
  while (bytes() > kMaxSmem && c.ring_slots > 1) --c.ring_slots;
  while (bytes() > kMaxSmem && c.sh.rows > 1) --c.sh.rows;
  c.sh.threads = threads * c.sh.rows;
  c.kept_at = c.sh.rows * c.ring_slots * slot;
  c.sums_at = c.kept_at + kept;
  c.smem = bytes();
  return c;
}

template <int DT>
Choice choose(const BlockFwdArgs& p, bool aligned, bool ln, int sms) {
  constexpr int VEC = Io<DT>::kVec;
  const int nv = groups_a_thread((p.H + VEC - 1) / VEC);
  if (!aligned) {
    switch (nv) {
      case 1: return make<DT, 1, true>(p, ln, sms);
      case 2: return make<DT, 2, true>(p, ln, sms);
      case 3: return make<DT, 3, true>(p, ln, sms);
      default: return make<DT, 4, true>(p, ln, sms);
    }
  }
  switch (nv) {
    case 1: return make<DT, 1, false>(p, ln, sms);
    case 2: return make<DT, 2, false>(p, ln, sms);
    case 3: return make<DT, 3, false>(p, ln, sms);
    default: return make<DT, 4, false>(p, ln, sms);
  }
}

}  // namespace

int resident_units(const void* f, const Shape& sh, int smem, const DeviceInfo& dev) {
  const Key key{f, dev.device, sh.threads, sh.C, smem};
  {
    std::lock_guard<std::mutex> g(g_mu);
    auto it = g_occ.find(key);
    if (it != g_occ.end()) return it->second;
  }
  int n = 0;
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024) {
    // raised once to what the device allows beside the kernel's static share
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, f);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               dev.smem_optin - static_cast<int>(fa.sharedSizeBytes));
  }
  if (e == cudaSuccess) {
    if (sh.C == 1) {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f, sh.threads, static_cast<size_t>(smem));
      n *= dev.sms;
    } else {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(sh.C * dev.sms));
      cfg.blockDim = dim3(static_cast<unsigned>(sh.threads));
      cfg.dynamicSmemBytes = static_cast<size_t>(smem);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(sh.C);
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&n, f, &cfg);
    }
  }
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_CUDA;
  }
  if (n < 1) return ADDLN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> g(g_mu);
  g_occ[key] = n;
  return n;
}

Walk walk_of(const Shape& sh) {
  Walk w;
  w.C = sh.C;
  w.slice = sh.slice;
  w.rows_per_cta = sh.rows;
  w.cta_warps = sh.threads / 32 / sh.rows;
  w.warps = w.cta_warps * sh.C;
  w.width = 1;
  while (w.width < w.warps && w.width < 32) w.width *= 2;
  return w;
}

}  // namespace blk

int launch_block_fwd(int dtype, bool aligned, bool layer_or_bias, const BlockFwdArgs& args,
                     const LaunchCtx& c) {
  using namespace blk;
  const Choice ch = dtype == kF32 ? choose<kF32>(args, aligned, layer_or_bias, c.dev.sms)
                    : dtype == kF16 ? choose<kF16>(args, aligned, layer_or_bias, c.dev.sms)
                                    : choose<kBF16>(args, aligned, layer_or_bias, c.dev.sms);
  BlockFwdArgs p = args;
  p.w = walk_of(ch.sh);
  p.kept_at = ch.kept_at;
  p.sums_at = ch.sums_at;
  p.ring_slots = ch.ring_slots;
  const int fit = resident_units(reinterpret_cast<const void*>(ch.k), ch.sh, ch.smem, c.dev);
  if (fit < 0) return fit;
  // Rows staged ahead: two, or one where every walker has more than eight
  // rows (us a pass with one / two: 2048x4096 fp16, 3 or 4 rows a walker,
  // 14.8 / 13.5; 32768x8192 bf16, 108 rows, 331 / 348).
  p.slots = p.rows > 8 * static_cast<int64_t>(fit) * ch.sh.rows ? 1 : ch.ring_slots;
  const int64_t need = (p.rows + ch.sh.rows - 1) / ch.sh.rows;
  const cudaError_t e = launch_units(ch.k, need < fit ? need : fit, ch.sh, ch.smem, c, p);
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_block_fwd)

}  // namespace addln
