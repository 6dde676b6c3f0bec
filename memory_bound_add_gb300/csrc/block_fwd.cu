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

// 1 / sqrt(mean square + eps) (in M2's place) and the mean that precedes it,
// of one row's slots; a layer norm leaves them shifted, an rms norm as they
// were (mean 0).
template <int VE, int NV, bool LN>
__device__ __forceinline__ RowStat row_norm(Exchange& ex, float2 (&v)[NV * VE / 2], const Cols<VE, NV>& cs, bool layer,
                                            float inv_h, float eps) {
  RowStat st{0.f, 0.f, 0.f};
  if (LN && layer) {
    st = walker_stats<VE, NV>(ex, v, cs);
  } else {
    // the slots of groups that do not exist hold zeros
    float2 q[2] = {dup2(0.f), dup2(0.f)};
#pragma unroll
    for (int j = 0; j < NV * VE / 2; ++j) q[j & 1] = fma2(v[j], v[j], q[j & 1]);
    q[0] = add2(q[0], q[1]);
    st.M2 = walker_sum(ex, q[0].x + q[0].y);
  }
  st.M2 = row_rstd(st.M2, inv_h, eps);
  return st;
}

// The parameters as the row's arithmetic uses them: w = s gate gamma and
// b = s gate beta of the post norm (gate: a per-channel one; without a post
// norm w = s gate, b = 0), and gamma and beta of the pre norm.
template <int VE, int NV, bool LN>
struct Params {
  static constexpr int P = NV * VE / 2;
  // they stay in registers where they are at most 64: loading them again for
  // every row costs more of L1's bandwidth than the row itself
  static constexpr bool kKept = NV * VE * (LN ? 4 : 2) <= (VE == 2 ? 32 : 64);
  static constexpr int Q = kKept ? P : (VE >= 2 ? VE / 2 : 1);
  float2 w[Q], b[LN ? Q : 1], g[Q], e[LN ? Q : 1];

  // slots of group k, at j of these arrays
  __device__ __forceinline__ void load_post(const BlockFwdArgs& p, uint32_t off, int k) {
    float2 gt[Q];
    const bool channel = p.gate_kind == ADDLN_GATE_CHANNEL;
    constexpr int n = VE >= 2 ? VE / 2 : 1;
    const int j0 = VE >= 2 ? k * VE / 2 : k / 2;
    if (channel) load_param<VE>(static_cast<const float*>(p.gate), off, gt, k);
    if (p.post != ADDLN_NORM_NONE) load_param<VE>(p.post_gamma, off, w, k);
    if (LN && p.post_beta) load_param<VE>(p.post_beta, off, b, k);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int j = j0 + i;
      if constexpr (VE >= 2) {
        float2 f = dup2(p.s);
        if (channel) f = mul2(f, gt[j]);
        w[j] = p.post != ADDLN_NORM_NONE ? mul2(f, w[j]) : f;
        if constexpr (LN) b[j] = p.post_beta ? mul2(f, b[j]) : dup2(0.f);
      } else {
        const float f = channel ? p.s * ((k & 1) ? gt[j].y : gt[j].x) : p.s;
        float& u = (k & 1) ? w[j].y : w[j].x;
        u = p.post != ADDLN_NORM_NONE ? f * u : f;
        if constexpr (LN) {
          float& c = (k & 1) ? b[j].y : b[j].x;
          c = p.post_beta ? f * c : 0.f;
        }
      }
    }
  }
  __device__ __forceinline__ void load_pre(const BlockFwdArgs& p, uint32_t off, int k) {
    load_param<VE>(p.pre_gamma, off, g, k);
    if constexpr (LN) {
      constexpr int n = VE >= 2 ? VE / 2 : 1;
      const int j0 = VE >= 2 ? k * VE / 2 : k / 2;
      if (p.pre_beta) {
        load_param<VE>(p.pre_beta, off, e, k);
      } else {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          if constexpr (VE >= 2)
            e[j0 + i] = dup2(0.f);
          else
            (k & 1 ? e[j0].y : e[j0].x) = 0.f;
        }
      }
    }
  }
};

// Registers a thread: with the parameters kept, 128-thread CTAs four to an SM.
// Caps of 96, 80 and 64 (5, 6 and 8 CTAs) spill or reload and measured slower:
// 2048x4096 fp16 rms/rms 13.3 us a pass at 128, 20.0 at 80, 22.7 at 64;
// 32768x8192 bf16 335, 471, 575.
template <int DT, int VE, int NV, bool LN, bool GR>
constexpr int fwd_regs() {
  return 128;
}

// The gate row of a row.
__device__ __forceinline__ int64_t gate_row_of(int64_t row, int64_t rpg, bool small) {
  return small ? static_cast<uint32_t>(row) / static_cast<uint32_t>(rpg) : row / rpg;
}

// LN: some norm of the call is a layer norm, or has a bias.  GR: a gate with
// rows.
template <int DT, int VE, int NV, bool LN, bool GR>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__((fwd_regs<DT, VE, NV, LN, GR>()))
    k_block_fwd(const __grid_constant__ BlockFwdArgs p) {
  constexpr int S = Io<DT>::kBytes;
  constexpr int P = NV * VE / 2;
  const int slots = Ring<DT, VE, NV, 2>::kAsync ? p.slots : 1;
  constexpr int GB = Grp<DT, VE>::kBytes;
  constexpr int NT = GR ? 3 : 2;
  constexpr int kStepBytes = Cols<VE, NV>::kStep * S;
  __shared__ float4 parts[2][kMaxWarps * kMaxCluster];
  extern __shared__ __align__(128) unsigned char smem[];
  const bool row_warp = p.w.rows_per_cta > 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.w.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.w.C);
  const int64_t stride = static_cast<int64_t>(gridDim.x / p.w.C) * p.w.rows_per_cta;
  int64_t row = static_cast<int64_t>(blockIdx.x / p.w.C) * p.w.rows_per_cta + (row_warp ? warp : 0);
  const int col0 = rank * p.w.slice;
  Exchange ex{parts, p.w, rank, 0};
  const bool leader = rank == 0 && lane == 0 && (row_warp || warp == 0);
  Ring<DT, VE, NV, NT> ring;
  ring.base = smem_addr(smem) + warp * Ring<DT, VE, NV, NT>::kWarp + lane * GB;
  Cols<VE, NV> cs;
  cs.init(row_warp ? 0 : warp, col0, min(p.w.slice, p.H - col0));
  // byte offset of this thread's group 0 in a row
  auto offset = [&](int64_t r) { return (r * p.H + cs.c0) * S; };

  auto fetch = [&](int slot, int64_t r) {
    if (r < p.rows) {
      const int64_t at = offset(r);
      const char* f = static_cast<const char*>(p.f) + at;
      const char* x = static_cast<const char*>(p.x) + at;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const bool in = ADDLN_IN(701, at + k * kStepBytes, cs.ok[k] ? GB : 0, f_rows_bytes(p, S));
        ring.fetch(slot, 0, k, f + k * kStepBytes, cs.ok[k] && in);
        ring.fetch(slot, 1, k, x + k * kStepBytes, cs.ok[k] && in);
      }
      if constexpr (GR) {
        const int64_t ga = (gate_row_of(r, p.rows_per_gate, p.rows <= 0x7fffffff) * p.gate_stride + cs.c0) * S;
        const char* g = static_cast<const char*>(p.gate) + ga;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const bool in = ADDLN_IN(705, ga + k * kStepBytes, cs.ok[k] ? GB : 0, f_gate_bytes(p, S));
          ring.fetch(slot, 2, k, g + k * kStepBytes, cs.ok[k] && in);
        }
      }
    }
    ring.commit();
  };
  // While the previous kernel of the stream may still be finishing, ask L2
  // for the first rows (a hint: nothing is read before the wait below, and
  // every SM's writes land in L2), where a walker has few of them.
  if (p.rows <= 8 * stride) {
    const int chunk0 = cs.c0 * S - lane * GB;  // the warp's chunk of a row
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
  Params<VE, NV, LN> par;
  constexpr bool kKept = Params<VE, NV, LN>::kKept;
  if constexpr (kKept) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ADDLN_IN(702, cs.par[k], 4 * VE, 4 * static_cast<int64_t>(p.H))) {
        par.load_post(p, cs.par[k], k);
        if (p.pre != ADDLN_NORM_NONE) par.load_pre(p, cs.par[k], k);
      }
  }

  for (int slot = 0; row < p.rows; row += stride, slot = slot + 1 == slots ? 0 : slot + 1) {
    if (slots == 1) ring.template wait<0>(); else ring.template wait<1>();
    float2 v[P];
    {
      Grp<DT, VE> r[NV];
      ring.template take<NV>(slot, 0, 0, r);
      to_slots<DT, VE, NV>(r, v);
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
      auto affine = [&](float2 u, float2 w, float2 b, float2 gt, float2 x) {
        if constexpr (LN) u = add2(u, negm);
        u = mul2(u, r2);
        const float2 ax = mul2(a2, x);
        if constexpr (GR) return fma2(LN ? fma2(u, w, b) : mul2(u, w), gt, ax);
        return fma2(u, w, LN ? add2(b, ax) : ax);
      };
      // groups that share slots in pairs (single elements) go two at a time
      constexpr int KU = VE >= 2 ? 1 : 2, n = VE >= 2 ? VE / 2 : 1;
#pragma unroll
      for (int k = 0; k < NV; k += KU) {
        Grp<DT, VE> rg[KU], rx[KU];
        float2 gt[n], x[n];
        ring.template take<KU>(slot, 1, k, rx);
        to_slots<DT, VE, KU>(rx, x);
        if constexpr (GR) {
          ring.template take<KU>(slot, 2, k, rg);
          to_slots<DT, VE, KU>(rg, gt);
        }
        if constexpr (!kKept)
          if (ADDLN_IN(711, cs.par[k], 4 * VE, 4 * static_cast<int64_t>(p.H))) par.load_post(p, cs.par[k], 0);
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const int j = (VE >= 2 ? k * VE / 2 : k / 2) + i, q = kKept ? j : i;
          v[j] = affine(v[j], par.w[q], LN ? par.b[LN ? q : 0] : dup2(0.f), GR ? gt[i] : dup2(1.f), x[i]);
        }
      }
    }
    cs.clear(v);
    fetch(slot, row + slots * stride);  // the slot has been read
    const int64_t off = offset(row);
    {
      char* h = static_cast<char*>(p.h) + off;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (cs.ok[k] && ADDLN_IN(706, off + k * kStepBytes, GB, f_rows_bytes(p, S)))
          store_group<DT, VE>(h + k * kStepBytes, v, k);
    }
    if (p.pre == ADDLN_NORM_NONE) continue;
    st = row_norm<VE, NV, LN>(ex, v, cs, p.pre == ADDLN_NORM_LAYER, p.inv_h, p.eps);
    if (leader && ADDLN_IN(707, 4 * row, 4, 4 * p.rows)) {
      if (p.pre_rstd) p.pre_rstd[row] = st.M2;
      if (LN && p.pre_mean) p.pre_mean[row] = st.mean;
    }
    char* y = static_cast<char*>(p.y) + off;
    const float2 negm = dup2(-st.m), r2 = dup2(st.M2);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!kKept && ADDLN_IN(708, cs.par[k], 4 * VE, 4 * static_cast<int64_t>(p.H))) par.load_pre(p, cs.par[k], 0);
      constexpr int n = VE >= 2 ? VE / 2 : 1;
      const int j0 = VE >= 2 ? k * VE / 2 : k / 2;
      if (VE >= 2 || (k & 1) == 0) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const int j = j0 + i, q = kKept ? j : i;
          if constexpr (LN)
            v[j] = fma2(mul2(add2(v[j], negm), r2), par.g[q], par.e[LN ? q : 0]);
          else
            v[j] = mul2(mul2(v[j], r2), par.g[q]);
        }
      }
      if (cs.ok[k] && ADDLN_IN(709, off + k * kStepBytes, GB, f_rows_bytes(p, S)))
        store_group<DT, VE>(y + k * kStepBytes, v, k);
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
  int smem = 0;
};

// Rows of `groups` groups of VE columns, NV groups a thread: a warp for a row
// where 32 threads hold it, four rows to a CTA; else a CTA of up to
// kMaxThreads; else a cluster.
template <int DT, int VE, int NV>
Choice make(const BlockFwdArgs& p, bool ln) {
  Choice c;
  const bool gr = p.gate_kind == ADDLN_GATE_ROWS;
  c.k = gr ? &k_block_fwd<DT, VE, NV, false, true> : &k_block_fwd<DT, VE, NV, false, false>;
  if constexpr (VE < 4 || NV < 4)  // layer norms keep more a column: fewer columns a thread
    if (ln) c.k = gr ? &k_block_fwd<DT, VE, NV, true, true> : &k_block_fwd<DT, VE, NV, true, false>;
  const int groups = p.H / VE;
  c.sh.C = (groups + NV * kMaxThreads - 1) / (NV * kMaxThreads);
  c.sh.slice = c.sh.C == 1 ? p.H : ((p.H + c.sh.C - 1) / c.sh.C + 15) / 16 * 16;
  const int threads = ((c.sh.slice / VE + NV - 1) / NV + 31) / 32 * 32;
  c.sh.rows = threads == 32 ? 4 : 1;
  c.sh.threads = threads * c.sh.rows;
  const int nt = p.gate_kind == ADDLN_GATE_ROWS ? 3 : 2;
  if (Grp<DT, VE>::kBytes >= 4) c.smem = kMaxSlots * nt * NV * c.sh.threads * Grp<DT, VE>::kBytes;
  return c;
}

// Groups a thread: the number (of 1 to 4 16-byte groups) that leaves the
// fewest of a row's threads' slots empty, the larger one where equal.
inline int groups_a_thread(int groups, int most) {
  int best = 1, waste = 1 << 30;
  for (int nv = 1; nv <= most; ++nv) {
    const int t = ((groups + nv - 1) / nv + 31) / 32 * 32;
    if (t * nv - groups <= waste) waste = t * nv - groups, best = nv;
  }
  return best;
}

template <int DT>
Choice choose(const BlockFwdArgs& p, int access, bool ln) {
  constexpr int VEC = Io<DT>::kVec;
  if (access == 16) {
    // beyond a warp's reach, no more than keeps the parameters in registers
    const int groups = p.H / VEC, most = !ln ? 4 : DT != kF32 && groups > 96 ? 2 : 3;
    switch (groups_a_thread(groups, most)) {
      case 1: return make<DT, VEC, 1>(p, ln);
      case 2: return make<DT, VEC, 2>(p, ln);
      case 3: return make<DT, VEC, 3>(p, ln);
      default: return make<DT, VEC, 4>(p, ln);
    }
  }
  if constexpr (DT != kF32)
    if (access == 4) return p.H <= 256 ? make<DT, 2, 4>(p, ln) : make<DT, 2, 8>(p, ln);
  return p.H <= 128 ? make<DT, 1, 4>(p, ln) : make<DT, 1, 8>(p, ln);
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

int launch_block_fwd(int dtype, int access, bool layer_or_bias, const BlockFwdArgs& args,
                     const LaunchCtx& c, const char** name) {
  using namespace blk;
  const Choice ch = dtype == kF32 ? choose<kF32>(args, access, layer_or_bias)
                    : dtype == kF16 ? choose<kF16>(args, access, layer_or_bias)
                                    : choose<kBF16>(args, access, layer_or_bias);
  *name = access == 16 ? "block_fwd_v16" : access == 4 ? "block_fwd_v4" : "block_fwd_v2";
  BlockFwdArgs p = args;
  p.w = walk_of(ch.sh);
  const int fit = resident_units(reinterpret_cast<const void*>(ch.k), ch.sh, ch.smem, c.dev);
  if (fit < 0) return fit;
  // Rows staged ahead: two, or one where every walker has more than eight
  // rows (us a pass with one / two: 2048x4096 fp16, 3 or 4 rows a walker,
  // 14.8 / 13.5; 32768x8192 bf16, 108 rows, 331 / 348).
  p.slots = p.rows > 8 * static_cast<int64_t>(fit) * ch.sh.rows ? 1 : 2;
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
