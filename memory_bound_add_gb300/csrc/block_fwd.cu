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

// 1 / sqrt(mean square + eps) and the shift and mean that precede it, of one
// row's slots; layer and rms norms in one form (K = m = 0 for rms).
template <int VE, bool LN>
__device__ __forceinline__ RowStat row_norm(Exchange& ex, const float2 (&v)[kE / 2],
                                            const bool (&ok)[kE / VE], int cnt, float inv_cnt,
                                            bool layer, float inv_h, float eps) {
  RowStat st{0.f, 0.f, 0.f};
  if (LN && layer) {
    st = walker_stats<VE>(ex, v, ok, cnt, inv_cnt);
  } else {
    // slots past the row's end hold zeros
    float2 q = dup2(0.f);
#pragma unroll
    for (int j = 0; j < kE / 2; ++j) q = fma2(v[j], v[j], q);
    st.M2 = walker_sum2(ex, make_float2(q.x + q.y, 0.f)).x;
  }
  st.M2 = row_rstd(st.M2, inv_h, eps);
  return st;
}

template <int DT, int VE, bool LN>
constexpr int fwd_regs() {
  return 80;
}

// LN: some norm of the call is a layer norm, or has a bias.
template <int DT, int VE, bool LN>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__((fwd_regs<DT, VE, LN>())) k_block_fwd(const BlockFwdArgs p) {
  constexpr int NV = kE / VE;
  [[maybe_unused]] constexpr int S = Io<DT>::kBytes;
  __shared__ float4 parts[2][kMaxWarps * kMaxCluster];
  const int T = blockDim.x, tid = threadIdx.x;
  const int rank = p.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.C);
  const int64_t walkers = gridDim.x / p.C;
  int64_t row = blockIdx.x / p.C;
  const int col0 = rank * p.slice;
  const int cols = min(p.slice, p.H - col0);
  Exchange ex{parts, T / 32 * p.C, T / 32, p.C, rank, 0};

  bool ok[NV];
  int cnt = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    ok[k] = (k * T + tid) * VE < cols;
    cnt += ok[k] ? VE : 0;
  }
  const float inv_cnt = cnt ? __frcp_rn(static_cast<float>(cnt)) : 0.f;
  auto col = [&](int k) { return col0 + (k * T + tid) * VE; };
  pdl_trigger();
  pdl_wait();

  for (; row < p.rows; row += walkers) {
    const int64_t base = row * p.H;
    Grp<DT, VE> rf[NV], rx[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rf[k].zero();
      rx[k].zero();
      if (ok[k] && ADDLN_IN(701, (base + col(k)) * S, VE * S, f_rows_bytes(p, S))) {
        rf[k].load(p.f, base + col(k));
        rx[k].load(p.x, base + col(k));
      }
    }
    float2 v[kE / 2];
    to_slots<DT, VE>(rf, v);
    if (p.post != ADDLN_NORM_NONE) {
      const RowStat st = row_norm<VE, LN>(ex, v, ok, cnt, inv_cnt, p.post == ADDLN_NORM_LAYER, p.inv_h, p.eps);
      const float2 negK = dup2(-st.K), negm = dup2(-st.m), r2 = dup2(st.M2);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float2 g[kE / 2], b[kE / 2];
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) g[j] = b[j] = dup2(0.f);
        if (ok[k] && ADDLN_IN(702, 4 * col(k), 4 * VE, 4 * static_cast<int64_t>(p.H))) {
          load_param<VE>(p.post_gamma, col(k), g, k);
          if (LN && p.post_beta) load_param<VE>(p.post_beta, col(k), b, k);
        }
        if constexpr (VE == 1) {
          float& u = (k & 1) ? v[k >> 1].y : v[k >> 1].x;
          u = fmaf(((u - st.K) - st.m) * st.M2, get_slot(g, k), get_slot(b, k));
        } else {
#pragma unroll
          for (int j = k * VE / 2; j < (k + 1) * VE / 2; ++j)
            v[j] = fma2(mul2(add2(add2(v[j], negK), negm), r2), g[j], b[j]);
        }
      }
      if (tid == 0 && rank == 0 && ADDLN_IN(703, 4 * row, 4, 4 * p.rows)) {
        if (p.post_rstd) p.post_rstd[row] = st.M2;
        if (LN && p.post_mean && p.post == ADDLN_NORM_LAYER) p.post_mean[row] = st.K + st.m;
      }
    }
    if (p.gate_kind == ADDLN_GATE_CHANNEL) {
      float2 g[kE / 2];
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) g[j] = dup2(0.f);
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (ok[k] && ADDLN_IN(704, 4 * col(k), 4 * VE, 4 * static_cast<int64_t>(p.H)))
          load_param<VE>(static_cast<const float*>(p.gate), col(k), g, k);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) v[j] = mul2(v[j], g[j]);
    } else if (p.gate_kind == ADDLN_GATE_ROWS) {
      const int64_t gbase = (row / p.rows_per_gate) * p.gate_stride;
      Grp<DT, VE> rg[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        rg[k].zero();
        if (ok[k] && ADDLN_IN(705, (gbase + col(k)) * S, VE * S, f_gate_bytes(p, S)))
          rg[k].load(p.gate, gbase + col(k));
      }
      float2 g[kE / 2];
      to_slots<DT, VE>(rg, g);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) v[j] = mul2(v[j], g[j]);
    }
    {
      float2 x[kE / 2];
      to_slots<DT, VE>(rx, x);
      const float2 a2 = dup2(p.a), s2 = dup2(p.s);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) v[j] = fma2(s2, v[j], mul2(a2, x[j]));
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ok[k] && ADDLN_IN(706, (base + col(k)) * S, VE * S, f_rows_bytes(p, S)))
        store_group<DT, VE>(p.h, base + col(k), v, k);
    if (p.pre == ADDLN_NORM_NONE) continue;
    // slots past the row's end: zeros, whatever the parameters were
    const RowStat st = row_norm<VE, LN>(ex, v, ok, cnt, inv_cnt, p.pre == ADDLN_NORM_LAYER, p.inv_h, p.eps);
    const float2 negK = dup2(-st.K), negm = dup2(-st.m), r2 = dup2(st.M2);
    if (tid == 0 && rank == 0 && ADDLN_IN(707, 4 * row, 4, 4 * p.rows)) {
      if (p.pre_rstd) p.pre_rstd[row] = st.M2;
      if (LN && p.pre_mean && p.pre == ADDLN_NORM_LAYER) p.pre_mean[row] = st.K + st.m;
    }
    float2 g[kE / 2], b[kE / 2];
#pragma unroll
    for (int j = 0; j < kE / 2; ++j) g[j] = b[j] = dup2(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ok[k] && ADDLN_IN(708, 4 * col(k), 4 * VE, 4 * static_cast<int64_t>(p.H))) {
        load_param<VE>(p.pre_gamma, col(k), g, k);
        if (LN && p.pre_beta) load_param<VE>(p.pre_beta, col(k), b, k);
      }
#pragma unroll
    for (int j = 0; j < kE / 2; ++j) v[j] = fma2(mul2(add2(add2(v[j], negK), negm), r2), g[j], b[j]);
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ok[k] && ADDLN_IN(709, (base + col(k)) * S, VE * S, f_rows_bytes(p, S)))
        store_group<DT, VE>(p.y, base + col(k), v, k);
  }
  // a CTA's shared memory has to outlive its peers' writes into it
  if (p.C > 1) cooperative_groups::this_cluster().sync();
}

// ------------------------------------------------------------------ host
namespace {

struct Key {
  const void* f;
  int device, threads, C;
  bool operator==(const Key& o) const {
    return f == o.f && device == o.device && threads == o.threads && C == o.C;
  }
};
struct KeyHash {
  size_t operator()(const Key& k) const {
    return std::hash<const void*>()(k.f) ^ (static_cast<size_t>(k.device) << 20) ^
           (static_cast<size_t>(k.threads) << 28) ^ (static_cast<size_t>(k.C) << 44);
  }
};
std::mutex g_mu;
std::unordered_map<Key, int, KeyHash> g_occ;

template <int DT, int VE>
auto pick(bool ln) {
  return ln ? &k_block_fwd<DT, VE, true> : &k_block_fwd<DT, VE, false>;
}

}  // namespace

int resident_walkers(const void* f, int threads, int C, const DeviceInfo& dev) {
  const Key key{f, dev.device, threads, C};
  {
    std::lock_guard<std::mutex> g(g_mu);
    auto it = g_occ.find(key);
    if (it != g_occ.end()) return it->second;
  }
  int n = 0;
  cudaError_t e;
  if (C == 1) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f, threads, 0);
    n *= dev.sms;
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(C * dev.sms));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, f, &cfg);
  }
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_CUDA;
  }
  if (n < 1) n = 1;
  std::lock_guard<std::mutex> g(g_mu);
  g_occ[key] = n;
  return n;
}

}  // namespace blk

int launch_block_fwd(int dtype, int access, bool layer_or_bias, const BlockFwdArgs& args,
                     const LaunchCtx& c, const char** name) {
  using namespace blk;
  void (*k)(BlockFwdArgs);
  if (dtype == kF32)
    k = access == 16 ? pick<kF32, 4>(layer_or_bias) : pick<kF32, 1>(layer_or_bias);
  else if (dtype == kF16)
    k = access == 16 ? pick<kF16, 8>(layer_or_bias) : access == 4 ? pick<kF16, 2>(layer_or_bias) : pick<kF16, 1>(layer_or_bias);
  else
    k = access == 16 ? pick<kBF16, 8>(layer_or_bias) : access == 4 ? pick<kBF16, 2>(layer_or_bias) : pick<kBF16, 1>(layer_or_bias);
  *name = access == 16 ? "block_fwd_v16" : access == 4 ? "block_fwd_v4" : "block_fwd_v2";
  const Shape sh = shape_of(args.H);
  BlockFwdArgs p = args;
  p.C = sh.C;
  p.slice = sh.slice;
  const int fit = resident_walkers(reinterpret_cast<const void*>(k), sh.threads, sh.C, c.dev);
  if (fit < 0) return fit;
  const cudaError_t e = launch_walkers(k, p.rows < fit ? p.rows : fit, sh, c, p);
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_block_fwd)

}  // namespace addln
