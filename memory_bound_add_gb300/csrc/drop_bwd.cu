// Backward of bias, dropout, residual sum and norm (drop_fwd.cu), in one pass
// over the rows.  With hhat = (h - mean) rstd and u = dy gamma:
//   D  = rstd (u - mean(u) - hhat mean(u hhat)) + dh    (rms: no mean(u))
//   dx = D,  df = keep ? D scale : 0
// and over the rows dgamma = sum dy hhat, dbeta = sum dy, dbias = sum df.
//
// Column sums.  A thread always has the same columns, so its sums stay in
// registers; the walkers of a CTA join them at the end, each CTA leaves one
// fp32 partial, and k_drop_sums adds the partials in a fixed order.
#include "philox.cuh"

namespace addln {
namespace blk {

// Sums of both parts of v over the walker's threads, the same bits in every
// one: a warp butterfly, then the warps' sums in a fixed order.
__device__ __forceinline__ float2 walker_sum2(Exchange<true>& ex, float2 v) {
  constexpr unsigned kAll = 0xffffffffu;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(kAll, v.x, off), __shfl_xor_sync(kAll, v.y, off)));
  if (ex.w.warps == 1) return v;
  const float4* b = ex(make_float4(v.x, v.y, 0.f, 0.f));
  const int width = ex.w.width;
  float2 t = dup2(0.f);
  for (int i = (threadIdx.x & 31) & (width - 1); i < ex.w.warps; i += 32) t = add2(t, make_float2(b[i].x, b[i].y));
  for (int off = 1; off < width; off <<= 1)
    t = add2(t, make_float2(__shfl_xor_sync(kAll, t.x, off), __shfl_xor_sync(kAll, t.y, off)));
  return t;
}

// Column sums of a kernel: dgamma, with FULL dbeta, with BIAS dbias.
__host__ __device__ constexpr int drop_sums(bool full, bool bias) { return 1 + full + bias; }

// Threads a CTA and registers a thread: 8 columns of a 16-bit type a thread fit 96
// registers, so that more rows are on an SM at once (us, 4096x768 fp16 layer with all
// gradients: 16 columns and 128 registers 15.2, 8 and 128 14.1, 8 and 96 13.3, 8 and
// 80 14.6); shifted rows, and three sums of edged ones, need more.
// (sums: column sums)
__host__ __device__ constexpr bool bwd_lean(int dt, int nv, int sums, int mode) {
  return dt != kF32 && nv == 1 && (mode == kAligned || (mode == kEdged && sums < 3));
}
__host__ __device__ constexpr int bwd_threads(int dt, int nv, int sums, int mode) {
  return bwd_lean(dt, nv, sums, mode) ? 640 : kMaxThreads;
}
template <int DT, int NV, int A, int MODE>
constexpr int bwd_regs() {
  return bwd_lean(DT, NV, A, MODE) ? 96 : 128;
}

// FULL: a layer norm, or dbeta is wanted.  BIAS: dbias is wanted.  MODE: how
// rows lie.
//
// The call moves 5 rows H elements with dy and dh.  Up to three column sums hold the
// registers that a second row a thread would need; an SM has one or two rows at a
// time.  With rms norms and many rows it is bound by memory: 32768x8192 bf16 419 us
// (6.4 TB/s, 0.96 of a copy), 8192x4096 58.0 (0.87), fp32 103 (0.98); layer norms with
// all gradients by instructions: 65.1 us (0.77), 65536x768 107 (0.56); rows of more
// than 4096 columns leave 10 to 16 warps an SM: 8192x5001 105 us (0.58; 8 columns a
// thread, 20 warps, 110).  Few rows pay for the sums: 4096x768 fp16 layer 14.2 us, of
// which joining them in a CTA and the second kernel take 4.3.
template <int DT, int NV, bool FULL, bool BIAS, int MODE>
__global__ void __launch_bounds__(bwd_threads(DT, NV, drop_sums(FULL, BIAS), MODE))
    __maxnreg__((bwd_regs<DT, NV, drop_sums(FULL, BIAS), MODE>()))
    k_drop_bwd(const __grid_constant__ DropBwdArgs p) {
  using IO = Io<DT>;
  constexpr bool SH = MODE == kShifted;
  constexpr int S = IO::kBytes, VE = IO::kVec, N = VE / 2;
  constexpr int A = drop_sums(FULL, BIAS), NT = 3;
  constexpr int P = NV * N;
  using R = Ring<DT, NV, NT, MODE>;
  extern __shared__ __align__(128) unsigned char smem[];
  if (p.w.C > 1) cluster_started();
  const int T = p.w.cta_warps * 32;
  const int side = p.w.rows_per_cta > 1 ? threadIdx.x / T : 0, tid = threadIdx.x - side * T;
  const int rank = p.w.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.w.C);
  const int64_t cta = blockIdx.x / p.w.C;
  const int64_t stride = static_cast<int64_t>(gridDim.x / p.w.C) * p.w.rows_per_cta;
  int64_t row = first_row<MODE>(cta, p.w.rows_per_cta, side);
  const int col0 = rank * p.w.slice;
  constexpr int slots = kMaxSlots;
  const int64_t extent = p.rows * static_cast<int64_t>(p.H) * S;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  R ring;
  ring.base = smem_addr(smem) + warp * kMaxSlots * R::kSlot + lane * 16;
  Kept<VE, NV> kept;  // gamma
  kept.base = smem_addr(smem) + p.kept_at + warp * Kept<VE, NV>::template bytes<1>() + lane * 16;
  Exchange<true> ex{p.w, p.sums_at + side * 2 * p.w.warps * 16, 0};
  Cols<VE, NV> cs;
  if constexpr (MODE == kEdged)
    cs.init_edged(tid >> 5, col0, p.w.slice, p.H, static_cast<int>(row * p.H & (VE - 1)));
  else
    cs.init(tid >> 5, col0, min(p.w.slice, p.H - col0));
  const bool has_dy = p.dy != nullptr, has_dh = p.dh != nullptr;

  auto offset = [&](int64_t r) { return (r * p.H + cs.c0) * S; };
  auto fetch = [&](int slot, int64_t r) {
    if (r < p.rows) {
      const int64_t at = offset(r);
      if (has_dy) {
        ring.template fetch<0>(cs, slot, p.dy, at, 780, extent);
        ring.template fetch<1>(cs, slot, p.h, at, 781, extent);
      }
      if (has_dh) ring.template fetch<2>(cs, slot, p.dh, at, 782, extent);
    }
    ring.commit();
  };
  float mean_n = 0.f, rstd_n = 0.f;  // of the next row
  auto stats = [&](int64_t r) {
    if (r >= p.rows || !has_dy || !ADDLN_IN(783, 4 * r, 4, 4 * p.rows)) return;
    rstd_n = __ldg(p.rstd + r);
    if constexpr (FULL)
      if (p.mean) mean_n = __ldg(p.mean + r);
  };
  // where a walker has few rows
  if (p.rows <= 8 * stride)
    for (int s = 0; s < slots && row + s * stride < p.rows; ++s) {
      const int64_t at = offset(row + s * stride);
      prefetch_row<S>(p.dy, at, cs, 779, extent);
      prefetch_row<S>(p.dy ? p.h : nullptr, at, cs, 779, extent);
      prefetch_row<S>(p.dh, at, cs, 779, extent);
    }
  pdl_trigger();
  pdl_wait();
  // a tensor that the call does not have is zeros, written once
  for (int s = 0; s < slots; ++s) {
    if (!has_dy) ring.template clear<0>(s), ring.template clear<1>(s);
    if (!has_dh) ring.template clear<2>(s);
  }
  for (int s = 0; s < slots; ++s) fetch(s, row + s * stride);
  Philox<(A < 3 && !bwd_lean(DT, NV, A, MODE))> rng;
  rng.init(p.drop);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float g[VE];
    load_params<VE, MODE>(has_dy ? p.gamma : nullptr, cs.col(k), p.H, 0.f, g, 784);
    kept.put(0, k, g);
  }
  stats(row);
  if (p.w.C > 1) cluster_wait_started();

  float2 sg[P], sb[FULL ? P : 1], sf[BIAS ? P : 1];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    sg[j] = dup2(0.f);
    if constexpr (FULL) sb[j] = dup2(0.f);
    if constexpr (BIAS) sf[j] = dup2(0.f);
  }
  const float2 scale = dup2(p.drop.scale);
  for (int slot = 0; row < p.rows; row += stride, slot = slot + 1 == slots ? 0 : slot + 1) {
    const int64_t off = offset(row);
    const uint64_t at = static_cast<uint64_t>(row * p.H + cs.c0);
    Mask<VE, NV, MODE> mask;
    if (p.drop.on) mask.row(rng, at, p.drop.above, p.drop.wide);
    ring.template wait<1>();
    ring.meet();
    const float2 nm = dup2(-mean_n), rs = dup2(rstd_n);
    stats(row + stride);
    int sh[NT] = {0, 0, 0};
    if constexpr (SH) sh[0] = low4(p.dy, off), sh[1] = low4(p.h, off), sh[2] = low4(p.dh, off);
    auto take = [&](int i, int k, float2 (&v)[N]) { IO::to_pairs(ring.take(slot, i, k, sh[i]), v); };
    auto hat = [&](int k, float2 (&v)[N]) {
      take(1, k, v);
      if (MODE == kEdged && k == 0) cs.clear_low(v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = mul2(FULL ? add2(v[j], nm) : v[j], rs);
    };
    float2 t[P];
    float2 q0 = dup2(0.f), q1 = dup2(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 hh[N], dy[N], d[N], u[N];
      const int j0 = k * N;
      hat(k, hh);
      take(0, k, dy);
      take(2, k, d);
      if (MODE == kEdged && k == 0) cs.clear_low(dy), cs.clear_low(d);
      kept.get(0, k, u);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        u[i] = mul2(u[i], dy[i]);
        sg[j0 + i] = fma2(dy[i], hh[i], sg[j0 + i]);
        q0 = fma2(u[i], hh[i], q0);
        if constexpr (FULL) {
          sb[j0 + i] = add2(sb[j0 + i], dy[i]);
          q1 = add2(q1, u[i]);
        }
        t[j0 + i] = fma2(rs, u[i], d[i]);
      }
    }
    float2 m = make_float2(q0.x + q0.y, q1.x + q1.y);
    if (has_dy) m = walker_sum2(ex, m);
    // rstd mean(u hhat), rstd mean(u)
    const float2 na2 = dup2(-rs.x * (m.x * p.inv_h));
    const float2 na1 = dup2(FULL && p.norm == ADDLN_NORM_LAYER ? -rs.x * (m.y * p.inv_h) : 0.f);
    Writer<DT, NV, MODE> dx, df;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 hh[N], o[N];
      hat(k, hh);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 v = t[k * N + i];
        o[i] = fma2(na2, hh[i], FULL ? add2(v, na1) : v);
      }
      if (p.dx != nullptr) dx.put(cs, p.dx, off, k, IO::from_pairs(o), 785, extent);
      if (p.drop.on) mask.apply(rng, at, k, p.drop.above, p.drop.wide, scale, o);
      if constexpr (BIAS) {
#pragma unroll
        for (int i = 0; i < N; ++i) sf[k * N + i] = add2(sf[k * N + i], o[i]);
      }
      df.put(cs, p.df, off, k, IO::from_pairs(o), 786, extent);
    }
    ring.meet();
    fetch(slot, row + slots * stride);
  }
  if (p.part != nullptr) {
    // the CTA's walkers join their sums in shared memory, halving their number
    // (the ring is free: what is in flight arrives first)
    int top = 1;
    while (top < p.w.rows_per_cta) top *= 2;
    if (top > 1) {
      ring.template wait<0>();
      __syncthreads();
    }
    for (int half = top / 2; half > 0; half /= 2) {
      const int to = side < half ? side : side - half;
      float* at = reinterpret_cast<float*>(smem) + static_cast<int64_t>(to) * A * 2 * P * T + tid;
      const bool gives = side >= half && side < 2 * half, gets = side < half && side + half < p.w.rows_per_cta;
      auto give = [&](const float2 (&v)[P], int a) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          at[(a * 2 * P + 2 * j) * T] = v[j].x;
          at[(a * 2 * P + 2 * j + 1) * T] = v[j].y;
        }
      };
      auto get = [&](float2 (&v)[P], int a) {
#pragma unroll
        for (int j = 0; j < P; ++j)
          v[j] = add2(v[j], make_float2(at[(a * 2 * P + 2 * j) * T], at[(a * 2 * P + 2 * j + 1) * T]));
      };
      if (gives) {
        give(sg, 0);
        if constexpr (FULL) give(sb, 1);
        if constexpr (BIAS) give(sf, A - 1);
      }
      __syncthreads();
      if (gets) {
        get(sg, 0);
        if constexpr (FULL) get(sb, 1);
        if constexpr (BIAS) get(sf, A - 1);
      }
      __syncthreads();
    }
    if (side == 0) {
      float* out = p.part + cta * A * p.Hp;
      store_cols<VE, NV, MODE>(out, cs, 787, p.Hp, sg);
      if constexpr (FULL) store_cols<VE, NV, MODE>(out + p.Hp, cs, 788, p.Hp, sb);
      if constexpr (BIAS) store_cols<VE, NV, MODE>(out + (A - 1) * p.Hp, cs, 789, p.Hp, sf);
    }
  }
  if (p.w.C > 1) cooperative_groups::this_cluster().sync();
}

// The CTAs' column sums of QUADS column quads, added in a fixed order.  Its time is a
// launch and its loads' latency.
template <bool FULL, bool BIAS, int QUADS, int THREADS>
__global__ void __launch_bounds__(THREADS) k_drop_sums(const __grid_constant__ DropBwdArgs p) {
  constexpr int A = drop_sums(FULL, BIAS);
  __shared__ float4 wsum[THREADS / 32][A][QUADS];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x;
  const int j = (blockIdx.x * QUADS + t % QUADS) * 4;  // the thread's first column
  float4 r[A];
  block_quad_sums<A, QUADS, THREADS>(p.part + j, p.parts, static_cast<int64_t>(A) * p.Hp, p.Hp, j < p.H,
                            (p.parts * A * p.Hp - j) * 4, wsum, r);
  if (t >= QUADS) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c = j + q;
    if (c >= p.H || !ADDLN_IN(790, 4 * c, 4, 4 * static_cast<int64_t>(p.H))) continue;
    auto at = [&](int a) { return q == 0 ? r[a].x : q == 1 ? r[a].y : q == 2 ? r[a].z : r[a].w; };
    if (p.dgamma) p.dgamma[c] = at(0);
    if (FULL && p.dbeta) p.dbeta[c] = at(FULL ? 1 : 0);
    if (BIAS && p.dbias) p.dbias[c] = at(A - 1);
  }
}

// ------------------------------------------------------------------ host
namespace {

using BwdKernel = void (*)(DropBwdArgs);

struct Choice {
  BwdKernel k = nullptr;
  Shape sh{};
  int smem = 0, kept_at = 0, sums_at = 0;
};

// NV groups of VE columns a thread; a CTA of up to bwd_threads threads for as
// many rows side by side as fit it, else one CTA for a row, else a cluster of
// as few CTAs as hold it.  Shared memory: the ring (at least what the walkers
// need to join their sums), gamma, the row sums.
template <int DT, int NV, bool FULL, bool BIAS, int MODE>
Choice make(int H, int64_t rows, int sms) {
  constexpr int VE = Io<DT>::kVec, kMost = bwd_threads(DT, NV, drop_sums(FULL, BIAS), MODE);
  Choice c;
  c.k = &k_drop_bwd<DT, NV, FULL, BIAS, MODE>;
  if (MODE == kEdged) H += VE - 1;
  const int groups = (H + VE - 1) / VE;
  c.sh.C = (groups + NV * kMost - 1) / (NV * kMost);
  c.sh.slice = c.sh.C == 1 ? H : ((H + c.sh.C - 1) / c.sh.C + 15) / 16 * 16;
  const int threads = ((c.sh.slice + VE - 1) / VE + 32 * NV - 1) / (32 * NV) * 32;
  c.sh.rows = c.sh.C > 1 ? 1 : rows_side_by_side(kMost / threads, rows, sms);
  c.sh.threads = threads * c.sh.rows;
  const int warps = c.sh.threads / 32;
  int ring = warps * kMaxSlots * static_cast<int>(Ring<DT, NV, 3, MODE>::kSlot);
  int half = 0;  // walkers that give their sums to another at once
  for (int top = 1; top < c.sh.rows; top *= 2) half = top;
  const int join = half * drop_sums(FULL, BIAS) * NV * VE * threads * 4;
  if (ring < join) ring = join;
  c.kept_at = ring;
  c.sums_at = c.kept_at + warps * static_cast<int>(Kept<VE, NV>::template bytes<1>());
  c.smem = c.sums_at + c.sh.rows * 2 * (threads / 32) * c.sh.C * 16;
  return c;
}

// The rows that walkers of 8 columns of a 16-bit type a thread have eight each of, in
// CTAs of up to `most` threads.
inline int64_t few_rows(int H, int sms, int most) {
  const int t = (H + 255) / 256 * 32;
  return t > most ? 0 : 8 * static_cast<int64_t>(sms) * (most / t);
}

// 16 columns of a 16-bit type a thread (8 of fp32) where a row is longer than a
// warp's 8 and a walker has more than eight rows (or none would fit one CTA); else 8
// (fp32: 4 for short rows).  us with 8 / 16: 4096x768 layer (6 rows to a walker)
// 13.3 / 15.2, 65536x768 124 / 111, 8192x2048 rms 44 / 33, 8192x4096 83 / 59.  Three
// column sums of shifted rows spill with 16.
template <int DT, bool FULL, bool BIAS, int MODE>
Choice choose(int H, int64_t rows, int sms) {
  if constexpr (!(FULL && BIAS && MODE == kShifted && DT != kF32)) {
    if (H > 32 * Io<DT>::kVec && (DT == kF32 || rows > few_rows(H, sms, bwd_threads(DT, 1, drop_sums(FULL, BIAS), MODE))))
      return make<DT, 2, FULL, BIAS, MODE>(H, rows, sms);
  }
  return make<DT, 1, FULL, BIAS, MODE>(H, rows, sms);
}

template <int DT, int MODE>
Choice choose(int H, bool full, bool bias, int64_t rows, int sms) {
  if (full) return bias ? choose<DT, true, true, MODE>(H, rows, sms) : choose<DT, true, false, MODE>(H, rows, sms);
  return bias ? choose<DT, false, true, MODE>(H, rows, sms) : choose<DT, false, false, MODE>(H, rows, sms);
}

template <int DT>
Choice choose(int H, int mode, bool full, bool bias, int64_t rows, int sms) {
  return mode == kAligned ? choose<DT, kAligned>(H, full, bias, rows, sms)
         : mode == kEdged ? choose<DT, kEdged>(H, full, bias, rows, sms)
                          : choose<DT, kShifted>(H, full, bias, rows, sms);
}

Choice choose(int dtype, int H, int mode, bool full, bool bias, int64_t rows, int sms) {
  return dtype == kF32   ? choose<kF32>(H, mode, full, bias, rows, sms)
         : dtype == kF16 ? choose<kF16>(H, mode, full, bias, rows, sms)
                         : choose<kBF16>(H, mode, full, bias, rows, sms);
}

int fit_of(const Choice& c, const DeviceInfo& dev) {
  return resident_units(reinterpret_cast<const void*>(c.k), c.sh, c.smem, dev);
}

int64_t part_bytes(int64_t parts, int sums, int64_t Hp) { return parts * sums * Hp * 4; }

template <bool FULL, bool BIAS>
BwdKernel pick_sums(int quads, int threads) {
  if (threads == 512) return quads == 8 ? &k_drop_sums<FULL, BIAS, 8, 512> : &k_drop_sums<FULL, BIAS, 4, 512>;
  return quads == 8 ? &k_drop_sums<FULL, BIAS, 8, 256> : &k_drop_sums<FULL, BIAS, 4, 256>;
}

}  // namespace
}  // namespace blk

// What any number of rows up to this one needs: their CTAs are no more than
// SMs, or than those of either kernel that fit with as many rows side by side as
// there is room for, and for edged rows as many again as make it a multiple of 8.
int64_t drop_bwd_workspace_bytes(int dtype, int mode, bool full, bool bias, int64_t rows, int H, const DeviceInfo& dev) {
  using namespace blk;
  int64_t units = dev.sms;
  for (const int64_t r : {few_rows(H, dev.sms, 640), few_rows(H, dev.sms, kMaxThreads), INT64_MAX / 2}) {
    if (r == 0) continue;  // wider than a CTA
    const int fit = fit_of(choose(dtype, H, mode, full, bias, r, dev.sms), dev);
    if (fit < 0) return fit;
    if (fit > units) units = fit;
  }
  if (units > rows) units = rows;
  if (mode == kEdged) units = (units + 7) / 8 * 8;
  return part_bytes(units, drop_sums(full, bias), (H + 3) / 4 * 4);
}

int launch_drop_bwd(int dtype, int mode, const DropBwdArgs& args, void* ws, int64_t ws_bytes, const LaunchCtx& c) {
  using namespace blk;
  DropBwdArgs p = args;
  const bool full = p.norm == ADDLN_NORM_LAYER || p.dbeta, bias = p.dbias != nullptr;
  const Choice ch = choose(dtype, p.H, mode, full, bias, p.rows, c.dev.sms);
  p.w = walk_of(ch.sh);
  const int fit = fit_of(ch, c.dev);
  if (fit < 0) return fit;
  if (mode == kEdged && fit < 8) return launch_drop_bwd(dtype, kShifted, args, ws, ws_bytes, c);
  p.parts = units_for((p.rows + ch.sh.rows - 1) / ch.sh.rows, fit, mode == kEdged);
  p.kept_at = ch.kept_at;
  p.sums_at = ch.sums_at;
  p.Hp = (p.H + 3) / 4 * 4;
  const bool cols = p.dgamma || p.dbeta || p.dbias;
  p.part = nullptr;
  if (cols) {
    if (ws == nullptr || ws_bytes < part_bytes(p.parts, drop_sums(full, bias), p.Hp) || (reinterpret_cast<uintptr_t>(ws) & 15u))
      return ADDLN_ERR_WORKSPACE;
    p.part = static_cast<float*>(ws);
  }
  cudaError_t e = launch_units(ch.k, p.parts, ch.sh, ch.smem, c, p);
  if (e == cudaSuccess && cols) {
    // 512 threads where each of 256 would have several partials; four quads a block
    // unless that makes more than two blocks an SM (us of a call with 256 and two quads,
    // 512 and four, 512 and eight: 4096x768 fp16 rms 13.2, 12.4, 12.6; 2048x4096 layer
    // 23.7, 23.0, 23.6; 4096x8192 rms 63.0, 62.1, 60.2; 64x768 fp32, 64 partials, with 256
    // / 512 and four 4.0 / 4.7).
    const int threads = p.parts > 128 ? 512 : 256, quads = p.Hp / 16 > 2 * c.dev.sms ? 8 : 4;
    const BwdKernel ks = full ? (bias ? pick_sums<true, true>(quads, threads) : pick_sums<true, false>(quads, threads))
                              : (bias ? pick_sums<false, true>(quads, threads) : pick_sums<false, false>(quads, threads));
    e = launch_kernel(ks, dim3(static_cast<unsigned>((p.Hp / 4 + quads - 1) / quads)), dim3(static_cast<unsigned>(threads)), 0,
                      c.stream, c.pdl, p);
  }
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_drop_bwd)

}  // namespace addln
