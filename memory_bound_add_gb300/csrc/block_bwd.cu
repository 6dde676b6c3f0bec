// Backward of the block boundary (block_fwd.cu), in one pass over the rows.
// With hhat = (h - mean_h) r_h, u = dy g, fhat = (f - mean_f) r_f:
//   D  = r_h (u - mean(u) - hhat mean(u hhat)) + dh     (rms: no mean(u))
//   dx = a D,  dn = s D gate
//   v  = dn pg,  df = r_f (v - mean(v) - fhat mean(v fhat))
// and over the rows dg = sum dy hhat, db = sum dy, dpg = sum dn fhat,
// dpb = sum dn, dgate = sum s D (fhat pg + pb).
//
// Column sums.  A walker takes a contiguous range of rows and a thread
// always the same columns, so its sums stay in registers.  Where one gate
// row serves all rows (or there is none) two sums give three gradients:
// with S1 = sum s D fhat and S0 = sum s D, dpg = gate S1, dpb = gate S0 and
// dgate = pg S1 + pb S0.  With gate rows the sums over a gate row's rows are
// written as soon as the range leaves it, rounded to the gate's type, when
// all its rows are the walker's; a gate row shared with other walkers leaves
// an fp32 partial.  k_block_sums adds all partials in a fixed order, so the
// result does not depend on scheduling.
#include "block.cuh"

#include "block.h"

namespace addln {
namespace blk {

constexpr int kE = 8;  // columns a thread
constexpr int kSlice = kE * kMaxThreads;

// First row of walker w's range.
__host__ __device__ __forceinline__ int64_t range_begin(int64_t w, int64_t rows, int64_t walkers) {
  const int64_t q = rows / walkers, r = rows - q * walkers;
  return w * q + (w < r ? w : r);
}

__device__ __forceinline__ int64_t b_rows_bytes(const BlockBwdArgs& p, int S) {
  return p.rows * static_cast<int64_t>(p.H) * S;
}
__device__ __forceinline__ int64_t b_gate_bytes(const BlockBwdArgs& p, int S) {
  return ((p.gate_rows - 1) * p.gate_stride + p.H) * S;
}

// Column sums a walker keeps: dgamma and sum(s D fhat) or dpg, and with FULL
// dbeta and sum(s D) or dpb.
__host__ __device__ constexpr int sums_of(bool full) { return full ? 4 : 2; }

template <int DT, int VE>
__device__ __forceinline__ void load_row(const void* t, int64_t base, const int (&col)[kE / VE],
                                         const bool (&ok)[kE / VE], int site, int64_t extent,
                                         Grp<DT, VE> (&r)[kE / VE]) {
#pragma unroll
  for (int k = 0; k < kE / VE; ++k) {
    r[k].zero();
    if (ok[k] && ADDLN_IN(site, (base + col[k]) * Io<DT>::kBytes, VE * Io<DT>::kBytes, extent))
      r[k].load(static_cast<const char*>(t) + (base + col[k]) * Io<DT>::kBytes);
  }
}

template <int VE>
__device__ __forceinline__ void load_cols(const float* t, const int (&col)[kE / VE], const bool (&ok)[kE / VE],
                                          int site, int H, float fill, float2 (&v)[kE / 2]) {
#pragma unroll
  for (int j = 0; j < kE / 2; ++j) v[j] = dup2(fill);
  if (t == nullptr) return;
#pragma unroll
  for (int k = 0; k < kE / VE; ++k)
    if (ok[k] && ADDLN_IN(site, 4 * col[k], 4 * VE, 4 * static_cast<int64_t>(H))) load_param<VE>(t, 4u * col[k], v, k);
}

// Stores slots as fp32 columns of an [Hp] vector.
template <int VE>
__device__ __forceinline__ void store_cols(float* t, const int (&col)[kE / VE], const bool (&ok)[kE / VE],
                                           int site, int Hp, const float2 (&v)[kE / 2]) {
#pragma unroll
  for (int k = 0; k < kE / VE; ++k) {
    if (!ok[k] || !ADDLN_IN(site, 4 * col[k], 4 * VE, 4 * static_cast<int64_t>(Hp))) continue;
    if constexpr (VE >= 4) {
#pragma unroll
      for (int q = 0; q < VE / 4; ++q)
        *reinterpret_cast<float4*>(t + col[k] + 4 * q) =
            make_float4(v[k * VE / 2 + 2 * q].x, v[k * VE / 2 + 2 * q].y, v[k * VE / 2 + 2 * q + 1].x,
                        v[k * VE / 2 + 2 * q + 1].y);
    } else if constexpr (VE == 2) {
      *reinterpret_cast<float2*>(t + col[k]) = v[k];
    } else {
      t[col[k]] = get_slot(v, k);
    }
  }
}

// FULL: some norm is a layer norm or has a bias.  GR: a gate with rows.
template <int DT, int VE, bool FULL, bool GR>
__global__ void __launch_bounds__(kMaxThreads) k_block_bwd(const __grid_constant__ BlockBwdArgs p) {
  constexpr int NV = kE / VE;
  [[maybe_unused]] constexpr int S = Io<DT>::kBytes;
  constexpr int A = sums_of(FULL);
  __shared__ float4 parts[2][kMaxWarps * kMaxCluster];
  const int T = blockDim.x, tid = threadIdx.x;
  const int rank = p.w.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.w.C);
  const int64_t walker = blockIdx.x / p.w.C;
  const int col0 = rank * p.w.slice;
  const int cols = min(p.w.slice, p.H - col0);
  Exchange ex{parts, p.w, rank, 0};
  bool ok[NV];
  int col[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    ok[k] = (k * T + tid) * VE < cols;
    col[k] = col0 + (k * T + tid) * VE;
  }
  pdl_trigger();
  pdl_wait();

  const int64_t r0 = range_begin(walker, p.rows, p.walkers);
  const int64_t r1 = range_begin(walker + 1, p.rows, p.walkers);
  const bool has_dy = p.dy != nullptr, has_dh = p.dh != nullptr;
  const bool post = p.post != ADDLN_NORM_NONE;
  const bool need_f = post || p.gate_kind != ADDLN_GATE_NONE;
  const int64_t extent = b_rows_bytes(p, S);

  float2 sg[kE / 2], sb[kE / 2], s1[kE / 2], s0[kE / 2], sd[kE / 2];
#pragma unroll
  for (int j = 0; j < kE / 2; ++j) sg[j] = sb[j] = s1[j] = s0[j] = sd[j] = dup2(0.f);
  int64_t g = 0, left = 0;  // gate row, rows left of it
  bool first = true;        // the gate row began before or at the range's begin
  if constexpr (GR) {
    g = r0 / p.rows_per_gate;
    left = (g + 1) * p.rows_per_gate - r0;
  }

  for (int64_t row = r0; row < r1; ++row) {
    const int64_t base = row * p.H;
    float2 D[kE / 2];
    if (has_dh) {
      Grp<DT, VE> r[NV];
      load_row<DT, VE>(p.dh, base, col, ok, 721, extent, r);
      to_slots<DT, VE, NV>(r, D);
    } else {
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) D[j] = dup2(0.f);
    }
    Grp<DT, VE> rf[NV];
    if (need_f) load_row<DT, VE>(p.f, base, col, ok, 722, extent, rf);
    if (has_dy) {
      float2 dy[kE / 2], hh[kE / 2], u[kE / 2];
      {
        Grp<DT, VE> r[NV];
        load_row<DT, VE>(p.dy, base, col, ok, 723, extent, r);
        to_slots<DT, VE, NV>(r, dy);
        load_row<DT, VE>(p.h, base, col, ok, 724, extent, r);
        to_slots<DT, VE, NV>(r, hh);
      }
      float mu = 0.f, rs = 0.f;
      if (ADDLN_IN(725, 4 * row, 4, 4 * p.rows)) {
        rs = __ldg(p.pre_rstd + row);
        if (FULL && p.pre == ADDLN_NORM_LAYER) mu = __ldg(p.pre_mean + row);
      }
      const float2 negmu = dup2(-mu), rs2 = dup2(rs);
      load_cols<VE>(p.pre_gamma, col, ok, 726, p.H, 0.f, u);
      float2 t1 = dup2(0.f), t2 = dup2(0.f);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) {
        hh[j] = mul2(add2(hh[j], negmu), rs2);
        u[j] = mul2(u[j], dy[j]);
        sg[j] = fma2(dy[j], hh[j], sg[j]);
        if constexpr (FULL) {
          sb[j] = add2(sb[j], dy[j]);
          t1 = add2(t1, u[j]);
        }
        t2 = fma2(u[j], hh[j], t2);
      }
      const float2 t = walker_sum2(ex, make_float2(t1.x + t1.y, t2.x + t2.y));
      const float2 nm = dup2(FULL && p.pre == ADDLN_NORM_LAYER ? -(t.x * p.inv_h) : 0.f);
      const float2 nmx = dup2(-(t.y * p.inv_h));
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) D[j] = fma2(rs2, add2(u[j], fma2(hh[j], nmx, nm)), D[j]);
    }
    {
      float2 o[kE / 2];
      const float2 a2 = dup2(p.a);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) o[j] = mul2(a2, D[j]);
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (ok[k] && ADDLN_IN(727, (base + col[k]) * S, VE * S, extent)) store_group<DT, VE>(static_cast<char*>(p.dx) + (base + col[k]) * S, o, k);
    }
    // D becomes s D, then dn
    const float2 sc = dup2(p.s);
#pragma unroll
    for (int j = 0; j < kE / 2; ++j) D[j] = mul2(sc, D[j]);
    float2 fh[kE / 2], pg[kE / 2];
    float pr = 1.f;
    if (need_f) {
      to_slots<DT, VE, NV>(rf, fh);
      if (post) {
        float pm = 0.f;
        if (ADDLN_IN(728, 4 * row, 4, 4 * p.rows)) {
          pr = __ldg(p.post_rstd + row);
          if (FULL && p.post == ADDLN_NORM_LAYER) pm = __ldg(p.post_mean + row);
        }
        const float2 npm = dup2(-pm), pr2 = dup2(pr);
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) fh[j] = mul2(add2(fh[j], npm), pr2);
      }
    }
    if (post) load_cols<VE>(p.post_gamma, col, ok, 729, p.H, 0.f, pg);
    if constexpr (GR) {
      // the gate's gradient s D n, then dn = s D gate
      float2 b[kE / 2];
      load_cols<VE>(FULL && post ? p.post_beta : nullptr, col, ok, 730, p.H, 0.f, b);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) {
        const float2 n = post ? fma2(fh[j], pg[j], b[j]) : fh[j];
        sd[j] = fma2(D[j], n, sd[j]);
      }
      Grp<DT, VE> rg[NV];
      load_row<DT, VE>(p.gate, g * p.gate_stride, col, ok, 731, b_gate_bytes(p, S), rg);
      float2 gt[kE / 2];
      to_slots<DT, VE, NV>(rg, gt);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) D[j] = mul2(D[j], gt[j]);
      if (--left == 0 || row + 1 == r1) {
        const bool begun_here = !first || g * p.rows_per_gate >= r0;
        const bool ends_here = left == 0 || row + 1 == p.rows;
        if (begun_here && ends_here) {
          const int64_t gb = g * p.H;
#pragma unroll
          for (int k = 0; k < NV && p.dgate != nullptr; ++k)
            if (ok[k] && ADDLN_IN(732, (gb + col[k]) * S, VE * S, p.gate_rows * static_cast<int64_t>(p.H) * S))
              store_group<DT, VE>(static_cast<char*>(p.dgate) + (gb + col[k]) * S, sd, k);
        } else if (p.seg != nullptr) {
          store_cols<VE>(p.seg + (2 * walker + (first ? 0 : 1)) * p.Hp, col, ok, 733, p.Hp, sd);
        }
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) sd[j] = dup2(0.f);
        first = false;
        left = p.rows_per_gate;
        ++g;
      }
    }
    // column sums of dn fhat and dn (GR), or of s D fhat and s D
    if (need_f) {
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) {
        s1[j] = fma2(D[j], fh[j], s1[j]);
        if constexpr (FULL) s0[j] = add2(s0[j], D[j]);
      }
    }
    if (!GR && p.gate_kind == ADDLN_GATE_CHANNEL) {
      float2 gt[kE / 2];
      load_cols<VE>(static_cast<const float*>(p.gate), col, ok, 734, p.H, 0.f, gt);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) D[j] = mul2(D[j], gt[j]);
    }
    if (post) {
      float2 t1 = dup2(0.f), t2 = dup2(0.f);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) {
        D[j] = mul2(D[j], pg[j]);
        if constexpr (FULL) t1 = add2(t1, D[j]);
        t2 = fma2(D[j], fh[j], t2);
      }
      const float2 t = walker_sum2(ex, make_float2(t1.x + t1.y, t2.x + t2.y));
      const float2 nm = dup2(FULL && p.post == ADDLN_NORM_LAYER ? -(t.x * p.inv_h) : 0.f);
      const float2 nmx = dup2(-(t.y * p.inv_h)), pr2 = dup2(pr);
#pragma unroll
      for (int j = 0; j < kE / 2; ++j) D[j] = mul2(pr2, add2(D[j], fma2(fh[j], nmx, nm)));
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ok[k] && ADDLN_IN(735, (base + col[k]) * S, VE * S, extent)) store_group<DT, VE>(static_cast<char*>(p.df) + (base + col[k]) * S, D, k);
  }
  if (p.part != nullptr) {
    float* out = p.part + walker * A * p.Hp;
    store_cols<VE>(out, col, ok, 736, p.Hp, sg);
    store_cols<VE>(out + p.Hp, col, ok, 737, p.Hp, s1);
    if constexpr (FULL) {
      store_cols<VE>(out + 2 * p.Hp, col, ok, 738, p.Hp, sb);
      store_cols<VE>(out + 3 * p.Hp, col, ok, 739, p.Hp, s0);
    }
  }
  if (p.w.C > 1) cooperative_groups::this_cluster().sync();
}

// ------------------------------------------------------------ joining sums
// blockIdx.y == 0: the walkers' column sums of kQuads column quads, added in
// a fixed order (thread t takes quad t % kQuads and the walkers t / kQuads,
// + kSlices, ...; then a butterfly over the warp's lanes of that quad and
// the warps in order), and from them the gradients of both norms and of a
// per-channel gate.  blockIdx.y > 0: the gate rows that several walkers
// share, the walkers in order.
constexpr int kSumThreads = 256, kQuads = 4, kSlices = kSumThreads / kQuads;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Sum over i < n of the quad at src + i * ld (in floats); every thread of the
// block takes part, the result is in the threads below kQuads.
__device__ __forceinline__ float4 block_quad_sum(const float* src, int64_t n, int64_t ld, bool in,
                                                 int64_t extent, float4 (*wsum)[kQuads]) {
  constexpr int kU = 8;  // loads in flight a thread
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in)
    for (int64_t i0 = t / kQuads; i0 < n; i0 += kSlices * kU) {
      float4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t i = i0 + u * kSlices;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n && ADDLN_IN(741, i * ld * 4, 16, extent))
          v[u] = __ldcg(reinterpret_cast<const float4*>(src + i * ld));
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) acc = add4(acc, v[u]);
    }
#pragma unroll
  for (int off = kQuads; off < 32; off <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
  }
  __syncthreads();  // the last call's sums have been read
  if (lane < kQuads) wsum[warp][lane] = acc;
  __syncthreads();
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (t < kQuads)
    for (int w = 0; w < kSumThreads / 32; ++w) r = add4(r, wsum[w][t]);
  return r;
}

// The gate rows that more than one walker shares.  Where walkers have at
// least as many rows as a gate row, a gate row meets at most one border
// between walkers, and border b (between walkers b - 1 and b) has one if it
// lies inside a gate row; otherwise every gate row is looked at.
__host__ __device__ __forceinline__ int64_t shared_candidates(int64_t rows, int64_t walkers,
                                                              int64_t gate_rows, int64_t rpg) {
  return rows / walkers >= rpg ? walkers - 1 : gate_rows;
}

template <int DT, bool FULL>
__global__ void __launch_bounds__(kSumThreads) k_block_sums(const BlockBwdArgs p) {
  constexpr int A = sums_of(FULL);
  __shared__ float4 wsum[kSumThreads / 32][kQuads];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x;
  const int j = (blockIdx.x * kQuads + t % kQuads) * 4;  // the thread's first column
  if (blockIdx.y == 0) {
    if (p.part == nullptr) return;
    float4 r[A];
#pragma unroll
    for (int a = 0; a < A; ++a)
      r[a] = block_quad_sum(p.part + a * static_cast<int64_t>(p.Hp) + j, p.walkers, static_cast<int64_t>(A) * p.Hp,
                            j < p.H, (p.walkers * A * p.Hp - a * static_cast<int64_t>(p.Hp) - j) * 4, wsum);
    if (t >= kQuads) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = j + q;
      if (c >= p.H || !ADDLN_IN(742, 4 * c, 4, 4 * static_cast<int64_t>(p.H))) continue;
      auto at = [&](int a) { return q == 0 ? r[a].x : q == 1 ? r[a].y : q == 2 ? r[a].z : r[a].w; };
      if (p.dpre_gamma) p.dpre_gamma[c] = at(0);
      if (FULL && p.dpre_beta) p.dpre_beta[c] = at(FULL ? 2 : 0);
      const bool channel = p.gate_kind == ADDLN_GATE_CHANNEL;
      const float gt = channel ? __ldg(static_cast<const float*>(p.gate) + c) : 1.f;
      if (p.dpost_gamma) p.dpost_gamma[c] = gt * at(1);
      if (FULL && p.dpost_beta) p.dpost_beta[c] = gt * at(FULL ? 3 : 1);
      if (channel && p.dgate) {
        float d = at(1);
        if (p.post != ADDLN_NORM_NONE) {
          d *= __ldg(p.post_gamma + c);
          if (FULL && p.post_beta) d = fmaf(__ldg(p.post_beta + c), at(FULL ? 3 : 1), d);
        }
        static_cast<float*>(p.dgate)[c] = d;
      }
    }
    return;
  }
  const int64_t rpg = p.rows_per_gate;
  int64_t g = blockIdx.y - 1;
  if (p.rows / p.walkers >= rpg) {
    const int64_t border = range_begin(blockIdx.y, p.rows, p.walkers);
    if (border % rpg == 0) return;
    g = border / rpg;
  }
  // walkers [w0, w1] with rows of gate row g: the first may hold it as its
  // last segment, the others as their first
  const int64_t b0 = g * rpg, b1 = min(p.rows, b0 + rpg);
  auto walker_of = [&](int64_t row) {
    const int64_t q = p.rows / p.walkers, r = p.rows - q * p.walkers;
    return row < r * (q + 1) ? row / (q + 1) : r + (row - r * (q + 1)) / q;
  };
  const int64_t w0 = walker_of(b0), w1 = walker_of(b1 - 1);
  if (w0 == w1) return;
  const bool head = range_begin(w0, p.rows, p.walkers) >= b0;
  const int64_t ex = p.walkers * 2 * p.Hp * 4;
  // walkers w0 + 1 .. w1 hold it in their first slot
  const float* src = p.seg + 2 * (w0 + 1) * p.Hp + j;
  const float4 rest = block_quad_sum(src, w1 - w0, 2 * static_cast<int64_t>(p.Hp), j < p.H,
                                     ex - (2 * (w0 + 1) * p.Hp + j) * 4, wsum);
  if (t >= kQuads || j >= p.H) return;
  const int64_t at0 = (2 * w0 + (head ? 0 : 1)) * p.Hp + j;
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ADDLN_IN(743, at0 * 4, 16, ex)) r = __ldcg(reinterpret_cast<const float4*>(p.seg + at0));
  r = add4(r, rest);
  const float o[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (j + q < p.H && ADDLN_IN(744, (g * p.H + j + q) * Io<DT>::kBytes, Io<DT>::kBytes,
                                p.gate_rows * static_cast<int64_t>(p.H) * Io<DT>::kBytes))
      Io<DT>::store1(p.dgate, g * p.H + j + q, o[q]);
}

// ------------------------------------------------------------------ host
namespace {

using BwdKernel = void (*)(BlockBwdArgs);

Shape shape_of(int H) {
  Shape s;
  s.C = (H + kSlice - 1) / kSlice;
  s.slice = s.C == 1 ? H : ((H + s.C - 1) / s.C + 15) / 16 * 16;
  s.threads = ((s.slice + kE - 1) / kE + 31) / 32 * 32;
  s.rows = 1;
  return s;
}

template <int DT, int VE>
BwdKernel pick_ve(bool full, bool gr) {
  if (full) return gr ? &k_block_bwd<DT, VE, true, true> : &k_block_bwd<DT, VE, true, false>;
  return gr ? &k_block_bwd<DT, VE, false, true> : &k_block_bwd<DT, VE, false, false>;
}

BwdKernel pick(int dtype, int access, bool full, bool gr) {
  if (dtype == kF32) return access == 16 ? pick_ve<kF32, 4>(full, gr) : pick_ve<kF32, 1>(full, gr);
  if (dtype == kF16)
    return access == 16 ? pick_ve<kF16, 8>(full, gr) : access == 4 ? pick_ve<kF16, 2>(full, gr) : pick_ve<kF16, 1>(full, gr);
  return access == 16 ? pick_ve<kBF16, 8>(full, gr) : access == 4 ? pick_ve<kBF16, 2>(full, gr) : pick_ve<kBF16, 1>(full, gr);
}

// Walkers of a launch: those that fit the device at once, no more than rows.
int64_t walkers_of(BwdKernel k, int64_t rows, const Shape& sh, const DeviceInfo& dev) {
  const int fit = resident_units(reinterpret_cast<const void*>(k), sh, 0, dev);
  if (fit < 0) return fit;
  return rows < fit ? rows : fit;
}

int64_t part_bytes(int64_t walkers, bool full, int64_t Hp) { return walkers * sums_of(full) * Hp * 4; }
int64_t seg_bytes(int64_t walkers, bool gr, int64_t rpg, int64_t Hp) {
  return gr && rpg > 1 ? walkers * 2 * Hp * 4 : 0;
}

template <int DT>
BwdKernel pick_sums(bool full) {
  return full ? &k_block_sums<DT, true> : &k_block_sums<DT, false>;
}

}  // namespace
}  // namespace blk

int64_t block_bwd_workspace_bytes(int dtype, int access, bool full, int64_t rows, int H, int gate_kind,
                                  int64_t rows_per_gate, const DeviceInfo& dev) {
  using namespace blk;
  const bool gr = gate_kind == ADDLN_GATE_ROWS;
  const Shape sh = shape_of(H);
  const int64_t w = walkers_of(pick(dtype, access, full, gr), rows, sh, dev);
  if (w < 0) return w;
  const int64_t Hp = (H + 3) / 4 * 4;
  return part_bytes(w, full, Hp) + seg_bytes(w, gr, rows_per_gate, Hp);
}

int launch_block_bwd(int dtype, int access, bool full, BlockBwdArgs p, void* ws, int64_t ws_bytes,
                     const LaunchCtx& c, const char** name) {
  using namespace blk;
  const bool gr = p.gate_kind == ADDLN_GATE_ROWS;
  const Shape sh = shape_of(p.H);
  const BwdKernel k = pick(dtype, access, full, gr);
  p.w = walk_of(sh);
  p.walkers = walkers_of(k, p.rows, sh, c.dev);
  if (p.walkers < 0) return static_cast<int>(p.walkers);
  p.Hp = (p.H + 3) / 4 * 4;
  const bool cols = p.dpre_gamma || p.dpre_beta || p.dpost_gamma || p.dpost_beta ||
                    (p.dgate && p.gate_kind == ADDLN_GATE_CHANNEL);
  const bool seg = gr && p.dgate != nullptr && p.rows_per_gate > 1 && p.walkers > 1;
  p.part = nullptr;
  p.seg = nullptr;
  if (cols || seg) {
    const int64_t pb = part_bytes(p.walkers, full, p.Hp);
    const int64_t need = pb + seg_bytes(p.walkers, gr, p.rows_per_gate, p.Hp);
    if (ws == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 15u)) return ADDLN_ERR_WORKSPACE;
    if (cols) p.part = static_cast<float*>(ws);
    if (seg) p.seg = reinterpret_cast<float*>(static_cast<char*>(ws) + pb);
  }
  *name = access == 16 ? "block_bwd_v16" : access == 4 ? "block_bwd_v4" : "block_bwd_v2";
  cudaError_t e = launch_units(k, p.walkers, sh, 0, c, p);
  if (e == cudaSuccess && (cols || seg)) {
    const BwdKernel ks = dtype == kF32 ? pick_sums<kF32>(full) : dtype == kF16 ? pick_sums<kF16>(full) : pick_sums<kBF16>(full);
    const int64_t ny = seg ? shared_candidates(p.rows, p.walkers, p.gate_rows, p.rows_per_gate) : 0;
    const dim3 grid(static_cast<unsigned>((p.Hp / 4 + kQuads - 1) / kQuads), static_cast<unsigned>(1 + ny));
    e = launch_kernel(ks, grid, dim3(kSumThreads), 0, c.stream, c.pdl, p);
  }
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_block_bwd)

}  // namespace addln
