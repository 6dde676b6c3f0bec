// Backward of the block boundary (block_fwd.cu), in one pass over the rows.
// With hhat = (h - mean_h) r_h, u = dy g, fhat = (f - mean_f) r_f and
// c = s gate pg (s gate without a post norm; the products' column factors):
//   t  = r_h u + dh
//   D  = t - r_h mean(u) - r_h mean(u hhat) hhat         (rms: no mean(u))
//   dx = a D,  v = c D,  df = r_f (v - mean(v) - fhat mean(v fhat))
// and over the rows dg = sum dy hhat, db = sum dy, and of D: dpg =
// s sum gate D fhat, dpb = s sum gate D, dgate = s sum D (fhat pg + pb).
//
// One exchange a row.  The means of v and v fhat are those of D, which needs
// the means of u and u hhat first; written out,
//   sum v      = sum c t      - r_h mean(u) sum c      - r_h mean(u hhat) sum c hhat
//   sum v fhat = sum c fhat t - r_h mean(u) sum c fhat - r_h mean(u hhat) sum c fhat hhat
// so all the sums a row needs (8, without layer norms 3) are taken together.
// Where dy's mean is large against its spread, D's elements carry a common error
// (of a mean(u) of that size), which a mean(v) of D itself would take out again and
// the written-out sum does not.  Error of df relative to 64 bits, so / by two
// exchanges, 64x4096 fp32 layer/layer, dy of spread 1 and mean 0, 10, 100:
// 7.1e-8 / 7.1e-8, 4.6e-7 / 2.8e-7, 5.0e-7 / 3.3e-7; dx, which has the common error
// either way, 5.1e-8, 4.4e-7, 5.1e-7.
//
// Column sums.  A walker takes a contiguous range of rows and a thread
// always the same columns, so its sums stay in registers.  Where one gate
// row serves all rows (or there is none) two sums give three gradients:
// with S1 = sum D fhat and S0 = sum D, dpg = s gate S1, dpb = s gate S0 and
// dgate = s (pg S1 + pb S0).  With gate rows the sums over a gate row's rows
// are written as soon as the range leaves it, rounded to the gate's type,
// when all its rows are the walker's; a gate row shared with other walkers
// leaves an fp32 partial.  k_block_sums adds all partials in a fixed order,
// so the result does not depend on scheduling.
//
// Several walkers share a CTA where a row needs few threads; they join their
// column sums at the end, so that there is one partial for each CTA.
#include "block.cuh"

#include "block.h"

namespace addln {
namespace blk {

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

// K sums (4 or 8) over the walker's threads, the same bits in every thread.
// Within a warp each step halves the sums a lane carries: 6 (9) exchanges
// instead of 5 K.
template <int K>
struct Sums {
  float* buf;  // [2][warps][K], this walker's
  const Walk& w;
  int rank, par, barrier;

  __device__ __forceinline__ void operator()(float (&v)[K]) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    constexpr int n = 32 / K;  // lanes that end up with the same sum
    float x[K];
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = v[i];
#pragma unroll
    for (int off = 16, m = K; m > 1; off >>= 1, m >>= 1) {
      const bool up = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < K / 2; ++i)
        if (i < m / 2) {
          const float mine = up ? x[i + m / 2] : x[i], other = up ? x[i] : x[i + m / 2];
          x[i] = mine + __shfl_xor_sync(kAll, other, off);
        }
    }
#pragma unroll
    for (int off = 16 / K; off > 0; off >>= 1) x[0] += __shfl_xor_sync(kAll, x[0], off);
    float t = x[0];
    // the sum a lane carries: its top bits
    const int at = lane / n;
    if (w.warps > 1) {
      float* b = buf + par * w.warps * K;
      par ^= 1;
      const int warp = (threadIdx.x >> 5) % w.cta_warps;
      if (w.C == 1) {
        if (lane % n == 0) b[warp * K + at] = t;
        asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(w.cta_warps * 32) : "memory");
      } else {
        namespace cg = cooperative_groups;
        cg::cluster_group cl = cg::this_cluster();
        if (lane % n == 0)
          for (int c = 0; c < w.C; ++c) cl.map_shared_rank(b, c)[(rank * w.cta_warps + warp) * K + at] = t;
        cl.sync();
      }
      // lane l adds sum l / n of the warps l % n, + n, ...
      t = 0.f;
      for (int i = lane % n; i < w.warps; i += n) t += b[i * K + at];
#pragma unroll
      for (int off = 16 / K; off > 0; off >>= 1) t += __shfl_xor_sync(kAll, t, off);
    }
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = __shfl_sync(kAll, t, i * (32 / K));
  }
};

// Threads a CTA, and the registers each may have.  Without gate rows, shifted
// rows of rms norms and 16-bit rows of layer norms that are not shifted fit
// 96: 640 threads, so that a row of 5120 columns takes one CTA instead of a
// cluster of two (us, cluster / CTA: 8192x5001 bf16 rms 296 / 177, 8192x5120
// bf16 layer 214 / 116; rows of up to 4096 columns 97 / 96).  The others spill.
__host__ __device__ constexpr bool bwd_lean(int dt, bool full, bool gr, bool sh) {
  return !gr && (sh ? !full : full && dt != kF32);
}
__host__ __device__ constexpr int bwd_threads(int dt, bool full, bool gr, bool sh) {
  return bwd_lean(dt, full, gr, sh) ? 640 : kMaxThreads;
}
template <int DT, bool FULL, bool GR, bool SH>
constexpr int bwd_regs() {
  return bwd_lean(DT, FULL, GR, SH) ? 96 : 128;
}

// FULL: some norm is a layer norm or has a bias.  GR: a gate with rows.  SH:
// some rows do not begin on 16-byte borders.
//
// The call moves 6 rows H elements.  With rms norms it is bound by memory where
// rows are many: 32768x8192 bf16 with gate rows 516 us (6.2 TB/s, 0.92 of a
// copy), 8192x4096 bf16 68 us (0.87).  The column sums take the registers for
// more rows at once: an SM has one CTA of 512 threads, whose warps meet once a
// row.  Short calls pay for that row's latency (about 2 us a row of a walker)
// and for the second kernel: 2048x4096 fp16 28.3 us (0.70).  Gate rows that serve
// a sequence each cost that kernel more than this one where they are many: below.  Layer norms need 8
// sums a row and twice the column sums, and are bound by instructions and that
// latency: 8192x4096 bf16 96 us (0.62), 4096x768 fp16 16.5 us (0.34).  A walker
// takes a contiguous range of rows, not a stride: a gate row then meets few
// walkers.
template <int DT, int NV, bool FULL, bool GR, bool SH>
__global__ void __launch_bounds__(bwd_threads(DT, FULL, GR, SH)) __maxnreg__((bwd_regs<DT, FULL, GR, SH>()))
    k_block_bwd(const __grid_constant__ BlockBwdArgs p) {
  using IO = Io<DT>;
  constexpr int S = IO::kBytes, VE = IO::kVec, N = VE / 2;
  constexpr int A = sums_of(FULL), K = FULL ? 8 : 4;
  constexpr int NT = GR ? 5 : 4, NP = FULL && GR ? 3 : 2;
  constexpr int P = NV * N;
  constexpr int kStepBytes = Cols<VE, NV>::kStep * S;
  using R = Ring<DT, NV, NT, SH>;
  extern __shared__ __align__(128) unsigned char smem[];
  if (p.w.C > 1) cluster_started();
  const int T = p.w.cta_warps * 32;
  const int side = p.w.rows_per_cta > 1 ? threadIdx.x / T : 0, tid = threadIdx.x - side * T;
  const int rank = p.w.C == 1 ? 0 : static_cast<int>(blockIdx.x % p.w.C);
  const int64_t cta = blockIdx.x / p.w.C;
  const int64_t walker = cta * p.w.rows_per_cta + side;
  const int col0 = rank * p.w.slice;
  constexpr int slots = kMaxSlots;
  R ring;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ring.base = smem_addr(smem) + warp * kMaxSlots * R::kSlot + lane * 16;
  // vector 0: gamma of the pre norm; 1: the factor c, or with gate rows s pg
  // (c is then that times the gate); 2: s pb
  Kept<VE, NV> kept;
  kept.base = smem_addr(smem) + p.kept_at + warp * Kept<VE, NV>::template bytes<NP>() + lane * 16;
  Sums<K> sums{reinterpret_cast<float*>(smem + p.sums_at) + side * 2 * p.w.warps * K, p.w, rank, 0, 1 + side};
  Cols<VE, NV> cs;
  cs.init(tid >> 5, col0, min(p.w.slice, p.H - col0));
  const bool has_dy = p.dy != nullptr, has_dh = p.dh != nullptr;
  const bool post = p.post != ADDLN_NORM_NONE;
  const bool need_f = post || p.gate_kind != ADDLN_GATE_NONE;
  const int64_t extent = b_rows_bytes(p, S);
  // a walker past the last has no rows
  const int64_t r0 = min(p.rows, range_begin(walker, p.rows, p.walkers));
  const int64_t r1 = min(p.rows, range_begin(walker + 1, p.rows, p.walkers));

  const int n = static_cast<int>(r1 - r0);  // rows of the walker
  const int row_bytes = p.H * S;
  // statistics of the next row, loaded a row ahead
  float hm_n = 0.f, hr_n = 0.f, fm_n = 0.f, fr_n = 1.f;
  auto stats = [&](int64_t r) {
    if (r >= r1 || !ADDLN_IN(725, 4 * r, 4, 4 * p.rows)) return;
    if (has_dy) hr_n = __ldg(p.pre_rstd + r);
    if (post) fr_n = __ldg(p.post_rstd + r);
    if constexpr (FULL) {
      if (p.pre_mean) hm_n = __ldg(p.pre_mean + r);
      if (p.post_mean) fm_n = __ldg(p.post_mean + r);
    }
  };
  // With gate rows: the byte offset of the gate row of the row to fetch next,
  // how many rows it still serves, and the first of them in the range.
  int gate_left = 0, gate_first = 0;
  int64_t gate_at = 0;
  auto clip = [](int64_t v) { return static_cast<int>(min(v, static_cast<int64_t>(0x7fffffff))); };
  auto gate_of = [&](int64_t r) {
    return p.rows <= 0x7fffffff ? static_cast<int64_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(p.rows_per_gate))
                                : r / p.rows_per_gate;
  };
  if constexpr (GR) {
    const int64_t g = gate_of(r0);
    gate_left = clip((g + 1) * p.rows_per_gate - r0);
    gate_at = (g * p.gate_stride + cs.c0) * S;
  }
  // Row number i of the range, whose group 0 of this thread is at byte `at`,
  // in two parts: dy and dh are read once, and their places are free again
  // before those of h, f and the gate.
  auto fetch_first = [&](int slot, int i, int64_t at) {
    if (i < n) {
      if (has_dy) ring.template fetch<0>(cs, slot, p.dy, at, 723, extent);
      if (has_dh) ring.template fetch<2>(cs, slot, p.dh, at, 721, extent);
    }
    ring.commit();
  };
  auto fetch_rest = [&](int slot, int i, int64_t at) {
    if (i < n) {
      if (has_dy) ring.template fetch<1>(cs, slot, p.h, at, 724, extent);
      if (need_f) ring.template fetch<3>(cs, slot, p.f, at, 722, extent);
      if constexpr (GR) {
        // a gate row that the slot's last row had is there already
        if (i - gate_first < slots) ring.template fetch<4>(cs, slot, p.gate, gate_at, 731, b_gate_bytes(p, S));
        if (--gate_left == 0) {
          gate_left = clip(p.rows_per_gate);
          gate_first = i + 1;
          gate_at += p.gate_stride * S;
        }
      }
    }
    ring.commit();
  };
  // While the previous kernel of the stream may still be finishing, ask L2
  // for the walker's first rows (hints alone, as in the forward).
  if (r0 < r1 && r1 - r0 <= 8) {
    const int ln = tid & 31, chunk0 = cs.c0 * S - ln * 16;
    const int bytes = min(NV * kStepBytes, (col0 + min(p.w.slice, p.H - col0)) * S - chunk0);
    for (int s = 0; s < slots && r0 + s < r1; ++s) {
      const int64_t at = (r0 + s) * p.H * S + chunk0 + ln * 128;
      if (ln * 128 >= bytes || !ADDLN_IN(720, at, 1, extent)) break;
      if (has_dy) prefetch_line(static_cast<const char*>(p.dy) + at), prefetch_line(static_cast<const char*>(p.h) + at);
      if (has_dh) prefetch_line(static_cast<const char*>(p.dh) + at);
      if (need_f) prefetch_line(static_cast<const char*>(p.f) + at);
    }
  }
  pdl_trigger();
  pdl_wait();
  // A tensor that the call does not have is zeros, written once: the rows'
  // arithmetic then needs no branches (u, hhat and dh are zeros, and rstd is
  // 0 or, for fhat, 1).
  for (int s = 0; s < slots; ++s) {
    if (!has_dy) ring.template clear<0>(s), ring.template clear<1>(s);
    if (!has_dh) ring.template clear<2>(s);
    if (!need_f) ring.template clear<3>(s);
  }
  for (int s = 0; s < slots; ++s) {
    const int64_t at = (r0 + s) * row_bytes + cs.c0 * S;
    fetch_first(s, s, at);
    fetch_rest(s, s, at);
  }

  // parameters, while the first rows arrive
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = cs.col(k);
    float g[VE], w[VE], b[VE], gt[VE];
    load_params<VE, SH>(has_dy ? p.pre_gamma : nullptr, c, p.H, 0.f, g, 726);
    load_params<VE, SH>(!GR && p.gate_kind == ADDLN_GATE_CHANNEL ? static_cast<const float*>(p.gate) : nullptr, c, p.H, 1.f, gt,
                    728);
    load_params<VE, SH>(p.post_gamma, c, p.H, 1.f, w, 729);
    load_params<VE, SH>(FULL && GR ? p.post_beta : nullptr, c, p.H, 0.f, b, 730);
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      w[e] *= p.s * gt[e];
      b[e] *= p.s;
      if (cs.valid(k) <= e) g[e] = w[e] = b[e] = 0.f;
    }
    kept.put(0, k, g);
    kept.put(1, k, w);
    if constexpr (FULL && GR) kept.put(2, k, b);
  }
  stats(r0);
  if (p.w.C > 1) cluster_wait_started();

  float2 sg[P], s1[P], sb[FULL ? P : 1], s0[FULL ? P : 1], sd[GR ? P : 1];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    sg[j] = s1[j] = dup2(0.f);
    if constexpr (FULL) sb[j] = s0[j] = dup2(0.f);
    if constexpr (GR) sd[j] = dup2(0.f);
  }
  // rows left of the current gate row
  int flush = 0;
  if constexpr (GR) flush = clip((gate_of(r0) + 1) * p.rows_per_gate - r0);

  int slot = 0;
  int64_t off = r0 * row_bytes + cs.c0 * S;
  for (int it = 0; it < n; ++it, off += row_bytes) {
    ring.template wait<2>();  // all but the next row's two parts
    ring.meet();
    const float2 nhm = dup2(-hm_n), hr = dup2(hr_n), nfm = dup2(-fm_n), fr = dup2(fr_n);
    stats(r0 + it + 1);
    // how far the row lies past 16-byte borders, tensor by tensor (of no
    // account for the zeros of a missing one)
    int sh[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) sh[i] = 0;
    if constexpr (SH) {
      sh[0] = low4(p.dy, off), sh[1] = low4(p.h, off), sh[2] = low4(p.dh, off), sh[3] = low4(p.f, off);
      if constexpr (GR) sh[4] = low4(p.gate, (gate_of(r0 + it) * p.gate_stride + cs.c0) * S);
    }
    auto take = [&](int i, int k, float2 (&v)[N]) { IO::to_pairs(ring.take(slot, i, k, sh[i]), v); };
    auto hat = [&](int i, int k, float2 negm, float2 r, float2 (&v)[N]) {
      take(i, k, v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = mul2(FULL ? add2(v[j], negm) : v[j], r);
    };

    float2 t[P];
    float2 q[K];
#pragma unroll
    for (int i = 0; i < K; ++i) q[i] = dup2(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 hh[N], fh[N], c[N], dy[N], d[N], u[N];
      const int j0 = k * N;
      hat(1, k, nhm, hr, hh);
      hat(3, k, nfm, fr, fh);
      take(0, k, dy);
      take(2, k, d);
      kept.get(0, k, u);
      kept.get(1, k, c);
      if constexpr (GR) {
        float2 gt[N];
        take(4, k, gt);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mul2(c[i], gt[i]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        u[i] = mul2(u[i], dy[i]);
        sg[j0 + i] = fma2(dy[i], hh[i], sg[j0 + i]);
        q[0] = fma2(u[i], hh[i], q[0]);
        const float2 tt = fma2(hr, u[i], d[i]);
        t[j0 + i] = tt;
        const float2 cf = mul2(c[i], fh[i]);
        q[1] = fma2(cf, tt, q[1]);
        q[2] = fma2(cf, hh[i], q[2]);
        if constexpr (FULL) {
          sb[j0 + i] = add2(sb[j0 + i], dy[i]);
          q[3] = add2(q[3], u[i]);
          q[4] = fma2(c[i], tt, q[4]);
          q[5] = fma2(c[i], hh[i], q[5]);
          q[6] = add2(q[6], c[i]);
          q[7] = add2(q[7], cf);
        }
      }
    }
    ring.meet();
    fetch_first(slot, it + slots, off + slots * row_bytes);
    float m[K];
#pragma unroll
    for (int i = 0; i < K; ++i) m[i] = q[i].x + q[i].y;
    if (has_dy || post) sums(m);
    // r_h mean(u hhat), r_h mean(u), mean(v fhat), mean(v)
    const float a2 = hr.x * (m[0] * p.inv_h);
    float a1 = 0.f, v2 = m[1] - a2 * m[2], v1 = 0.f;
    if constexpr (FULL) {
      if (p.pre == ADDLN_NORM_LAYER) a1 = hr.x * (m[FULL ? 3 : 0] * p.inv_h);
      v2 -= a1 * m[FULL ? 7 : 0];
      if (p.post == ADDLN_NORM_LAYER) v1 = (m[FULL ? 4 : 0] - a2 * m[FULL ? 5 : 0] - a1 * m[FULL ? 6 : 0]) * p.inv_h;
    }
    v2 *= p.inv_h;
    const float2 na2 = dup2(-a2), na1 = dup2(-a1), nv2 = dup2(-v2), nv1 = dup2(-v1), pa = dup2(p.a);
    Writer<DT, NV, SH> dx, df;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 hh[N], fh[N], c[N], o[N];
      const int j0 = k * N;
      hat(1, k, nhm, hr, hh);
      hat(3, k, nfm, fr, fh);
      kept.get(1, k, c);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        t[j0 + i] = fma2(na2, hh[i], FULL ? add2(t[j0 + i], na1) : t[j0 + i]);
        o[i] = mul2(pa, t[j0 + i]);
      }
      dx.put(cs, p.dx, off, k, IO::from_pairs(o), 727, extent);
      if constexpr (GR) {
        // the gate's own gradient D (fhat w + b), and D times the gate
        float2 b[N], gt[N];
        if constexpr (FULL) kept.get(2, k, b);
        take(4, k, gt);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 D = t[j0 + i];
          const float2 nn = FULL ? fma2(fh[i], c[i], b[i]) : mul2(fh[i], c[i]);
          sd[j0 + i] = fma2(D, nn, sd[j0 + i]);
          t[j0 + i] = mul2(D, gt[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s1[j0 + i] = fma2(t[j0 + i], fh[i], s1[j0 + i]);
        if constexpr (FULL) s0[j0 + i] = add2(s0[j0 + i], t[j0 + i]);
        o[i] = mul2(c[i], t[j0 + i]);
      }
      if (post)
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = mul2(fr, fma2(fh[i], nv2, FULL ? add2(o[i], nv1) : o[i]));
      df.put(cs, p.df, off, k, IO::from_pairs(o), 735, extent);
    }
    ring.meet();
    fetch_rest(slot, it + slots, off + slots * row_bytes);
    slot = slot + 1 == slots ? 0 : slot + 1;
    if constexpr (GR) {
      if (--flush == 0 || it + 1 == n) {
        const int64_t row = r0 + it, g = gate_of(row), begin = g * p.rows_per_gate;
        const bool whole = begin >= r0 && row + 1 == min(p.rows, begin + p.rows_per_gate);
        if (whole) {
          if (p.dgate != nullptr) {
            Writer<DT, NV, SH> out;
#pragma unroll
            for (int k = 0; k < NV; ++k)
              out.put(cs, p.dgate, (g * p.H + cs.c0) * S, k, IO::from_pairs(sd + k * N), 732,
                      p.gate_rows * static_cast<int64_t>(p.H) * S);
          }
        } else if (p.seg != nullptr) {
          // the range's first gate row, or its last
          store_cols<VE, NV>(p.seg + (2 * walker + (begin <= r0 ? 0 : 1)) * p.Hp, cs, 733, p.Hp, sd);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) sd[j] = dup2(0.f);
        flush = clip(p.rows_per_gate);
      }
    }
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
        give(s1, 1);
        if constexpr (FULL) give(sb, 2), give(s0, 3);
      }
      __syncthreads();
      if (gets) {
        get(sg, 0);
        get(s1, 1);
        if constexpr (FULL) get(sb, 2), get(s0, 3);
      }
      __syncthreads();
    }
    if (side == 0) {
      float* out = p.part + cta * A * p.Hp;
      store_cols<VE, NV>(out, cs, 736, p.Hp, sg);
      store_cols<VE, NV>(out + p.Hp, cs, 737, p.Hp, s1);
      if constexpr (FULL) {
        store_cols<VE, NV>(out + 2 * p.Hp, cs, 738, p.Hp, sb);
        store_cols<VE, NV>(out + 3 * p.Hp, cs, 739, p.Hp, s0);
      }
    }
  }
  if (p.w.C > 1) cooperative_groups::this_cluster().sync();
}

// ------------------------------------------------------------ joining sums
// blockIdx.y == 0: the CTAs' column sums of QUADS column quads, added in a
// fixed order (thread t takes quad t % QUADS and the partials t / QUADS,
// + kSumThreads / QUADS, ...; then a butterfly over the warp's lanes of that
// quad and the warps in order), and from them the gradients of both norms
// and of a per-channel gate.  blockIdx.y > 0: the gate rows that several
// walkers share, the walkers in order.  The partials sit in L2 (2 to 10 MB) and
// without shared gate rows the kernel's time is its latency (64x768 fp32 2.6 us
// behind the rows' kernel, 4096x768 fp16 3.8, 2048x4096 fp16 5.0), so a thread's
// loads of all A sums are in flight together.
//
// Shared gate rows are another matter: each that may be shared has Hp / 4 / QUADS
// CTAs, which add a few partials or none, and their number is what the kernel then
// takes (us of the rows' kernel / the column sums / the gate rows' CTAs, and
// how many of these; bf16 but for the last): 32768x8192 rms, 4096 rows a gate row,
// 494 / 7 / 15, 4096; 65536x1152, 256 rows, rms 172 / 6 / 58, 18432, layer 233 / 5 /
// 135, 36864; 8192x4096, 64 rows, rms 65 / 6 / 102, 32768, layer 100 / 6 / 241, 65536;
// 2048x4096 fp16 rms, 2 rows, 21 / 6 / 147, 77568.
// The gate rows that more than one walker shares.  Where walkers have at
// least as many rows as a gate row, a gate row meets at most one border
// between walkers, and border b (between walkers b - 1 and b) has one if it
// lies inside a gate row; otherwise every gate row is looked at.
__host__ __device__ __forceinline__ int64_t shared_candidates(int64_t rows, int64_t walkers,
                                                              int64_t gate_rows, int64_t rpg) {
  return rows / walkers >= rpg ? walkers - 1 : gate_rows;
}

template <int DT, bool FULL, int QUADS>
__global__ void __launch_bounds__(kSumThreads) k_block_sums(const __grid_constant__ BlockBwdArgs p) {
  constexpr int A = sums_of(FULL);
  __shared__ float4 wsum[kSumThreads / 32][A][QUADS];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x;
  const int j = (blockIdx.x * QUADS + t % QUADS) * 4;  // the thread's first column
  if (blockIdx.y == 0) {
    if (p.part == nullptr) return;
    float4 r[A];
    block_quad_sums<A, QUADS>(p.part + j, p.parts, static_cast<int64_t>(A) * p.Hp, p.Hp, j < p.H,
                              (p.parts * A * p.Hp - j) * 4, wsum, r);
    if (t >= QUADS) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = j + q;
      if (c >= p.H || !ADDLN_IN(742, 4 * c, 4, 4 * static_cast<int64_t>(p.H))) continue;
      auto at = [&](int a) { return q == 0 ? r[a].x : q == 1 ? r[a].y : q == 2 ? r[a].z : r[a].w; };
      if (p.dpre_gamma) p.dpre_gamma[c] = at(0);
      if (FULL && p.dpre_beta) p.dpre_beta[c] = at(FULL ? 2 : 0);
      const bool channel = p.gate_kind == ADDLN_GATE_CHANNEL;
      const float gt = channel ? p.s * __ldg(static_cast<const float*>(p.gate) + c) : p.s;
      if (p.dpost_gamma) p.dpost_gamma[c] = gt * at(1);
      if (FULL && p.dpost_beta) p.dpost_beta[c] = gt * at(FULL ? 3 : 1);
      if (channel && p.dgate) {
        float d = p.s * at(1);
        if (p.post != ADDLN_NORM_NONE) {
          d *= __ldg(p.post_gamma + c);
          if (FULL && p.post_beta) d = fmaf(p.s * __ldg(p.post_beta + c), at(FULL ? 3 : 1), d);
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
  float4 rest[1];
  block_quad_sums<1, QUADS>(src, w1 - w0, 2 * static_cast<int64_t>(p.Hp), 0, j < p.H,
                            ex - (2 * (w0 + 1) * p.Hp + j) * 4, reinterpret_cast<float4(*)[1][QUADS]>(wsum), rest);
  if (t >= QUADS || j >= p.H) return;
  const int64_t at0 = (2 * w0 + (head ? 0 : 1)) * p.Hp + j;
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ADDLN_IN(743, at0 * 4, 16, ex)) r = __ldcg(reinterpret_cast<const float4*>(p.seg + at0));
  r = add4(r, rest[0]);
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

struct Choice {
  BwdKernel k = nullptr;
  Shape sh{};
  int smem = 0, kept_at = 0, sums_at = 0;
};

// NV groups of VE columns a thread; a CTA of up to kSideThreads threads for as
// many rows side by side as fit it, else one CTA for a row, else a cluster of
// as few CTAs as hold it: its barrier costs more than several clusters to an
// SM give back (8192x6144 bf16 layer, clusters of 2 / 4 / 8: 230, 265, 400 us;
// 8192x5120 fp32 rms 168, 268, 421).  Shared memory: the ring (at least what
// the walkers need to join their sums), the parameters, the row sums.
constexpr int kSideThreads = 512;

template <int DT, int NV, bool FULL, bool GR, bool SH>
Choice make(int H, int64_t rows, int sms) {
  constexpr int VE = Io<DT>::kVec, kMost = bwd_threads(DT, FULL, GR, SH);
  Choice c;
  c.k = &k_block_bwd<DT, NV, FULL, GR, SH>;
  const int groups = (H + VE - 1) / VE;
  c.sh.C = (groups + NV * kMost - 1) / (NV * kMost);
  c.sh.slice = c.sh.C == 1 ? H : ((H + c.sh.C - 1) / c.sh.C + 15) / 16 * 16;
  const int threads = ((c.sh.slice + VE - 1) / VE + 32 * NV - 1) / (32 * NV) * 32;
  c.sh.rows = c.sh.C > 1 || threads > kSideThreads / 2 ? 1 : kSideThreads / threads;
  c.sh.rows = rows_side_by_side(c.sh.rows, rows, sms);
  c.sh.threads = threads * c.sh.rows;
  const int warps = c.sh.threads / 32;
  int ring = warps * kMaxSlots * static_cast<int>(Ring<DT, NV, GR ? 5 : 4, SH>::kSlot);
  int half = 0;  // walkers that give their sums to another at once
  for (int top = 1; top < c.sh.rows; top *= 2) half = top;
  const int join = half * sums_of(FULL) * NV * VE * threads * 4;
  if (ring < join) ring = join;
  c.kept_at = ring;
  c.sums_at = c.kept_at + warps * static_cast<int>(Kept<VE, NV>::template bytes<FULL && GR ? 3 : 2>());
  c.smem = c.sums_at + c.sh.rows * 2 * (threads / 32) * c.sh.C * (FULL ? 8 : 4) * 4;
  return c;
}

// The rows that walkers of VE columns a thread have eight each of.
inline int64_t few_rows(int H, int VE, int sms) {
  return 8 * static_cast<int64_t>(sms) * (kSideThreads / ((H + 32 * VE - 1) / (32 * VE) * 32));
}

// 16 columns of a 16-bit type a thread where the sums are two or three for a
// column, rows are not shifted and, with 8 a thread, longer than a warp's and
// more than eight to a walker; else 8 (4 of fp32 where 8 spill).  us with 8 /
// 16: 300x768 bf16 rms 5.2 / 7.0, 8192x512 (7 rows to a walker) 14.2 / 14.9,
// 8192x1024 (13 rows) 23.8 / 21.5, 2048x4096 fp16 (13 rows) 32.7 / 28.4,
// 32768x256 (a warp's) 21.9 / 28.1.
template <int DT, bool FULL, bool GR, bool SH>
Choice choose(int H, int64_t rows, int sms) {
  constexpr int VEC = Io<DT>::kVec;
  if constexpr (DT == kF32) {
    return make<DT, SH && FULL && GR ? 1 : 2, FULL, GR, SH>(H, rows, sms);
  } else {
    if constexpr (!SH && !FULL) {
      if (H > 32 * VEC && rows > few_rows(H, VEC, sms)) return make<DT, 2, FULL, GR, SH>(H, rows, sms);
    }
    return make<DT, 1, FULL, GR, SH>(H, rows, sms);
  }
}

template <int DT, bool FULL>
Choice choose(int H, bool aligned, bool gr, int64_t rows, int sms) {
  if (aligned) return gr ? choose<DT, FULL, true, false>(H, rows, sms) : choose<DT, FULL, false, false>(H, rows, sms);
  return gr ? choose<DT, FULL, true, true>(H, rows, sms) : choose<DT, FULL, false, true>(H, rows, sms);
}

Choice choose(int dtype, int H, bool aligned, bool full, bool gr, int64_t rows, int sms) {
  if (dtype == kF32) return full ? choose<kF32, true>(H, aligned, gr, rows, sms) : choose<kF32, false>(H, aligned, gr, rows, sms);
  if (dtype == kF16) return full ? choose<kF16, true>(H, aligned, gr, rows, sms) : choose<kF16, false>(H, aligned, gr, rows, sms);
  return full ? choose<kBF16, true>(H, aligned, gr, rows, sms) : choose<kBF16, false>(H, aligned, gr, rows, sms);
}

// Units (CTAs or clusters) of a launch: those that fit the device at once, no
// more than the rows need.
int64_t units_of(const Choice& c, int64_t rows, const DeviceInfo& dev) {
  const int fit = resident_units(reinterpret_cast<const void*>(c.k), c.sh, c.smem, dev);
  if (fit < 0) return fit;
  const int64_t need = (rows + c.sh.rows - 1) / c.sh.rows;
  return need < fit ? need : fit;
}

int64_t part_bytes(int64_t parts, bool full, int64_t Hp) { return parts * sums_of(full) * Hp * 4; }
int64_t seg_bytes(int64_t walkers, bool gr, int64_t rpg, int64_t Hp) {
  return gr && rpg > 1 ? walkers * 2 * Hp * 4 : 0;
}

// Quads a block: the most (of 2, 4, 8) whose partials a thread still loads in
// one round (us of the backward with 2 / 8 throughout: 64x768 fp32 5.3 / 5.0,
// 4096x768 fp16 16.5 / 17.7, 32768x256 bf16 21.7 / 23.3).
inline int sums_quads(int64_t parts, bool full) {
  const int64_t one_round = kSumThreads * (8 / sums_of(full));
  return 8 * parts <= one_round ? 8 : 4 * parts <= one_round ? 4 : 2;
}

template <int DT>
BwdKernel pick_sums(bool full, int quads) {
  if (full) return quads == 8 ? &k_block_sums<DT, true, 8> : quads == 4 ? &k_block_sums<DT, true, 4> : &k_block_sums<DT, true, 2>;
  return quads == 8 ? &k_block_sums<DT, false, 8> : quads == 4 ? &k_block_sums<DT, false, 4> : &k_block_sums<DT, false, 2>;
}

}  // namespace
}  // namespace blk

// What any number of rows up to this one needs, so that a workspace serves
// shorter calls too: their CTAs are no more than SMs, or than those of either
// kernel, with as many rows side by side as there is room for, that fit.
int64_t block_bwd_workspace_bytes(int dtype, bool aligned, bool full, int64_t rows, int H, int gate_kind,
                                  int64_t rows_per_gate, const DeviceInfo& dev) {
  using namespace blk;
  const bool gr = gate_kind == ADDLN_GATE_ROWS;
  int64_t units = dev.sms, side = 1;
  for (const int64_t r : {few_rows(H, dtype == kF32 ? 4 : 8, dev.sms), INT64_MAX / 2}) {
    if (r == 0) continue;  // wider than one CTA
    const Choice ch = choose(dtype, H, aligned, full, gr, r, dev.sms);
    const int64_t fit = units_of(ch, INT64_MAX / 2, dev);
    if (fit < 0) return fit;
    units = units > fit ? units : fit;
    side = side > ch.sh.rows ? side : ch.sh.rows;
  }
  if (units > rows) units = rows;
  const int64_t Hp = (H + 3) / 4 * 4;
  return part_bytes(units, full, Hp) + seg_bytes(units * side, gr, rows_per_gate, Hp);
}

int launch_block_bwd(int dtype, bool aligned, bool full, BlockBwdArgs p, void* ws, int64_t ws_bytes,
                     const LaunchCtx& c) {
  using namespace blk;
  const bool gr = p.gate_kind == ADDLN_GATE_ROWS;
  const Choice ch = choose(dtype, p.H, aligned, full, gr, p.rows, c.dev.sms);
  p.w = walk_of(ch.sh);
  p.parts = units_of(ch, p.rows, c.dev);
  if (p.parts < 0) return static_cast<int>(p.parts);
  p.walkers = p.parts * ch.sh.rows;
  if (p.walkers > p.rows) p.walkers = p.rows;
  p.kept_at = ch.kept_at;
  p.sums_at = ch.sums_at;
  p.Hp = (p.H + 3) / 4 * 4;
  const bool cols = p.dpre_gamma || p.dpre_beta || p.dpost_gamma || p.dpost_beta ||
                    (p.dgate && p.gate_kind == ADDLN_GATE_CHANNEL);
  const bool seg = gr && p.dgate != nullptr && p.rows_per_gate > 1 && p.walkers > 1;
  p.part = nullptr;
  p.seg = nullptr;
  if (cols || seg) {
    const int64_t pb = part_bytes(p.parts, full, p.Hp);
    const int64_t need = pb + seg_bytes(p.parts * ch.sh.rows, gr, p.rows_per_gate, p.Hp);
    if (ws == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 15u)) return ADDLN_ERR_WORKSPACE;
    if (cols) p.part = static_cast<float*>(ws);
    if (seg) p.seg = reinterpret_cast<float*>(static_cast<char*>(ws) + pb);
  }
  cudaError_t e = launch_units(ch.k, p.parts, ch.sh, ch.smem, c, p);
  if (e == cudaSuccess && (cols || seg)) {
    const int quads = sums_quads(p.parts, full);
    const BwdKernel ks = dtype == kF32   ? pick_sums<kF32>(full, quads)
                         : dtype == kF16 ? pick_sums<kF16>(full, quads)
                                         : pick_sums<kBF16>(full, quads);
    const int64_t ny = seg ? shared_candidates(p.rows, p.walkers, p.gate_rows, p.rows_per_gate) : 0;
    const dim3 grid(static_cast<unsigned>((p.Hp / 4 + quads - 1) / quads), static_cast<unsigned>(1 + ny));
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
