// Shared by the block-boundary kernels (block_fwd.cu, block_bwd.cu): how a
// row is spread over threads, how its elements reach them, and the row
// reductions over a warp, a CTA or the CTAs of a cluster.
//
// Layout.  One walker handles one row at a time: a warp, a CTA, or for the
// longest rows a cluster of C CTAs that each own a slice of the columns.  A
// warp owns 32 NV groups of VE neighbouring columns, of which lane l has
// groups l, l + 32, ...: the addresses of a thread's groups are constants
// apart.  VE follows the alignment that all buffers of a call share: 16-byte
// accesses, or 4-byte, or single elements.
#pragma once

#include <cooperative_groups.h>

#include "../../include/addln_block.h"
#include "block.h"
#include "common.cuh"

namespace addln {
namespace blk {

constexpr int kMaxThreads = 512;  // threads a CTA
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxCluster = 8;    // the portable cluster size
constexpr int kMaxSmem = 227 * 1024;  // dynamic shared memory of a CTA

// VE elements of DT at p (element offset i), as 32-bit words or one 16-bit
// value, and their fp32 values in slots [k VE, (k + 1) VE) of float2 v[NV VE / 2].
template <int DT, int VE>
struct Grp {
  using IO = Io<DT>;
  static constexpr int S = IO::kBytes;
  static constexpr int kBytes = VE * S;
  static constexpr int W = kBytes >= 4 ? kBytes / 4 : 1;  // words held
  uint32_t w[W];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = 0u;
  }
  __device__ __forceinline__ void load(const char* q) {
    if constexpr (kBytes == 16) {
      const uint4 u = ld_stream_v4(q);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else if constexpr (kBytes == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
    } else {
      w[0] = __ldg(reinterpret_cast<const unsigned short*>(q));
    }
  }
  // value of element e of the group
  __device__ __forceinline__ float get(int e) const {
    if constexpr (DT == kF32) return __uint_as_float(w[e]);
    const unsigned short b = static_cast<unsigned short>((e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu);
    if constexpr (DT == kF16) return __half2float(__ushort_as_half(b));
    return __bfloat162float(__ushort_as_bfloat16(b));
  }
};

template <int DT, int VE, int NV>
__device__ __forceinline__ void to_slots(const Grp<DT, VE> (&g)[NV], float2 (&v)[NV * VE / 2]) {
  if constexpr (VE >= 2) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int q = 0; q < VE / 2; ++q) {
        if constexpr (DT == kF32)
          v[k * VE / 2 + q] = make_float2(__uint_as_float(g[k].w[2 * q]), __uint_as_float(g[k].w[2 * q + 1]));
        else
          v[k * VE / 2 + q] = Io<DT>::w2f(g[k].w[q]);
      }
  } else {
#pragma unroll
    for (int q = 0; q < NV / 2; ++q) v[q] = make_float2(g[2 * q].get(0), g[2 * q + 1].get(0));
  }
}

// Stores group k of the slots, rounded to DT, at q.
template <int DT, int VE, int P>
__device__ __forceinline__ void store_group(char* q, const float2 (&v)[P], int k) {
  if constexpr (VE * Io<DT>::kBytes == 16) {
    st_stream_v4(q, Io<DT>::from_pairs(&v[k * VE / 2]));
  } else if constexpr (VE == 2) {  // 16-bit pair
    *reinterpret_cast<uint32_t*>(q) = Io<DT>::f2w(v[k].x, v[k].y);
  } else {
    Io<DT>::store1(q, 0, (k & 1) ? v[k >> 1].y : v[k >> 1].x);
  }
}

// VE fp32 parameters at byte offset `off`; `fill` where there are none.
template <int VE>
__device__ __forceinline__ void load_params(const float* p, uint32_t off, float fill, float (&v)[VE], int site,
                                            int64_t extent) {
#pragma unroll
  for (int e = 0; e < VE; ++e) v[e] = fill;
  if (p == nullptr || !ADDLN_IN(site, off, 4 * VE, extent)) return;
  const char* q = reinterpret_cast<const char*>(p) + off;
  if constexpr (VE >= 4) {
#pragma unroll
    for (int h = 0; h < VE / 4; ++h) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(q) + h);
      v[4 * h] = u.x, v[4 * h + 1] = u.y, v[4 * h + 2] = u.z, v[4 * h + 3] = u.w;
    }
  } else if constexpr (VE == 2) {
    const float2 u = __ldg(reinterpret_cast<const float2*>(q));
    v[0] = u.x, v[1] = u.y;
  } else {
    v[0] = __ldg(reinterpret_cast<const float*>(q));
  }
}

template <int P>
__device__ __forceinline__ float get_slot(const float2 (&v)[P], int e) {
  return (e & 1) ? v[e >> 1].y : v[e >> 1].x;
}

// Asks L2 for the 128-byte line at p (a hint).
__device__ __forceinline__ void prefetch_line(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// A thread's groups of a row.  A group past the end of the slice does not
// exist: it is fetched as zeros and never stored, and reads the parameters of
// the slice's last group.
template <int VE, int NV>
struct Cols {
  static constexpr int kStep = 32 * VE;  // columns between a thread's groups
  int c0;           // first column of group 0
  bool ok[NV];
  bool all;         // every group of the warp exists
  float n, inv_n;   // columns of the warp, 1 / n (0 for none)
  uint32_t par[NV]; // byte offset of each group in an fp32 vector of H columns

  __device__ __forceinline__ void init(int warp, int col0, int cols) {
    const int at0 = warp * NV * kStep + (threadIdx.x & 31) * VE;
    c0 = col0 + at0;
    const int own = min(max(cols - warp * NV * kStep, 0), NV * kStep);
    n = static_cast<float>(own);
    inv_n = own ? __frcp_rn(n) : 0.f;
    bool full = true;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int at = at0 + k * kStep;
      ok[k] = at < cols;
      full = full && ok[k];
      par[k] = 4u * static_cast<uint32_t>(col0 + (ok[k] ? at : cols - VE));
    }
    all = __all_sync(0xffffffffu, full);
  }
  __device__ __forceinline__ int col(int k) const { return c0 + k * kStep; }
  // zeros in the slots of groups that do not exist
  __device__ __forceinline__ void clear(float2 (&v)[NV * VE / 2]) const {
    if (all) return;
#pragma unroll
    for (int e = 0; e < NV * VE; ++e) {
      float& u = (e & 1) ? v[e >> 1].y : v[e >> 1].x;
      u = ok[e / VE] ? u : 0.f;
    }
  }
};

// --------------------------------------------------------------- staging
// A thread's groups of the rows ahead, in a ring of slots of its own in
// shared memory: it copies them itself (cp.async, 16 or 4 bytes at a time,
// zeros for a group that does not exist) and alone reads them, so no barrier
// is needed, and no register holds them.  A warp's ring is one piece,
// [slot][tensor][group][lane], so that all its addresses are constants apart.
// Two-byte groups cannot be copied that way; they wait in registers, two in
// each (one slot).
constexpr int kMaxSlots = 2;

template <int DT, int VE, int NV, int NT>
struct Ring {
  static constexpr int kBytes = Grp<DT, VE>::kBytes;
  static constexpr bool kAsync = kBytes >= 4;
  static constexpr uint32_t kStep = 32 * kBytes;                    // between groups
  static constexpr uint32_t kSlot = kAsync ? NT * NV * kStep : 0;  // bytes of a warp's slot
  uint32_t base;  // this thread's first group of slot 0
  uint32_t held[kAsync ? 1 : NT][kAsync ? 1 : NV / 2];

  __device__ __forceinline__ uint32_t at(int slot, int i, int k) const {
    return base + static_cast<uint32_t>(slot) * (NT * NV * kStep) + static_cast<uint32_t>(i * NV + k) * kStep;
  }
  // group k of tensor i from src, if it exists
  __device__ __forceinline__ void fetch(int slot, int i, int k, const char* src, bool ok) {
    if constexpr (kAsync) {
      const uint32_t dst = at(slot, i, k);
      const int n = ok ? kBytes : 0;
      if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    } else {
      Grp<DT, VE> g;
      g.zero();
      if (ok) g.load(src);
      held[i][k >> 1] = (k & 1) ? __byte_perm(held[i][k >> 1], g.w[0], 0x5410) : g.w[0];
    }
  }
  // zeros for tensor i
  __device__ __forceinline__ void clear(int slot, int i) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if constexpr (kAsync) {
        const uint32_t dst = at(slot, i, k);
#pragma unroll
        for (int b = 0; b < kBytes; b += 4)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + b), "r"(0) : "memory");
      } else {
        held[i][k >> 1] = 0u;
      }
    }
  }
  __device__ __forceinline__ void commit() {
    if constexpr (kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // all but the AHEAD groups of copies committed last have arrived
  template <int AHEAD>
  __device__ __forceinline__ void wait() {
    if constexpr (kAsync) asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
  }
  // groups k0 .. k0 + N - 1 of tensor i
  template <int N>
  __device__ __forceinline__ void take(int slot, int i, int k0, Grp<DT, VE> (&g)[N]) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (kAsync) {
        const uint32_t src = at(slot, i, k0 + k);
        if constexpr (kBytes == 16) {
          const uint4 u = ld_shared_v4(src);
          g[k].w[0] = u.x, g[k].w[1] = u.y, g[k].w[2] = u.z, g[k].w[3] = u.w;
        } else {
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(g[k].w[0]) : "r"(src));
        }
      } else {
        g[k].w[0] = ((k0 + k) & 1) ? held[i][(k0 + k) >> 1] >> 16 : held[i][(k0 + k) >> 1] & 0xffffu;
      }
    }
  }
};

// Parameters in shared memory, each thread's columns in places of its own (a
// warp's in one piece [vector][group][part][lane]), so that a read costs half
// of what a 16-byte load through L1 does.
template <int VE, int NV>
struct Kept {
  static constexpr int kPart = VE >= 4 ? 16 : VE * 4;
  static constexpr int Q = VE * 4 / kPart;
  static constexpr uint32_t kStep = 32 * kPart;
  template <int NP>
  __device__ static constexpr uint32_t bytes() {
    return NP * NV * Q * kStep;
  }
  uint32_t base;

  __device__ __forceinline__ uint32_t at(int i, int k, int q) const {
    return base + static_cast<uint32_t>((i * NV + k) * Q + q) * kStep;
  }
  __device__ __forceinline__ void put(int i, int k, const float (&v)[VE]) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if constexpr (VE >= 4)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at(i, k, q)), "f"(v[4 * q]), "f"(v[4 * q + 1]),
                     "f"(v[4 * q + 2]), "f"(v[4 * q + 3]) : "memory");
      else if constexpr (VE == 2)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at(i, k, q)), "f"(v[0]), "f"(v[1]) : "memory");
      else
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at(i, k, q)), "f"(v[0]) : "memory");
    }
  }
  // N groups from k0 on
  template <int N>
  __device__ __forceinline__ void get(int i, int k0, float2 (&v)[N * VE / 2]) const {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if constexpr (VE >= 4) {
          const uint4 u = ld_shared_v4(at(i, k0 + k, q));
          v[k * VE / 2 + 2 * q] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
          v[k * VE / 2 + 2 * q + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        } else if constexpr (VE == 2) {
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v[k].x), "=f"(v[k].y) : "r"(at(i, k0 + k, q)));
        } else {
          float f;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(at(i, k0 + k, q)));
          if (k & 1) v[k >> 1].y = f; else v[k >> 1].x = f;
        }
      }
  }
};

// --------------------------------------------------------- row reductions
// Every warp publishes one float4; after exchange() every thread of the
// walker may read all of them, in the same order.  Two buffers in turn: a
// warp can write exchange i + 2's values only after the barrier of exchange
// i + 1, which every warp passes only when it has read those of exchange i.
// SIDES: a CTA may have walkers of several warps side by side, each with a
// barrier of its own (a kernel that names barriers by number takes all 16 of
// them, so that only four of its CTAs fit an SM).
template <bool SIDES>
struct Exchange {
  const Walk& w;
  int at;  // byte offset in shared memory of [2][warps], this walker's
  int par;

  __device__ __forceinline__ const float4* operator()(float4 v) {
    extern __shared__ __align__(128) unsigned char smem[];
    float4* b = reinterpret_cast<float4*>(smem + at) + par * w.warps;
    par ^= 1;
    const int lane = threadIdx.x & 31, side = SIDES ? (threadIdx.x >> 5) / w.cta_warps : 0;
    const int warp = (threadIdx.x >> 5) - side * w.cta_warps;
    if (w.C == 1) {
      if (lane == 0) b[warp] = v;
      if constexpr (SIDES)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + side), "r"(w.cta_warps * 32) : "memory");
      else
        __syncthreads();
    } else {
      namespace cg = cooperative_groups;
      cg::cluster_group cl = cg::this_cluster();
      const int rank = static_cast<int>(blockIdx.x % w.C);
      if (lane < w.C) cl.map_shared_rank(b, lane)[rank * w.cta_warps + warp] = v;
      cl.sync();
    }
    return b;
  }
};

// Sum over the walker, the same bits in every thread: a warp butterfly, then
// the warps' sums in a fixed order.
template <bool SIDES>
__device__ __forceinline__ float walker_sum(Exchange<SIDES>& ex, float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (ex.w.warps == 1) return v;
  const float4* b = ex(make_float4(v, 0.f, 0.f, 0.f));
  // groups of `width` lanes (a power of two of at least n, at most 32) add
  // the same n sums in the same order
  const int width = ex.w.width;
  float t = 0.f;
  for (int i = (threadIdx.x & 31) & (width - 1); i < ex.w.warps; i += 32) t += b[i].x;
  for (int off = 1; off < width; off <<= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  return t;
}

// Mean and sum of squared deviations of the walker's row.  Each warp takes
// the mean of its own values, K_w, off them (a row whose mean is large
// against its spread then loses nothing to it), and v is left that way; the
// little that is left of the mean and the squares are summed around K_w, and
// the warps' parts are put on the first warp's K_0.  Returns the mean, the
// mean on this warp's shift, and M2.
//
// Two different fp32 values of size K differ by 2^-24 K or more, so an M2
// below a quarter of that square is the rounding of K_w in a row of equal
// values: such a row is made exact (all deviations and M2 zero).
struct RowStat {
  float mean, m, M2;
};

template <int VE, int NV, bool SIDES>
__device__ __forceinline__ RowStat walker_stats(Exchange<SIDES>& ex, float2 (&v)[NV * VE / 2], const Cols<VE, NV>& cs) {
  constexpr int P = NV * VE / 2;
  constexpr unsigned kAll = 0xffffffffu;
  float2 s[2] = {dup2(0.f), dup2(0.f)}, q[2] = {dup2(0.f), dup2(0.f)};
  cs.clear(v);
#pragma unroll
  for (int j = 0; j < P; ++j) s[j & 1] = add2(s[j & 1], v[j]);
  s[0] = add2(s[0], s[1]);
  float sum = s[0].x + s[0].y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
  const float K = sum * cs.inv_n;
  const float2 negK = dup2(-K);
#pragma unroll
  for (int j = 0; j < P; ++j) v[j] = add2(v[j], negK);
  cs.clear(v);
  s[0] = s[1] = dup2(0.f);
#pragma unroll
  for (int j = 0; j < P; ++j) {
    s[j & 1] = add2(s[j & 1], v[j]);
    q[j & 1] = fma2(v[j], v[j], q[j & 1]);
  }
  s[0] = add2(s[0], s[1]);
  q[0] = add2(q[0], q[1]);
  float2 w = make_float2(s[0].x + s[0].y, q[0].x + q[0].y);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    w = add2(w, make_float2(__shfl_xor_sync(kAll, w.x, off), __shfl_xor_sync(kAll, w.y, off)));
  const float m = w.x * cs.inv_n;
  Part t{cs.n, m, fmaxf(fmaf(-w.x, m, w.y), 0.f) + (w.y - w.y)};  // a NaN stays
  float K0 = K;
  if (ex.w.warps > 1) {
    const float4* b = ex(make_float4(K, t.n, t.m, t.M2));
    const int width = ex.w.width;
    K0 = b[0].x;
    t = Part{0.f, 0.f, 0.f};
    for (int i = (threadIdx.x & 31) & (width - 1); i < ex.w.warps; i += width) {
      const float4 u = b[i];
      t = merge<false>(t, Part{u.y, (u.x - K0) + u.z, u.w});
    }
    for (int off = 1; off < width; off <<= 1)
      t = merge<false>(t, Part{__shfl_xor_sync(kAll, t.n, off), __shfl_xor_sync(kAll, t.m, off),
                               __shfl_xor_sync(kAll, t.M2, off)});
  }
  RowStat st{K0 + t.m, t.m - (K - K0), t.M2};
  const float least = 0x1p-25f * K0;
  if (t.M2 < least * least) {
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = dup2(0.f);
    st.m = st.M2 = 0.f;
  }
  return st;
}

// ------------------------------------------------------------------ host
// How a call's rows are spread over threads and CTAs.
struct Shape {
  int threads;   // threads of a CTA
  int rows;      // rows a CTA walks side by side, a warp for each; 1: a walker is a CTA or cluster
  int C;         // CTAs of a row
  int slice;     // columns a CTA owns, a multiple of 16
};

// Units (CTAs, or clusters of C CTAs) of kernel f that fit the device at
// once; cached per kernel, device, threads, cluster and shared memory.
// Negative: a CUDA error.
int resident_units(const void* f, const Shape& sh, int smem, const DeviceInfo& dev);

Walk walk_of(const Shape& sh);

// Launches kernel(args...) as units * C CTAs.
template <typename Args>
cudaError_t launch_units(void (*kernel)(Args), int64_t units, const Shape& sh, int smem, const LaunchCtx& c,
                         const Args& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.gridDim = dim3(static_cast<unsigned>(units * sh.C));
  cfg.blockDim = dim3(static_cast<unsigned>(sh.threads));
  cfg.stream = static_cast<cudaStream_t>(c.stream);
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (sh.C > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(sh.C);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (c.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(n);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace blk
}  // namespace addln
