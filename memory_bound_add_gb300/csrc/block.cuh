// Shared by the block-boundary kernels (block_fwd.cu, block_bwd.cu): how a
// row is spread over threads, loads and stores of VE neighbouring elements,
// and the row reductions over a CTA or over the CTAs of a cluster.
//
// Layout.  One walker handles one row at a time: a CTA, or for rows of more
// than kSlice columns a cluster of C CTAs that each own a slice of the
// columns.  A thread owns E = 8 columns of its CTA's slice, as NV = E / VE
// groups of VE neighbours: group k starts at (k T + tid) VE of T threads.
// VE follows the alignment that all buffers of a call share: 16-byte
// accesses, or 4-byte, or single elements.  Eight columns a thread keep the
// thread's share of four column sums, the row's values and the parameters in
// registers at 512 threads a CTA, so that one kernel serves every width.
#pragma once

#include <cooperative_groups.h>

#include "../../include/addln_block.h"
#include "common.cuh"

namespace addln {
namespace blk {

constexpr int kE = 8;             // columns a thread
constexpr int kMaxThreads = 512;  // threads a CTA
constexpr int kSlice = kE * kMaxThreads;
constexpr int kMaxCluster = 8;    // the portable cluster size: 8 * 4096 columns
constexpr int kMaxWarps = kMaxThreads / 32;

// VE elements of DT at p (element offset i), as 32-bit words or one 16-bit
// value, and their fp32 values in slots [k VE, (k + 1) VE) of float2 v[E/2].
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
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const char* q = static_cast<const char*>(p) + i * S;
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

template <int DT, int VE>
__device__ __forceinline__ void to_slots(const Grp<DT, VE> (&g)[kE / VE], float2 (&v)[kE / 2]) {
  if constexpr (VE >= 2) {
#pragma unroll
    for (int k = 0; k < kE / VE; ++k)
#pragma unroll
      for (int q = 0; q < VE / 2; ++q) {
        if constexpr (DT == kF32)
          v[k * VE / 2 + q] = make_float2(__uint_as_float(g[k].w[2 * q]), __uint_as_float(g[k].w[2 * q + 1]));
        else
          v[k * VE / 2 + q] = Io<DT>::w2f(g[k].w[q]);
      }
  } else {
#pragma unroll
    for (int q = 0; q < kE / 2; ++q) v[q] = make_float2(g[2 * q].get(0), g[2 * q + 1].get(0));
  }
}

// Stores group k of the slots (rounded to DT) at element offset i.
template <int DT, int VE>
__device__ __forceinline__ void store_group(void* p, int64_t i, const float2 (&v)[kE / 2], int k) {
  char* q = static_cast<char*>(p) + i * Io<DT>::kBytes;
  if constexpr (VE * Io<DT>::kBytes == 16) {
    st_stream_v4(q, Io<DT>::from_pairs(&v[k * VE / 2]));
  } else if constexpr (VE == 2) {  // 16-bit pair
    *reinterpret_cast<uint32_t*>(q) = Io<DT>::f2w(v[k].x, v[k].y);
  } else {
    Io<DT>::store1(q, 0, (k & 1) ? v[k >> 1].y : v[k >> 1].x);
  }
}

// VE fp32 parameters at column c into the slots of group k.
template <int VE>
__device__ __forceinline__ void load_param(const float* p, int c, float2 (&v)[kE / 2], int k) {
  if constexpr (VE >= 4) {
#pragma unroll
    for (int q = 0; q < VE / 4; ++q) {
      const float4 t = ld_param_f4(p + c + 4 * q);
      v[k * VE / 2 + 2 * q] = make_float2(t.x, t.y);
      v[k * VE / 2 + 2 * q + 1] = make_float2(t.z, t.w);
    }
  } else if constexpr (VE == 2) {
    v[k] = __ldg(reinterpret_cast<const float2*>(p + c));
  } else {
    const float t = __ldg(p + c);
    if (k & 1) v[k >> 1].y = t; else v[k >> 1].x = t;
  }
}

__device__ __forceinline__ float get_slot(const float2 (&v)[kE / 2], int e) {
  return (e & 1) ? v[e >> 1].y : v[e >> 1].x;
}

// --------------------------------------------------------- row reductions
// Every warp publishes one float4; after exchange() every thread of the
// walker may read all n of them, in the same order.  Two buffers in turn: a
// warp can write exchange i + 2's values only after the barrier of exchange
// i + 1, which every warp passes only when it has read those of exchange i.
struct Exchange {
  float4 (*buf)[kMaxWarps * kMaxCluster];  // [2][...]
  int n;       // warps of the walker
  int nw;      // warps of this CTA
  int C;       // CTAs of the walker
  int rank;    // this CTA's place among them
  int par;

  __device__ __forceinline__ const float4* operator()(float4 v) {
    float4* b = buf[par];
    par ^= 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (C == 1) {
      if (lane == 0) b[warp] = v;
      __syncthreads();
    } else {
      namespace cg = cooperative_groups;
      cg::cluster_group cl = cg::this_cluster();
      if (lane < C) cl.map_shared_rank(b, lane)[rank * nw + warp] = v;
      cl.sync();
    }
    return b;
  }
};

// Sum of (a, b) over the walker, the same bits in every thread: a warp
// butterfly, then the warps' sums in a fixed order.
__device__ __forceinline__ float2 walker_sum2(Exchange& ex, float2 v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, off), __shfl_xor_sync(0xffffffffu, v.y, off)));
  if (ex.n == 1) return v;
  const float4* b = ex(make_float4(v.x, v.y, 0.f, 0.f));
  const int lane = threadIdx.x & 31;
  float2 t = dup2(0.f);
  for (int i = lane; i < ex.n; i += 32) t = add2(t, *reinterpret_cast<const float2*>(b + i));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    t = add2(t, make_float2(__shfl_xor_sync(0xffffffffu, t.x, off), __shfl_xor_sync(0xffffffffu, t.y, off)));
  return t;
}

// Mean and sum of squared deviations of the walker's row.  Each warp works
// on values shifted by its own first value K_w (a row whose mean is large
// against its spread then loses nothing); the warps' parts are put on the
// first warp's shift, K_w - K_0 being a difference of two values of the row.
// v: this thread's slots (ok: which exist; the others hold anything finite);
// inv_cnt: 1 / cnt of this thread, 0 for none.  Returns K_0 in .n's place
// beside the mean and M2 relative to it.
struct RowStat {
  float K, m, M2;
};

template <int VE>
__device__ __forceinline__ RowStat walker_stats(Exchange& ex, const float2 (&v)[kE / 2],
                                                const bool (&ok)[kE / VE], int cnt, float inv_cnt) {
  const float K = __shfl_sync(0xffffffffu, v[0].x, 0);
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) sum += ok[e / VE] ? get_slot(v, e) - K : 0.f;
  Part p;
  p.n = static_cast<float>(cnt);
  p.m = sum * inv_cnt;
  p.M2 = 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float d = ok[e / VE] ? (get_slot(v, e) - K) - p.m : 0.f;
    p.M2 = fmaf(d, d, p.M2);
  }
  p = butterfly<false, 32>(p);
  if (ex.n == 1) return {K, p.m, p.M2};
  const float4* b = ex(make_float4(K, p.n, p.m, p.M2));
  const int lane = threadIdx.x & 31;
  const float K0 = b[0].x;
  Part t{0.f, 0.f, 0.f};
  for (int i = lane; i < ex.n; i += 32) {
    const float4 u = b[i];
    t = merge<false>(t, Part{u.y, (u.x - K0) + u.z, u.w});
  }
  t = butterfly<false, 32>(t);
  return {K0, t.m, t.M2};
}

// ------------------------------------------------------------------ host
// How a call's rows are spread: VE, threads, cluster and slice.
struct Shape {
  int threads;
  int C;
  int slice;  // columns a CTA owns, a multiple of 8
};

inline Shape shape_of(int H) {
  Shape s;
  s.C = (H + kSlice - 1) / kSlice;
  s.slice = s.C == 1 ? H : ((H + s.C - 1) / s.C + 7) / 8 * 8;
  s.threads = ((s.slice + kE - 1) / kE + 31) / 32 * 32;
  return s;
}

inline int elem_size(int dtype) { return dtype == kF32 ? 4 : 2; }

// Walkers (CTAs or clusters) of kernel f that fit the device at once; cached
// per kernel, device, threads and cluster.  Negative: a CUDA error.
int resident_walkers(const void* f, int threads, int C, const DeviceInfo& dev);

// Launches kernel(args...) as walkers * C CTAs.
template <typename Args>
cudaError_t launch_walkers(void (*kernel)(Args), int64_t walkers, const Shape& sh, const LaunchCtx& c,
                           const Args& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(walkers * sh.C));
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
