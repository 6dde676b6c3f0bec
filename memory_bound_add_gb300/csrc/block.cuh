// Shared by the block-boundary kernels (block_fwd.cu, block_bwd.cu): how a
// row is spread over threads, how its elements reach them, and the row
// reductions over a warp, a CTA or the CTAs of a cluster.
//
// Layout.  One walker handles one row at a time: a warp, a CTA, or for the
// longest rows a cluster of C CTAs that each own a slice of the columns.  A
// warp owns 32 NV groups of VE neighbouring columns (16 bytes of the I/O
// type), of which lane l has groups l, l + 32, ...: the addresses of a
// thread's groups are constants apart.
//
// Rows that do not begin on 16-byte borders (SH: odd widths, offsets into a
// buffer) move in 16-byte granules all the same: a lane copies the granule
// that its group begins in, takes its group out of that and its neighbour's,
// and writes the granule that holds its group's begin together with the end
// of its neighbour's, which it gets by shuffle.  Accesses of single elements
// (2 bytes each) took twice as long: 8192x5001 bf16 rms/rms forward 204 us,
// with granules 99; backward 404 and 177.
#pragma once

#include <cooperative_groups.h>

#include "../../include/addln_block.h"
#include "block.h"
#include "common.cuh"

namespace addln {
namespace blk {

constexpr int kMaxThreads = 512;  // threads a CTA
constexpr int kMaxCluster = 8;    // the portable cluster size
constexpr int kMaxSmem = 227 * 1024;  // dynamic shared memory of a CTA

// VE fp32 parameters from column c on, of H; `fill` for a missing vector and
// past the end.  SH: any address, and the end may lie within the group.
template <int VE, bool SH>
__device__ __forceinline__ void load_params(const float* p, int c, int H, float fill, float (&v)[VE], int site) {
#pragma unroll
  for (int e = 0; e < VE; ++e) v[e] = fill;
  if (p == nullptr) return;
  p += c;
  if constexpr (SH) {
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (c + e < H && ADDLN_IN(site, 4 * (c + e), 4, 4 * static_cast<int64_t>(H))) v[e] = __ldg(p + e);
  } else {
    if (c >= H || !ADDLN_IN(site, 4 * c, 4 * VE, 4 * static_cast<int64_t>(H))) return;
#pragma unroll
    for (int h = 0; h < VE / 4; ++h) {
      const float4 u = ld_param_f4(p + 4 * h);
      v[4 * h] = u.x, v[4 * h + 1] = u.y, v[4 * h + 2] = u.z, v[4 * h + 3] = u.w;
    }
  }
}

// Asks L2 for the 128-byte line at p (a hint).
__device__ __forceinline__ void prefetch_line(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// A thread's groups of a row.  A group past the end of the slice does not
// exist: it is fetched as zeros and never stored, and its parameters are
// zeros.  With SH the slice's last group may hold fewer than VE columns.
template <int VE, int NV>
struct Cols {
  static constexpr int kStep = 32 * VE;  // columns between a thread's groups
  static constexpr int P = NV * VE / 2;
  int c0;           // first column of group 0
  int left;         // columns of the slice from c0 on (may be 0 or less)
  bool all;         // every group of the warp is whole
  float n, inv_n;   // columns of the warp, 1 / n (0 for none)

  __device__ __forceinline__ void init(int warp, int col0, int cols) {
    const int at0 = warp * NV * kStep + (threadIdx.x & 31) * VE;
    c0 = col0 + at0;
    left = cols - at0;
    const int own = min(max(cols - warp * NV * kStep, 0), NV * kStep);
    n = static_cast<float>(own);
    inv_n = own ? __frcp_rn(n) : 0.f;
    all = own == NV * kStep;
  }
  __device__ __forceinline__ int col(int k) const { return c0 + k * kStep; }
  __device__ __forceinline__ bool ok(int k) const { return left > k * kStep; }
  // columns of group k that exist
  __device__ __forceinline__ int valid(int k) const { return min(max(left - k * kStep, 0), VE); }
  // zeros in the slots of columns that do not exist
  __device__ __forceinline__ void clear(float2 (&v)[P]) const {
    if (all) return;
#pragma unroll
    for (int e = 0; e < NV * VE; ++e) {
      float& u = (e & 1) ? v[e >> 1].y : v[e >> 1].x;
      u = left > (e / VE) * kStep + e % VE ? u : 0.f;
    }
  }
};

// ------------------------------------------------------- shifted granules
// Bytes [sh, sh + 16) of the 32 bytes lo, hi; sh < 16, a multiple of 2.
__device__ __forceinline__ uint4 window(const uint4& lo, const uint4& hi, int sh) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (sh & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (sh & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const int bits = (sh & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

__device__ __forceinline__ int low4(const void* p, int64_t off) {
  return (static_cast<int>(reinterpret_cast<uintptr_t>(p)) + static_cast<int>(off)) & 15;
}

// Element e (a constant) of a group, as it is stored.
template <int S>
__device__ __forceinline__ void store_element(char* p, const uint4& v, int e) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (S == 4)
    *reinterpret_cast<uint32_t*>(p) = w[e];
  else
    *reinterpret_cast<unsigned short*>(p) = static_cast<unsigned short>((e & 1) ? w[e >> 1] >> 16 : w[e >> 1]);
}

// Writes a row's groups in the order of k, 0 to NV - 1, to `base + off` of a
// tensor of `extent` bytes.
template <int DT, int NV, bool SH>
struct Writer {
  static constexpr int S = Io<DT>::kBytes, VE = Io<DT>::kVec;
  uint4 prev;  // the last group, of lane 31

  __device__ __forceinline__ void put(const Cols<VE, NV>& cs, void* base, int64_t off, int k, const uint4& v, int site,
                                      int64_t extent) {
    off += k * (cs.kStep * S);
    char* p = static_cast<char*>(base) + off;
    if constexpr (!SH) {
      if (cs.ok(k) && ADDLN_IN(site, off, 16, extent)) st_stream_v4(p, v);
      return;
    } else {
      constexpr unsigned kAll = 0xffffffffu;
      const int lane = threadIdx.x & 31;
      const int s = low4(p, 0);  // bytes past the border, the same for the warp
      uint4 w = v;
      int lo = 0, hi = cs.valid(k);  // elements of the granule to write
      if (s != 0) {
        uint4 n;
        const uint4 send = lane == 31 && k > 0 ? prev : v;
        n.x = __shfl_sync(kAll, send.x, (lane + 31) & 31);
        n.y = __shfl_sync(kAll, send.y, (lane + 31) & 31);
        n.z = __shfl_sync(kAll, send.z, (lane + 31) & 31);
        n.w = __shfl_sync(kAll, send.w, (lane + 31) & 31);
        prev = v;
        w = window(n, v, 16 - s);
        const int own = s / S;  // the first of this lane's elements in it
        // the neighbour's group is there from the warp's second on
        const bool has = k > 0 || lane > 0;
        const int before = min(max(cs.left - (k * cs.kStep - VE), 0), VE) - (VE - own);
        lo = has ? 0 : own;
        hi = hi > 0 ? own + min(hi, VE - own) : has ? max(before, 0) : 0;
        p -= s;
        off -= s;
      }
      if (lo == 0 && hi == VE) {
        if (ADDLN_IN(site, off, 16, extent)) st_stream_v4(p, w);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (e >= lo && e < hi && ADDLN_IN(site, off + e * S, S, extent)) store_element<S>(p + e * S, w, e);
      }
      // nobody follows the warp's last group: its own end
      if (s != 0 && k == NV - 1 && lane == 31) {
        const int own = s / S;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (e >= VE - own && e < cs.valid(k) && ADDLN_IN(site, off + s + e * S, S, extent))
            store_element<S>(p + s + e * S, v, e);
      }
    }
  }
};

// --------------------------------------------------------------- staging
// A warp's groups of the rows ahead, in a ring of slots of its own in shared
// memory, copied by cp.async, 16 bytes a lane (zeros for what does not
// exist).  Without SH a lane alone reads what it has copied, so no barrier is
// needed; with SH a group may reach into the next lane's granule, and the
// warp meets before it reads and before it copies anew.  A warp's ring is one
// piece, [slot][tensor][group][lane], with SH one granule more a tensor.
constexpr int kMaxSlots = 2;

template <int DT, int NV, int NT, bool SH>
struct Ring {
  static constexpr int S = Io<DT>::kBytes, VE = Io<DT>::kVec;
  static constexpr uint32_t kTensor = (NV * 32 + (SH ? 1 : 0)) * 16;
  static constexpr uint32_t kSlot = NT * kTensor;  // bytes of a warp's slot
  uint32_t base;  // this thread's granule of group 0 of slot 0

  __device__ __forceinline__ uint32_t at(int slot, int i, int k) const {
    return base + static_cast<uint32_t>(slot) * kSlot + static_cast<uint32_t>(i) * kTensor + static_cast<uint32_t>(k) * 512u;
  }
  // n of the 16 bytes at src, zeros for the rest
  __device__ __forceinline__ static void copy(uint32_t dst, const char* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  }
  // A row of tensor I: group 0 of this thread at byte off of t.
  template <int I>
  __device__ __forceinline__ void fetch(const Cols<VE, NV>& cs, int slot, const void* t, int64_t off, int site,
                                        int64_t extent) {
    const char* p = static_cast<const char*>(t) + off;
    if constexpr (!SH) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const bool in = cs.ok(k) && ADDLN_IN(site, off + k * (cs.kStep * S), 16, extent);
        copy(at(slot, I, k), p + k * (cs.kStep * S), in ? 16 : 0);
      }
    } else {
      const int s = low4(p, 0);
      // bytes of the row's slice from this granule on; what lies past them is
      // not read.  A granule that begins before the row has the bytes before
      // it read along, which are the tensor's (the row before), but for the
      // tensor's own first granule.
      const int bytes = cs.left * S + s;
      p -= s;
      off -= s;
#pragma unroll
      for (int k = 0; k <= NV; ++k) {
        if (k == NV && (threadIdx.x & 31) != 0) continue;  // the granule after the last lane's
        const int n = min(max(bytes - k * (cs.kStep * S), 0), 16);
        const int64_t o = off + k * (cs.kStep * S);
        if (k == 0 && o < 0) {
          // zeros first: the row may end within this granule
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at(slot, I, 0)), "r"(0) : "memory");
#pragma unroll
          for (int b = 0; b < 16; b += S)
            if (b >= s && b < n && ADDLN_IN(site, o + b, S, extent)) {
              if constexpr (S == 4)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at(slot, I, 0) + b),
                             "r"(__ldcg(reinterpret_cast<const uint32_t*>(p + b))) : "memory");
              else
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at(slot, I, 0) + b),
                             "h"(__ldcg(reinterpret_cast<const unsigned short*>(p + b))) : "memory");
            }
        } else {
          copy(at(slot, I, k), p + k * (cs.kStep * S), n > 0 && ADDLN_IN(site, o, n, extent) ? n : 0);
        }
      }
    }
  }
  // zeros for tensor I
  template <int I>
  __device__ __forceinline__ void clear(int slot) {
#pragma unroll
    for (int k = 0; k <= (SH ? NV : NV - 1); ++k) {
      if (k == NV && (threadIdx.x & 31) != 0) continue;
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at(slot, I, k)), "r"(0) : "memory");
    }
  }
  __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // all but the AHEAD groups of copies committed last have arrived
  template <int AHEAD>
  __device__ __forceinline__ static void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
  }
  // before the first read of a slot, and before it is copied into again
  __device__ __forceinline__ static void meet() {
    if constexpr (SH) __syncwarp();
  }
  // Group k of tensor i, whose row lies s bytes past the borders.
  __device__ __forceinline__ uint4 take(int slot, int i, int k, int s) const {
    const uint32_t a = at(slot, i, k);
    const uint4 v = ld_shared_v4(a);
    if constexpr (!SH) return v;
    if (s == 0) return v;
    return window(v, ld_shared_v4(a + 16), s);
  }
};

// Parameters in shared memory, each thread's columns in places of its own (a
// warp's in one piece [vector][group][part][lane]), so that a read costs half
// of what a 16-byte load through L1 does.
template <int VE, int NV>
struct Kept {
  static constexpr int Q = VE / 4;  // 16-byte parts of a group
  static constexpr uint32_t kStep = 32 * 16;
  template <int NP>
  __host__ __device__ static constexpr uint32_t bytes() {
    return NP * NV * Q * kStep;
  }
  uint32_t base;

  __device__ __forceinline__ uint32_t at(int i, int k, int q) const {
    return base + static_cast<uint32_t>((i * NV + k) * Q + q) * kStep;
  }
  __device__ __forceinline__ void put(int i, int k, const float (&v)[VE]) const {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at(i, k, q)), "f"(v[4 * q]), "f"(v[4 * q + 1]),
                   "f"(v[4 * q + 2]), "f"(v[4 * q + 3]) : "memory");
  }
  __device__ __forceinline__ void get(int i, int k, float2 (&v)[VE / 2]) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint4 u = ld_shared_v4(at(i, k, q));
      v[2 * q] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      v[2 * q + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
};

// A CTA of a cluster may write into a peer's shared memory only once the peer
// has started: every thread arrives when it begins, and waits before its first
// exchange, behind the row's copies and the parameters, which take longer.
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

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

// Rows to put side by side in a CTA that has room for `most`: where the call's
// rows are few, the least power of two that needs no more CTAs than SMs (us,
// with `most` / so: forward 64x768 layer 4.4 / 2.9, 300x1024 layer 5.0 / 3.4;
// backward 64x768 fp32 6.6 / 5.0, 300x256 bf16 layer 6.8 / 5.5).
inline int rows_side_by_side(int most, int64_t rows, int sms) {
  int n = 1;
  while (n < most && static_cast<int64_t>(n) * sms < rows) n *= 2;
  return n < most ? n : most;
}

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
