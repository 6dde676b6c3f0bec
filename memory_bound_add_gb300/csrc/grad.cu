// Global gradient norm and clipping over many tensors (include/addln_grad.h).
//
// The table of tensors travels in the launch's parameters (up to 1000
// tensors a launch), so a call needs no copy to the device and can be
// captured.  The memory of all tensors is cut into chunks of 16 KB on 16-byte
// borders, which the CTAs of a persistent grid take in turn: 4 vectors a
// thread, the next chunk's loads issued before the current one is used.  A
// thread adds the squares of a chunk's share (at most 32 elements) in fp32
// and the shares as an unevaluated sum of two fp32 values; a CTA leaves one
// partial.  The kernel that scales adds the partials itself, in a fixed
// order, in every CTA, and takes the chunks from the last to the first: what
// the first kernel read last is in L2 still.
#include <math.h>

#include <algorithm>
#include <vector>

#include <cuda_runtime.h>

#include "../../include/addln_grad.h"
#include "abi.h"
#include "block.h"
#include "common.cuh"

namespace addln {
namespace gr {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;
constexpr int kMaxCtas = 2048;  // partials a launch may leave
// Tensors of a launch's table: one of 4 KB where that holds them all, else 32 KB
// (9 tensors: the larger table costs the host 6 us a call, the GPU nothing).
constexpr int kManyTensors = 1000, kFewTensors = 120;
// 16-byte vectors a thread has of a chunk (us with 2, 4, 8: one block of fp32 in
// place 13.5, 11.8, 13.9; 1.75e9 bf16 1683, 1585, 1956).
constexpr int kVecs = 4;
constexpr int kChunk = kThreads * kVecs * 16;

struct Entry {
  const void* g;
  void* out;
  int64_t n;
  uint32_t first;  // chunks of the tensors before this one
  uint8_t dtype, out_dtype;
};

template <int N>
struct Table {
  Entry e[N];
  int count;
  uint32_t chunks;
};

// hi + lo, lo being what the roundings of hi left.  (fp64 would do, but has
// a 64th of the rate: adding a few hundred partials in every CTA took it
// longer than the memory traffic of a small model.)
struct Two {
  float hi, lo;
  __device__ __forceinline__ void add(float s, float s_lo) {
    const float sum = __fadd_rn(hi, s), b = __fadd_rn(sum, -hi);
    const float err = __fadd_rn(__fadd_rn(hi, -__fadd_rn(sum, -b)), __fadd_rn(s, -b));
    lo = __fadd_rn(lo, __fadd_rn(err, s_lo));
    hi = sum;
  }
};

// A CTA's sum of squares: hi + lo, and in fp64 the shares that leave fp32's
// range.
struct alignas(16) Partial {
  Two s;
  double wide;
};

struct ClipArgs {
  const Partial* part;  // partials to add (nparts of them), or nullptr: *norm is there already
  int nparts;
  float* norm_out;     // written from the partials by the first CTA, or nullptr
  const float* norm;
  float scale, max_norm;
};

// The tensor that chunk c belongs to (tensors without elements have no chunk).
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, uint32_t c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Which elements of a chunk are the tensor's: the chunk's element r (counted
// from its 16-byte border) is element begin + r of the tensor, for r in
// [lo, hi); `mis` of the tensor's first elements' places on that border are
// not its own.  one: the element before the first or after the last whole
// vector that this thread has (thread q of the first warp has r = lo + q,
// thread q of the second r = hi / VEC VEC + q), or -1.
template <int S>  // bytes of an element
struct Share {
  static constexpr int VEC = 16 / S;
  int64_t begin;
  int lo, hi;

  __device__ __forceinline__ Share(const Entry& e, uint32_t chunk) {
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(e.g) & 15u) / S;
    begin = static_cast<int64_t>(chunk) * (kChunk / S) - mis;
    lo = chunk == 0 ? mis : 0;
    hi = static_cast<int>(min(static_cast<int64_t>(kChunk / S), e.n - begin));
  }
  __device__ __forceinline__ bool whole(int r) const { return r >= lo && r + VEC <= hi; }
  __device__ __forceinline__ int one() const {
    const int t = threadIdx.x, q = t & 31, first = (lo + VEC - 1) / VEC * VEC, last = max(first, hi / VEC * VEC);
    if (t < 32 && lo + q < min(first, hi)) return lo + q;
    if (t >= 32 && t < 64 && last + q < hi) return last + q;
    return -1;
  }
};

struct Piece {
  int k;           // tensor
  uint32_t chunk;  // its chunk
  uint4 v[kVecs];  // vector j: elements (threadIdx.x + j kThreads) VEC on, zeros if not all are the tensor's
  uint32_t e;      // the one element, or 0
};

// Loads past L1: in place, this kernel writes what it reads.
template <int S>
__device__ __forceinline__ void load_share(const Entry& e, Piece& p) {
  const Share<S> s(e, p.chunk);
  const char* g = static_cast<const char*>(e.g) + s.begin * S;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int r = (threadIdx.x + j * kThreads) * s.VEC;
    p.v[j] = make_uint4(0, 0, 0, 0);
    if (s.whole(r) && ADDLN_IN(801, (s.begin + r) * S, 16, e.n * S))
      p.v[j] = __ldcg(reinterpret_cast<const uint4*>(g + r * S));
  }
  p.e = 0;
  const int r = s.one();
  if (r >= 0 && ADDLN_IN(802, (s.begin + r) * S, S, e.n * S)) {
    if constexpr (S == 4)
      p.e = __ldcg(reinterpret_cast<const uint32_t*>(g) + r);
    else
      p.e = __ldcg(reinterpret_cast<const unsigned short*>(g) + r);
  }
}

template <int N>
__device__ __forceinline__ void load_piece(const Table<N>& t, uint32_t c, Piece& p) {
  const Entry& e = t.e[p.k];
  p.chunk = c - e.first;
  if (e.dtype == kF32)
    load_share<4>(e, p);
  else
    load_share<2>(e, p);
}

template <int DT>
__device__ __forceinline__ float value_of(uint32_t raw) {
  if constexpr (DT == kF32) return __uint_as_float(raw);
  const unsigned short b = static_cast<unsigned short>(raw);
  return DT == kF16 ? __half2float(__ushort_as_half(b)) : __bfloat162float(__ushort_as_bfloat16(b));
}

// Sum of squares of a thread's share.  At most 33 elements, so fp32 keeps it
// to a few roundings.  Where the sum is below 1e-30, squares may have been lost
// to fp32's range, and 2^43 elements (the most a call takes) in shares of up to
// 1e25 each stay below 1e38, within it: beyond either end 0 is returned and
// *lost set, unless all elements are zeros.  (Sums of fp16 squares are below
// 2e11; only a NaN or an infinity leaves the range.)
template <int DT>
__device__ __forceinline__ float squares(const Piece& p, bool* lost) {
  using IO = Io<DT>;
  constexpr int VEC = IO::kVec;
  const float one = value_of<DT>(p.e);
  float2 acc[2] = {make_float2(one * one, 0.f), dup2(0.f)};
  uint32_t any = p.e;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float2 f[VEC / 2];
    IO::to_pairs(p.v[j], f);
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) acc[q & 1] = fma2(f[q], f[q], acc[q & 1]);
    any |= p.v[j].x | p.v[j].y | p.v[j].z | p.v[j].w;
  }
  const float s = (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
  if (DT == kF16 ? s <= 1e25f : s >= 1e-30f && s <= 1e25f) return s;
  *lost = (any & (DT == kF32 ? 0x7fffffffu : 0x7fff7fffu)) != 0;
  return 0.f;
}

template <int DT>
__device__ __forceinline__ double squares_wide(const Piece& p) {
  using IO = Io<DT>;
  constexpr int VEC = IO::kVec;
  const double one = value_of<DT>(p.e);
  double d = one * one;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[VEC];
    IO::unpack(p.v[j], f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) d = fma(static_cast<double>(f[e]), static_cast<double>(f[e]), d);
  }
  return d;
}

__device__ __forceinline__ float squares_of(int dt, const Piece& p, bool* lost) {
  return dt == kF32 ? squares<kF32>(p, lost) : dt == kF16 ? squares<kF16>(p, lost) : squares<kBF16>(p, lost);
}

// Reads every gradient once and is bound by that.  With the kernel that adds the
// partials: 260 MB of fp16 41 us (6.3 TB/s), 3.5 GB of bf16 492 us (7.1 TB/s),
// 28 MB of fp32 8.8 us, most of it the two launches and the first loads.
template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_grad_squares(const __grid_constant__ Table<N> t, Partial* part) {
  constexpr int kWarps = kThreads / 32;
  __shared__ Partial sums[kWarps];
  pdl_trigger();
  pdl_wait();
  Two sum{0.f, 0.f};
  Piece next;
  next.k = tensor_of(t, blockIdx.x);
  bool have = false, again = false;
  for (uint32_t c = blockIdx.x;; c += gridDim.x) {
    // the next chunk's loads, before the current one is used
    const Piece cur = next;
    const bool more = c < t.chunks;
    if (more) {
      while (next.k + 1 < t.count && t.e[next.k + 1].first <= c) ++next.k;
      load_piece(t, c, next);
    }
    if (have) {
      bool lost = false;
      sum.add(squares_of(t.e[cur.k].dtype, cur, &lost), 0.f);
      again |= lost;
    }
    if (!more) break;
    have = true;
  }
  // shares that fp32 cannot hold (NaN, infinite, very large or small), again
  double wide = 0.0;
  const bool redo = __syncthreads_or(again);
  if (redo) {
    Piece p;
    p.k = tensor_of(t, blockIdx.x);
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
      while (p.k + 1 < t.count && t.e[p.k + 1].first <= c) ++p.k;
      load_piece(t, c, p);
      const int dt = t.e[p.k].dtype;
      bool lost = false;
      squares_of(dt, p, &lost);
      if (lost) wide += dt == kF32 ? squares_wide<kF32>(p) : dt == kF16 ? squares_wide<kF16>(p) : squares_wide<kBF16>(p);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) wide += __shfl_down_sync(0xffffffffu, wide, off);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float hi = __shfl_down_sync(0xffffffffu, sum.hi, off), lo = __shfl_down_sync(0xffffffffu, sum.lo, off);
    sum.add(hi, lo);
  }
  if (lane == 0) sums[warp] = Partial{sum, wide};
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) {
      sum.add(sums[w].s.hi, sums[w].s.lo);
      if (redo) wide += sums[w].wide;
    }
    part[blockIdx.x] = Partial{sum, wide};
  }
}

// norm from the partials, added in a fixed order; the same value in every
// thread of every CTA.
__device__ __forceinline__ float norm_of(const Partial* part, int n, float scale, Partial* shared) {
  constexpr int kWarps = kThreads / 32;
  Two sum{0.f, 0.f};
  double wide = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads * 4) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (i + u * kThreads < n) v[u] = __ldcg(reinterpret_cast<const uint4*>(part + i + u * kThreads));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      sum.add(__uint_as_float(v[u].x), __uint_as_float(v[u].y));
      if ((v[u].z | v[u].w) != 0) wide += __hiloint2double(static_cast<int>(v[u].w), static_cast<int>(v[u].z));
    }
  }
  const bool any = __syncthreads_or(wide != 0.0);  // true for a NaN
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float hi = __shfl_down_sync(0xffffffffu, sum.hi, off), lo = __shfl_down_sync(0xffffffffu, sum.lo, off);
    sum.add(hi, lo);
    if (any) wide += __shfl_down_sync(0xffffffffu, wide, off);
  }
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = Partial{sum, wide};
  __syncthreads();
  // every thread joins the warps' sums itself
  sum = shared[0].s;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) sum.add(shared[w].s.hi, shared[w].s.lo);
  if (!any) return scale * __fsqrt_rn(__fadd_rn(sum.hi, sum.lo));
  wide = shared[0].wide;
  for (int w = 1; w < kWarps; ++w) wide += shared[w].wide;
  return static_cast<float>(static_cast<double>(scale) * sqrt((static_cast<double>(sum.hi) + sum.lo) + wide));
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const Partial* part, int n, float scale, float* norm) {
  __shared__ Partial shared[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const float v = norm_of(part, n, scale, shared);
  if (threadIdx.x == 0) *norm = v;
}

// 32 bytes at q, 32-byte aligned (evict-first, as st_stream_v4).
__device__ __forceinline__ void st_stream_v8(void* q, const uint4& a, const uint4& b) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// out = g factor for a thread's share of a chunk.
template <int DT, int OUT>
__device__ __forceinline__ void scale_share(const Entry& e, const Piece& p, float factor) {
  using IO = Io<DT>;
  using OO = Io<OUT>;
  constexpr int VEC = IO::kVec, OV = OO::kVec, OS = OO::kBytes;
  const Share<IO::kBytes> s(e, p.chunk);
  char* out = static_cast<char*>(e.out) + s.begin * OS;
  const float2 f2 = dup2(factor);
  // out's vectors begin where g's do on a border of their own size (16 bytes,
  // or 32 for two of fp32)
  const bool wide = (reinterpret_cast<uintptr_t>(out) & (VEC * OS - 1)) == 0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int r = (threadIdx.x + j * kThreads) * VEC;
    if (!s.whole(r) || !ADDLN_IN(813, s.begin + r, VEC, e.n)) continue;
    float2 f[VEC / 2];
    IO::to_pairs(p.v[j], f);
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) f[q] = mul2(f[q], f2);
    if (wide) {
      if constexpr (VEC == OV)
        st_stream_v4(out + r * OS, OO::from_pairs(f));
      else
        st_stream_v8(out + r * OS, OO::from_pairs(f), OO::from_pairs(f + OV / 2));
    } else {
#pragma unroll
      for (int q = 0; q < VEC; ++q) OO::store1(out, r + q, (q & 1) ? f[q >> 1].y : f[q >> 1].x);
    }
  }
  const int r = s.one();
  if (r >= 0 && ADDLN_IN(814, s.begin + r, 1, e.n)) OO::store1(out, r, value_of<DT>(p.e) * factor);
}

// Reads every gradient a second time (what L2 no longer holds, from memory) and
// writes it.  Both kernels: 260 MB of fp16 into fp32 173 us (779 MB of
// algorithmic traffic 0.66 of a copy; with the second read 0.89), 3.5 GB of
// bf16 1570 us (0.66; with it 0.99), 28 MB of fp32 in place with nothing to scale
// 11.8 us.  Gradients of less than L2's 129 MB are there still; of larger ones the
// end is, hence from the last chunk to the first (first to last: 1% slower).
// This kernel alone, scaling in place by a norm that is given: 28 MB of fp32 10.8
// us, 260 MB of fp16 83 (6.2 TB/s), 3.5 GB of bf16 1080 (6.5 TB/s).  Outs whose
// vectors do not begin where the gradients' do are written element by element:
// 260 MB of fp16 at odd places of a buffer into fp32 tensors of their own, both
// kernels, 551 us.
template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_grad_clip(const __grid_constant__ Table<N> t, const ClipArgs a) {
  __shared__ Partial shared[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  float norm;
  if (a.part != nullptr) {
    norm = norm_of(a.part, a.nparts, a.scale, shared);
    if (a.norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.norm_out = norm;
  } else {
    norm = __ldcg(a.norm);
  }
  // without a limit nothing is scaled down, an infinite norm no more than another
  const float coef = isinf(a.max_norm) && !isnan(norm) ? 1.f : a.max_norm / (norm + 1e-6f);
  const float factor = a.scale * (coef > 1.f ? 1.f : coef);  // a NaN stays
  // from the last chunk to the first; in place with factor 1 there is
  // nothing to write
  if (blockIdx.x >= t.chunks) return;
  auto skip = [&](int k) { return factor == 1.f && t.e[k].g == t.e[k].out; };
  Piece next;
  next.k = tensor_of(t, t.chunks - 1 - blockIdx.x);
  bool have = false;
  for (int64_t left = static_cast<int64_t>(t.chunks) - 1 - blockIdx.x;; left -= gridDim.x) {
    const Piece cur = next;
    const bool more = left >= 0;
    if (more) {
      const uint32_t c = static_cast<uint32_t>(left);
      while (t.e[next.k].first > c) --next.k;
      if (!skip(next.k)) load_piece(t, c, next);
    }
    if (have && !skip(cur.k)) {
      const Entry& e = t.e[cur.k];
      if (e.dtype == kF32)
        scale_share<kF32, kF32>(e, cur, factor);
      else if (e.dtype == kF16)
        e.out_dtype == kF32 ? scale_share<kF16, kF32>(e, cur, factor) : scale_share<kF16, kF16>(e, cur, factor);
      else
        e.out_dtype == kF32 ? scale_share<kBF16, kF32>(e, cur, factor) : scale_share<kBF16, kBF16>(e, cur, factor);
    }
    if (!more) break;
    have = true;
  }
}

// ------------------------------------------------------------------ host
namespace {

using namespace addln::abi;

struct Lists {
  const void* const* grads;
  void* const* outs;
  const int64_t* sizes;
  const int* dtypes;
  const int* out_dtypes;
  int64_t count;
  void* out(int64_t i) const { return outs ? outs[i] : const_cast<void*>(grads[i]); }
  int out_dtype(int64_t i) const { return outs ? out_dtypes[i] : dtypes[i]; }
};

// More elements than any memory holds; chunk numbers stay within 32 bits.
constexpr int64_t kMaxTotal = int64_t{1} << 43;

struct Span {
  uintptr_t lo, hi;
  bool out;
};

// scaled: the outs are written, so they are checked too.
int check(const Lists& l, bool scaled, float scale, float max_norm) {
  if (l.count < 0) return ADDLN_ERR_SHAPE;
  if (!(scale > 0.f) || isinf(scale) || !(max_norm >= 0.f)) return ADDLN_ERR_SCALE;
  if (l.count == 0) return ADDLN_OK;
  if (!l.grads || !l.sizes || !l.dtypes || (scaled && l.outs && !l.out_dtypes)) return ADDLN_ERR_NULL;
  int64_t total = 0;
  for (int64_t i = 0; i < l.count; ++i) {
    if (!valid_dtype(l.dtypes[i])) return ADDLN_ERR_DTYPE;
    if (l.sizes[i] < 0 || l.sizes[i] > kMaxTotal - total) return ADDLN_ERR_SHAPE;
    total += l.sizes[i];
    if (scaled && l.out_dtype(i) != l.dtypes[i] && l.out_dtype(i) != ADDLN_FP32) return ADDLN_ERR_DTYPE;
    if (l.sizes[i] == 0) continue;
    if (!l.grads[i] || (scaled && !l.out(i))) return ADDLN_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(l.grads[i]) & (elem_bytes(l.dtypes[i]) - 1)) return ADDLN_ERR_ALIGN;
    if (scaled && (reinterpret_cast<uintptr_t>(l.out(i)) & (elem_bytes(l.out_dtype(i)) - 1))) return ADDLN_ERR_ALIGN;
  }
  return ADDLN_OK;
}

// Whether some out meets a gradient other than its own in place, or another
// out.  extra: [lo, hi) of one more output (the norm), or empty.
int check_overlap(const Lists& l, bool scaled, const Range& norm, bool norm_is_out, const Range& ws) {
  std::vector<Span> v;
  v.reserve(static_cast<size_t>(l.count) * 2 + 2);
  for (int64_t i = 0; i < l.count; ++i) {
    if (l.sizes[i] == 0) continue;
    const Range g = range_of(l.grads[i], l.sizes[i] * elem_bytes(l.dtypes[i]));
    if (scaled) {
      const Range o = range_of(l.out(i), l.sizes[i] * elem_bytes(l.out_dtype(i)));
      v.push_back({o.lo, o.hi, true});
      if (o.lo == g.lo && o.hi == g.hi) continue;
    }
    v.push_back({g.lo, g.hi, false});
  }
  if (norm.present) v.push_back({norm.lo, norm.hi, norm_is_out});
  if (ws.present) v.push_back({ws.lo, ws.hi, true});
  auto less = [](const Span& a, const Span& b) { return a.lo < b.lo; };
  if (!std::is_sorted(v.begin(), v.end(), less)) std::sort(v.begin(), v.end(), less);
  uintptr_t any_hi = 0, out_hi = 0;
  for (const Span& s : v) {
    if ((s.out ? any_hi : out_hi) > s.lo) return ADDLN_ERR_ALIAS;
    any_hi = std::max(any_hi, s.hi);
    if (s.out) out_hi = std::max(out_hi, s.hi);
  }
  return ADDLN_OK;
}

// One launch's share of the lists, from tensor `from` on; returns the next
// that has elements, or count.
template <int N>
int64_t fill(const Lists& l, int64_t from, bool scaled, Table<N>* t) {
  t->count = 0;
  int64_t chunks = 0, i = from;
  for (; i < l.count; ++i) {
    if (l.sizes[i] == 0) continue;
    if (t->count == N) break;
    t->e[t->count++] = {l.grads[i], scaled ? l.out(i) : nullptr, l.sizes[i], static_cast<uint32_t>(chunks),
                        static_cast<uint8_t>(l.dtypes[i]), static_cast<uint8_t>(scaled ? l.out_dtype(i) : 0)};
    const int64_t bytes = l.sizes[i] * elem_bytes(l.dtypes[i]) + (reinterpret_cast<uintptr_t>(l.grads[i]) & 15u);
    chunks += (bytes - 1) / kChunk + 1;
  }
  t->chunks = static_cast<uint32_t>(chunks);
  return i;
}

int launched(cudaError_t e) {
  if (e == cudaSuccess) return ADDLN_OK;
  note_cuda_error(static_cast<int>(e));
  return ADDLN_ERR_LAUNCH;
}

unsigned ctas_of(uint32_t chunks, int sms) {
  const uint32_t wave = static_cast<uint32_t>(std::min(kMaxCtas, sms * kCtasPerSm));
  return std::min(chunks, wave);
}

template <int N>
int run(const Lists& l, bool want_norm, bool scaled, float scale, float max_norm, float* norm, Partial* part,
        const LaunchCtx& c) {
  Table<N> t;
  int nparts = 0, launches = 0;
  if (want_norm) {
    for (int64_t i = 0; i < l.count;) {
      i = fill(l, i, scaled, &t);
      if (t.chunks == 0) continue;
      const unsigned ctas = ctas_of(t.chunks, c.dev.sms);
      const int rc = launched(launch_kernel(k_grad_squares<N>, dim3(ctas), dim3(kThreads), 0, c.stream, c.pdl, t,
                                            part + nparts));
      if (rc != ADDLN_OK) return rc;
      nparts += static_cast<int>(ctas);
      ++launches;
    }
    // one launch's partials are added by the scaling kernel's CTAs themselves
    if (!scaled || launches != 1) {
      const int rc = launched(launch_kernel(k_grad_norm, dim3(1), dim3(kThreads), 0, c.stream, c.pdl,
                                            static_cast<const Partial*>(part), nparts, scale, norm));
      if (rc != ADDLN_OK) return rc;
    }
  }
  if (!scaled) return ADDLN_OK;
  const bool join = want_norm && launches == 1;
  for (int64_t i = 0; i < l.count;) {
    if (!join) i = fill(l, i, true, &t);
    else i = l.count;  // the table is the one just launched
    if (t.chunks == 0) continue;
    const ClipArgs a{join ? part : nullptr, nparts, join ? norm : nullptr, norm, scale, max_norm};
    const int rc = launched(launch_kernel(k_grad_clip<N>, dim3(ctas_of(t.chunks, c.dev.sms)), dim3(kThreads), 0,
                                          c.stream, c.pdl, t, a));
    if (rc != ADDLN_OK) return rc;
  }
  return ADDLN_OK;
}

int64_t workspace_size(int64_t count) {
  if (count < 0 || count > INT64_MAX / 1024) return ADDLN_ERR_SHAPE;
  // every launch but the last takes at least kFewTensors tensors
  return (count / kFewTensors + 1) * kMaxCtas * static_cast<int64_t>(sizeof(Partial));
}

int call(const Lists& l, bool want_norm, bool scaled, float scale, float max_norm, float* norm, void* ws,
         int64_t ws_bytes, void* stream) {
  int rc = check(l, scaled, scale, max_norm);
  if (rc != ADDLN_OK) return rc;
  if (!norm) return ADDLN_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(norm) & 3u) return ADDLN_ERR_ALIGN;
  if (want_norm && (!ws || (reinterpret_cast<uintptr_t>(ws) & 15u) || ws_bytes < workspace_size(l.count)))
    return ADDLN_ERR_WORKSPACE;
  rc = check_overlap(l, scaled, range_of(norm, 4), want_norm, range_of(want_norm ? ws : nullptr, ws_bytes));
  if (rc != ADDLN_OK) return rc;
  LaunchCtx c;
  rc = launch_context(stream, &c);
  if (rc != ADDLN_OK) return rc;
  Partial* part = static_cast<Partial*>(ws);
  return l.count <= kFewTensors ? run<kFewTensors>(l, want_norm, scaled, scale, max_norm, norm, part, c)
                                : run<kManyTensors>(l, want_norm, scaled, scale, max_norm, norm, part, c);
}

}  // namespace
}  // namespace gr

ADDLN_BOUNDS_READER(read_bounds_grad)

}  // namespace addln

extern "C" {

int64_t grad_norm_workspace_size(int64_t count) { return addln::gr::workspace_size(count); }

int grad_norm(const void* const* grads, const int64_t* sizes, const int* dtypes, int64_t count, float scale,
              float* norm, void* workspace, int64_t workspace_bytes, void* stream) try {
  return addln::gr::call({grads, nullptr, sizes, dtypes, nullptr, count}, true, false, scale, 0.f, norm, workspace,
                         workspace_bytes, stream);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int grad_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes,
              const int* out_dtypes, int64_t count, float scale, float max_norm, const float* norm,
              void* stream) try {
  return addln::gr::call({grads, outs, sizes, dtypes, out_dtypes, count}, false, true, scale, max_norm,
                         const_cast<float*>(norm), nullptr, 0, stream);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

int grad_norm_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int* dtypes,
                   const int* out_dtypes, int64_t count, float scale, float max_norm, float* norm, void* workspace,
                   int64_t workspace_bytes, void* stream) try {
  return addln::gr::call({grads, outs, sizes, dtypes, out_dtypes, count}, true, true, scale, max_norm, norm,
                         workspace, workspace_bytes, stream);
} catch (...) {
  return ADDLN_ERR_HOST_MEMORY;
}

}  // extern "C"
