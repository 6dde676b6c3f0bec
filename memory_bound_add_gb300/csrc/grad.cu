// Global gradient norm and clipping over many tensors (include/addln_grad.h).
//
// The table of tensors travels in the launch's parameters (up to 1000
// tensors a launch), so a call needs no copy to the device and can be
// captured.  The elements of all tensors are cut into chunks, which the CTAs
// of a persistent grid take in turn; a CTA sums squares in fp32 within a
// thread's share of a chunk and in fp64 beyond, and leaves one fp64 partial.
// The kernel that scales adds the partials itself, in a fixed order, in every
// CTA, and takes the chunks from the last to the first: what the first kernel
// read last is in L2 still.
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
constexpr int kManyTensors = 1000, kFewTensors = 120;

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
  int chunk;  // elements, a multiple of 8
};

struct ClipArgs {
  const double* part;  // partials to add (nparts of them), or nullptr: *norm is there already
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

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += red[w];
  return t;
}

// Sum of squares of elements [0, n) at g (n at most one chunk), this
// thread's share.  The share is at most a few dozen elements, so fp32 keeps
// it to a few roundings; where it leaves [1e-30, 1e30], squares may have been
// lost to fp32's range, and the share is summed again in fp64.
template <int DT>
__device__ __forceinline__ double chunk_squares(const char* g, int n, int64_t left_bytes) {
  using IO = Io<DT>;
  constexpr int S = IO::kBytes, VEC = IO::kVec;
  const int tid = threadIdx.x;
  const int head = min(n, static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(g) & 15u)) & 15u) / S));
  const int nv = (n - head) / VEC;
  const int tail = n - head - nv * VEC;
  const char* body = g + head * S;
  float2 acc[2] = {dup2(0.f), dup2(0.f)};
  uint32_t any = 0;
  auto vec = [&](const uint4& u) {
    float2 f[VEC / 2];
    IO::to_pairs(u, f);
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) acc[q & 1] = fma2(f[q], f[q], acc[q & 1]);
    any |= u.x | u.y | u.z | u.w;
  };
  constexpr int kU = 4;  // 16-byte loads in flight a thread
  int i = tid;
  for (; i + (kU - 1) * kThreads < nv; i += kU * kThreads) {
    uint4 u[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      u[k] = make_uint4(0, 0, 0, 0);
      if (ADDLN_IN(801, (i + k * kThreads) * 16 + head * S, 16, left_bytes))
        u[k] = __ldg(reinterpret_cast<const uint4*>(body) + i + k * kThreads);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) vec(u[k]);
  }
  for (; i < nv; i += kThreads)
    if (ADDLN_IN(802, i * 16 + head * S, 16, left_bytes)) vec(__ldg(reinterpret_cast<const uint4*>(body) + i));
  // the elements before the first and after the last 16-byte vector
  const int extra = tid < head ? tid : tid - head < tail ? n - tail + (tid - head) : -1;
  if (extra >= 0 && ADDLN_IN(803, extra * S, S, left_bytes)) {
    const float v = IO::load1(g, extra);
    acc[0].x = fmaf(v, v, acc[0].x);
    any |= v != 0.f;
  }
  const float s = (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
  if (DT == kF16 || (s >= 1e-30f && s <= 1e30f)) return s;
  const uint32_t mask = DT == kF32 ? 0x7fffffffu : 0x7fff7fffu;
  if ((any & mask) == 0) return 0.0;
  double d = 0.0;
  for (int j = tid; j < nv; j += kThreads)
    if (ADDLN_IN(804, j * 16 + head * S, 16, left_bytes)) {
      float f[VEC];
      IO::unpack(__ldg(reinterpret_cast<const uint4*>(body) + j), f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) d = fma(static_cast<double>(f[e]), static_cast<double>(f[e]), d);
    }
  if (extra >= 0 && ADDLN_IN(805, extra * S, S, left_bytes)) {
    const double v = IO::load1(g, extra);
    d = fma(v, v, d);
  }
  return d;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_grad_squares(const __grid_constant__ Table<N> t, double* part) {
  __shared__ double red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  double sum = 0.0;
  {
    int k = tensor_of(t, blockIdx.x);
    for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
      while (k + 1 < t.count && t.e[k + 1].first <= c) ++k;
      const int64_t at = static_cast<int64_t>(c - t.e[k].first) * t.chunk;
      const int64_t rest = t.e[k].n - at;
      const int n = static_cast<int>(rest < t.chunk ? rest : t.chunk);
      const int dt = t.e[k].dtype;
      const char* g = static_cast<const char*>(t.e[k].g) + at * (dt == kF32 ? 4 : 2);
      if (dt == kF32)
        sum += chunk_squares<kF32>(g, n, rest * 4);
      else if (dt == kF16)
        sum += chunk_squares<kF16>(g, n, rest * 2);
      else
        sum += chunk_squares<kBF16>(g, n, rest * 2);
    }
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// norm from the partials: every thread of every CTA gets the same value.
__device__ __forceinline__ float norm_of(const double* part, int n, float scale, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += __ldcg(part + i);
  s = block_sum(s, red);
  return static_cast<float>(static_cast<double>(scale) * sqrt(s));
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const double* part, int n, float scale, float* norm) {
  __shared__ double red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const float v = norm_of(part, n, scale, red);
  if (threadIdx.x == 0) *norm = v;
}

// out = g factor for elements [0, n) of one chunk.
template <int DT, int OUT>
__device__ __forceinline__ void chunk_scale(const char* g, char* out, int n, float factor, int64_t left) {
  using IO = Io<DT>;
  using OO = Io<OUT>;
  constexpr int S = IO::kBytes, VEC = IO::kVec, OV = OO::kVec, OS = OO::kBytes;
  const int tid = threadIdx.x;
  int head = min(n, static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(g) & 15u)) & 15u) / S));
  if ((reinterpret_cast<uintptr_t>(out + head * OS) & 15u) != 0) {
    // no common place for 16-byte accesses: element by element
    for (int i = tid; i < n; i += kThreads)
      if (ADDLN_IN(811, i, 1, left)) OO::store1(out, i, IO::load1(g, i) * factor);
    return;
  }
  const int nv = (n - head) / VEC;
  const int tail = n - head - nv * VEC;
  const char* body = g + head * S;
  char* obody = out + head * OS;
  const float2 f2 = dup2(factor);
  auto store = [&](int i, const uint4& u) {
    float2 f[VEC / 2];
    IO::to_pairs(u, f);
#pragma unroll
    for (int q = 0; q < VEC / 2; ++q) f[q] = mul2(f[q], f2);
#pragma unroll
    for (int q = 0; q < VEC / OV; ++q)
      st_stream_v4(obody + (static_cast<int64_t>(i) * VEC + q * OV) * OS, OO::from_pairs(f + q * OV / 2));
  };
  constexpr int kU = 4;
  int i = tid;
  for (; i + (kU - 1) * kThreads < nv; i += kU * kThreads) {
    uint4 u[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      u[k] = make_uint4(0, 0, 0, 0);
      if (ADDLN_IN(812, (i + k * kThreads) * VEC + head, VEC, left))
        u[k] = ld_stream_v4(body + static_cast<int64_t>(i + k * kThreads) * 16);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k)
      if (ADDLN_IN(813, (i + k * kThreads) * VEC + head, VEC, left)) store(i + k * kThreads, u[k]);
  }
  for (; i < nv; i += kThreads)
    if (ADDLN_IN(814, i * VEC + head, VEC, left)) store(i, ld_stream_v4(body + static_cast<int64_t>(i) * 16));
  const int extra = tid < head ? tid : tid - head < tail ? n - tail + (tid - head) : -1;
  if (extra >= 0 && ADDLN_IN(815, extra, 1, left)) OO::store1(out, extra, IO::load1(g, extra) * factor);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_grad_clip(const __grid_constant__ Table<N> t, const ClipArgs a) {
  __shared__ double red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  float norm;
  if (a.part != nullptr) {
    norm = norm_of(a.part, a.nparts, a.scale, red);
    if (a.norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.norm_out = norm;
  } else {
    norm = __ldcg(a.norm);
  }
  const float coef = a.max_norm / (norm + 1e-6f);
  const float factor = a.scale * (coef > 1.f ? 1.f : coef);  // a NaN stays
  if (blockIdx.x >= t.chunks) return;
  int k = tensor_of(t, t.chunks - 1 - blockIdx.x);
  for (int64_t left = static_cast<int64_t>(t.chunks) - 1 - blockIdx.x; left >= 0; left -= gridDim.x) {
    const uint32_t c = static_cast<uint32_t>(left);
    while (t.e[k].first > c) --k;
    const int64_t at = static_cast<int64_t>(c - t.e[k].first) * t.chunk;
    const int64_t rest = t.e[k].n - at;
    const int n = static_cast<int>(rest < t.chunk ? rest : t.chunk);
    const int dt = t.e[k].dtype, od = t.e[k].out_dtype;
    const char* g = static_cast<const char*>(t.e[k].g) + at * (dt == kF32 ? 4 : 2);
    char* out = static_cast<char*>(t.e[k].out) + at * (od == kF32 ? 4 : 2);
    if (factor == 1.f && g == out) continue;  // in place, nothing to scale
    if (dt == kF32)
      chunk_scale<kF32, kF32>(g, out, n, factor, rest);
    else if (dt == kF16)
      od == kF32 ? chunk_scale<kF16, kF32>(g, out, n, factor, rest) : chunk_scale<kF16, kF16>(g, out, n, factor, rest);
    else
      od == kF32 ? chunk_scale<kBF16, kF32>(g, out, n, factor, rest) : chunk_scale<kBF16, kBF16>(g, out, n, factor, rest);
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
constexpr int64_t kMaxTotal = int64_t{1} << 45;

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

// Elements a chunk: about sixteen chunks a CTA of one full wave, so that the
// CTAs come out even, between 2048 (8 elements a thread) and 16384 (64).
int chunk_of(int64_t total, int sms) {
  const int64_t want = total / (static_cast<int64_t>(sms) * kCtasPerSm * 16);
  int64_t c = 2048;
  while (c < 16384 && c < want) c *= 2;
  return static_cast<int>(c);
}

// One launch's share of the lists, from tensor `from` on; returns the next
// that has elements, or count.
template <int N>
int64_t fill(const Lists& l, int64_t from, int chunk, bool scaled, Table<N>* t) {
  t->count = 0;
  t->chunk = chunk;
  int64_t chunks = 0, i = from;
  for (; i < l.count; ++i) {
    if (l.sizes[i] == 0) continue;
    if (t->count == N) break;
    t->e[t->count++] = {l.grads[i], scaled ? l.out(i) : nullptr, l.sizes[i], static_cast<uint32_t>(chunks),
                        static_cast<uint8_t>(l.dtypes[i]), static_cast<uint8_t>(scaled ? l.out_dtype(i) : 0)};
    chunks += (l.sizes[i] - 1) / chunk + 1;
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
int run(const Lists& l, bool want_norm, bool scaled, float scale, float max_norm, float* norm, double* part,
        const LaunchCtx& c) {
  int64_t total = 0;
  for (int64_t i = 0; i < l.count; ++i) total += l.sizes[i];
  const int chunk = chunk_of(total, c.dev.sms);
  Table<N> t;
  int nparts = 0, launches = 0;
  if (want_norm) {
    for (int64_t i = 0; i < l.count;) {
      i = fill(l, i, chunk, scaled, &t);
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
                                            static_cast<const double*>(part), nparts, scale, norm));
      if (rc != ADDLN_OK) return rc;
    }
  }
  if (!scaled) return ADDLN_OK;
  const bool join = want_norm && launches == 1;
  for (int64_t i = 0; i < l.count;) {
    if (!join) i = fill(l, i, chunk, true, &t);
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
  if (count < 0 || count > INT64_MAX / 64) return ADDLN_ERR_SHAPE;
  // every launch but the last takes at least kFewTensors tensors
  return (count / kFewTensors + 1) * kMaxCtas * static_cast<int64_t>(sizeof(double));
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
  double* part = static_cast<double*>(ws);
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
