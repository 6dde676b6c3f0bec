// y = dropout(x), element by element: 2 S bytes and an eighth of a block of random
// bits an element.  Bound by memory where the tensor is large: 32768x8192 bf16 158 us
// (6.8 TB/s, 1.02 of a copy), 8192x4096 fp32 41 us (0.98); 4096x768 fp16 3.3 us, a
// launch and 13 MB.  17.5 instructions an element of bf16 leave a quarter of the issue
// slots empty.  Tensors off 16-byte borders go element by element, a thread's eight side
// by side, so that a warp's accesses lie 16 bytes apart: 32768x8192 bf16 645 us (0.25),
// 8192x4096 fp32 141 (0.28), 4096x768 fp16 9.8.
#include "philox.cuh"

namespace addln {
namespace blk {

constexpr int kThreads = 256;

// VEC: x and y lie on 16-byte borders.  A thread has kBlocks blocks of 8
// elements, a CTA's threads apart and all in flight; the tensor's last block may be
// shorter.
template <int DT, bool VEC, int kBlocks>
__global__ void __launch_bounds__(kThreads) k_dropout(const void* x, void* y, int64_t n, const DropSpec d) {
  using IO = Io<DT>;
  constexpr int S = IO::kBytes, U = S / 2;  // 16-byte vectors a block
  const int64_t b0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kBlocks) + threadIdx.x;
  // a short tensor's lines asked of L2 while the kernel before may be finishing
  if (kBlocks == 1 && (threadIdx.x & (16 / S - 1)) == 0 && b0 * 8 < n && ADDLN_IN(764, b0 * 8 * S, 1, n * S))
    prefetch_line(static_cast<const char*>(x) + b0 * 8 * S);
  pdl_trigger();
  pdl_wait();
  const float2 scale = dup2(d.scale);
  const int64_t whole = VEC ? n / 8 : 0;
  [[maybe_unused]] const int64_t extent = n * S;
  uint4 v[kBlocks][U];
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int64_t b = b0 + j * kThreads;
    if (b >= whole) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[j][u] = make_uint4(0, 0, 0, 0);
      const int64_t at = b * 8 * S + 16 * u;
      // not the read-only path: y may be x
      if (ADDLN_IN(761, at, 16, extent)) v[j][u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at));
    }
  }
  Philox<false> rng;
  rng.init(d);
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int64_t b = b0 + j * kThreads;
    if (b * 8 >= n) break;
    uint4 w = make_uint4(0, 0, 0, 0);
    uint32_t above = d.above;
    if (d.on) w = rng(b, 0, d.wide);
    const uint32_t t[4] = {w.x, w.y, w.z, w.w};
    if (b < whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint4 o = v[j][u];
        if (d.on) {
          float2 f[IO::kVec / 2];
          IO::to_pairs(o, f);
#pragma unroll
          for (int i = 0; i < IO::kVec / 2; ++i) {
            const uint32_t ww = t[u * (IO::kVec / 2) + i];
            const float2 s = mul2(f[i], scale);
            f[i] = make_float2(keep_lo(ww, above) ? s.x : 0.f, keep_hi(ww, above) ? s.y : 0.f);
          }
          o = IO::from_pairs(f);
        }
        const int64_t at = b * 8 * S + 16 * u;
        if (ADDLN_IN(762, at, 16, extent)) st_stream_v4(static_cast<char*>(y) + at, o);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t i = b * 8 + e;
        if (i >= n || !ADDLN_IN(763, i * S, S, extent)) continue;
        const bool keep = (e & 1) ? keep_hi(t[e >> 1], above) : keep_lo(t[e >> 1], above);
        if constexpr (DT == kF32) {
          const float f = __ldcs(static_cast<const float*>(x) + i);
          static_cast<float*>(y)[i] = !d.on ? f : keep ? f * d.scale : 0.f;
        } else {
          const unsigned short h = __ldcs(static_cast<const unsigned short*>(x) + i);
          const float f = DT == kF16 ? __half2float(__ushort_as_half(h)) : __bfloat162float(__ushort_as_bfloat16(h));
          if (d.on)
            IO::store1(y, i, keep ? f * d.scale : 0.f);
          else
            static_cast<unsigned short*>(y)[i] = h;
        }
      }
    }
  }
}

namespace {
using DropKernel = void (*)(const void*, void*, int64_t, const DropSpec);
template <int DT>
DropKernel pick(bool vec, bool many) {
  if (vec) return many ? &k_dropout<DT, true, 4> : &k_dropout<DT, true, 1>;
  return many ? &k_dropout<DT, false, 4> : &k_dropout<DT, false, 1>;
}
}  // namespace
}  // namespace blk

int launch_dropout(int dtype, const void* x, void* y, int64_t n, const DropSpec& drop, const LaunchCtx& c) {
  using namespace blk;
  const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 15) == 0;
  // One block a thread up to twice as many as the GPU has threads for, else four
  // (us with one / four, bf16: 256x768 1.2 / 1.9, 4096x768 3.7 / 4.9, 8192x4096 24.7 /
  // 22.1, 16384x8192 94 / 81).
  const int64_t blocks = n / 8 + (n % 8 != 0);
  const bool many = blocks > int64_t{2 * 2048} * c.dev.sms;
  const DropKernel k = dtype == kF32 ? pick<kF32>(vec, many) : dtype == kF16 ? pick<kF16>(vec, many) : pick<kBF16>(vec, many);
  const int64_t per = kThreads * (many ? 4 : 1), ctas = (blocks + per - 1) / per;
  if (ctas > 0x7fffffff) return ADDLN_ERR_SHAPE;
  const cudaError_t e = launch_kernel(k, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, c.stream, c.pdl, x, y, n, drop);
  if (e != cudaSuccess) {
    note_cuda_error(static_cast<int>(e));
    return ADDLN_ERR_LAUNCH;
  }
  return ADDLN_OK;
}

ADDLN_BOUNDS_READER(read_bounds_drop)

}  // namespace addln
