// The random bits of a dropout mask: Philox 4x32 with 10 rounds, from its
// authors' description (Salmon, Moraes, Dror, Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", 2011).  A round multiplies two of the four words by
// constants, 32 x 32 to 64 bits, and swaps and xors the halves with the other
// two and with the key, which grows by a constant a round.
//
// One block of bits serves 8 elements with 16 each: 20 wide products and as
// many three-way xors, some 8 issue slots an element.  A plain dropout of 16-bit
// elements, which moves 4 bytes each, has about 22 slots an element at the
// bandwidth of a copy; with 32 bits an element the generator alone would take
// most of them.
#pragma once

#include "block.cuh"
#include "drop.h"

namespace addln {
namespace blk {

struct Philox {
  uint32_t k0, k1, o0, o1;  // key, upper half of the counter

  __device__ __forceinline__ void init(const DropSpec& d) {
    uint64_t seed = d.seed, offset = d.offset;
    if (d.rng != nullptr && ADDLN_IN(760, 0, 16, 16)) {
      seed = __ldcg(reinterpret_cast<const unsigned long long*>(d.rng));
      offset = __ldcg(reinterpret_cast<const unsigned long long*>(d.rng) + 1);
    }
    k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    o0 = static_cast<uint32_t>(offset), o1 = static_cast<uint32_t>(offset >> 32);
  }
  // the four words of block `at`
  __device__ __forceinline__ uint4 operator()(uint64_t at) const {
    uint32_t c0 = static_cast<uint32_t>(at), c1 = static_cast<uint32_t>(at >> 32), c2 = o0, c3 = o1;
    uint32_t a = k0, b = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
      c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ a;
      c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ b;
      c1 = static_cast<uint32_t>(p1), c3 = static_cast<uint32_t>(p0);
      a += 0x9E3779B9u, b += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
  }
};

// Whether the elements of the low and the high half of a word are kept.
__device__ __forceinline__ bool keep_lo(uint32_t w, uint32_t above) { return (w << 16) > above; }
__device__ __forceinline__ bool keep_hi(uint32_t w, uint32_t above) { return w > above; }

// Bit e: element e of the block is kept.
__device__ __forceinline__ uint32_t keep_bits(const uint4& w, uint32_t above) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m |= keep_lo(v[i], above) ? 1u << (2 * i) : 0u;
    m |= keep_hi(v[i], above) ? 2u << (2 * i) : 0u;
  }
  return m;
}

// The mask of a thread's groups of one row.  Rows on 16-byte borders: a group
// of 8 is a block of bits, one of 4 (fp32) a half of one.  Other rows (SH): a
// group may lie in two blocks, its own and the next one, which is the next
// lane's, or lane 0's of the next k, or behind the warp's last group a block of
// its own; so all groups' bits are made first, 8 a group, and exchanged.
template <int VE, int NV, bool SH>
struct Mask {
  uint32_t bits;  // SH: of group k from bit 8 k on

  // at: index in the tensor of this thread's first column of group 0
  __device__ __forceinline__ void row(const Philox& rng, uint64_t at, uint32_t above) {
    if constexpr (SH) {
      constexpr unsigned kAll = 0xffffffffu;
      const int lane = threadIdx.x & 31;
      uint32_t own = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) own |= keep_bits(rng((at + k * 32 * VE) >> 3), above) << (8 * k);
      const uint32_t end = keep_bits(rng((at + ((NV - 1) * 32 + 1) * VE) >> 3), above);
      uint32_t next = __shfl_sync(kAll, own, (lane + 1) & 31);
      if (lane == 31) next = (NV > 1 ? next >> 8 : 0u) | end << (8 * (NV - 1));
      const int s = static_cast<int>(at & 7);
      bits = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t two = ((own >> (8 * k)) & 0xffu) | ((next >> (8 * k)) & 0xffu) << 8;
        bits |= ((two >> s) & 0xffu) << (8 * k);
      }
    }
  }
  // v[i] of group k: kept ones times `scale`, dropped ones 0
  __device__ __forceinline__ void apply(const Philox& rng, uint64_t at, int k, uint32_t above, float2 scale,
                                        float2 (&v)[VE / 2]) const {
    if constexpr (SH) {
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) {
        const float2 u = mul2(v[i], scale);
        v[i].x = (bits >> (8 * k + 2 * i)) & 1u ? u.x : 0.f;
        v[i].y = (bits >> (8 * k + 2 * i)) & 2u ? u.y : 0.f;
      }
    } else {
      const uint4 w = rng((at + k * 32 * VE) >> 3);
      uint32_t t[4] = {w.x, w.y, w.z, w.w};
      if constexpr (VE == 4) {
        const bool up = ((at >> 2) & 1) != 0;
        t[0] = up ? w.z : w.x, t[1] = up ? w.w : w.y;
      }
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) {
        const float2 u = mul2(v[i], scale);
        v[i].x = keep_lo(t[i], above) ? u.x : 0.f;
        v[i].y = keep_hi(t[i], above) ? u.y : 0.f;
      }
    }
  }
};

}  // namespace blk
}  // namespace addln
