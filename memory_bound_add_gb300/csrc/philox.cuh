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

// What the first two rounds make of the offset, of the counter's second word
// (the upper half of the block's number) and of the key is the same for all
// blocks that share that word: two of the 20 products, and the xors beside them,
// are made once, which leaves 18 products a block.  The keys are the same for the
// whole grid: a warp reduction says so to the compiler, which then keeps them in
// uniform registers.  Both together: 32768x8192 bf16 dropout 187 us to 159, the
// boundary forward 347 to 320.
//
// KEYS: the other rounds' keys are reduced too, or the compiler adds them up anew for
// every block (85 instructions a block with all, so 69): worth 16 reductions where a
// thread makes many blocks and registers are left (boundary forward 8192x4096 bf16
// 43.8 us to 42.9, backward 32768x8192 427 to 418; dropout with its four blocks a
// thread 159 to 170).
template <bool KEYS>
struct Philox {
  uint32_t k0, k1, o0, o1;      // key, upper half of the counter
  uint32_t hi, a0, a2, b0, b3;  // second word, and what it gives
  uint32_t ka[KEYS ? 8 : 1], kb[KEYS ? 8 : 1];

  __device__ __forceinline__ static void mul(uint32_t a, uint32_t m, uint32_t& h, uint32_t& l) {
    const uint64_t p = static_cast<uint64_t>(a) * m;
    h = static_cast<uint32_t>(p >> 32), l = static_cast<uint32_t>(p);
  }
  __device__ __forceinline__ void head(uint32_t second) {
    uint32_t h, l, c0;
    hi = second;
    mul(o0, kM1, h, l);
    c0 = h ^ hi ^ k0;         // round 0: words 0 and 1 are c0 and l
    a2 = o1 ^ k1;             // word 2: the product's upper half ^ a2
    a0 = l ^ (k0 + kW0);      // round 1: word 0
    mul(c0, kM0, h, b3);      // word 3
    b0 = h ^ (k1 + kW1);      // word 2: round 0's word 3 ^ b0
  }
  // every thread of the warp takes part
  __device__ __forceinline__ void init(const DropSpec& d) {
    uint64_t seed = d.seed, offset = d.offset;
    if (d.rng != nullptr && ADDLN_IN(760, 0, 16, 16)) {
      // by way of L1: every warp of the grid reads these, and one slice of L2 would
      // have them all (4096x768 fp16 dropout 7.2 us, so 3.3)
      seed = __ldg(reinterpret_cast<const unsigned long long*>(d.rng));
      offset = __ldg(reinterpret_cast<const unsigned long long*>(d.rng) + 1);
    }
    auto same = [](uint64_t v) { return __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(v)); };
    k0 = same(seed), k1 = same(seed >> 32);
    o0 = same(offset), o1 = same(offset >> 32);
    head(0);
    if constexpr (KEYS) {
#pragma unroll
      for (uint32_t r = 2; r < 10; ++r) ka[r - 2] = same(k0 + r * kW0), kb[r - 2] = same(k1 + r * kW1);
    }
  }
  // the four words of block `at` + `more`; wide: its number may have an upper half
  __device__ __forceinline__ uint4 operator()(uint64_t at, uint32_t more, bool wide) {
    if (wide) {
      const uint32_t second = static_cast<uint32_t>((at + more) >> 32);
      if (second != hi) head(second);
    }
    uint32_t h, l, c0, c1, c2, c3;
    mul(static_cast<uint32_t>(at) + more, kM0, h, l);
    c2 = h ^ a2;
    mul(c2, kM1, h, c1);
    c0 = h ^ a0, c2 = l ^ b0, c3 = b3;
#pragma unroll
    for (uint32_t r = 2; r < 10; ++r) {
      uint32_t h0, l0, h1, l1;
      mul(c0, kM0, h0, l0);
      mul(c2, kM1, h1, l1);
      c0 = h1 ^ c1 ^ (KEYS ? ka[KEYS ? r - 2 : 0] : k0 + r * kW0);
      c2 = h0 ^ c3 ^ (KEYS ? kb[KEYS ? r - 2 : 0] : k1 + r * kW1);
      c1 = l1, c3 = l0;
    }
    return make_uint4(c0, c1, c2, c3);
  }
  static constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u, kW0 = 0x9E3779B9u, kW1 = 0xBB67AE85u;
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

// The mask of a thread's groups of one row.  Rows on 16-byte borders, and edged
// ones: a group of 8 is a block of bits, one of 4 (fp32) a half of one.  Shifted
// rows: a
// group may lie in two blocks, its own and the next one, which is the next
// lane's, or lane 0's of the next k, or behind the warp's last group a block of
// its own; so all groups' bits are made first, 8 a group, and exchanged.
template <int VE, int NV, int MODE>
struct Mask {
  static constexpr bool SH = MODE == kShifted;
  uint32_t bits;  // SH: of group k from bit 8 k on

  // at: index in the tensor of this thread's first column of group 0
  template <typename P>
  __device__ __forceinline__ void row(P& rng, uint64_t at, uint32_t above, bool wide) {
    if constexpr (SH) {
      constexpr unsigned kAll = 0xffffffffu;
      const int lane = threadIdx.x & 31;
      uint32_t own = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) own |= keep_bits(rng(at >> 3, k * 4 * VE, wide), above) << (8 * k);
      const uint32_t end = keep_bits(rng((at + VE) >> 3, (NV - 1) * 4 * VE, wide), above);
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
  template <typename P>
  __device__ __forceinline__ void apply(P& rng, uint64_t at, int k, uint32_t above, bool wide, float2 scale,
                                        float2 (&v)[VE / 2]) const {
    if constexpr (SH) {
#pragma unroll
      for (int i = 0; i < VE / 2; ++i) {
        const float2 u = mul2(v[i], scale);
        v[i].x = (bits >> (8 * k + 2 * i)) & 1u ? u.x : 0.f;
        v[i].y = (bits >> (8 * k + 2 * i)) & 2u ? u.y : 0.f;
      }
    } else {
      const uint4 w = rng(at >> 3, k * 4 * VE, wide);
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
