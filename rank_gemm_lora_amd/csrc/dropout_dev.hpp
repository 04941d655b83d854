// Dropout from a counter-based generator: whether element (t, k) of a [T, K] tensor is kept is a function of (seed,
// offset, t, k) alone, formed wherever it is needed and never stored.
#pragma once

#include "common.hpp"
#include "step.hpp"

namespace lora {
namespace {

// Philox-4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11) with 7 rounds, the
// fewest that pass the paper's BigCrush tests. One call gives the 8 elements 8 n .. 8 n + 7 of the flattened tensor
// (K is a multiple of 8) 16 bits each: element 2 i + h takes bits 16 h .. + 15 of word i.
__device__ __forceinline__ u32x4 philox7(uint64_t n, uint64_t seed, uint64_t offset) {
  uint32_t a = static_cast<uint32_t>(n), b = static_cast<uint32_t>(n >> 32);
  uint32_t c = static_cast<uint32_t>(offset), d = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * a, q = static_cast<uint64_t>(0xCD9E8D57u) * c;
    a = static_cast<uint32_t>(q >> 32) ^ b ^ k0;
    b = static_cast<uint32_t>(q);
    c = static_cast<uint32_t>(p >> 32) ^ d ^ k1;
    d = static_cast<uint32_t>(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{a, b, c, d};
}

// The generator of one launch (its state read once per workgroup where it lies on the device).
struct Dropper {
  uint64_t seed, offset;
  uint32_t thr2;   // thr in both halves: kept where the 16 bits are at least thr
  int64_t blocks;  // calls per row, K / 8
  __device__ __forceinline__ void init(const Drop& d, int64_t K) {
    seed = d.rng != nullptr ? d.rng[0] : d.seed;
    offset = d.rng != nullptr ? d.rng[1] : d.offset;
    thr2 = d.thr | (d.thr << 16);
    blocks = K / 8;
  }
  // 0xffff in each half whose 16 bits keep their element
  __device__ __forceinline__ uint32_t mask(uint32_t w) const {
    const u16x2 r = __builtin_bit_cast(u16x2, w), t = __builtin_bit_cast(u16x2, thr2);
    const u16x2 one = {1, 1};
    // thr - r, saturated: zero exactly where r >= thr
    const u16x2 lost = __builtin_elementwise_min(__builtin_elementwise_sub_sat(t, r), one);
    return __builtin_bit_cast(uint32_t, lost - one);
  }
  // the 8 elements of block kb (of 8 columns) of row t, as four masks of two
  __device__ __forceinline__ u32x4 masks(int64_t t, int64_t kb) const {
    const u32x4 w = philox7(static_cast<uint64_t>(t * blocks + kb), seed, offset);
    return u32x4{mask(w[0]), mask(w[1]), mask(w[2]), mask(w[3])};
  }
};

}  // namespace
}  // namespace lora
