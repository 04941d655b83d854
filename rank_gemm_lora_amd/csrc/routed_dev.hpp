// Device helpers of the routed kernels (routed.hip, gemm.hip).
#pragma once

#include "common.hpp"
#include "routed.hpp"

namespace lora {

// The adapter of token t and its scale; -1 (the base output) past the last token, for an index outside
// the pool, a zero scale or a rank of zero.
__device__ __forceinline__ int route(const Routing& rt, int64_t t, int64_t T, float& s) {
  s = 0.f;
  if (t >= T || rt.n_adapters == 0) return -1;
  const int a = rt.token_adapter[t];
  if (static_cast<uint32_t>(a) >= static_cast<uint32_t>(rt.n_adapters)) return -1;
  s = rt.scales[a];
  if (rt.token_scale != nullptr) s *= rt.token_scale[t];
  if (s == 0.f || (rt.ranks != nullptr && rt.ranks[a] <= 0)) return -1;
  return a;
}

// Rank of adapter a in its slot, a multiple of 8 (a is wave-uniform).
__device__ __forceinline__ int route_rank(const int32_t* ranks, int rank, int a) {
  return ranks != nullptr ? __builtin_amdgcn_readfirstlane((min(ranks[a], rank) + 7) & ~7) : rank;
}

// Its rank itself: what lies behind is zeros in t, whatever x and the scale are (an infinite x times the zeros
// that pad a rank to 8, to the slot or to 64 would be NaN there, and so would the token's outputs).
__device__ __forceinline__ int route_live(const int32_t* ranks, int rank, int a) {
  return ranks != nullptr ? min(ranks[a], rank) : rank;
}

typedef __attribute__((address_space(3))) void lds_void;

// s_waitcnt immediate: at most n vector memory operations outstanding, other counters not waited for.
constexpr int waitcnt_vmem(int n) { return (n & 0xf) | ((n >> 4) << 14) | 0x70 | 0xf00; }

// Workgroup barrier that does not wait for the loads of later stages (__syncthreads would); this wave's
// LDS reads are complete before it arrives.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xc07f);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// A bf16 pair with zero in place of what is infinite or NaN.
__device__ __forceinline__ uint32_t finite_pair(uint32_t v) {
  if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
  if ((v & 0x7f800000u) == 0x7f800000u) v &= 0xffffu;
  return v;
}

// NV consecutive values v of one token, scaled by s, from rank q (at element `at`) on, zeros from rank `live` on, as bf16: hi + mid, or hi + mid + lo, which
// together hold all 24 bits of t (each the nearest bf16 of what the ones before it leave; nothing behind a
// value that is not finite). NV is 2 or 4.
template <int NV>
__device__ __forceinline__ void put_rank_wide(const RoutedDown& p, int64_t at, int q, int live, const float (&v)[NV], float s) {
  uint32_t w[3][NV / 2];
#pragma unroll
  for (int e = 0; e < NV; e += 2) {
    float a = q + e < live ? v[e] * s : 0.f, b = q + e + 1 < live ? v[e + 1] * s : 0.f;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t h = pack_bf16x2(a, b);
      w[k][e / 2] = h;
      const float ha = __uint_as_float(h << 16), hb = __uint_as_float(h & 0xffff0000u);
      a = __builtin_isfinite(ha) ? a - ha : 0.f;
      b = __builtin_isfinite(hb) ? b - hb : 0.f;
    }
  }
  uint16_t* const dst[3] = {p.hi, p.mid, p.lo};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k == p.terms) break;
    if constexpr (NV == 4) *reinterpret_cast<uint2*>(dst[k] + at) = uint2{w[k][0], w[k][1]};
    else *reinterpret_cast<uint32_t*>(dst[k] + at) = w[k][0];
  }
}

}  // namespace lora
