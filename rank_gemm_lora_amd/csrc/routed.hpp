// Internal interface of the routed kernels (routed.hip): a linear layer whose tokens take their
// adapters from a pool.
#pragma once

#include "launch.hpp"

namespace lora {

// Rank-wide producer: t = s_t . x[t] A_a^T of every token's own adapter a, as hi = RN_bf16(t) and,
// where lo is not null, RN_bf16(t - hi). Writes eid and blk (RoutedGemm) too.
struct RoutedDown {
  const uint16_t* x; int64_t ldx;
  int64_t T, K;
  const uint16_t* A;   // [n_adapters, rank, K]
  Routing rt;
  uint16_t* hi;        // [T, ldt]; a token's row is written up to its adapter's rank, then zeros to a
  uint16_t* lo;        // multiple of 64; not at all without an adapter
  int64_t ldt;         // rank_pad(rank)
  int32_t* eid;        // [T]
  int32_t* blk;        // [ceil(T / 16)]
};
hipError_t launch_routed_down(const RoutedDown& p, hipStream_t s);

// Tokens sorted by adapter (in token order within one), and the work items of a contraction over
// them: sorted positions are cut into chunks of `chunk`, an item is one adapter's part of one chunk.
// Item z = a + (index of its chunk), so every item has a place known without counting; items[z] is
// empty (lo == hi) where adapter and chunk do not meet.
struct RouteItem {
  int32_t adapter, lo, hi;
  int32_t part;  // where its partial sums go: -1 straight to the gradient (the adapter has one item), else a slot
};
struct RoutePlan {
  const int32_t* eid; int64_t T;
  int32_t n_adapters;
  int32_t chunk;
  int32_t* perm;       // [T]
  int32_t* off;        // [n_adapters + 1]
  RouteItem* items;    // [n_items]
  int64_t n_items;     // route_items(T, n_adapters, chunk)
};
constexpr int kRouteMaxChunk = 4096;  // positions of an item that a workgroup keeps in LDS
inline int64_t route_chunks(int64_t T, int64_t chunk) { return (T + chunk - 1) / chunk; }
inline int64_t route_items(int64_t T, int64_t n, int64_t chunk) { return n + T / chunk + 1; }
// Slots of partial sums: a chunk holds at most two items of adapters with more than one (the end of
// one, the start of another).
inline int64_t route_parts(int64_t T, int64_t chunk) { return 2 * route_chunks(T, chunk); }
hipError_t launch_route_plan(const RoutePlan& p, hipStream_t s);

// Contraction chunk for outputs of `tiles` workgroups each (the wider of the two gradients).
constexpr int kRtI = 256, kRtJ = 64, kRtT = 64;
inline int32_t route_chunk(int64_t T, int64_t tiles) {
  int64_t s = 1024 / (tiles > 0 ? tiles : 1);
  s = s < 1 ? 1 : (s > 64 ? 64 : s);
  int64_t c = (T + s - 1) / s;
  c = (c + kRtT - 1) / kRtT * kRtT;
  return static_cast<int32_t>(c < 256 ? 256 : (c > kRouteMaxChunk ? kRouteMaxChunk : c));
}

// out[a] = sum over a's tokens of P[t] (x) (hi + lo)[t]: [M, rank] row-major, or [rank, M] with
// transpose. Adapters without tokens get zeros.
struct RoutedContract {
  const uint16_t* P; int64_t ldp, M;
  const uint16_t *hi, *lo; int64_t ldt;
  int32_t rank;
  const RoutePlan* plan;
  float* part;         // [route_parts, M, rank_pad]
  float* out;
  bool transpose;
};
hipError_t launch_routed_contract(const RoutedContract& p, hipStream_t s);

}  // namespace lora
