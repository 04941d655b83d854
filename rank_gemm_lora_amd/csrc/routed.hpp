// Internal interface of the routed kernels (routed.hip): a linear layer whose tokens take their
// adapters from a pool.
#pragma once

#include "launch.hpp"

namespace lora {

// Rank-wide producer: t = s_t . x[t] A_a^T of every token's own adapter a, as hi = RN_bf16(t), mid =
// RN_bf16(t - hi) and, with three terms, the rest of its 24 bits in lo. The layer's second product takes two
// terms (hi alone left 2^-8 of every rank's part in an output that two terms round once; as the base product's
// operands they are multiplied exactly), the gradients' contractions three. Writes eid and blk (RoutedGemm) too.
// With many tokens (splits > 0) a block of 128 tokens with up to kRingAdapters is multiplied by a ring of
// LDS stages, once per adapter, K in `splits` parts of ks stages of 64; the other blocks, and all blocks of
// fewer tokens, 16 tokens at a time straight from memory.
// (9000 tokens that take 6 adapters in turn, 8960 -> 1536, rank 64: 367 us with all of a block's adapters in the ring,
// 926 with blocks of more than four left to the 16-token form; 16 instead of 8 costs the launches of others 1%)
constexpr int kRingAdapters = 8;
struct RoutedDown {
  const uint16_t* x; int64_t ldx;
  int64_t T, K;
  const uint16_t* A;   // [n_adapters, rank, K]
  Routing rt;
  uint16_t* hi;        // [T, ldt]; the row of a token with an adapter is written whole (zeros behind the
  uint16_t *mid, *lo;  // adapter's rank), another token's not at all
  int terms;           // 2: hi and mid, 3: lo too
  int64_t ldt;         // rank_pad(rank)
  int32_t* eid;        // [T]
  int32_t* blk;        // [ceil(T / 16)]
  int splits, ks;      // of the ring (0: not used)
  int parts;           // without the ring: workgroups that share K (1: none)
  int32_t* ring;       // [ceil(T / 128)]: adapters of the block's tokens, -1: more than kRingAdapters
  float* tpart;        // splits > 1, parts > 1: partial sums [splits or parts, T, ldt]
  int32_t* order;      // not null (sorts_tokens(T)): the tokens sorted by adapter go there, [2, T]: the token of
                       // each place, then its adapter; in token order within one adapter, those without an
                       // adapter last. The blocks of 16 are of this order
};
// Few tokens: t~ (as hi and mid) and the base product over a ring of LDS stages in one launch, then the sum.
// Above it the hot GEMM: with every token on one adapter it would be a little faster from somewhere between 192 and
// 256 tokens on (4096 -> 14336, rank 16: 66 against 59 us, 67 against 71), with mixed ones it is slower there and
// beyond (256 tokens: of 8 adapters 81 against 72 us, of 64 136 against 86).
constexpr int64_t kFewMaxT = 256;
// (one block of 16 is as good in any order)
inline bool sorts_tokens(int64_t T) { return T > kRouteBlock && T <= kFewMaxT; }
constexpr int kRingBlock = 128;
constexpr int64_t kRingMinT = 1025;
inline int64_t ring_blocks(int64_t T) { return T >= kRingMinT ? (T + kRingBlock - 1) / kRingBlock : 0; }
// The ring's split of K, from T and K alone: the time goes as the rounds of 256 workgroups over the splits (a
// compute unit holds two, and a block makes about two, one for each of its adapters; rounds of 512 measured 40
// against 36 us for 4977 tokens, K 8960); each split adds its partial sums (taken as 4%). At least 4 stages a
// split.
inline void ring_plan(int64_t T, int64_t K, int* splits, int* ks) {
  *splits = *ks = 0;
  if (T < kRingMinT) return;
  const int64_t mt = ring_blocks(T), nk = (K * 2 + 127) / 128;
  double best = 0;
  for (int s = 1; s <= kMaxProducerSplits && (s == 1 || nk / s >= 4); ++s) {
    const double cost = static_cast<double>((mt * s + 255) / 256) / s * (1 + 0.04 * (s - 1));
    if (s > 1 && cost >= best) continue;
    best = cost;
    *ks = static_cast<int>((nk + s - 1) / s);
    *splits = static_cast<int>((nk + *ks - 1) / *ks);
  }
}
inline size_t ring_bytes(int64_t T, int64_t K, int64_t ldt) {
  int S, ks;
  ring_plan(T, K, &S, &ks);
  return S > 1 ? static_cast<size_t>(S) * static_cast<size_t>(T) * static_cast<size_t>(ldt) * 4 : 0;
}
// Workgroups that share the adapters of a block of 16 tokens: as many as it can hold, in sorted blocks (which
// hold about as many adapters together as there are blocks and adapters) one more than `times` their mean.
inline int down_slots(int64_t T, int n_adapters, bool sorted, int times) {
  const int64_t m = T < kRouteBlock ? T : kRouteBlock, blocks = (T + kRouteBlock - 1) / kRouteBlock;
  const int64_t n = n_adapters < m ? (n_adapters > 0 ? n_adapters : 1) : m;
  const int64_t mean = times * ((n_adapters + blocks - 1) / blocks) + 1;
  return static_cast<int>(sorted && mean < n ? mean : n);
}
// Parts of K of the producer without the ring: the fewest estimated microseconds. A wave has 256 k (128 above
// 32 ranks) in flight, each such round about 1.5 us; joining parts takes a launch of 3.5 us; more than 256
// workgroups do not help (sorted blocks hold about as many adapters as there are blocks and adapters).
inline int down_parts(int64_t T, int64_t K, int64_t rank, int n_adapters) {
  if (T >= kRingMinT) return 1;
  const int64_t blocks = (T + kRouteBlock - 1) / kRouteBlock, slots = down_slots(T, n_adapters, sorts_tokens(T), 1);
  const int64_t units = blocks * slots < blocks + n_adapters ? blocks * slots : blocks + n_adapters;
  const int64_t wgs = units * ((rank + 63) / 64), round = 8 * (rank > 32 ? 128 : 256);
  int best = 1;
  double cost = 1.5 * static_cast<double>((K + round - 1) / round);
  for (int s = 2; s <= 8 && s * wgs <= 256; ++s) {
    const double c = 1.5 * static_cast<double>((K + s * round - 1) / (s * round)) + 3.5;
    if (c < cost) best = s, cost = c;
  }
  return best;
}
// Of K inputs beside a base product of K0 inputs and N outputs: one part if its time passes there, else the fewest
// estimated microseconds. Beside the weight's stream and with fewer loads in flight (256 k up to 16 ranks, 128 up
// to 32, else 64) a round is about 4 us up to 16 ranks, 2.5 above; the launch that joins parts 5.
// (256 tokens, 8960 -> 1536, rank 64: 95 us in one part, 42 in five.)
inline int down_parts_beside(int64_t K, int64_t K0, int64_t N, int64_t rank) {
  const int64_t round = 8 * (rank > 32 ? 64 : (rank > 16 ? 128 : 256));
  const double each = rank > 16 ? 2.5 : 4.0, base = 4 + static_cast<double>(K0 * N * 2) / 3.5e6;
  int best = 1;
  double cost = 0;
  for (int s = 1; s <= 8; ++s) {
    const double over = each * static_cast<double>((K + s * round - 1) / (s * round)) - base;
    const double c = (over < 0 ? 0 : over) + (s > 1 ? 5 : 0);
    if (s == 1 || c < cost) best = s, cost = c;
  }
  return best;
}
inline size_t part_bytes(int parts, int64_t T, int64_t rank) {
  return parts > 1 ? static_cast<size_t>(parts) * static_cast<size_t>(T) * static_cast<size_t>(rank_pad(rank)) * 4 : 0;
}
// One product, or two of the same tokens and routing (x against A, dy against B^T) in the same launches. z0:
// the first's share of the grid's z; slots: workgroups that share a block's adapters without the ring.
struct RoutedDowns {
  RoutedDown d[2];
  int n, z0, slots;
};
hipError_t launch_routed_ring(RoutedDowns p, hipStream_t s);  // (gemm.hip)
hipError_t launch_routed_down(RoutedDowns p, hipStream_t s);

constexpr int kDownWaves = 8;
// From kFewMaxT up to 1024 tokens the few-token kernels still take outputs so narrow that the hot GEMM's 128 x 128
// tiles would leave half of the compute units without one (tokens as they come, not sorted).
inline bool few_path(int64_t T, int64_t N) {
  return T <= kFewMaxT || (T < kRingMinT && (T + 127) / 128 * ((N + 127) / 128) <= 128);
}
// Parts that one workgroup of the base product writes: halves of a stage's k up to 32 tokens.
constexpr int few_halves(int bm) { return bm < 64 ? 2 : 1; }
struct FewPlan {
  int bm;            // tokens of a tile
  int token_tiles;
  int64_t tiles;     // all tiles (64 outputs each)
  int splits, stages;  // parts of K, 64-k stages of each
  int parts;           // partial sums of an output
};
// Token tiles of 16, 32, 64 or 128; K in as many parts as bring two workgroups to each of 256 compute
// units, at least 4 stages each.
inline FewPlan few_plan(int64_t T, int64_t K, int64_t N) {
  FewPlan f;
  f.bm = T <= 16 ? 16 : (T <= 32 ? 32 : (T <= 64 ? 64 : 128));
  f.token_tiles = static_cast<int>((T + f.bm - 1) / f.bm);
  f.tiles = (N + 63) / 64 * f.token_tiles;
  const int64_t nk = (K + 63) / 64;
  int64_t s = 512 / f.tiles;
  s = s > 8 ? 8 : s;
  s = s > nk / 4 ? nk / 4 : s;
  s = s < 1 ? 1 : s;
  f.stages = static_cast<int>((nk + s - 1) / s);
  f.splits = static_cast<int>((nk + f.stages - 1) / f.stages);
  f.parts = f.splits * few_halves(f.bm);
  return f;
}
inline size_t few_part_bytes(const FewPlan& f, int64_t T) {
  return static_cast<size_t>(f.tiles / f.token_tiles) * f.parts * static_cast<size_t>(T) * 64 * 4;
}
struct RoutedFew {
  const uint16_t* x; int64_t ldx;
  const uint16_t* W;
  const uint16_t* bias;
  uint16_t* y; int64_t ldy;
  int64_t T, K, N;
  const uint16_t *hi, *mid; int64_t ldt;
  RoutedGemm rt;
  const int32_t* order;  // [2, T]: the producer's, null without one
  float* part;           // [ceil(N / 64), parts, T, 64]
};
hipError_t launch_routed_few(const RoutedFew& p, const RoutedDowns& downs, hipStream_t s);

// Tokens sorted by adapter (in token order within one), and the work items of a contraction over them: an
// adapter's tokens in ceil(count / chunk) items of nearly equal length (one, empty, without tokens), the
// items of all adapters one behind the other.
struct RouteItem {
  int32_t adapter, lo, hi;
  int32_t part;  // where its partial sums go: -1 straight to the gradient (the adapter's only item), else a slot
};
struct RouteTable {
  int32_t chunk;
  int32_t* first;      // [n_adapters + 1]: the first item of each adapter
  RouteItem* items;    // [n_items], the places behind the last item empty
  int64_t n_items;     // route_items(T, n_adapters, chunk)
};
struct RoutePlan {
  Routing rt; int64_t T;
  const int32_t* eid;  // the producer's, or null: the plan looks up the tokens' adapters itself
  int32_t n_adapters;  // 0: no plan
  int32_t* perm;       // [T]
  RouteTable table[2]; // one for each gradient: their widths ask for chunks of their own
};
constexpr int kRouteMaxChunk = 4096;  // positions of an item that a workgroup keeps in LDS
inline int64_t route_items(int64_t T, int64_t n, int64_t chunk) { return n + T / chunk + 1; }
// Slots of partial sums, counted over the items of adapters with more than one: k > 1 items hold more than
// (k - 1) chunk >= k chunk / 2 tokens, so there are at most 2 T / chunk.
inline int64_t route_parts(int64_t T, int64_t chunk) { return 2 * (T / chunk) + 1; }
// dst[i] [C, R] = src[i] [R, C] transposed for i < slots; contiguous, 16-byte aligned, R and C multiples of 8.
struct TransposeStack {
  const uint16_t* src;
  uint16_t* dst;
  int64_t R, C, slots;
};
constexpr int kTransposeStacks = 3;
// The plan from eid; or n <= kTransposeStacks stacks; or both in one launch, for which the plan does without eid:
// up to 1024 tokens (a load of each wave's): 333 tokens 7.8 us against 6.3 + 6.1 apart. With more its chains of
// look-ups are longer than the transposes (18871 tokens: 44 us against 20.5 + 12.8) and it follows the producer.
constexpr int64_t kPlanFirstT = 1024;
hipError_t launch_route_prepare(const RoutePlan& p, const TransposeStack* stacks, int n, hipStream_t s);

// Most tokens of an item for an output of `tiles` workgroups: about two
// workgroups for each of 256 compute units if the adapters were one, and items long enough that the partial
// sums of adapters with several stay few.
constexpr int kRtI = 256, kRtJ = 64, kRtT = 64;
inline int32_t route_chunk(int64_t T, int64_t tiles) {
  int64_t c = (T * tiles / 512 + kRtT - 1) / kRtT * kRtT;
  return static_cast<int32_t>(c < 512 ? 512 : (c > kRouteMaxChunk ? kRouteMaxChunk : c));
}

// out[a] = sum over a's tokens of P[t] (x) (hi + mid + lo)[t]: [M, rank] row-major, or [rank, M] with
// transpose. Adapters without tokens get zeros. One contraction, or two of the same pool in the same launches.
struct RoutedContract {
  const uint16_t* P; int64_t ldp, M;
  const uint16_t* q[3]; int64_t ldt;  // hi, mid, lo
  RouteTable table;
  float* part;         // [route_parts, M, rank]
  float* out;
  bool transpose;
};
struct RoutedContracts {
  RoutedContract c[2];
  int n, tiles0;       // tiles0: the first's share of the grid's x
  int32_t rank, n_adapters;
  const int32_t* ranks;  // of each adapter, or null
  const int32_t* perm;
};
hipError_t launch_routed_contract(RoutedContracts p, hipStream_t s);

}  // namespace lora
