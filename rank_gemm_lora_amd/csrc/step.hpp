// Internal interface of the kernels of a fine-tuning step (step.hip: linear layers with dropout before the adapter and
// the gated feed-forward; loss.hip: the vocabulary loss) for the C-ABI host code (step_api.cpp).
#pragma once

#include "launch.hpp"

namespace lora {

// Dropout of an adapter's input. thr of 65536 outcomes drop an element; 0: none.
struct Drop {
  uint32_t thr;
  uint64_t seed, offset;
  const uint64_t* rng;  // device {seed, offset} in place of the two, or null
};

// A rank-wide product's row: R columns (the adapters side by side) as two bf16 terms, hi = RN(v) then mid = RN(v - hi),
// zeros up to a multiple of 64. (One term alone leaves 2^-9 of every rank's part in an output that is rounded once.)
inline int64_t pair_ld(int64_t R) { return (2 * R + 63) / 64 * 64; }

// ---------------------------------------------------------------- rank-wide products
// tt[t] = scale . x[t] . A^T (x masked by drop when given) for up to two adapters side by side, or with `nn`
// scale . x[t] . B for B [K, rank] (the gradient's side: one adapter).
struct RankProduct {
  const uint16_t* x; int64_t ldx;
  const uint16_t* A[2];   // [rank, K], or nn: [K, rank]
  int rank[2];            // rank[1] 0: one adapter
  float scale[2];
  int64_t T, K;
  Drop drop;
  float* part;            // [S, T, R]
  uint16_t* tt;           // [T, pair_ld(R)]
};
// Few tokens and ranks, and a K of up to 16 steps of 32 for each of 16 waves: the product in one launch, without partial sums
// in memory, every 16 tokens reading all of A. Up to 65536 elements of the result and 4096 tokens. Whole dropout steps, this
// against the ring and its finishing launch, rank 16: 333 tokens 1536 -> 1536 59 against 66 us, 2500 tokens 75 against 82,
// 4000 tokens 4096 -> 4096 279 against 285 (1500 tokens 8192 -> 1536: 164 against 159); rank 64: 600 tokens 8192 -> 8192 341
// against 344, 2000 tokens 1536 -> 1536 95 against 87, 4000 130 against 120. With 8960 inputs the ring is as fast.
constexpr int64_t kRankFewT = 4096, kRankFewK = 8192, kRankFewElements = 65536;
constexpr int64_t kRankFewR = 64;  // columns of one workgroup
inline bool rank_few(int64_t T, int64_t K, int64_t R) {
  return T <= kRankFewT && K <= kRankFewK && R <= kRankFewR && T * R <= kRankFewElements;
}
// Splits of K, fixed by the sizes: as few rounds of workgroups of 128 tokens, two on each of 256 compute units, as make
// the least stages of 64 one after the other (3 more for each round's start); a split's sums cost a write and a read.
// (18871 tokens, 8960 inputs, masked: 94 us; 3 splits, 444 workgroups one to a unit in two rounds, took 116.)
constexpr int kRankMaxSplits = 16;
inline void rank_plan(int64_t T, int64_t K, int64_t tasks, int* S, int* ks) {
  const int64_t mt = (T + 127) / 128 * tasks, nk = (K + 63) / 64;
  int64_t least = 0;
  *S = 1;
  *ks = static_cast<int>(nk);
  for (int64_t s = 1; s <= kRankMaxSplits; ++s) {
    const int64_t k = (nk + s - 1) / s;
    if (s > 1 && (k < 3 || (nk + k - 1) / k != s)) continue;
    const int64_t est = (mt * s + 511) / 512 * (k + 3);
    if (least == 0 || est < least) {
      least = est;
      *S = static_cast<int>(s);
      *ks = static_cast<int>(k);
    }
  }
}
inline int64_t rank_tasks(int64_t R, bool nn) { return nn ? (R + 127) / 128 : R <= 64 ? 1 : 2 * ((R + 127) / 128); }
inline size_t rank_part_bytes(int64_t T, int64_t K, int64_t R, bool nn) {
  int S, ks;
  rank_plan(T, K, rank_tasks(R, nn), &S, &ks);
  return static_cast<size_t>(S) * static_cast<size_t>(T) * static_cast<size_t>(R) * 4;
}
// Either or both (null: not there), of the same tokens; each with partial sums of its own.
hipError_t launch_rank_products(const RankProduct* nt, const RankProduct* nn, hipStream_t s);

// ---------------------------------------------------------------- ring GEMMs
// y [T, N] = sum over segments of x_i . W_i (NT: W [N, K], NN: W [K, N]) + tt . [E; E] (tt as above; NT: E_i [N, rank_i],
// NN: E_i [rank_i, N]) + bias. With `drop` (NN) the extension's part is masked as the [T, N] tensor it is a gradient of.
struct RingArgs {
  const uint16_t* x[2]; int64_t ldx;
  const uint16_t* W[2];
  int64_t K[2]; int n_seg;
  const uint16_t* tt; int64_t ldt;
  const uint16_t* E[2]; int re[2];
  const uint16_t* bias[2];
  int64_t T, N;
  uint16_t* y; int64_t ldy;
  Drop drop;
  int terms;      // kTerms: the x_i have second terms (below); tt has zeros there
  float* part;    // partial sums of the split tiles
  int full, S, ks;  // RingPlan
  float* saved;   // gated: where the forward leaves g and u, or null
  int act;
};
inline int64_t ring_stages(const RingArgs& p) {
  int64_t n = p.tt != nullptr ? p.ldt / 64 : 0;
  for (int i = 0; i < p.n_seg; ++i) n += (p.K[i] + 63) / 64;
  return n;
}
// How a layer's tiles are run: 256 x 256 tiles, one on a compute unit, or 128 x 128, two; the tiles of the last round,
// which would leave units idle, each cut along the contraction into S parts of ks stages whose fp32 sums a second launch
// joins. Chosen by an estimate of the time in microseconds (256 units; measured on MI355X: a stage of 64 indices takes a
// 256 x 256 tile 1.7, two 128 x 128 tiles side by side 1.0; filling the ring and the epilogue take 8 and 5; the second
// launch 6, and a sum is written and read at 4 TB/s). 4352 tokens, dx of 4096 -> 14336 in two segments: 272 tiles are one
// round and 16 tiles; whole, 1222 us (in 128 x 128 tiles); the 16 cut into 15 parts each, 901 and 15 for the joining.
struct RingPlan {
  bool big;
  int64_t tiles;
  int64_t full;  // tiles that are run whole; the others in S parts
  int S, ks;
};
constexpr int kRingUnits = 256, kRingMaxSplits = 16, kRingMinStages = 4;
inline RingPlan ring_plan(int64_t T, int64_t N, int64_t stages) {
  RingPlan best = {false, 0, 0, 1, static_cast<int>(stages > 0 ? stages : 1)};
  double least = 0.0;
  for (int big = 0; big < 2; ++big) {
    const int64_t bm = big ? 256 : 128, slots = big ? kRingUnits : 2 * kRingUnits;
    const int64_t tiles = (T + bm - 1) / bm * ((N + bm - 1) / bm);
    const double stage = big ? 1.7 : 1.0, ends = big ? 8.0 : 5.0;
    for (int s = 1; s <= kRingMaxSplits; ++s) {
      const int64_t ks = (stages + s - 1) / s;
      if (s > 1 && (ks < kRingMinStages || (stages + ks - 1) / ks != s)) continue;
      const int64_t full = s > 1 ? tiles / slots * slots : tiles, rem = tiles - full;
      if (s > 1 && rem == 0) continue;
      const double whole = static_cast<double>((full + slots - 1) / slots) * (static_cast<double>(stages) * stage + ends);
      const double tail = rem > 0 ? static_cast<double>((rem * s + slots - 1) / slots) * (static_cast<double>(ks) * stage + ends) +
                                        6.0 + static_cast<double>(rem * s * bm * bm) * 8.0 / 4e6
                                  : 0.0;
      if (best.tiles == 0 || whole + tail < least) {
        least = whole + tail;
        best = RingPlan{big != 0, tiles, full, s, static_cast<int>(ks)};
      }
    }
  }
  return best;
}
// x of two bf16 terms, for up to 64 tokens: the second terms are 64 rows behind the first and pass as tokens of their own in
// the same 128-token tile; the joining launch adds the two. (The gated gradients are rounded to bf16 for dx and dB, which
// brings those 1.4 times the error of their own rounding alone; over few values the ratio strays from that, and for few
// tokens the second term costs nothing.)
constexpr int kTerms = 64;
inline int64_t term_rows(int64_t T) { return T <= kTerms ? kTerms + T : T; }
inline RingPlan terms_plan(int64_t N, int64_t stages) {  // every tile in parts, two workgroups a unit
  const int64_t tiles = (N + 127) / 128;
  int64_t s = 2 * kRingUnits / tiles;
  s = s > kRingMaxSplits ? kRingMaxSplits : s;
  s = s > stages / kRingMinStages ? stages / kRingMinStages : s;
  s = s < 1 ? 1 : s;
  const int64_t ks = (stages + s - 1) / s;
  return RingPlan{false, tiles, 0, static_cast<int>((stages + ks - 1) / ks), static_cast<int>(ks)};
}
inline size_t terms_part_bytes(int64_t N, int64_t stages) {
  const RingPlan p = terms_plan(N, stages);
  return static_cast<size_t>(p.tiles * p.S) * 128 * 128 * 4;
}
inline size_t ring_part_bytes(int64_t T, int64_t N, int64_t stages) {
  const RingPlan p = ring_plan(T, N, stages);
  const int64_t bm = p.big ? 256 : 128;
  return p.S > 1 ? static_cast<size_t>((p.tiles - p.full) * p.S) * static_cast<size_t>(bm * bm) * 4 : 0;
}
hipError_t launch_ring(const RingArgs& p, bool nn, hipStream_t s);  // (p.part: ring_part_bytes(T, N, ring_stages))
// h = act(g) . u: W[0], E[0], bias[0] the gate's, [1] the up projection's; N columns of each; one segment.
// (p.part: ring_part_bytes(T, 2 N, ring_stages))
hipError_t launch_gated(const RingArgs& p, hipStream_t s);

// The same for few tokens: x against both weights and both adapters' A in one launch, each product whole or its
// contraction in S parts, fp32 sums to memory; the second launch adds the adapters and the activation. Reading the weights
// is the whole cost, and the products of A pass beside it, where the other way has them before it.
struct GatedFew {
  const uint16_t* x; int64_t ldx;
  const uint16_t *W[2], *A[2], *B[2], *bias[2];
  int rank[2];
  float scale[2];
  int64_t T, K, F;
  uint16_t* h; int64_t ldh;
  int act;
  float* part;     // [S, T, few_ld]
  int S, ks;
};
// Up to 64 tokens, and up to 128 (one tile) where the weights are long: whole calls, this against the other way, 4096 ->
// 14336: 1 token 66 against 86 us, 64 tokens 72 against 88, 65 71 against 88, 128 79 against 90; 1536 -> 8960: 1 token 21
// against 28, 64 tokens 26 against 30, 65 27 against 29, 100 32 against 30. (Long: between these two layers, of 2^23.7 and
// 2^25.8 elements; the crossing itself was not located.)
constexpr int64_t kGatedFewT = 64, kGatedFewLongT = 128, kGatedFewLong = int64_t(1) << 25;
inline bool gated_few(int64_t T, int64_t K, int64_t F) {
  return T <= kGatedFewT || (T <= kGatedFewLongT && K * F >= kGatedFewLong);
}
inline int64_t few_cols(int64_t F) { return (F + 3) / 4 * 4; }
inline int64_t few_ld(int64_t F, int64_t R) { return 2 * few_cols(F) + R; }
// Parts of the contraction: the weights at 5.2 TB/s, or a workgroup's stages one after the other (0.45 us each and 4 for
// the ring's start), whichever takes longer, and the sums written and read. (One token, 1536 -> 8960: 17.7 us whole, 140
// workgroups with a long way each, against 13.7. 48 tokens, 4096 -> 14336, were 68 us in 1 to 4 parts alike.)
inline void few_plan(int64_t T, int64_t K, int64_t F, int64_t R, int* S, int* ks) {
  const int64_t nk = (K + 63) / 64;
  const double read = 4.0 * static_cast<double>(F) * static_cast<double>(K) / 5.2e6;
  double least = 0.0;
  *S = 1;
  *ks = static_cast<int>(nk);
  for (int64_t s = 1; s <= 16; ++s) {
    const int64_t k = (nk + s - 1) / s;
    if (s > 1 && (k < 3 || (nk + k - 1) / k != s)) continue;
    const double chain = static_cast<double>(k) * 0.45 + 4.0;
    const double est = (read > chain ? read : chain) + static_cast<double>(s * T * few_ld(F, R)) * 8.0 / 4e6;
    if (least == 0.0 || est < least) {
      least = est;
      *S = static_cast<int>(s);
      *ks = static_cast<int>(k);
    }
  }
}
inline size_t few_part_bytes(int64_t T, int64_t K, int64_t F, int64_t R) {
  int S, ks;
  few_plan(T, K, F, R, &S, &ks);
  return static_cast<size_t>(S) * static_cast<size_t>(T) * static_cast<size_t>(few_ld(F, R)) * 4;
}
hipError_t launch_gated_few(const GatedFew& p, hipStream_t s);

// g and u as the forward keeps them: fp32, in blocks of 16 tokens x 16 columns as the MFMA leaves them (block (a, b):
// 256 values of g, then 256 of u; lane l = 16 q + r holds token r, columns 4 q .. + 3).
inline int64_t gated_blocks(int64_t n) { return (n + 15) / 16; }
inline size_t gated_saved_bytes(int64_t T, int64_t F) {
  return static_cast<size_t>(gated_blocks(T)) * static_cast<size_t>(gated_blocks(F)) * 512 * 4;
}
// dg = dh . u . act'(g) and du = dh . act(g), bf16 [T, F] each (up to 64 tokens two terms of each: [term_rows, F]), and with
// v (whose x is not used) the rank-wide product of them, dg . B_gate beside du . B_up, formed from the values as they pass
// before that rounding, in S parts of `per` runs of 64 columns. (From the rounded values the gradients of A had 1.5 times
// the error of their own rounding.) Workgroups of 64 tokens, four to each of 256 units where F and 32 parts allow it.
inline int64_t grad_blocks(int64_t R0, int64_t R1) { return (R0 + 15) / 16 + (R1 + 15) / 16; }
inline void grad_plan(int64_t T, int64_t F, int* S, int* per) {
  const int64_t mt = (T + 63) / 64, runs = (F + 63) / 64;
  int64_t s = (1024 + mt - 1) / mt;
  s = s > 32 ? 32 : s;
  s = s > runs ? runs : s;
  *per = static_cast<int>((runs + s - 1) / s);
  *S = static_cast<int>((runs + *per - 1) / *per);
}
inline size_t grad_part_bytes(int64_t T, int64_t F, int64_t R) {
  int S, per;
  grad_plan(T, F, &S, &per);
  return static_cast<size_t>(S) * static_cast<size_t>(T) * static_cast<size_t>(R) * 4;
}
hipError_t launch_gated_grad(const float* saved, const uint16_t* dh, int64_t lddh, int64_t T, int64_t F, int act,
                             uint16_t* dg, uint16_t* du, const RankProduct* v, hipStream_t s);

// ---------------------------------------------------------------- token contractions
// out_i [J, M] (transposed: one adapter's rows behind the other's) or [M, J] = P^T . Q over the tokens, Q the columns
// q_col .. of a rank-wide product's rows (both terms). P masked by drop when given.
struct ContractTask {
  const uint16_t* P; int64_t ldp, M;
  const uint16_t* tt; int64_t ldt;
  int R;            // where the second term's columns begin
  int q_col, J;
  bool transposed, masked;
  void* out[2];     // transposed: rows [0, split) and [split, J); else out[0]
  int split;
  int terms;        // kTerms: P has second terms that many rows behind the first
};
constexpr int kMaxContract = 3;
struct Contract {
  ContractTask task[kMaxContract]; int n_tasks;
  int64_t T;
  Drop drop;        // of the masked tasks' P
  bool out_bf16;
  int halves;       // 2: some task has second terms (the others have none of its half of the parts)
  float* part;      // [task][halves S, M, J]
};
constexpr int kCtI = 256, kCtJ = 64, kCtT = 32;
inline int64_t contract_tiles(int64_t M, int64_t J) { return (M + kCtI - 1) / kCtI * ((J + kCtJ - 1) / kCtJ); }
// Token chunks: as rank_plan, tiles of 256 x 64 two to a compute unit, at most 64 chunks of whole stages of 32 tokens.
inline void contract_plan(int64_t T, int64_t tiles, int* S, int64_t* chunk) {
  const int64_t nst = (T + kCtT - 1) / kCtT;
  int64_t least = 0;
  *S = 1;
  *chunk = (nst > 0 ? nst : 1) * kCtT;
  for (int64_t s = 1; s <= 64 && s <= nst; ++s) {
    const int64_t k = (nst + s - 1) / s;
    if ((nst + k - 1) / k != s) continue;
    // (a chunk's sums, 64 KB, cost about as much as four stages' reads)
    const int64_t est = (tiles * s + 511) / 512 * (k + 7);
    if (least == 0 || est < least) {
      least = est;
      *S = static_cast<int>(s);
      *chunk = k * kCtT;
    }
  }
}
inline size_t contract_part_bytes(int64_t T, int64_t tiles, int64_t elements) {  // elements: M J of all tasks
  int S;
  int64_t c;
  contract_plan(T, tiles, &S, &c);
  return static_cast<size_t>(S) * static_cast<size_t>(elements) * 4;
}
hipError_t launch_contract(const Contract& p, hipStream_t s);

}  // namespace lora
