// Internal interface of the vocabulary loss (loss.hip) for the C-ABI host code (step_api.cpp).
#pragma once

#include "step.hpp"

namespace lora {

struct VocabLoss {
  const uint16_t* h; int64_t ldh;     // [T, K]
  const uint16_t* W;                  // [V, K]
  const int64_t* target;              // [T]
  const float* dloss;                 // [T] or null (1)
  int64_t T, K, V;
  float *loss, *lse;                  // [T], each may be null
  uint16_t* dh; int64_t lddh;         // [T, K], or null: the loss alone
  float *ref, *sum;                   // [blocks, T]: a block of columns' power of two c, and its sum of 2^(l log2 e - c)
  float *tlogit;                      // [T]
  float *top;                         // [T]: the largest c so far (the sums over shares are relative to 2^top)
  float *fade;                        // [T]: 2^(top before the piece - top now)
  float *rest, *scale;                // [T]: 1 - p[target], and 2^top / sum of all exponentials
  uint16_t* share; int64_t piece;     // [T, piece]: a piece's 2^(l log2 e - c of their block), without the targets'
  uint8_t* shift;                     // [blocks of a piece, shift_ld]: top - c, where dh_kernel's lanes find it
  float* part;                        // parts of dh's tiles
};

// Columns of the vocabulary per piece: the shares of a piece take at most 1 GiB, and the sums over a piece are added to
// those before it in memory (T K 8 bytes per piece, which a piece of 8192 columns outweighs eight times over in its
// products).
inline int64_t loss_piece(int64_t T, int64_t V) {
  int64_t p = (int64_t(1) << 29) / (T > 0 ? T : 1) / 256 * 256;
  p = p < 4096 ? 4096 : (p > 524288 ? 524288 : p);  // (its row stride stays below 4 MB)
  const int64_t all = (V + 255) / 256 * 256;
  return p < all ? p : all;
}
// Blocks of columns for which a power of two and a sum are kept: 64 at a time with the smaller tile, 128 with the larger.
inline int64_t loss_blocks(int64_t V) { return (V + 127) / 128 * 2; }
inline int64_t shift_ld(int64_t T) { return (T + 255) / 256 * 256; }
// The tiles of dh: as a layer's where one piece holds the vocabulary, else each in parts that later pieces are added to.
inline RingPlan loss_plan(int64_t T, int64_t K, int64_t V) {
  const int64_t piece = loss_piece(T, V);
  RingPlan p = ring_plan(T, K, ((V < piece ? V : piece) + 63) / 64);
  if (V > piece) p.full = 0;
  return p;
}
inline size_t loss_part_bytes(int64_t T, int64_t K, int64_t V) {
  const RingPlan p = loss_plan(T, K, V);
  const int64_t bm = p.big ? 256 : 128;
  return static_cast<size_t>((p.tiles - p.full) * p.S) * static_cast<size_t>(bm * bm) * 4;
}
hipError_t launch_vocab_loss(const VocabLoss& p, hipStream_t s);

}  // namespace lora
