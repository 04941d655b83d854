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
  float *stat_m, *stat_s;             // [blocks, T]: largest logit of a block of columns, and the sum of exp(l - it)
  float *tlogit;                      // [T]
  float *wlse, *rest;                 // [T]: lse, and 1 - p[target]
  uint16_t* share; int64_t piece;     // [T, piece]: a piece's shares p, without the targets'
  float* acc;                         // [S, T, K]
};

// Columns of the vocabulary per piece: the shares of a piece take at most 1 GiB, and a piece's sums are added to fp32
// accumulators in memory (T K 8 bytes per piece, which a piece of 8192 columns outweighs eight times over in its products).
inline int64_t loss_piece(int64_t T, int64_t V) {
  int64_t p = (int64_t(1) << 29) / (T > 0 ? T : 1) / 256 * 256;
  p = p < 4096 ? 4096 : (p > 524288 ? 524288 : p);  // (its row stride stays below 4 MB)
  const int64_t all = (V + 255) / 256 * 256;
  return p < all ? p : all;
}
// Blocks of columns for which statistics are kept: 64 at a time with the smaller tile, 128 with the larger.
inline int64_t loss_blocks(int64_t V) { return (V + 127) / 128 * 2; }
inline void loss_splits(int64_t T, int64_t K, int64_t stages, int* S, int* ks) {
  const int64_t tiles = (T + 127) / 128 * ((K + 127) / 128);
  int64_t s = tiles > 0 ? 512 / tiles : 1;
  const int64_t smax = stages / 8 > 1 ? stages / 8 : 1;
  s = s < 1 ? 1 : (s > 16 ? 16 : s);
  s = s > smax ? smax : s;
  *ks = static_cast<int>((stages + s - 1) / s);
  if (*ks < 1) *ks = 1;
  *S = static_cast<int>((stages + *ks - 1) / *ks);
}
inline size_t loss_acc_bytes(int64_t T, int64_t K, int64_t piece) {
  int S, ks;
  loss_splits(T, K, (piece + 63) / 64, &S, &ks);
  return static_cast<size_t>(S) * static_cast<size_t>(T) * static_cast<size_t>(K) * 4;
}
hipError_t launch_vocab_loss(const VocabLoss& p, hipStream_t s);

}  // namespace lora
