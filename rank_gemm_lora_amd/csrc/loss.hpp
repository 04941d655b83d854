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

// Columns of the vocabulary per piece: as few pieces of equal width as keep the shares of one at 1 GiB (above 131072 tokens
// at 8192 bytes a token: 4096 columns). From the second piece on, the sums of every tile of dh pass through memory once
// each way per piece (T K 8 bytes and those of the cut tiles), which a piece of 4096 columns outweighs six times over in
// its products.
inline int64_t loss_piece(int64_t T, int64_t V) {
  int64_t most = (int64_t(1) << 29) / (T > 0 ? T : 1) / 256 * 256;
  most = most < 4096 ? 4096 : (most > 524288 ? 524288 : most);  // (its row stride stays below 4 MB)
  const int64_t n = (V + most - 1) / most;
  return ((V + n - 1) / n + 255) / 256 * 256;
}
// Blocks of columns for which a power of two and a sum are kept: 64 at a time with the smaller tile, 128 with the larger.
inline int64_t loss_blocks(int64_t V) { return (V + 127) / 128 * 2; }
inline int64_t shift_ld(int64_t T) { return (T + 255) / 256 * 256; }
// The tiles of dh: as a layer's of a piece's stages. Where there are several pieces the whole tiles have sums in memory too,
// one part each behind the parts of the cut ones.
inline RingPlan loss_plan(int64_t T, int64_t K, int64_t V) {
  const int64_t piece = loss_piece(T, V);
  return ring_plan(T, K, ((V < piece ? V : piece) + 63) / 64);
}
inline size_t loss_part_bytes(int64_t T, int64_t K, int64_t V) {
  const RingPlan p = loss_plan(T, K, V);
  const int64_t bm = p.big ? 256 : 128, whole = V > loss_piece(T, V) ? p.full : 0;
  return static_cast<size_t>((p.tiles - p.full) * p.S + whole) * static_cast<size_t>(bm * bm) * 4;
}
hipError_t launch_vocab_loss(const VocabLoss& p, hipStream_t s);

}  // namespace lora
