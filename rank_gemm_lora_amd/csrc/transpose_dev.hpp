// Device transpose through LDS (backward.hip, routed.hip).
#pragma once

#include "common.hpp"

namespace lora {

// dst[c][r] = src[r][c] of one 64 x 64 tile by 256 threads (tid), with 16-byte accesses: a thread reads one 8-element piece of a source row
// (8 threads per 64-element tile row, 32 rows per pass) and writes one 8-element piece of a
// destination row, gathered from 8 rows of the tile in LDS (rows padded to 72 elements so that
// 16-byte stores of consecutive rows stay aligned). Needs C, ld and Rpad multiples of 8 and
// 16-byte aligned src and dst. Measured on MI355X: B^T of 8960 x 64 2.6 against 5.3 us, W^T of
// 8960 x 1536 11.6 against 18.7 us; the same bytes.
__device__ __forceinline__ void transpose_tile16(const bf16_bits* __restrict__ src, int64_t lds_, int64_t R, int64_t C,
                                                 bf16_bits* __restrict__ dst, int64_t Rpad, int64_t Cpad, int64_t r0,
                                                 int64_t c0, bf16_bits (&tile)[64][72], int tid) {
  const int pc = tid & 7, rr = tid >> 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = rr + 32 * h;
    const int64_t r = r0 + i, c = c0 + pc * 8;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (r < R && c < C) v = *reinterpret_cast<const u32x4*>(src + r * lds_ + c);
    *reinterpret_cast<u32x4*>(&tile[i][pc * 8]) = v;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = rr + 32 * h;  // destination row c0 + j, elements r0 + 8 pc .. + 7
    const int64_t c = c0 + j, r = r0 + pc * 8;
    if (c < Cpad && r < Rpad) {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = static_cast<uint32_t>(tile[pc * 8 + 2 * e][j]) |
               (static_cast<uint32_t>(tile[pc * 8 + 2 * e + 1][j]) << 16);
      *reinterpret_cast<u32x4*>(dst + c * Rpad + r) = o;
    }
  }
}

}  // namespace lora
