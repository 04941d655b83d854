// Kernels of a fine-tuning step, bf16: the linear layer with dropout before its adapter, and the gated half of a
// feed-forward block whose two projections carry adapters, forward and backward, the base weights frozen.
//
//   dropout   t = s x' A^T, x' = x . keep                      rank_kernel (the mask formed on its x fragments)
//             y = x W^T + b + t B^T                            ring_kernel NT, t as extension stages
//             u = s dy B                                       rank_kernel
//             dx = dy W + keep . (u A)                         ring_kernel NN, the mask between extension and base stages
//             dA = u^T x', dB = dy^T t                         contract_kernel (the mask on the staged x)
//   gated     h = act(x Wg^T + bg + tg Bg^T) . (x Wu^T + bu + tu Bu^T)      gated_kernel: one GEMM, one rounding
//             dg = dh u act'(g), du = dh act(g)                gated_grad_kernel, from g and u as the forward kept them
//             v = s d B, dx = dg Wg + du Wu + vg Ag + vu Au, dA = v^T x, dB = d^T t        as above
//
// Rank-wide rows are two bf16 terms (step.hpp); every sum is fp32.
#include "common.hpp"
#include "dropout_dev.hpp"
#include "launch.hpp"
#include "ring_ops.hpp"
#include "step.hpp"

namespace lora {
namespace {
using namespace pipe;

// ---------------------------------------------------------------------------
// Rank-wide product over rows contiguous along the contraction (the forward's): 128 tokens and BN adapter rows per
// workgroup through the LDS ring of the one-adapter producer, K in splits; fp32 partial sums. HBM-bound: x is read once
// (R <= 128). Two workgroups on a compute unit, so that the generator's arithmetic in one (as long as the reads) does not
// keep the other's copies waiting. 18871 tokens, 8960 inputs, rank 64, masked: 94 us, x at 3.6 TB/s (one workgroup a unit:
// 116); 12288 tokens, 4096 inputs, two of rank 32, unmasked: 24 us, 4.2 TB/s.
using RankNarrow = PCfg<128, 64, 32, 64, 128, 3>;   // up to 64 columns
using RankWide = PCfg<128, 128, 32, 128, 128, 4>;

template <class P, bool DROP>
__device__ __forceinline__ void rank_nt(const RankProduct& p, int ks, int bx, int by, int bz, char* smem) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm0 = wave * P::WM;
  const int R = p.rank[0] + p.rank[1], q0 = by * P::BN;
  const int64_t m0 = static_cast<int64_t>(bx) * P::BM;
  const int rows_m = static_cast<int>(min<int64_t>(P::BM, p.T - m0));
  const int kb_total = static_cast<int>(p.K * 2), nk = (kb_total + P::RB - 1) / P::RB;
  const bool k_tail = kb_total % P::RB != 0;
  const uint32_t ldx_b = static_cast<uint32_t>(p.ldx * 2), lda_b = static_cast<uint32_t>(p.K * 2);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + m0 * p.ldx, static_cast<uint32_t>(rows_m) * ldx_b);
  const __amdgpu_buffer_rsrc_t ar0 = make_rsrc(p.A[0], static_cast<uint32_t>(p.rank[0]) * lda_b);
  const __amdgpu_buffer_rsrc_t ar1 = make_rsrc(p.A[1], static_cast<uint32_t>(p.rank[1]) * lda_b);
  TileOffsets<P, P::BM> ox;
  ox.init(ldx_b, 0, rows_m, 0);
  // adapter rows q0 .. : a copy instruction takes 8 of them, all of one adapter (ranks are multiples of 8)
  constexpr int NA = TileOffsets<P, P::BN>::N;
  uint32_t va[NA];
#pragma unroll
  for (int l = 0; l < NA; ++l) {
    const int row = (l * P::WAVES + wave) * 8 + (lane >> 3), g = q0 + row;
    const uint32_t c = static_cast<uint32_t>(((lane & 7) ^ ((row >> 1) & 7)) * 16);
    va[l] = g < R ? static_cast<uint32_t>(g < p.rank[0] ? g : g - p.rank[0]) * lda_b + c : 0x80000000u;
  }
  const int s_lo = bz * ks, ns = min(nk, s_lo + ks) - s_lo;
  auto issue = [&](int s) {
    char* bx = smem + (s % P::S) * P::STAGE_BYTES;
    const int kb = (s_lo + s) * P::RB;
    const bool tail = k_tail && s_lo + s == nk - 1;
    ox.load(bx, xr, kb, tail, kb_total);
#pragma unroll
    for (int l = 0; l < NA; ++l) {
      const int slot0 = (l * P::WAVES + wave) * 64;
      uint32_t v = va[l];
      if (tail) {
        const int row = (l * P::WAVES + wave) * 8 + (lane >> 3);
        if (kb + ((lane & 7) ^ ((row >> 1) & 7)) * 16 >= kb_total) v = 0x80000000u;
      }
      const bool second = q0 + (l * P::WAVES + wave) * 8 >= p.rank[0];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(second ? ar1 : ar0, (lds_void*)(bx + P::X_BYTES + slot0 * 16), 16, v, kb,
                                               0, 0);
    }
  };
  f32x16 acc[P::NI][P::NJ];
  if constexpr (DROP) {
    // lane (r, h) holds block 2 kk + h (of 8) of the stage of token wm0 + r: one call of the generator
    Dropper d;
    d.init(p.drop, p.K);
    const int64_t row0 = (m0 + wm0 + (lane & 31)) * d.blocks + s_lo * 8 + (lane >> 5);
    auto touch = [&](Frags<P>& f, int s, int kk) {
      const u32x4 w = philox7(static_cast<uint64_t>(row0 + s * 8 + kk * 2), d.seed, d.offset);
      u32x4 v = __builtin_bit_cast(u32x4, f.b[0]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] &= d.mask(w[e]);
      f.b[0] = __builtin_bit_cast(bf16x8, v);
    };
    static_assert(P::NJ == 1, "one token per lane");
    pipe_loop<P>(acc, smem, ns, issue, 0, wm0, lane, touch);
  } else {
    pipe_loop<P>(acc, smem, ns, issue, 0, wm0, lane);
  }
  // lane (r, h) holds adapter rows q0 + 32 i + 8 g + 4 h + e of token wm0 + r
  const int r = lane & 31, h = lane >> 5;
  const int64_t m = m0 + wm0 + r;
  if (m >= p.T) return;
  float* row = p.part + (static_cast<int64_t>(bz) * p.T + m) * R;
#pragma unroll
  for (int i = 0; i < P::NI; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int q = q0 + i * 32 + g * 8 + h * 4;
      if (q < R)
        *reinterpret_cast<f32x4*>(row + q) =
            f32x4{acc[i][0][g * 4], acc[i][0][g * 4 + 1], acc[i][0][g * 4 + 2], acc[i][0][g * 4 + 3]};
    }
}

// tt = the two terms of scale . sum of the splits, in order; zeros behind them. 4 columns per thread.
// (`terms`: rows of zeros that many behind.)
__device__ __forceinline__ void rank_finish(const RankProduct& p, int S, int64_t bx, int terms = 0) {
  const int R = p.rank[0] + p.rank[1], ldt = static_cast<int>((2 * R + 63) / 64 * 64), quads = ldt / 4;
  const int64_t idx = bx * 256 + threadIdx.x;
  if (idx >= p.T * quads) return;
  const int64_t t = idx / quads;
  const int c = static_cast<int>(idx - t * quads) * 4;
  uint2 w = {0u, 0u};
  if (c < 2 * R) {
    const bool mid = c >= R;
    const int q = mid ? c - R : c;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int z = 0; z < S; ++z) v += *reinterpret_cast<const f32x4*>(p.part + (z * p.T + t) * R + q);
    v *= q < p.rank[0] ? p.scale[0] : p.scale[1];
    w = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    if (mid) {
      // (a sum that overflows has its infinity in the first term: the second is zero there, not inf - inf)
      float lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t b = e < 2 ? w.x : w.y;
        const float hi = __uint_as_float(e & 1 ? b & 0xffff0000u : b << 16);
        lo[e] = __builtin_isfinite(hi) ? v[e] - hi : 0.f;
      }
      w = uint2{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3])};
    }
  }
  *reinterpret_cast<uint2*>(p.tt + t * ldt + c) = w;
  if (terms > 0) *reinterpret_cast<uint2*>(p.tt + (terms + t) * ldt + c) = uint2{0u, 0u};
}

__global__ __launch_bounds__(256) void rank_finish_kernel(RankProduct a, int Sa, int blocks, RankProduct b, int Sb) {
  if (static_cast<int>(blockIdx.x) < blocks) rank_finish(a, Sa, blockIdx.x);
  else rank_finish(b, Sb, blockIdx.x - blocks);
}

__global__ __launch_bounds__(256) void grad_rank_finish_kernel(RankProduct v, int S, int terms) {
  rank_finish(v, S, blockIdx.x, terms);
}

// Few tokens: 16 tokens by up to 64 columns per workgroup of 16 waves that share K, 32 indices at a time in turn, straight
// from memory three steps ahead (two at 64 columns: 128 registers a lane). Rows along the contraction (A) are loaded as
// the MFMA takes them; rows across it (B [K, rank]) go through a piece of LDS per wave and its transposing read. The
// waves' sums are added in order in LDS, and the two terms written. Bound by the way to memory, once or twice over.
constexpr int kFewWaves = 16;

template <bool NN, bool DROP, int NB>
__device__ __forceinline__ void rank_few_sum(f32x4 (&acc)[NB], const uint16_t* x, int64_t ldx, const uint16_t* const (&A)[2],
                                             const int (&rank)[2], int64_t K, int64_t T, const Dropper& d, int64_t m0,
                                             char* st) {
  const int lane = threadIdx.x & 63, wave = ring_wave(), r = lane & 15, q = lane >> 4;
  const int R = rank[0] + rank[1];
  const int rows_m = static_cast<int>(min<int64_t>(16, T - m0));
  const uint32_t ldx_b = static_cast<uint32_t>(ldx * 2);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(x + m0 * ldx, static_cast<uint32_t>(rows_m) * ldx_b);
  const int nst = static_cast<int>((K + 31) / 32);
  constexpr int D = NB == 4 ? 3 : 4;
  u32x4 xv[D], av[D][NB];
  // Lane's rows of A from its first index on. Columns that are not there read another's: no sum of theirs is used.
  const uint16_t* rows[NB];
  int64_t kin[NB];  // an index beyond K reads the last ones, and is zero below
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if constexpr (!NN) {
      const int g = min(i * 16 + r, R - 1);  // (one adapter's rows behind the other's)
      rows[i] = g < rank[0] ? A[0] + static_cast<int64_t>(g) * K : A[1] + static_cast<int64_t>(g - rank[0]) * K;
      kin[i] = 8 * q;
    } else {
      const int pc = i * 64 + lane;  // 32 rows of 16 NB columns, in pieces of 8
      rows[i] = A[0] + min(pc % (NB * 2) * 8, R - 8);
      kin[i] = pc / (NB * 2);
    }
  }
  auto load = [&](int b, int s) {
    const int64_t k = static_cast<int64_t>(s) * 32;
    xv[b] = __builtin_amdgcn_raw_buffer_load_b128(
        xr, k + 8 * q < K ? static_cast<uint32_t>(r) * ldx_b + static_cast<uint32_t>(k + 8 * q) * 2 : kMissing, 0, 0);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int64_t at = min(k + kin[i], NN ? K - 1 : K - 8);
      av[b][i] = *reinterpret_cast<const u32x4*>(rows[i] + (NN ? at * R : at));
    }
  };
  auto there = [&](const u32x4& v, int i, int64_t k) { return k + kin[i] < K ? v : u32x4{0u, 0u, 0u, 0u}; };
#pragma unroll
  for (int i = 0; i < NB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int b = 0; b < D - 1; ++b) load(b, b * kFewWaves + wave);
  for (int s0 = wave; s0 < nst; s0 += kFewWaves * D) {
#pragma unroll
    for (int b = 0; b < D; ++b) {
      const int s = s0 + b * kFewWaves;
      load((b + D - 1) % D, s + (D - 1) * kFewWaves);
      u32x4 xb = xv[b];
      if constexpr (DROP) {
        if (s < nst) xb &= d.masks(m0 + r, static_cast<int64_t>(s) * 4 + q);
      }
      const int64_t k = static_cast<int64_t>(s) * 32;
      bf16x8 af[NB];
      if constexpr (NN) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int pc = i * 64 + lane, per = NB * 2, row = pc / per, c = pc % per;
          // (granules of 16 columns; rows of NB granules)
          *reinterpret_cast<u32x4*>(st + row * NB * 32 + c * 16) = there(av[b][i], i, k);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const char* at = st + (8 * q + (r >> 2)) * NB * 32 + i * 32 + (r & 3) * 8;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * NB * 32));
          af[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
      } else {
#pragma unroll
        for (int i = 0; i < NB; ++i) af[i] = __builtin_bit_cast(bf16x8, there(av[b][i], i, k));
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], __builtin_bit_cast(bf16x8, xb), acc[i], 0, 0, 0);
    }
  }
}

// A product's sums, then the two terms in the rows of tt and zeros behind them.
template <bool NN, bool DROP, int NB>
__device__ __forceinline__ void rank_few(const RankProduct& p, int64_t m0, char* smem) {
  const int lane = threadIdx.x & 63, wave = ring_wave(), r = lane & 15, q = lane >> 4;
  const int R = p.rank[0] + p.rank[1];
  Dropper d;
  d.blocks = p.K / 8;
  if constexpr (DROP) d.init(p.drop, p.K);
  f32x4 acc[NB];
  rank_few_sum<NN, DROP, NB>(acc, p.x, p.ldx, p.A, p.rank, p.K, p.T, d, m0, smem + wave * NB * 1024);
  __syncthreads();  // (the waves' pieces become their sums)
  float* sums = reinterpret_cast<float*>(smem);  // [wave][16 NB columns][16 tokens]
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[(wave * NB * 16 + i * 16 + 4 * q + e) * 16 + r] = acc[i][e];
  __syncthreads();
  const int ldt = (2 * R + 63) / 64 * 64;
  for (int idx = threadIdx.x; idx < 16 * R; idx += kFewWaves * 64) {
    const int t = idx / R, c = idx - t * R;
    if (m0 + t >= p.T) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += sums[(w * NB * 16 + c) * 16 + t];
    v *= c < p.rank[0] ? p.scale[0] : p.scale[1];
    const uint16_t hi = f32_to_bf16_rne(v);
    const float h = bf16_to_f32(hi);
    uint16_t* row = p.tt + (m0 + t) * ldt + c;
    row[0] = hi;
    row[R] = __builtin_isfinite(h) ? f32_to_bf16_rne(v - h) : static_cast<uint16_t>(0);
  }
  const int z = ldt - 2 * R;
  for (int idx = threadIdx.x; idx < 16 * z; idx += kFewWaves * 64) {
    const int t = idx / z;
    if (m0 + t < p.T) p.tt[(m0 + t) * ldt + 2 * R + idx - t * z] = 0;
  }
}

template <bool NN, bool DROP>
__device__ __forceinline__ void rank_few_nb(const RankProduct& p, int64_t m0, char* smem) {
  const int R = p.rank[0] + p.rank[1];
  if (R <= 16) rank_few<NN, DROP, 1>(p, m0, smem);
  else if (R <= 32) rank_few<NN, DROP, 2>(p, m0, smem);
  else rank_few<NN, DROP, 4>(p, m0, smem);
}

// Grid (blocks of 16 tokens, products): a's (where it is there), then b's.
template <bool DROP>
__global__ __launch_bounds__(kFewWaves * 64) void rank_few_kernel(RankProduct a, int n_a, RankProduct b) {
  __shared__ __attribute__((aligned(1024))) char smem[kFewWaves * 4 * 1024];
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  if (static_cast<int>(blockIdx.y) < n_a) rank_few_nb<false, DROP>(a, m0, smem);
  else rank_few_nb<true, false>(b, m0, smem);
}

// (NJ: blocks of 16 tokens from m0 on)
template <class P, int NJ>
__device__ __forceinline__ void store_block(const f32x4 (&acc)[P::NI][NJ], const RingArgs& p, int64_t m0, int64_t n0,
                                            char* smem) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  BlockOut<NJ * 16, P::WN> out{smem + ring_wave() * NJ * 16 * P::WN * 2};
#pragma unroll
  for (int i = 0; i < P::NI; ++i) {
    float bv[4];
    load_bias4(bv, p.bias[0], n0 + i * 16 + q * 4, p.N);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      out.put(j * 16 + r, i * 16 + q * 4, pack_bf16x2(acc[i][j][0] + bv[0], acc[i][j][1] + bv[1]),
              pack_bf16x2(acc[i][j][2] + bv[2], acc[i][j][3] + bv[3]));
    __builtin_amdgcn_sched_barrier(0);
  }
  if (m0 < p.T && n0 < p.N)
    out.store(p.y + m0 * p.ldy + n0, p.ldy, static_cast<int>(min<int64_t>(NJ * 16, p.T - m0)),
              static_cast<int>(min<int64_t>(P::WN, p.N - n0)));
}

// acc = 0 where the element of the [T, N] tensor is dropped. A lane holds 4 columns, half of a call's 8: lanes of rows q
// and q ^ 1 make the calls of blocks i and i + 1, and two swaps of 16-lane rows bring each the halves that it needs (a
// row's own first words and its neighbour's, block i; the same of the other, block i + 1).
template <class P>
__device__ __forceinline__ void drop_block(f32x4 (&acc)[P::NI][P::NJ], const Dropper& d, int64_t m0, int64_t n0) {
  const int lane = opaque_int(threadIdx.x & 63), r = lane & 15, q = lane >> 4;
  const uint32_t thr = d.thr2 & 0xffffu;
#pragma unroll
  for (int j = 0; j < P::NJ; ++j) {
    const int64_t row = (m0 + j * 16 + r) * d.blocks + n0 / 8 + (q >> 1) + (q & 1) * 2;
#pragma unroll
    for (int i = 0; i < P::NI; i += 2) {
      const u32x4 w = philox7(static_cast<uint64_t>(row + i * 2), d.seed, d.offset);
      // odd rows of the first operand change places with the even rows before them of the second
      const auto lo = __builtin_amdgcn_permlane16_swap(w[0], w[2], false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(w[1], w[3], false, false);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w0 = lo[h], w1 = hi[h];
        f32x4& v = acc[i + h][j];
        v[0] = (w0 & 0xffffu) >= thr ? v[0] : 0.f;
        v[1] = (w0 >> 16) >= thr ? v[1] : 0.f;
        v[2] = (w1 & 0xffffu) >= thr ? v[2] : 0.f;
        v[3] = (w1 >> 16) >= thr ? v[3] : 0.f;
#if defined(__HIP_DEVICE_COMPILE__)
        if constexpr (P::BM == 256) asm volatile("" : "+a"(v));  // (back to where the MFMAs keep it)
#endif
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <class P>
struct DropNnOp : NnOp<P, 1, 1> {
  Dropper d;
  int64_t mw, nw;
  __device__ __forceinline__ void between(f32x4 (&acc)[P::NI][P::NJ]) const { drop_block<P>(acc, d, mw, nw); }
};

enum { kFormNt = 0, kFormNn = 1, kFormNn2 = 2, kFormNnDrop = 3 };  // (Nn2: two segments, two adapters)

// One layer: a workgroup per whole tile, then one per part of the others. Bound by the matrix pipes and the power they may
// draw. NT, 18871 tokens, 8960 -> 1536: 464 us, 1.12 PFLOP/s (444 whole tiles, 1.7 rounds of 256 units); NN, the gated
// dx of 4352 tokens, two times 14336 -> 4096: 901 us, 1.13; NN masked, dx of 18871 tokens, 1536 -> 8960: 651 us, of which
// the masks are 66.
template <class P, int FORM>
__global__ __launch_bounds__(P::THREADS, P::OCC) void ring_kernel(RingArgs p, int mt, int nt, int NS) {
  __shared__ __attribute__((aligned(1024))) char smem[P::SLOTS * P::SLOT_BYTES];
  const RingWork work(blockIdx.x, p.full, mt * nt, p.S, p.ks, NS);
  const RingTile tile(work.tile, mt, nt, P::GROUP_M);
  const int wave = ring_wave();
  const int wm0 = (wave % P::WAVES_M) * P::WM, wn0 = (wave / P::WAVES_M) * P::WN;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM, n0 = static_cast<int64_t>(tile.n) * P::BN;
  const int ns = work.hi - work.lo;
  f32x4 acc[P::NI][P::NJ];
  if constexpr (FORM == kFormNt) {
    NtOp<P, false> op;
    op.init(p, m0, n0, work.lo, work.hi);
    ring_run<P, false>(acc, op, ns, smem, wm0, wn0);
  } else if constexpr (FORM != kFormNnDrop) {
    NnOp<P, FORM == kFormNn2 ? 2 : 1, FORM == kFormNn2 ? 2 : 1> op;
    op.init(p.x, p.ldx, p.W, p.K, FORM == kFormNn2 ? p.T + p.terms : p.T, p.N, m0, n0, work.lo, work.hi);
    op.extend(p, m0, n0);
    ring_run<P, true>(acc, op, ns, smem, wm0, wn0);
  } else {
    DropNnOp<P> op;
    op.init(p.x, p.ldx, p.W, p.K, p.T, p.N, m0, n0, work.lo, work.hi);
    op.extend(p, m0, n0);
    op.d.init(p.drop, p.N);
    op.mw = m0 + wm0;
    op.nw = n0 + wn0;
    const int at = op.NE - work.lo;  // the first stage behind the extension
    ring_run<P, true, true>(acc, op, ns, smem, wm0, wn0, at);
    if (at >= ns) drop_block<P>(acc, op.d, op.mw, op.nw);  // (this part ends before the base stages)
  }
  if (work.unit >= 0) put_part<P>(acc, p.part, work.unit);
  else store_block<P, P::NJ>(acc, p, m0 + wm0, n0 + wn0, smem);
}

// The tiles that were cut: grid (tiles, column blocks of a wave).
template <class P>
__global__ __launch_bounds__(P::THREADS) void ring_join_kernel(RingArgs p, int mt, int nt) {
  __shared__ __attribute__((aligned(16))) char smem[P::WAVES * 16 * P::WN * 2];
  const RingTile tile(p.full + blockIdx.x, mt, nt, P::GROUP_M);
  const int wave = ring_wave(), j = blockIdx.y;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM + (wave % P::WAVES_M) * P::WM + j * 16;
  const int64_t n0 = static_cast<int64_t>(tile.n) * P::BN + (wave / P::WAVES_M) * P::WN;
  f32x4 acc[P::NI][1];
  sum_parts<P>(acc, p.part, blockIdx.x, p.S, j);
  if constexpr (P::BM == 2 * kTerms && P::WM == kTerms) {
    if (p.terms > 0) {  // the second terms are the next wave's tokens
      if (wave % P::WAVES_M != 0) return;
      f32x4 mid[P::NI][1];
      sum_parts<P>(mid, p.part, blockIdx.x, p.S, j, 1);
#pragma unroll
      for (int i = 0; i < P::NI; ++i) acc[i][0] += mid[i][0];
    }
  }
  store_block<P, 1>(acc, p, m0, n0, smem);
}

// Rank-wide product over rows of the contraction (the gradient's, B [K, rank] as it lies): 128 tokens and up to 128
// columns per workgroup, K in splits. Most of the MFMA's columns are empty for small ranks; the kernel is bound by
// reading x.
__device__ __forceinline__ void rank_nn(const RankProduct& p, int ks, int bx, int by, int bz, char* smem) {
  using P = Ring128;
  const int wave = ring_wave();
  const int wm0 = (wave % P::WAVES_M) * P::WM, wn0 = (wave / P::WAVES_M) * P::WN;
  const int64_t m0 = static_cast<int64_t>(bx) * P::BM, n0 = static_cast<int64_t>(by) * P::BN;
  const int NS = static_cast<int>((p.K + 63) / 64), s_lo = bz * ks, s_hi = min(NS, s_lo + ks);
  NnOp<P, 1, 0> op;
  op.init(&p.x, p.ldx, &p.A[0], &p.K, p.T, p.rank[0], m0, n0, s_lo, s_hi);
  f32x4 acc[P::NI][P::NJ];
  ring_run<P, true>(acc, op, s_hi - s_lo, smem, wm0, wn0);
  const int R = p.rank[0];
  store_part<P>(acc, p.part + static_cast<int64_t>(bz) * p.T * R, R, m0 + wm0, n0 + wn0, p.T, R);
}

// The first n_nt workgroups make the one product (grid (m-tiles, rows, splits) counted x first), the others the other.
template <class P, bool DROP>
__global__ __launch_bounds__(256, P::BN == 64 ? 2 : 1) void rank_kernel(RankProduct a, int ks_a, int n_nt, int chunks_a,
                                                                        RankProduct b, int ks_b, int chunks_b) {
  static_assert(P::THREADS == 256 && Ring128::THREADS == 256, "one block size");
  constexpr int kNt = P::S * P::STAGE_BYTES, kNn = Ring128::SLOTS * Ring128::SLOT_BYTES;
  __shared__ __attribute__((aligned(1024))) char smem[kNt > kNn ? kNt : kNn];
  const int id = blockIdx.x;
  if (id < n_nt) {
    const int mt = static_cast<int>((a.T + 127) / 128), rest = id / mt;
    rank_nt<P, DROP>(a, ks_a, id - rest * mt, rest % chunks_a, rest / chunks_a, smem);
  } else {
    const int mt = static_cast<int>((b.T + 127) / 128), i = id - n_nt, rest = i / mt;
    rank_nn(b, ks_b, i - rest * mt, rest % chunks_b, rest / chunks_b, smem);
  }
}

// ---------------------------------------------------------------------------
// The gated feed-forward.

// act(g) and act'(g). exp2 and the reciprocal are the hardware's (within 1 last bit of fp32 each).
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896f); }

template <int ACT, bool GRAD>
__device__ __forceinline__ void act_of(float g, float& a, float& da) {
  if constexpr (ACT == 0) {  // g sigmoid(g)
    const float s = __builtin_amdgcn_rcpf(1.f + fast_exp(-g));
    a = g * s;
    if (GRAD) da = s * (1.f + g * (1.f - s));
  } else if constexpr (ACT == 1) {
    // g Phi(g): the tail Phi(-|g|) = erfc(z) / 2, z = |g| / sqrt 2, whose exponential is also the derivative's density.
    // erfc(z) exp(z^2) = t P(t), t = 1 / (1 + z / 2): P of degree 8 fitted to the least relative error over z in [0, 10]
    // (1.3e-7 with these coefficients; 4e-7 with fp32's roundings), so that the tail keeps its digits however small it is.
    const float z = __builtin_fabsf(g) * 0.70710678118655f;
    const float t = __builtin_amdgcn_rcpf(1.f + 0.5f * z), e = fast_exp(-z * z);
    constexpr float kP[9] = {2.82088987e-01f, 2.82322961e-01f, 2.43534581e-01f, 2.00811248e-01f, -2.18574236e-02f,
                             2.70748975e-01f, -4.80521969e-01f, 2.81239052e-01f, -5.83664508e-02f};
    float poly = kP[8];
#pragma unroll
    for (int k = 7; k >= 0; --k) poly = fmaf(poly, t, kP[k]);
    const float tail = 0.5f * t * poly * e, cdf = g < 0.f ? tail : 1.f - tail;
    a = g * cdf;
    if (GRAD) da = cdf + g * e * 0.39894228040143f;
  } else {  // g sigmoid(2 c (g + 0.044715 g^3)), which is g (1 + tanh(c (..))) / 2
    const float c2 = 1.59576912160573f, g2 = fminf(g * g, 1e4f);  // (far beyond, s is 0 or 1: no infinity below)
    const float s = __builtin_amdgcn_rcpf(1.f + fast_exp(-c2 * g * (1.f + 0.044715f * g2)));
    a = g * s;
    if (GRAD) da = s + g * s * (1.f - s) * c2 * (1.f + 0.134145f * g2);
  }
}

template <class P, int ACT, int NJ>
__device__ __forceinline__ void gated_store(const f32x4 (&acc)[P::NI][NJ], const RingArgs& p, int64_t m0, int64_t n0,
                                            char* smem) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  BlockOut<NJ * 16, P::WN / 2> out{smem + ring_wave() * NJ * 16 * P::WN};
  const int64_t fb = (p.N + 15) / 16;
#pragma unroll
  for (int i = 0; i < P::NI / 2; ++i) {
    float bg[4], bu[4];
    const int64_t n = n0 + i * 16 + q * 4;
    load_bias4(bg, p.bias[0], n, p.N);
    load_bias4(bu, p.bias[1], n, p.N);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      f32x4 g, u;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = acc[2 * i][j][e] + bg[e];
        u[e] = acc[2 * i + 1][j][e] + bu[e];
        float a, da;
        act_of<ACT, false>(g[e], a, da);
        v[e] = a * u[e];
      }
      out.put(j * 16 + r, i * 16 + q * 4, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      if (p.saved != nullptr && m0 + j * 16 < p.T && n0 + i * 16 < p.N) {
        float* b = p.saved + (((m0 >> 4) + j) * fb + (n0 >> 4) + i) * 512 + lane * 4;
        __builtin_nontemporal_store(g, reinterpret_cast<f32x4*>(b));
        __builtin_nontemporal_store(u, reinterpret_cast<f32x4*>(b + 256));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (p.y != nullptr && m0 < p.T && n0 < p.N)
    out.store(p.y + m0 * p.ldy + n0, p.ldy, static_cast<int>(min<int64_t>(NJ * 16, p.T - m0)),
              static_cast<int>(min<int64_t>(P::WN / 2, p.N - n0)));
}

// BN / 2 outputs per tile: gate and up blocks of 16 rows in turn, so that a lane has g and u of the same outputs and the
// activation needs no exchange. Bound by the matrix pipes: 12288 tokens, 4096 -> 14336: 2.15 to 2.25 ms by the card, 1.28 to
// 1.34 PFLOP/s (2.40 ms under the profiler); pipes 68% busy at 1.8 GHz. A tile's start and epilogue are 15 of its 115 us
// (ring filling 4, activation and stores 10); a stage takes 1.5, 1.1 of it MFMAs. All operands from L2 made it 4% faster;
// what a stage computes for the next, spread between its MFMAs instead of before them, 1% slower.
template <class P, int ACT>
__global__ __launch_bounds__(P::THREADS, P::OCC) void gated_kernel(RingArgs p, int mt, int nt, int NS) {
  __shared__ __attribute__((aligned(1024))) char smem[P::SLOTS * P::SLOT_BYTES];
  const RingWork work(blockIdx.x, p.full, mt * nt, p.S, p.ks, NS);
  const RingTile tile(work.tile, mt, nt, P::GROUP_M);
  const int wave = ring_wave();
  const int wm0 = (wave % P::WAVES_M) * P::WM, wn0 = (wave / P::WAVES_M) * P::WN;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM, n0 = static_cast<int64_t>(tile.n) * (P::BN / 2);
  f32x4 acc[P::NI][P::NJ];
  NtOp<P, true> op;
  op.init(p, m0, n0, work.lo, work.hi);
  ring_run<P, false>(acc, op, work.hi - work.lo, smem, wm0, wn0);
  if (work.unit >= 0) put_part<P>(acc, p.part, work.unit);
  else gated_store<P, ACT, P::NJ>(acc, p, m0 + wm0, n0 + wn0 / 2, smem);
}

template <class P, int ACT>
__global__ __launch_bounds__(P::THREADS) void gated_join_kernel(RingArgs p, int mt, int nt) {
  __shared__ __attribute__((aligned(16))) char smem[P::WAVES * 16 * P::WN];
  const RingTile tile(p.full + blockIdx.x, mt, nt, P::GROUP_M);
  const int wave = ring_wave(), j = blockIdx.y;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM + (wave % P::WAVES_M) * P::WM + j * 16;
  const int64_t n0 = static_cast<int64_t>(tile.n) * (P::BN / 2) + (wave / P::WAVES_M) * (P::WN / 2);
  f32x4 acc[P::NI][1];
  sum_parts<P>(acc, p.part, blockIdx.x, p.S, j);
  gated_store<P, ACT, 1>(acc, p, m0, n0, smem);
}

// Few tokens: grid (128-row tiles of gate, up, A_gate, A_up, one behind the other; parts of the contraction). Bound by
// reading the weights: 48 tokens, 4096 -> 14336: 58 us from memory (42 where the Infinity Cache holds a part), 235 MB.
__global__ __launch_bounds__(Ring128::THREADS, Ring128::OCC) void gated_few_kernel(GatedFew p) {
  using P = Ring128;
  __shared__ __attribute__((aligned(1024))) char smem[P::SLOTS * P::SLOT_BYTES];
  const int nf = static_cast<int>((p.F + 127) / 128), na = (p.rank[0] + 127) / 128;
  int id = blockIdx.x;
  const int64_t fc = (p.F + 3) / 4 * 4, ld = 2 * fc + p.rank[0] + p.rank[1];
  RingArgs g = {};
  g.x[0] = p.x; g.ldx = p.ldx; g.K[0] = p.K; g.T = p.T;
  int64_t col;
  if (id < 2 * nf) {
    const int side = id >= nf ? 1 : 0;
    g.W[0] = p.W[side];
    g.N = p.F;
    col = side * fc;
    id -= side * nf;
  } else {
    id -= 2 * nf;
    const int side = id >= na ? 1 : 0;
    g.W[0] = p.A[side];
    g.N = p.rank[side];
    col = 2 * fc + (side ? p.rank[0] : 0);
    id -= side * na;
  }
  const int wave = ring_wave();
  const int wm0 = (wave % P::WAVES_M) * P::WM, wn0 = (wave / P::WAVES_M) * P::WN;
  const int64_t n0 = static_cast<int64_t>(id) * P::BN;
  const int NS = static_cast<int>((p.K + 63) / 64), lo = static_cast<int>(blockIdx.y) * p.ks, hi = min(NS, lo + p.ks);
  f32x4 acc[P::NI][P::NJ];
  NtOp<P, false> op;
  op.init(g, 0, n0, lo, hi);
  ring_run<P, false>(acc, op, hi - lo, smem, wm0, wn0);
  store_part<P>(acc, p.part + static_cast<int64_t>(blockIdx.y) * p.T * ld + col, ld, wm0, n0 + wn0, p.T, g.N);
}

// h of 4 tokens and 256 columns per workgroup; the rank-wide products stay in fp32.
template <int ACT>
__global__ __launch_bounds__(256) void gated_few_finish_kernel(GatedFew p) {
  extern __shared__ __attribute__((aligned(16))) float tt[];  // [4][R]
  const int R = p.rank[0] + p.rank[1];
  const int64_t fc = (p.F + 3) / 4 * 4, ld = 2 * fc + R;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 4, n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t nn = min<int64_t>(n, p.F - 1);
  float g[4], u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = u[i] = 0.f;
  for (int z = 0; z < p.S; ++z)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* row = p.part + (z * p.T + min<int64_t>(t0 + i, p.T - 1)) * ld + nn;
      g[i] += row[0];
      u[i] += row[fc];
    }
  for (int c = threadIdx.x; c < 4 * R; c += 256) {
    const int i = c / R, q = c - i * R;
    const float* row = p.part + min<int64_t>(t0 + i, p.T - 1) * ld + 2 * fc + q;
    float v = 0.f;
    for (int z = 0; z < p.S; ++z) v += row[z * p.T * ld];
    tt[c] = v * (q < p.rank[0] ? p.scale[0] : p.scale[1]);
  }
  __syncthreads();
  if (n >= p.F) return;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    float (&v)[4] = side ? u : g;
    const int r = p.rank[side];
    const uint16_t* b = p.B[side] + n * r;
    const float* t = tt + (side ? p.rank[0] : 0);
    for (int q = 0; q < r; q += 8) {  // (ranks are multiples of 8, B 16-byte aligned)
      const u32x4 w = *reinterpret_cast<const u32x4*>(b + q);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t pair = w[e >> 1];
        const float bv = __uint_as_float(e & 1 ? pair & 0xffff0000u : pair << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(t[i * R + q + e], bv, v[i]);
      }
    }
    if (p.bias[side] != nullptr) {
      const float bv = bf16_to_f32(p.bias[side][n]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += bv;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t0 + i >= p.T) break;
    float a, da;
    act_of<ACT, false>(g[i], a, da);
    p.h[(t0 + i) * p.ldh + n] = f32_to_bf16_rne(a * u[i]);
  }
}

// dg and du, and v = dg . B_gate beside du . B_up (NB blocks of 16 of its columns; 0: none): 64 tokens per workgroup, 16 to
// a wave, `per` runs of 64 columns one after the other, from the blocks that the forward kept. A wave's values go through
// LDS as two bf16 terms each, which the MFMAs take from there, against the run's rows of both B, read across with the
// transposing read; the first terms are stored (up to 64 tokens both). More blocks than eight are further grid layers,
// which form the values again and store none. HBM-bound: 4352 tokens, 14336 wide, ranks 32 and 32: 204 us, 873 MB at
// 4.3 TB/s (without second terms 189); a product of its own, from the stored values, took 75 us beside 195.
template <int ACT, int NB>
__global__ __launch_bounds__(256) void gated_grad_kernel(const float* __restrict__ saved, const uint16_t* __restrict__ dh,
                                                         int64_t lddh, int64_t T, int64_t F, uint16_t* __restrict__ dg,
                                                         uint16_t* __restrict__ du, RankProduct v, int per) {
  constexpr int PPR = NB > 0 ? 2 * NB : 1;  // 16-byte pieces of a run's row of B
  __shared__ __attribute__((aligned(16))) char smem[4][2][2][16 * 64 * 2], sb[64 * PPR * 16];  // [wave][side][term]
  const int lane = threadIdx.x & 63, wave = ring_wave(), r = lane & 15, q = lane >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 64 + wave * 16;
  const int ng = (v.rank[0] + 15) / 16, first = static_cast<int>(blockIdx.z) * NB;
  const int64_t run0 = static_cast<int64_t>(blockIdx.y) * per, run1 = min<int64_t>((F + 63) / 64, run0 + per);
  const bool here = m0 < T, both = T <= kTerms;  // (a wave without tokens still stages B)
  const bool stores = blockIdx.z == 0;
  const int64_t fb = (F + 15) / 16, m = min<int64_t>(m0 + r, T - 1);
  f32x4 g[4], u[4];
  uint2 d[4];
  auto load = [&](int64_t n0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + i * 16;
      if (n >= F) continue;
      const float* b = saved + ((m0 >> 4) * fb + (n >> 4)) * 512 + lane * 4;
      g[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(b));
      u[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(b + 256));
      // (F is a multiple of 8, and so is the row stride: 8 bytes never cross the end)
      d[i] = n + q * 4 < F ? *reinterpret_cast<const uint2*>(dh + m * lddh + n + q * 4) : uint2{0u, 0u};
    }
  };
  auto put = [&](int side, int col, const float (&x)[4]) {
    BlockOut<16, 64> hi{smem[wave][side][0]}, mid{smem[wave][side][1]};
    const uint32_t lo2 = pack_bf16x2(x[0], x[1]), hi2 = pack_bf16x2(x[2], x[3]);
    hi.put(r, col, lo2, hi2);
    if (NB == 0 && !both) return;
    float rest[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // (nothing behind an infinity)
      const uint32_t w = e < 2 ? lo2 : hi2;
      const float h = __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
      rest[e] = __builtin_isfinite(h) ? x[e] - h : 0.f;
    }
    mid.put(r, col, pack_bf16x2(rest[0], rest[1]), pack_bf16x2(rest[2], rest[3]));
  };
  auto form = [&](int64_t n0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n0 + i * 16 >= F) continue;
      const float dv[4] = {__uint_as_float(d[i].x << 16), __uint_as_float(d[i].x & 0xffff0000u),
                           __uint_as_float(d[i].y << 16), __uint_as_float(d[i].y & 0xffff0000u)};
      float vg[4], vu[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, da;
        act_of<ACT, true>(g[i][e], a, da);
        vg[e] = dv[e] * u[i][e] * da;
        vu[e] = dv[e] * a;
      }
      put(0, i * 16 + q * 4, vg);
      put(1, i * 16 + q * 4, vu);
    }
  };
  // this thread's pieces of a run's rows of B (zeros where a column is none of an adapter's)
  constexpr int NP = NB > 0 ? (64 * PPR + 255) / 256 : 1;
  u32x4 bv[NP];
  auto load_b = [&](int64_t n0) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int id = i * 256 + threadIdx.x, row = id / PPR, pc = id - row * PPR, blk = first + pc / 2;
      const int side = blk >= ng ? 1 : 0, col = (side ? blk - ng : blk) * 16 + (pc & 1) * 8;
      bv[i] = row < 64 && n0 + row < F && col < v.rank[side]
                  ? *reinterpret_cast<const u32x4*>(v.A[side] + (n0 + row) * v.rank[side] + col)
                  : u32x4{0u, 0u, 0u, 0u};
    }
  };
  f32x4 acc[NB > 0 ? NB : 1];
#pragma unroll
  for (int i = 0; i < NB; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (NB > 0) load_b(run0 * 64);
  if (here) load(run0 * 64);
  for (int64_t run = run0; run < run1; ++run) {
    const int64_t n0 = run * 64;
    if (NB > 0) {
      __syncthreads();  // (the last run's B has been read)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int id = i * 256 + threadIdx.x;
        if (id < 64 * PPR) *reinterpret_cast<u32x4*>(sb + id * 16) = bv[i];
      }
    }
    if (here) form(n0);
    if (run + 1 < run1) {  // (on their way while this run is multiplied and stored)
      if (NB > 0) load_b(n0 + 64);
      if (here) load(n0 + 64);
    }
    if (NB > 0) __syncthreads();
    if (!here) continue;
    if constexpr (NB > 0) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const bool in = n0 + kk * 32 + 8 * q < F;
        bf16x8 x[2][2];
#pragma unroll
        for (int side = 0; side < 2; ++side)
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(smem[wave][side][term] + BlockOut<16, 64>::at(r, kk * 4 + q));
            x[side][term] = __builtin_bit_cast(bf16x8, in ? w : u32x4{0u, 0u, 0u, 0u});
          }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const char* at = sb + (kk * 32 + 8 * q + (r >> 2)) * NB * 32 + i * 32 + (r & 3) * 8;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * NB * 32));
          const bf16x8 a = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
          const bool up = first + i >= ng;
#pragma unroll
          for (int term = 0; term < 2; ++term)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, up ? x[1][term] : x[0][term], acc[i], 0, 0, 0);
        }
      }
    }
    if (!stores) continue;
    const int rows = static_cast<int>(min<int64_t>(16, T - m0)), cols = static_cast<int>(min<int64_t>(64, F - n0));
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        if (term > 0 && !both) continue;
        const BlockOut<16, 64> out{smem[wave][side][term]};
        out.store((side ? du : dg) + (m0 + term * kTerms) * F + n0, F, rows, cols);
      }
  }
  if (NB == 0 || m0 + r >= T) return;
  const int R = v.rank[0] + v.rank[1];
  float* row = v.part + (static_cast<int64_t>(blockIdx.y) * T + m0 + r) * R;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int blk = first + i, side = blk >= ng ? 1 : 0, c = (side ? blk - ng : blk) * 16 + 4 * q;
    if (c < v.rank[side]) *reinterpret_cast<f32x4*>(row + (side ? v.rank[0] : 0) + c) = acc[i];
  }
}

// ---------------------------------------------------------------------------
// Token contraction: 256 rows of P^T x 64 columns of Q per workgroup, 32 tokens per stage, a ring of three stages
// [32 t][256] of P and [32 t][64 first terms | 64 second terms] of Q, both read with the transposing LDS read, two
// workgroups on a compute unit. Token chunks over grid y leave fp32 partial sums that contract_reduce_kernel adds in
// order. HBM-bound: P is read once (and, masked, the generator's arithmetic takes about as long): 285 MB of x, dg and du
// (4352 tokens, 4096 -> 14336) in 58 us, 4.9 TB/s; 396 MB of x and dy (18871 tokens, 8960 -> 1536) in 85, masked 130.
constexpr int kCtP = kCtT * kCtI * 2, kCtQ = kCtT * 2 * kCtJ * 2, kCtStage = kCtP + kCtQ;

__device__ __forceinline__ bf16x8 tr_frag(const char* at, int row4) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + row4));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// NB blocks of 16 columns. (restrict: the copies in flight go to other slots; see ring_stage)
template <int NB>
__device__ __forceinline__ void contract_stage(f32x4 (&acc)[4][kCtJ / 16], const char* __restrict__ pb,
                                               const char* __restrict__ qb, uint32_t pa, uint32_t qa) {
  bf16x8 af[4], bq[NB][2];
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) af[ib] = tr_frag(pb + (pa ^ static_cast<uint32_t>(ib << 5)), 4 * 512);
#pragma unroll
  for (int jb = 0; jb < NB; ++jb)
#pragma unroll
    for (int term = 0; term < 2; ++term)
      bq[jb][term] = tr_frag(qb + (qa ^ static_cast<uint32_t>((term * 4 + jb) << 5)), 4 * 256);
#pragma unroll
  for (int jb = 0; jb < NB; ++jb)
#pragma unroll
    for (int term = 0; term < 2; ++term)
#pragma unroll
      for (int ib = 0; ib < 4; ++ib)
        acc[ib][jb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[ib], bq[jb][term], acc[ib][jb], 0, 0, 0);
}

template <bool DROP>
__global__ __launch_bounds__(256, 2) void contract_kernel(Contract p, int S, int64_t chunk) {
  __shared__ __attribute__((aligned(1024))) char smem[3 * kCtStage];
  const int lane = threadIdx.x & 63, wave = ring_wave(), r = lane & 15, q = lane >> 4;
  int ti = 0, id = blockIdx.x;
  int64_t before = 0;  // elements of the tasks before this one
  while (ti + 1 < p.n_tasks) {
    const int n = static_cast<int>((p.task[ti].M + kCtI - 1) / kCtI) * ((p.task[ti].J + kCtJ - 1) / kCtJ);
    if (id < n) break;
    id -= n;
    before += p.task[ti].M * p.task[ti].J;
    ++ti;
  }
  const ContractTask& k = p.task[ti];
  const int it = static_cast<int>((k.M + kCtI - 1) / kCtI);
  const int j0 = id / it * kCtJ, jn = min(kCtJ, k.J - j0), nj = (jn + 15) / 16;
  const int64_t i0 = static_cast<int64_t>(id % it) * kCtI;
  const int cols = static_cast<int>(min<int64_t>(kCtI, k.M - i0));
  const int z = blockIdx.y, S1 = S / p.halves, half = z >= S1 ? 1 : 0;
  const int64_t t_lo = (z - half * S1) * chunk, t_hi = min<int64_t>(p.T, t_lo + chunk);
  const bool none = half > 0 && k.terms == 0;
  const int nst = t_hi > t_lo && !none ? static_cast<int>((t_hi - t_lo + kCtT - 1) / kCtT) : 0;
  const uint16_t* P = k.P + (half ? k.terms * k.ldp : 0);
  const uint32_t ldp_b = static_cast<uint32_t>(k.ldp * 2), ldt_b = static_cast<uint32_t>(k.ldt * 2);
  // per-lane offsets: 4 instructions of P (2 rows of 512 bytes each), 2 of Q (4 rows of 256)
  uint32_t vp[4], vq[2];
  int prow[4], pcol[4];
#pragma unroll
  for (int l = 0; l < 4; ++l) {
    const int sl = (l * 4 + wave) * 64 + lane, t = sl / 32, pc = sl % 32, f = (t & 3) | (((t >> 3) & 1) << 2);
    const int col = (((pc >> 1) ^ f) * 2 + (pc & 1)) * 8;
    vp[l] = col < cols ? static_cast<uint32_t>(t) * ldp_b + col * 2 : kMissing;
    prow[l] = t;
    pcol[l] = col;
  }
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    const int sl = (l * 4 + wave) * 64 + lane, t = sl / 16, pc = sl % 16, f = (t & 3) | (((t >> 3) & 1) << 2);
    const int col = (((pc >> 1) ^ f) * 2 + (pc & 1)) * 8, c = col & 63;
    vq[l] = c < jn ? static_cast<uint32_t>(t) * ldt_b + static_cast<uint32_t>((col < 64 ? 0 : k.R) + k.q_col + j0 + c) * 2
                   : kMissing;
  }
  auto issue = [&](int s) {
    char* b = smem + (s % 3) * kCtStage;
    const int64_t t0 = t_lo + static_cast<int64_t>(s) * kCtT;
    const int rows = s < nst ? static_cast<int>(min<int64_t>(kCtT, t_hi - t0)) : 0;
    const int64_t at = rows > 0 ? t0 : 0;
    const __amdgpu_buffer_rsrc_t pr = make_rsrc(
        P + at * k.ldp + i0, rows > 0 ? static_cast<uint32_t>(rows - 1) * ldp_b + static_cast<uint32_t>(cols) * 2 : 0u);
    const __amdgpu_buffer_rsrc_t qr = make_rsrc(k.tt + at * k.ldt, static_cast<uint32_t>(rows) * ldt_b);
#pragma unroll
    for (int l = 0; l < 4; ++l)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(pr, (lds_void*)(b + (l * 4 + wave) * 1024), 16, vp[l], 0, 0, 0);
#pragma unroll
    for (int l = 0; l < 2; ++l)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(qr, (lds_void*)(b + kCtP + (l * 4 + wave) * 1024), 16, vq[l], 0, 0, 0);
  };
  Dropper d;
  const bool masked = DROP && k.masked;
  if constexpr (DROP) d.init(p.drop, k.M);
  f32x4 acc[4][kCtJ / 16];
#pragma unroll
  for (int ib = 0; ib < 4; ++ib)
#pragma unroll
    for (int jb = 0; jb < kCtJ / 16; ++jb) acc[ib][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int f = (r >> 2) | ((q & 1) << 2);
  const uint32_t pa = static_cast<uint32_t>((8 * q + (r >> 2)) * 512 + (((wave * 4) ^ f) * 32) + (r & 3) * 8);
  const uint32_t qa = static_cast<uint32_t>((8 * q + (r >> 2)) * 256 + f * 32 + (r & 3) * 8);
  issue(0);
  issue(1);
  for (int s = 0; s < nst; ++s) {
    u32x4 mask[4];
    if (masked) {  // (needs no data: formed while the stage's copies are on their way)
#pragma unroll
      for (int l = 0; l < 4; ++l)
        mask[l] = d.masks(t_lo + static_cast<int64_t>(s) * kCtT + prow[l], (i0 + pcol[l]) / 8);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(6));  // this wave's copies of stage s landed; s + 1's may be in flight
    char* b = smem + (s % 3) * kCtStage;
    if (masked) {  // (each wave masks what it copied)
#pragma unroll
      for (int l = 0; l < 4; ++l) *reinterpret_cast<u32x4*>(b + ((l * 4 + wave) * 64 + lane) * 16) &= mask[l];
    }
    stage_barrier();  // stage s is there for every wave, and every wave is done reading stage s - 1
    issue(s + 2);
    if (nj == 4) contract_stage<4>(acc, b, b + kCtP, pa, qa);
    else if (nj == 3) contract_stage<3>(acc, b, b + kCtP, pa, qa);
    else if (nj == 2) contract_stage<2>(acc, b, b + kCtP, pa, qa);
    else contract_stage<1>(acc, b, b + kCtP, pa, qa);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  // lane (r, q) of block (ib, jb): rows i = 64 wave + 16 ib + 4 q + e of P^T, column j = 16 jb + r
  float* part = p.part + (before * S + z * k.M * k.J);
#pragma unroll
  for (int jb = 0; jb < kCtJ / 16; ++jb) {
    const int j = j0 + jb * 16 + r;
    if (j >= k.J || jb >= nj) continue;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
      const int64_t i = i0 + wave * 64 + ib * 16 + 4 * q;
      if (i >= k.M) continue;  // (M is a multiple of 8: four rows exist together)
      if (k.transposed) {
        *reinterpret_cast<f32x4*>(part + static_cast<int64_t>(j) * k.M + i) = acc[ib][jb];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) part[(i + e) * k.J + j] = acc[ib][jb][e];
      }
    }
  }
}

// The chunks' sum in order, 4 elements per thread (M and J are multiples of 8). Grid y: task.
__global__ __launch_bounds__(256) void contract_reduce_kernel(Contract p, int S) {
  const int ti = blockIdx.y;
  const ContractTask& k = p.task[ti];
  const int64_t n = k.M * k.J, idx = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (idx >= n) return;
  int64_t before = 0;
  for (int i = 0; i < ti; ++i) before += p.task[i].M * p.task[i].J;
  const float* src = p.part + before * S + idx;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int z = 0; z < S; ++z) v += *reinterpret_cast<const f32x4*>(src + z * n);
  const int64_t cut = k.transposed ? static_cast<int64_t>(k.split) * k.M : n;
  void* out = idx < cut ? k.out[0] : k.out[1];
  const int64_t at = idx < cut ? idx : idx - cut;
  if (out == nullptr) return;
  if (p.out_bf16) {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (reinterpret_cast<uintptr_t>(o) % 8 == 0) {
      *reinterpret_cast<uint2*>(o) = uint2{lo, hi};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = static_cast<uint16_t>((e < 2 ? lo : hi) >> (16 * (e & 1)));
    }
  } else {
    float* o = static_cast<float*>(out) + at;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = v[e];
  }
}

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

}  // namespace

hipError_t launch_rank_products(const RankProduct* nt, const RankProduct* nn, hipStream_t s) {
  RankProduct a = {}, b = {};
  int Sa = 0, ka = 1, n_nt = 0, ca = 1, Sb = 0, kb = 1, n_nn = 0, cb = 1;
  bool narrow = true, drop = false, few = true;
  if (nt != nullptr) {
    a = *nt;
    const int64_t R = a.rank[0] + a.rank[1];
    narrow = R <= 64;
    drop = a.drop.thr != 0;
    few = rank_few(a.T, a.K, R);
    rank_plan(a.T, a.K, rank_tasks(R, false), &Sa, &ka);
    ca = static_cast<int>(narrow ? 1 : (R + 127) / 128);
    n_nt = static_cast<int>((a.T + 127) / 128) * ca * Sa;
  }
  if (nn != nullptr) {
    b = *nn;
    few = few && rank_few(b.T, b.K, b.rank[0]);
    cb = static_cast<int>(rank_tasks(b.rank[0], true));
    rank_plan(b.T, b.K, cb, &Sb, &kb);
    n_nn = static_cast<int>((b.T + 127) / 128) * cb * Sb;
  }
  if (few) {
    const unsigned na = nt != nullptr ? 1 : 0, nb = nn != nullptr ? 1 : 0;
    const dim3 fg(blocks_of(nt != nullptr ? a.T : b.T, 16), na + nb), fb(kFewWaves * 64);
    if (drop) hipLaunchKernelGGL(rank_few_kernel<true>, fg, fb, 0, s, a, static_cast<int>(na), b);
    else hipLaunchKernelGGL(rank_few_kernel<false>, fg, fb, 0, s, a, static_cast<int>(na), b);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(n_nt + n_nn)), block(256);
  if (narrow && drop) hipLaunchKernelGGL((rank_kernel<RankNarrow, true>), grid, block, 0, s, a, ka, n_nt, ca, b, kb, cb);
  else if (narrow) hipLaunchKernelGGL((rank_kernel<RankNarrow, false>), grid, block, 0, s, a, ka, n_nt, ca, b, kb, cb);
  else if (drop) hipLaunchKernelGGL((rank_kernel<RankWide, true>), grid, block, 0, s, a, ka, n_nt, ca, b, kb, cb);
  else hipLaunchKernelGGL((rank_kernel<RankWide, false>), grid, block, 0, s, a, ka, n_nt, ca, b, kb, cb);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  auto blocks = [](const RankProduct& p, int S) {
    return S > 0 ? blocks_of(p.T * (pair_ld(p.rank[0] + p.rank[1]) / 4), 256) : 0u;
  };
  const unsigned ba = blocks(a, Sa), bb = blocks(b, Sb);
  hipLaunchKernelGGL(rank_finish_kernel, dim3(ba + bb), dim3(256), 0, s, a, Sa, static_cast<int>(ba), b, Sb);
  return hipGetLastError();
}

template <class P, int FORM>
hipError_t launch_ring_cfg(const RingArgs& p, int NS, hipStream_t s) {
  const int mt = static_cast<int>((p.T + p.terms + P::BM - 1) / P::BM), nt = static_cast<int>((p.N + P::BN - 1) / P::BN);
  const int rem = mt * nt - p.full;
  hipLaunchKernelGGL((ring_kernel<P, FORM>), dim3(static_cast<unsigned>(p.full + rem * p.S)), dim3(P::THREADS), 0, s, p, mt,
                     nt, NS);
  if (rem > 0)
    hipLaunchKernelGGL(ring_join_kernel<P>, dim3(static_cast<unsigned>(rem), P::NJ), dim3(P::THREADS), 0, s, p, mt, nt);
  return hipGetLastError();
}

hipError_t launch_ring(const RingArgs& a, bool nn, hipStream_t s) {
  RingArgs p = a;
  const int NS = static_cast<int>(ring_stages(p));
  const RingPlan plan = p.terms > 0 ? terms_plan(p.N, NS) : ring_plan(p.T, p.N, NS);
  p.full = static_cast<int>(plan.full);
  p.S = plan.S;
  p.ks = plan.ks;
  const bool big = plan.big;
  if (!nn) return big ? launch_ring_cfg<Ring256, kFormNt>(p, NS, s) : launch_ring_cfg<Ring128, kFormNt>(p, NS, s);
  if (p.n_seg > 1) return big ? launch_ring_cfg<Ring256, kFormNn2>(p, NS, s) : launch_ring_cfg<Ring128, kFormNn2>(p, NS, s);
  if (p.drop.thr == 0) return big ? launch_ring_cfg<Ring256, kFormNn>(p, NS, s) : launch_ring_cfg<Ring128, kFormNn>(p, NS, s);
  return big ? launch_ring_cfg<Ring256, kFormNnDrop>(p, NS, s) : launch_ring_cfg<Ring128, kFormNnDrop>(p, NS, s);
}

template <class P, int ACT>
hipError_t launch_gated_cfg(const RingArgs& p, int NS, hipStream_t s) {
  const int mt = static_cast<int>((p.T + P::BM - 1) / P::BM), nt = static_cast<int>((2 * p.N + P::BN - 1) / P::BN);
  const int rem = mt * nt - p.full;
  hipLaunchKernelGGL((gated_kernel<P, ACT>), dim3(static_cast<unsigned>(p.full + rem * p.S)), dim3(P::THREADS), 0, s, p, mt,
                     nt, NS);
  if (rem > 0)
    hipLaunchKernelGGL((gated_join_kernel<P, ACT>), dim3(static_cast<unsigned>(rem), P::NJ), dim3(P::THREADS), 0, s, p, mt,
                       nt);
  return hipGetLastError();
}

hipError_t launch_gated(const RingArgs& a, hipStream_t s) {
  RingArgs p = a;
  const int NS = static_cast<int>(ring_stages(p));
  const RingPlan plan = ring_plan(p.T, 2 * p.N, NS);
  p.full = static_cast<int>(plan.full);
  p.S = plan.S;
  p.ks = plan.ks;
  if (p.act == 0) return plan.big ? launch_gated_cfg<Ring256, 0>(p, NS, s) : launch_gated_cfg<Ring128, 0>(p, NS, s);
  if (p.act == 1) return plan.big ? launch_gated_cfg<Ring256, 1>(p, NS, s) : launch_gated_cfg<Ring128, 1>(p, NS, s);
  return plan.big ? launch_gated_cfg<Ring256, 2>(p, NS, s) : launch_gated_cfg<Ring128, 2>(p, NS, s);
}

hipError_t launch_gated_few(const GatedFew& a, hipStream_t s) {
  GatedFew p = a;
  const int R = p.rank[0] + p.rank[1];
  few_plan(p.T, p.K, p.F, R, &p.S, &p.ks);
  const int tiles = static_cast<int>(2 * ((p.F + 127) / 128)) + (p.rank[0] + 127) / 128 + (p.rank[1] + 127) / 128;
  hipLaunchKernelGGL(gated_few_kernel, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(p.S)), dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(blocks_of(p.F, 256), blocks_of(p.T, 4)), block(256);
  const size_t lds = static_cast<size_t>(4 * R) * 4;  // (at most 2048 ranks: 32 KB)
  if (p.act == 0) hipLaunchKernelGGL(gated_few_finish_kernel<0>, grid, block, lds, s, p);
  else if (p.act == 1) hipLaunchKernelGGL(gated_few_finish_kernel<1>, grid, block, lds, s, p);
  else hipLaunchKernelGGL(gated_few_finish_kernel<2>, grid, block, lds, s, p);
  return hipGetLastError();
}

template <int ACT>
static hipError_t launch_gated_grad_act(const float* saved, const uint16_t* dh, int64_t lddh, int64_t T, int64_t F,
                                        uint16_t* dg, uint16_t* du, const RankProduct* v, hipStream_t s) {
  int S, per;
  grad_plan(T, F, &S, &per);
  const RankProduct p = v != nullptr ? *v : RankProduct{};
  const unsigned nb = v != nullptr ? static_cast<unsigned>(grad_blocks(p.rank[0], p.rank[1])) : 0;
  const dim3 grid(blocks_of(T, 64), static_cast<unsigned>(S), nb > 8 ? (nb + 7) / 8 : 1), block(256);
  if (nb == 0) hipLaunchKernelGGL((gated_grad_kernel<ACT, 0>), grid, block, 0, s, saved, dh, lddh, T, F, dg, du, p, per);
  else if (nb == 1) hipLaunchKernelGGL((gated_grad_kernel<ACT, 1>), grid, block, 0, s, saved, dh, lddh, T, F, dg, du, p, per);
  else if (nb == 2) hipLaunchKernelGGL((gated_grad_kernel<ACT, 2>), grid, block, 0, s, saved, dh, lddh, T, F, dg, du, p, per);
  else if (nb <= 4) hipLaunchKernelGGL((gated_grad_kernel<ACT, 4>), grid, block, 0, s, saved, dh, lddh, T, F, dg, du, p, per);
  else hipLaunchKernelGGL((gated_grad_kernel<ACT, 8>), grid, block, 0, s, saved, dh, lddh, T, F, dg, du, p, per);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || v == nullptr) return e;
  hipLaunchKernelGGL(grad_rank_finish_kernel, dim3(blocks_of(T * (pair_ld(p.rank[0] + p.rank[1]) / 4), 256)), dim3(256), 0, s,
                     p, S, T <= kTerms ? kTerms : 0);
  return hipGetLastError();
}

hipError_t launch_gated_grad(const float* saved, const uint16_t* dh, int64_t lddh, int64_t T, int64_t F, int act,
                             uint16_t* dg, uint16_t* du, const RankProduct* v, hipStream_t s) {
  if (act == 0) return launch_gated_grad_act<0>(saved, dh, lddh, T, F, dg, du, v, s);
  if (act == 1) return launch_gated_grad_act<1>(saved, dh, lddh, T, F, dg, du, v, s);
  return launch_gated_grad_act<2>(saved, dh, lddh, T, F, dg, du, v, s);
}

hipError_t launch_contract(const Contract& p, hipStream_t s) {
  int64_t tiles = 0, most = 0;
  bool drop = false;
  for (int i = 0; i < p.n_tasks; ++i) {
    tiles += contract_tiles(p.task[i].M, p.task[i].J);
    most = p.task[i].M * p.task[i].J > most ? p.task[i].M * p.task[i].J : most;
    drop = drop || (p.task[i].masked && p.drop.thr != 0);
  }
  int S;
  int64_t chunk;
  contract_plan(p.T, tiles, &S, &chunk);
  S *= p.halves;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(S));
  if (drop) hipLaunchKernelGGL(contract_kernel<true>, grid, dim3(256), 0, s, p, S, chunk);
  else hipLaunchKernelGGL(contract_kernel<false>, grid, dim3(256), 0, s, p, S, chunk);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(contract_reduce_kernel, dim3(blocks_of(most, 1024), static_cast<unsigned>(p.n_tasks)), dim3(256), 0, s,
                     p, S);
  return hipGetLastError();
}

}  // namespace lora
