// Softmax cross entropy over a vocabulary straight from hidden states h [T, K] and the output weight W [V, K], bf16:
//
//   l = h W^T (never kept),  lse = log sum exp(l),  loss = lse - l[target]
//   dh = dloss (sum over v != target of p_v W_v  -  (1 - p_target) W_target),  p = exp(l - lse)
//
// The target is held apart from the other tokens throughout: p_target - 1 is minus the others' sum, where the difference
// of a share rounded to bf16 and one would lose what a sure token has left.
//
//   logits_kernel<stats>   l of a tile in the accumulators; per token and block of columns the largest logit and the sum
//   lse_kernel             blocks -> lse, loss, 1 - p_target
//   logits_kernel<share>   l of a piece of the vocabulary again, p to memory in bf16
//   dh_kernel              sums over a piece of p W, fp32, added to the pieces' before it
//   dh_finish_kernel       the target's part, dloss, one rounding
#include "common.hpp"
#include "loss.hpp"
#include "ring_ops.hpp"

namespace lora {
namespace {

constexpr float kLog2e = 1.44269504088896f;
__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }

enum { kStats = 0, kShare = 1 };

// l of the columns v0 .. v0 + cols of the vocabulary.
template <class P, int MODE>
__global__ __launch_bounds__(P::THREADS, P::OCC) void logits_kernel(VocabLoss p, int64_t v0, int64_t cols, int mt, int nt) {
  __shared__ __attribute__((aligned(1024))) char smem[P::SLOTS * P::SLOT_BYTES];
  const RingTile tile(xcd_remap(blockIdx.x, mt * nt), mt, nt, P::GROUP_M);
  const int wave = ring_wave();
  const int wm0 = (wave % P::WAVES_M) * P::WM, wn0 = (wave / P::WAVES_M) * P::WN;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM, n0 = static_cast<int64_t>(tile.n) * P::BN;
  const int NS = static_cast<int>((p.K + 63) / 64);
  RingArgs g = {};
  g.x[0] = p.h; g.ldx = p.ldh; g.W[0] = p.W + v0 * p.K; g.K[0] = p.K; g.n_seg = 1; g.T = p.T; g.N = cols;
  f32x4 acc[P::NI][P::NJ];
  NtOp<P, false> op;
  op.init(g, m0, n0, 0, NS);
  ring_run<P, false>(acc, op, NS, smem, wm0, wn0);
  const int lane = opaque_int(threadIdx.x & 63), r = lane & 15, q = lane >> 4;
  const int64_t mw = m0 + wm0, nw = n0 + wn0;  // of this wave's block (columns within the piece)
  if (nw >= cols) return;
  const int left = static_cast<int>(min<int64_t>(P::WN, cols - nw));
  if constexpr (MODE == kStats) {
    const int64_t block = (v0 + nw) / P::WN;
#pragma unroll
    for (int j = 0; j < P::NJ; ++j) {
      const int64_t m = mw + j * 16 + r;
      const int64_t at = p.target[min<int64_t>(m, p.T - 1)] - v0 - nw;  // the target's column within the block
      const int tc = at >= 0 && at < left ? static_cast<int>(at) : -1;
      float top = -__builtin_inff(), mine = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < P::NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = i * 16 + q * 4 + e;
          if (c == tc) mine = acc[i][j][e];
          else if (c < left) top = fmaxf(top, acc[i][j][e]);
        }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float base = top > -__builtin_inff() ? top : 0.f;
#pragma unroll
      for (int i = 0; i < P::NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = i * 16 + q * 4 + e;
          if (c != tc && c < left) sum += exp_of(acc[i][j][e] - base);
        }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (m < p.T) {
        if (q == 0) {
          p.stat_m[block * p.T + m] = top;
          p.stat_s[block * p.T + m] = sum;
        }
        if (tc >= 0 && (tc & 15) >> 2 == q) p.tlogit[m] = mine;
      }
    }
  } else {
    BlockOut<P::WM, P::WN> out{smem + wave * P::WM * P::WN * 2};
#pragma unroll
    for (int j = 0; j < P::NJ; ++j) {
      const int64_t m = min<int64_t>(mw + j * 16 + r, p.T - 1);
      const int64_t at = p.target[m] - v0 - nw;
      const int tc = at >= 0 && at < left ? static_cast<int>(at) : -1;
      const float lse = p.wlse[m];
#pragma unroll
      for (int i = 0; i < P::NI; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = i * 16 + q * 4 + e;
          v[e] = c != tc && c < left ? exp_of(acc[i][j][e] - lse) : 0.f;
        }
        out.put(j * 16 + r, i * 16 + q * 4, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // (zeros up to the next 8 columns: a copied chunk is whole)
    if (mw < p.T)
      out.store(p.share + mw * p.piece + nw, p.piece, static_cast<int>(min<int64_t>(P::WM, p.T - mw)), (left + 7) / 8 * 8);
  }
}

// 16 tokens per workgroup, 16 threads each: the blocks' statistics joined. A token without a target (one outside the
// vocabulary) has loss 0 and, by rest < 0, no gradient.
__global__ __launch_bounds__(256) void lse_kernel(VocabLoss p, int64_t blocks) {
  __shared__ float sm[16][17], ss[16][17];
  const int lt = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 16 + lt, tt = min<int64_t>(t, p.T - 1);
  float top = -__builtin_inff(), sum = 0.f;
  for (int64_t b = part; b < blocks; b += 16) {
    const float m = p.stat_m[b * p.T + tt], s = p.stat_s[b * p.T + tt];
    const float now = fmaxf(top, m);
    const float base = now > -__builtin_inff() ? now : 0.f;
    sum = sum * exp_of(top - base) + s * exp_of(m - base);
    top = now;
  }
  sm[part][lt] = top;
  ss[part][lt] = sum;
  __syncthreads();
  if (part != 0 || t >= p.T) return;
  const int64_t target = p.target[t];
  const bool some = target >= 0 && target < p.V;
  const float mine = some ? p.tlogit[t] : -__builtin_inff();
  float all = mine;
  for (int i = 0; i < 16; ++i) all = fmaxf(all, sm[i][lt]);
  const float base = all > -__builtin_inff() ? all : 0.f;
  float others = 0.f;
  for (int i = 0; i < 16; ++i) others += ss[i][lt] * exp_of(sm[i][lt] - base);
  const float total = others + exp_of(mine - base);
  const float lse = base + __builtin_logf(total);
  if (p.lse != nullptr) p.lse[t] = lse;
  // loss = log(total) - (l_target - base), which loses nothing where the target is the largest
  if (p.loss != nullptr) p.loss[t] = some ? (mine == base ? log1pf(others) : lse - mine) : 0.f;
  p.wlse[t] = lse;
  p.rest[t] = some ? others / total : -1.f;
}

// acc += p W over a piece: grid (tiles, splits), a split's stages summed into its own [T, K].
template <class P>
__global__ __launch_bounds__(P::THREADS, P::OCC) void dh_kernel(VocabLoss p, int64_t v0, int64_t cols, int ks, bool first,
                                                                int mt, int nt) {
  __shared__ __attribute__((aligned(1024))) char smem[P::SLOTS * P::SLOT_BYTES];
  const RingTile tile(xcd_remap(blockIdx.x, mt * nt), mt, nt, P::GROUP_M);
  const int wave = ring_wave();
  const int wm0 = (wave % P::WAVES_M) * P::WM, wn0 = (wave / P::WAVES_M) * P::WN;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM, n0 = static_cast<int64_t>(tile.n) * P::BN;
  const int NS = static_cast<int>((cols + 63) / 64), s_lo = static_cast<int>(blockIdx.y) * ks, s_hi = min(NS, s_lo + ks);
  float* mine = p.acc + static_cast<int64_t>(blockIdx.y) * p.T * p.K;
  if (s_lo >= s_hi && !first) return;
  const uint16_t *x = p.share, *W = p.W + v0 * p.K;
  NnOp<P, 1, 0> op;
  op.init(&x, p.piece, &W, &cols, p.T, p.K, m0, n0, s_lo, s_hi);
  f32x4 acc[P::NI][P::NJ];
  ring_run<P, true>(acc, op, max(0, s_hi - s_lo), smem, wm0, wn0);
  store_part<P>(acc, mine, p.K, m0 + wm0, n0 + wn0, p.T, p.K, !first);
}

// dh = dloss (sum of the splits - (1 - p_target) W_target); 4 columns per thread.
__global__ __launch_bounds__(256) void dh_finish_kernel(VocabLoss p, int S) {
  const int64_t quads = p.K / 4, idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= p.T * quads) return;
  const int64_t t = idx / quads, k = (idx - t * quads) * 4;
  const float rest = p.rest[t];
  uint2 w = {0u, 0u};
  if (!(rest == -1.f)) {  // (a NaN goes on)
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int z = 0; z < S; ++z) v += *reinterpret_cast<const f32x4*>(p.acc + (z * p.T + t) * p.K + k);
    const uint2 wt = *reinterpret_cast<const uint2*>(p.W + p.target[t] * p.K + k);
    const float g = p.dloss != nullptr ? p.dloss[t] : 1.f;
    const float o[4] = {g * (v[0] - rest * __uint_as_float(wt.x << 16)), g * (v[1] - rest * __uint_as_float(wt.x & 0xffff0000u)),
                        g * (v[2] - rest * __uint_as_float(wt.y << 16)), g * (v[3] - rest * __uint_as_float(wt.y & 0xffff0000u))};
    w = uint2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
  }
  uint16_t* dst = p.dh + t * p.lddh + k;
  if (reinterpret_cast<uintptr_t>(dst) % 8 == 0) {
    *reinterpret_cast<uint2*>(dst) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) dst[e] = static_cast<uint16_t>((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
  }
}

int loss_cus() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  return n;
}

template <class P, int MODE>
hipError_t launch_logits(const VocabLoss& p, int64_t v0, int64_t cols, hipStream_t s) {
  const int mt = static_cast<int>((p.T + P::BM - 1) / P::BM), nt = static_cast<int>((cols + P::BN - 1) / P::BN);
  hipLaunchKernelGGL((logits_kernel<P, MODE>), dim3(static_cast<unsigned>(mt * nt)), dim3(P::THREADS), 0, s, p, v0, cols,
                     mt, nt);
  return hipGetLastError();
}

template <class P>
hipError_t launch_dh(const VocabLoss& p, int64_t v0, int64_t cols, int S, int ks, hipStream_t s) {
  const int mt = static_cast<int>((p.T + P::BM - 1) / P::BM), nt = static_cast<int>((p.K + P::BN - 1) / P::BN);
  hipLaunchKernelGGL(dh_kernel<P>, dim3(static_cast<unsigned>(mt * nt), static_cast<unsigned>(S)), dim3(P::THREADS), 0, s, p,
                     v0, cols, ks, v0 == 0, mt, nt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_vocab_loss(const VocabLoss& p, hipStream_t s) {
  const int cus = loss_cus();
  const bool small = small_tile(p.T, p.V, cus);
  hipError_t e = small ? launch_logits<Ring128, kStats>(p, 0, p.V, s) : launch_logits<Ring256, kStats>(p, 0, p.V, s);
  if (e != hipSuccess) return e;
  const int64_t wn = small ? Ring128::WN : Ring256::WN;
  hipLaunchKernelGGL(lse_kernel, dim3(static_cast<unsigned>((p.T + 15) / 16)), dim3(256), 0, s, p, (p.V + wn - 1) / wn);
  e = hipGetLastError();
  if (e != hipSuccess || p.dh == nullptr) return e;
  int S, ks;
  loss_splits(p.T, p.K, (p.piece + 63) / 64, &S, &ks);
  const bool narrow = S > 1 || small_tile(p.T, p.K, cus);
  for (int64_t v0 = 0; v0 < p.V; v0 += p.piece) {
    const int64_t cols = p.piece < p.V - v0 ? p.piece : p.V - v0;
    e = small ? launch_logits<Ring128, kShare>(p, v0, cols, s) : launch_logits<Ring256, kShare>(p, v0, cols, s);
    if (e != hipSuccess) return e;
    e = narrow ? launch_dh<Ring128>(p, v0, cols, S, ks, s) : launch_dh<Ring256>(p, v0, cols, S, ks, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(dh_finish_kernel, dim3(static_cast<unsigned>((p.T * (p.K / 4) + 255) / 256)), dim3(256), 0, s, p, S);
  return hipGetLastError();
}

}  // namespace lora
