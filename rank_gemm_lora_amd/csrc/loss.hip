// Softmax cross entropy over a vocabulary straight from hidden states h [T, K] and the output weight W [V, K], bf16:
//
//   l = h W^T (never kept),  lse = log sum exp(l),  loss = lse - l[target]
//   dh = dloss (sum over v != target of p_v W_v  -  (1 - p_target) W_target),  p = exp(l - lse)
//
// One pass over the logits, though lse is known only behind it: a block of columns leaves its exponentials relative to a
// power of two 2^c of its own, c = ceil(log2 of the token's largest exponential in the block), so that none overflows and
// the largest lies in (1/2, 1]. Bringing a block to the largest c of its token is then a subtraction from bf16 exponents,
// exact (what falls below the smallest number is lost, at most 2^-126 of the largest term), which dh_kernel makes on the
// fragments it multiplies. Forming p anew from a second pass over the logits, with lse known, took 9.8 ms against 7.1
// (4096 tokens, 4096 inputs, 128017 words: logits 3.6 ms, 1.20 PFLOP/s, dh 3.7, 1.16; the matrix pipes bound both).
//
// The target is held apart from the other tokens throughout: p_target - 1 is minus the others' sum, where the difference
// of a share rounded to bf16 and one would lose what a sure token has left.
//
//   logits_kernel    l of a piece of the vocabulary in the accumulators; c and the sum per token and block, and the shares
//                    2^(l log2 e - c) in bf16 (for the loss alone: no shares)
//   piece_kernel     the token's largest c so far, and every block's distance from it; in the end lse, loss, 1 - p_target
//   dh_kernel        sums over the piece of shares . W, fp32; where a piece is not the first, added to those before it
//   dh_join_kernel   the parts' sum, the target's part, dloss, one rounding (a whole tile of a single piece does so itself)
#include "common.hpp"
#include "loss.hpp"
#include "ring_ops.hpp"

namespace lora {
namespace {

constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.69314718055995f;
constexpr float kNoTerm = -1e37f;  // c of a block without terms: further below any other than exponents reach
__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// l of the columns v0 .. v0 + cols of the vocabulary.
template <class P, bool SHARE>
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
  const int64_t block = (v0 + nw) / P::WN;
  BlockOut<P::WM, P::WN> out{smem + wave * P::WM * P::WN * 2};
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
    const float c2 = fmaxf(__builtin_ceilf(top * kLog2e), kNoTerm);
#pragma unroll
    for (int i = 0; i < P::NI; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = i * 16 + q * 4 + e;
        v[e] = c != tc && c < left ? exp2_of(fmaf(acc[i][j][e], kLog2e, -c2)) : 0.f;
        sum += v[e];
      }
      if (SHARE) out.put(j * 16 + r, i * 16 + q * 4, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (m < p.T) {
      if (q == 0) {
        p.ref[block * p.T + m] = c2;
        p.sum[block * p.T + m] = sum;
      }
      if (tc >= 0 && (tc & 15) >> 2 == q) p.tlogit[m] = mine;
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // (zeros up to the next 8 columns: a copied chunk is whole)
  if (SHARE && mw < p.T)
    out.store(p.share + mw * p.piece + nw, p.piece, static_cast<int>(min<int64_t>(P::WM, p.T - mw)), (left + 7) / 8 * 8);
}

// Where dh_kernel's lane (r, ..) finds the shifts of its tokens j * 16 + r of a wave's WM, side by side.
__device__ __forceinline__ int64_t shift_at(int64_t t, int wm) {
  const int64_t base = t / wm * wm;
  const int in = static_cast<int>(t - base);
  return base + (in & 15) * (wm / 16) + (in >> 4);
}

// 16 tokens per workgroup (64 bytes of each block's row), 64 threads each: the largest c of the piece's blocks [b0, b1) and
// before, every block's distance from it where there are shares; behind the last piece (all its blocks: [0, b1)) lse and
// what comes of it. A token without a target (one outside the vocabulary) has loss 0 and, by rest < 0, no gradient.
// Bound by the reads' latency.
template <bool SHARE, bool LAST>
__global__ __launch_bounds__(1024) void piece_kernel(VocabLoss p, int64_t b0, int64_t b1, int wm, int64_t ld) {
  __shared__ float s[2][16][16];
  const int lt = threadIdx.x & 15, part = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 16 + lt, tt = min<int64_t>(t, p.T - 1);
  auto join = [&](float v, int which, auto op) {  // of the 64 threads of a token, in one order
    v = op(v, __shfl_xor(v, 16));
    v = op(v, __shfl_xor(v, 32));
    if ((part & 3) == 0) s[which][wave][lt] = v;
    __syncthreads();
    v = s[which][0][lt];
#pragma unroll
    for (int w = 1; w < 16; ++w) v = op(v, s[which][w][lt]);
    return v;
  };
  const float before = b0 == 0 ? kNoTerm : p.top[tt];
  float top = before;
#pragma unroll 4
  for (int64_t b = b0 + part; b < b1; b += 64) top = fmaxf(top, p.ref[b * p.T + tt]);
  top = join(top, 0, [](float x, float y) { return fmaxf(x, y); });
  if (SHARE && t < p.T) {
    if (part == 0) {
      p.top[t] = top;
      p.fade[t] = exp2_of(before - top);
    }
    const int64_t at = shift_at(t, wm);
#pragma unroll 4
    for (int64_t b = b0 + part; b < b1; b += 64)
      p.shift[(b - b0) * ld + at] = static_cast<uint8_t>(fminf(top - p.ref[b * p.T + t], 255.f));
  }
  if (!LAST) return;
  float others = 0.f;  // relative to 2^top
#pragma unroll 4
  for (int64_t b = part; b < b1; b += 64) others += p.sum[b * p.T + tt] * exp2_of(p.ref[b * p.T + tt] - top);
  others = join(others, 1, [](float x, float y) { return x + y; });
  if (part != 0 || t >= p.T) return;
  const int64_t target = p.target[t];
  const bool some = target >= 0 && target < p.V;
  const float mine = some ? p.tlogit[t] : 0.f;
  // with the target: relative to 2^base, the larger of the two
  const float mine2 = some ? mine * kLog2e : kNoTerm, base = fmaxf(top, __builtin_ceilf(mine2));
  const float far = others * exp2_of(top - base), own = some ? exp2_of(mine2 - base) : 0.f, total = far + own;
  const float lse = base * kLn2 + __builtin_logf(total);
  if (p.lse != nullptr) p.lse[t] = lse;
  // loss = log(1 + the others relative to the target), which loses nothing where the target is far ahead, while that exists
  if (p.loss != nullptr) {
    const float ahead = mine2 - top;
    p.loss[t] = !some ? 0.f : (ahead > -10.f ? log1pf(others * exp2_of(-ahead)) : lse - mine);
  }
  p.rest[t] = some ? far / total : -1.f;
  p.scale[t] = exp2_of(top - base) / total;
}

// The shares of a stage's block are brought to the token's largest c: 128 per step off a bf16's bits, kept at zero.
template <class P>
struct ShareOp : NnOp<P, 1, 0> {
  const uint8_t* sh;  // this lane's first byte of the piece's first block
  int64_t ld;
  int psh;            // a block has 1 << psh stages
  uint32_t now[P::NJ / 4], then[P::NJ / 4];
  __device__ __forceinline__ void fetch(int t) {
    const int s = this->lo + t;
    const uint32_t* at = reinterpret_cast<const uint32_t*>(sh + static_cast<int64_t>((s < this->hi ? s : this->lo) >> psh) * ld);
#pragma unroll
    for (int w = 0; w < P::NJ / 4; ++w) then[w] = at[w];
  }
  __device__ __forceinline__ void next() {
#pragma unroll
    for (int w = 0; w < P::NJ / 4; ++w) now[w] = then[w];
  }
  __device__ __forceinline__ void touch(bf16x8& b, int j) const {
    const uint32_t by = (now[j / 4] >> (8 * (j % 4)) & 0xffu) << 7;
    const u16x2 off = __builtin_bit_cast(u16x2, by | by << 16);
    u32x4 v = __builtin_bit_cast(u32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = v[e];  // (a bit_cast of the element itself reads the vector's first)
      v[e] = __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, w), off));
    }
    b = __builtin_bit_cast(bf16x8, v);
  }
};

// dh of a wave's block (NJ blocks of 16 tokens from m0 on): dloss (scale . sum - rest . W_target).
template <class P, int NJ>
__device__ __forceinline__ void store_dh(const f32x4 (&acc)[P::NI][NJ], const VocabLoss& p, int64_t m0, int64_t n0,
                                         char* smem) {
  const int lane = opaque_int(threadIdx.x & 63), r = lane & 15, q = lane >> 4;
  BlockOut<NJ * 16, P::WN> out{smem + ring_wave() * NJ * 16 * P::WN * 2};
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t m = min<int64_t>(m0 + j * 16 + r, p.T - 1);
    const float rest = p.rest[m], g = p.dloss != nullptr ? p.dloss[m] : 1.f, gs = g * p.scale[m], gr = g * rest;
    const bool none = rest == -1.f;  // (a NaN goes on)
    const uint16_t* wt = p.W + (none ? 0 : p.target[m] * p.K) + n0;
#pragma unroll
    for (int i = 0; i < P::NI; ++i) {
      const int c = i * 16 + q * 4;
      // (K is a multiple of 8: four columns exist together)
      const uint2 w = !none && n0 + c < p.K ? *reinterpret_cast<const uint2*>(wt + c) : uint2{0u, 0u};
      const float o[4] = {gs * acc[i][j][0] - gr * __uint_as_float(w.x << 16),
                          gs * acc[i][j][1] - gr * __uint_as_float(w.x & 0xffff0000u),
                          gs * acc[i][j][2] - gr * __uint_as_float(w.y << 16),
                          gs * acc[i][j][3] - gr * __uint_as_float(w.y & 0xffff0000u)};
      out.put(j * 16 + r, c, none ? 0u : pack_bf16x2(o[0], o[1]), none ? 0u : pack_bf16x2(o[2], o[3]));
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if (m0 < p.T && n0 < p.K)
    out.store(p.dh + m0 * p.lddh + n0, p.lddh, static_cast<int>(min<int64_t>(NJ * 16, p.T - m0)),
              static_cast<int>(min<int64_t>(P::WN, p.K - n0)));
}

// The sums over the piece's columns v0 .. v0 + cols; bw: columns per block of shares.
template <class P>
__global__ __launch_bounds__(P::THREADS, P::OCC) void dh_kernel(VocabLoss p, int64_t v0, int64_t cols, int full, int S,
                                                                int ks, int bw, int mt, int nt) {
  __shared__ __attribute__((aligned(1024))) char smem[P::SLOTS * P::SLOT_BYTES];
  const int NS = static_cast<int>((cols + 63) / 64);
  const RingWork work(blockIdx.x, full, mt * nt, S, ks, NS);
  const RingTile tile(work.tile, mt, nt, P::GROUP_M);
  const int wave = ring_wave();
  const int wm0 = (wave % P::WAVES_M) * P::WM, wn0 = (wave / P::WAVES_M) * P::WN;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM, n0 = static_cast<int64_t>(tile.n) * P::BN;
  const int unit = work.unit < 0 && p.piece < p.V ? (mt * nt - full) * S + work.tile : work.unit;
  const int ns = max(0, work.hi - work.lo);  // (a last piece may have none for the last parts; theirs still fade)
  const uint16_t *x = p.share, *W = p.W + v0 * p.K;
  f32x4 acc[P::NI][P::NJ];
  ShareOp<P> op;
  op.init(&x, p.piece, &W, &cols, p.T, p.K, m0, n0, work.lo, work.hi);
  op.ld = (p.T + 255) / 256 * 256;
  op.psh = bw / 128;
  op.sh = p.shift + m0 + wm0 + (threadIdx.x & 15) * P::NJ;
  ring_run<P, true, false, true>(acc, op, ns, smem, wm0, wn0);
  const VocabLoss a = late_args<VocabLoss>();
  if (unit < 0) {
    store_dh<P, P::NJ>(acc, a, m0 + wm0, n0 + wn0, smem);
    return;
  }
  const int lane = opaque_int(threadIdx.x & 63), r = lane & 15;
#pragma unroll
  for (int j = 0; j < P::NJ; ++j) {
    const float f = v0 == 0 ? 0.f : a.fade[min<int64_t>(m0 + wm0 + j * 16 + r, a.T - 1)];
#pragma unroll
    for (int i = 0; i < P::NI; ++i) {
      f32x4* at = part_at<P>(a.part, unit, j, i) + lane;
      if (v0 == 0) *at = acc[i][j];
      else *at = *at * f + acc[i][j];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The tiles with sums in memory: grid (tiles, column blocks of a wave). All of them behind several pieces, else the cut ones.
template <class P>
__global__ __launch_bounds__(P::THREADS) void dh_join_kernel(VocabLoss p, int full, int S, int mt, int nt) {
  __shared__ __attribute__((aligned(16))) char smem[P::WAVES * 16 * P::WN * 2];
  const int L = (p.piece < p.V ? 0 : full) + static_cast<int>(blockIdx.x);
  const RingTile tile(L, mt, nt, P::GROUP_M);
  const int wave = ring_wave(), j = blockIdx.y;
  const int64_t m0 = static_cast<int64_t>(tile.m) * P::BM + (wave % P::WAVES_M) * P::WM + j * 16;
  const int64_t n0 = static_cast<int64_t>(tile.n) * P::BN + (wave / P::WAVES_M) * P::WN;
  f32x4 acc[P::NI][1];
  if (L < full) sum_parts<P>(acc, p.part, (mt * nt - full) * S + L, 1, j);
  else sum_parts<P>(acc, p.part, L - full, S, j);
  store_dh<P, 1>(acc, p, m0, n0, smem);
}

template <class P>
hipError_t launch_logits(const VocabLoss& p, int64_t v0, int64_t cols, bool share, hipStream_t s) {
  const int mt = static_cast<int>((p.T + P::BM - 1) / P::BM), nt = static_cast<int>((cols + P::BN - 1) / P::BN);
  const dim3 grid(static_cast<unsigned>(mt * nt)), block(P::THREADS);
  if (share) hipLaunchKernelGGL((logits_kernel<P, true>), grid, block, 0, s, p, v0, cols, mt, nt);
  else hipLaunchKernelGGL((logits_kernel<P, false>), grid, block, 0, s, p, v0, cols, mt, nt);
  return hipGetLastError();
}

template <class P>
hipError_t launch_dh(const VocabLoss& p, int64_t v0, int64_t cols, const RingPlan& r, int bw, bool last, hipStream_t s) {
  const int mt = static_cast<int>((p.T + P::BM - 1) / P::BM), nt = static_cast<int>((p.K + P::BN - 1) / P::BN);
  const int full = static_cast<int>(r.full), rem = mt * nt - full;
  hipLaunchKernelGGL(dh_kernel<P>, dim3(static_cast<unsigned>(full + rem * r.S)), dim3(P::THREADS), 0, s, p, v0, cols, full,
                     r.S, r.ks, bw, mt, nt);
  const int join = p.piece < p.V ? mt * nt : rem;
  if (last && join > 0)
    hipLaunchKernelGGL(dh_join_kernel<P>, dim3(static_cast<unsigned>(join), P::NJ), dim3(P::THREADS), 0, s, p, full, r.S, mt,
                       nt);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_vocab_loss(const VocabLoss& p, hipStream_t s) {
  const unsigned tok16 = static_cast<unsigned>((p.T + 15) / 16);
  const bool grad = p.dh != nullptr;
  const int64_t piece = grad ? p.piece : p.V;
  // (The estimate may count a cut of the last round, which the logits do not make: 13 of 560 sizes tried take a tile that it
  // puts 2 to 18% behind the other without cuts, 512 tokens of 5120 inputs over 50257 words the smaller one.)
  const bool big = ring_plan(p.T, piece < p.V ? piece : p.V, (p.K + 63) / 64).big;
  const int bw = big ? Ring256::WN : Ring128::WN;
  const RingPlan r = loss_plan(p.T, p.K, p.V);
  const int wm = r.big ? Ring256::WM : Ring128::WM;
  for (int64_t v0 = 0; v0 < p.V; v0 += piece) {
    const int64_t cols = piece < p.V - v0 ? piece : p.V - v0;
    const bool last = v0 + cols >= p.V;
    hipError_t e = big ? launch_logits<Ring256>(p, v0, cols, grad, s) : launch_logits<Ring128>(p, v0, cols, grad, s);
    if (e != hipSuccess) return e;
    const int64_t b0 = v0 / bw, b1 = (v0 + cols + bw - 1) / bw, ld = shift_ld(p.T);
    if (!grad) hipLaunchKernelGGL((piece_kernel<false, true>), dim3(tok16), dim3(1024), 0, s, p, b0, b1, wm, ld);
    else if (last) hipLaunchKernelGGL((piece_kernel<true, true>), dim3(tok16), dim3(1024), 0, s, p, b0, b1, wm, ld);
    else hipLaunchKernelGGL((piece_kernel<true, false>), dim3(tok16), dim3(1024), 0, s, p, b0, b1, wm, ld);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!grad) continue;
    e = r.big ? launch_dh<Ring256>(p, v0, cols, r, bw, last, s) : launch_dh<Ring128>(p, v0, cols, r, bw, last, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lora
