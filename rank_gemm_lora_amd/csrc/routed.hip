// A linear layer whose tokens take their adapters from a pool (multi-adapter serving and training on
// one frozen base weight):
//
//   y[t] = x[t].W^T + b + s_t . (x[t].A_a^T).B_a^T,   a = token_adapter[t],  s_t = scales[a] . token_scale[t]
//
// (SGLang PR #43501, Modifications: the scale multiplies the rank-wide intermediate and is honoured per
// request; here the adapter is per request too.) The rank-wide products run here; the base product with
// the second adapter product in its accumulator is gemm.hip's hot kernel.
#include "routed.hpp"

#include "common.hpp"

namespace lora {
namespace {

constexpr uint32_t kOutOfRange = 0x80000000u;  // a buffer offset past every range: the load returns zeros

// The adapter of token t and its scale; -1 (the base output) past the last token, for an index outside
// the pool, a zero scale or a rank of zero.
__device__ __forceinline__ int route(const Routing& rt, int64_t t, int64_t T, float& s) {
  s = 0.f;
  if (t >= T || rt.n_adapters == 0) return -1;
  const int a = rt.token_adapter[t];
  if (static_cast<uint32_t>(a) >= static_cast<uint32_t>(rt.n_adapters)) return -1;
  s = rt.scales[a];
  if (rt.token_scale != nullptr) s *= rt.token_scale[t];
  if (s == 0.f || (rt.ranks != nullptr && rt.ranks[a] <= 0)) return -1;
  return a;
}

// ---------------------------------------------------------------------------
// Rank-wide producer. Workgroup: one block of 16 tokens, 64 ranks, every gridDim.z-th of the block's
// distinct adapters; 8 waves split K and add their sums through LDS in wave order. Operands go from
// global memory straight into MFMA fragments (lane (r, q): 8 consecutive k of adapter row r / token r);
// all 16 tokens are multiplied, and the rows of the adapter's own tokens are kept.
constexpr int kDownWaves = 8;

__global__ __launch_bounds__(64 * kDownWaves) void routed_down_kernel(RoutedDown p) {
  __shared__ f32x4 red[kDownWaves][4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRouteBlock;
  const int rows = static_cast<int>(min<int64_t>(kRouteBlock, p.T - t0));
  float s;
  const int id = route(p.rt, t0 + r, p.T, s);
  uint32_t todo = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(id >= 0)) & 0xffffu;
  if (wave == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    if (q == 0 && r < rows) p.eid[t0 + r] = id;
    const int first = __builtin_amdgcn_readfirstlane(id);
    const bool same = __builtin_amdgcn_ballot_w64(r < rows && id != first) == 0;
    if (lane == 0) p.blk[blockIdx.x] = same ? first : -2;
  }
  const int q0 = blockIdx.y * 64;
  const int64_t kper = ((p.K + kDownWaves - 1) / kDownWaves + 31) / 32 * 32;
  const int64_t k_lo = wave * kper, k_hi = min<int64_t>(p.K, k_lo + kper);
  const uint32_t ldx_b = static_cast<uint32_t>(p.ldx * 2), lda_b = static_cast<uint32_t>(p.K * 2);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + t0 * p.ldx, static_cast<uint32_t>(rows) * ldx_b);
  int nth = 0;
  while (todo != 0) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    todo &= ~static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(id == a));
    if (nth++ % static_cast<int>(gridDim.z) != static_cast<int>(blockIdx.z)) continue;
    const int rank =
        p.rt.ranks != nullptr ? __builtin_amdgcn_readfirstlane((min(p.rt.ranks[a], p.rt.rank) + 7) & ~7) : p.rt.rank;
    const int rows_a = max(0, min(64, rank - q0));
    const int nrb = (rows_a + 15) / 16;
    const __amdgpu_buffer_rsrc_t ar =
        make_rsrc(p.A + (static_cast<int64_t>(a) * p.rt.rank + q0) * p.K, static_cast<uint32_t>(rows_a) * lda_b);
    f32x4 acc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t kg = k_lo; kg < k_hi; kg += 128) {
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        const int64_t k = kg + 32 * st + 8 * q;
        const bool in = k < k_hi;
        const bf16x8 xf = __builtin_bit_cast(
            bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                        xr, in ? static_cast<uint32_t>(r) * ldx_b + static_cast<uint32_t>(k * 2) : kOutOfRange, 0, 0));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (b >= nrb) continue;
          const uint32_t off = static_cast<uint32_t>(b * 16 + r) * lda_b + static_cast<uint32_t>(k * 2);
          const bf16x8 af = __builtin_bit_cast(
              bf16x8, __builtin_amdgcn_raw_buffer_load_b128(ar, in ? off : kOutOfRange, 0, 0));
          acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, xf, acc[b], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) red[wave][b][lane] = acc[b];
    __syncthreads();
    // thread (b, lane): ranks q0 + 16 b + 4 q .. +3 of token t0 + r
    if (wave < 4 && id == a) {
      f32x4 v = red[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kDownWaves; ++w) v += red[w][wave][lane];
      v *= s;
      uint2 hi;
      hi.x = pack_bf16x2(v[0], v[1]);
      hi.y = pack_bf16x2(v[2], v[3]);
      const int64_t at = (t0 + r) * p.ldt + q0 + wave * 16 + 4 * q;
      *reinterpret_cast<uint2*>(p.hi + at) = hi;
      if (p.lo != nullptr) {
        float l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t h = e < 2 ? hi.x : hi.y;
          const float hf = __uint_as_float(e & 1 ? h & 0xffff0000u : h << 16);
          l[e] = __builtin_isfinite(hf) ? v[e] - hf : 0.f;
        }
        *reinterpret_cast<uint2*>(p.lo + at) = uint2{pack_bf16x2(l[0], l[1]), pack_bf16x2(l[2], l[3])};
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Tokens sorted by adapter: workgroup a finds its adapter's tokens. The 16 waves take consecutive
// stretches of the tokens; a first pass counts (tokens of lower adapters give the start, wave counts the
// places), a second writes. No atomics: the order is the tokens' own.
__global__ __launch_bounds__(1024) void route_plan_kernel(RoutePlan p) {
  __shared__ int below[16], mine[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int a = blockIdx.x;
  const int64_t per = ((p.T + 15) / 16 + 63) / 64 * 64;
  const int64_t lo = wave * per, hi = min<int64_t>(p.T, lo + per);
  int nb = 0, nm = 0;
  for (int64_t t = lo; t < hi; t += 64) {
    const int id = t + lane < hi ? p.eid[t + lane] : -1;
    nb += __popcll(__builtin_amdgcn_ballot_w64(id >= 0 && id < a));
    nm += __popcll(__builtin_amdgcn_ballot_w64(id == a));
  }
  if (lane == 0) below[wave] = nb, mine[wave] = nm;
  __syncthreads();
  int start = 0, count = 0, at = 0;
  for (int w = 0; w < 16; ++w) {
    start += below[w];
    if (w < wave) at += mine[w];
    count += mine[w];
  }
  at += start;
  for (int64_t t = lo; t < hi; t += 64) {
    const int id = t + lane < hi ? p.eid[t + lane] : -1;
    const uint64_t m = __builtin_amdgcn_ballot_w64(id == a);
    if (id == a) p.perm[at + __popcll(m & ((1ull << lane) - 1))] = static_cast<int32_t>(t + lane);
    at += __popcll(m);
  }
  const int end = start + count, c = p.chunk;
  if (threadIdx.x == 0) {
    p.off[a] = start;
    if (a == p.n_adapters - 1) p.off[a + 1] = end;
  }
  // items a + j for the chunks j from the one that holds `start` to the one that holds `end`: the next
  // adapter's first item follows, so the items of all adapters fill their table without a gap
  const int j0 = start / c, j1 = end / c;
  const bool several = count > 0 && (end - 1) / c != j0;
  for (int j = j0 + threadIdx.x; j <= j1; j += 1024) {
    RouteItem it;
    it.adapter = a;
    it.lo = max(start, j * c);
    it.hi = max(it.lo, min(end, (j + 1) * c));
    it.part = several ? 2 * j + (j == j0 ? 1 : 0) : -1;
    p.items[a + j] = it;
  }
  if (a == p.n_adapters - 1) {  // places behind the last item (tokens without an adapter)
    for (int64_t z = static_cast<int64_t>(a) + j1 + 1 + threadIdx.x; z < p.n_items; z += 1024) p.items[z] = RouteItem{0, 0, 0, -1};
  }
}

// ---------------------------------------------------------------------------
// Contraction over an adapter's tokens: grid (256 columns of P, item, 64 ranks), tokens in steps of 64
// gathered through perm. Both operands are token-major and are transposed on the way to LDS (a thread
// turns 8 tokens x 8 columns in registers); lane (r, q) of the MFMA then reads 8 consecutive tokens of
// one column. The rank-wide operand is hi + lo, both multiplied into the same fp32 sum: gradients keep
// about 16 bits of it.
__device__ __forceinline__ int tsw(int row, int piece) { return row * 8 + (piece ^ ((row ^ (row >> 3)) & 7)); }

__device__ __forceinline__ void transpose_to_lds(char* dst, const u32x4 (&v)[8], int c, int g) {
#pragma unroll
  for (int ii = 0; ii < 8; ++ii) {  // row 8 c + ii: tokens 8 g .. 8 g + 7
    u32x4 o;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const uint32_t lo = v[2 * m][ii >> 1], hi = v[2 * m + 1][ii >> 1];
      o[m] = (ii & 1) ? ((lo >> 16) | (hi & 0xffff0000u)) : ((lo & 0xffffu) | (hi << 16));
    }
    *reinterpret_cast<u32x4*>(dst + tsw(8 * c + ii, g) * 16) = o;
  }
}

struct ContractArgs {
  const bf16_bits* P; int64_t ldp, M;
  const bf16_bits *hi, *lo; int64_t ldt;
  int rank;
  const int32_t* perm;
  const RouteItem* items;
  float *part, *out;
};

template <bool TRANSPOSE>
__global__ __launch_bounds__(256, 2) void routed_tn_kernel(ContractArgs p) {
  __shared__ __attribute__((aligned(256))) char pb[kRtI * kRtT * 2];
  __shared__ __attribute__((aligned(256))) char qb[2][kRtJ * kRtT * 2];
  __shared__ int32_t tok[kRouteMaxChunk];
  const RouteItem it = p.items[blockIdx.y];
  const int cnt = it.hi - it.lo;
  if (cnt <= 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kRtI;
  const int j0 = blockIdx.z * kRtJ;
  const int nj = (min(kRtJ, p.rank - j0) + 15) / 16;
  for (int i = threadIdx.x; i < cnt; i += 256) tok[i] = p.perm[it.lo + i];
  __syncthreads();
  const int nsteps = (cnt + kRtT - 1) / kRtT;
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;  // P: columns i0 + 8 c .. +7, tokens 8 g .. +7 of the step
  const bool pcol = i0 + 8 * c < p.M;
  const bf16_bits* pcolp = p.P + i0 + 8 * c;
  const int qc = threadIdx.x & 7, qg = (threadIdx.x >> 3) & 7;  // threads < 128: hi (wave 0), lo (wave 1)
  const bf16_bits* qcolp = (wave == 0 ? p.hi : p.lo) + j0 + 8 * qc;
  u32x4 pv[8], qv[8];
  auto load = [&](int step) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = step * kRtT + 8 * g + e;
      pv[e] = u32x4{0u, 0u, 0u, 0u};
      if (pcol && i < cnt) pv[e] = *reinterpret_cast<const u32x4*>(pcolp + tok[i] * p.ldp);
    }
    if (wave < 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = step * kRtT + 8 * qg + e;
        qv[e] = u32x4{0u, 0u, 0u, 0u};
        if (i < cnt) qv[e] = *reinterpret_cast<const u32x4*>(qcolp + tok[i] * p.ldt);
      }
    }
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int ib = 0; ib < 4; ++ib)
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) acc[ib][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
  load(0);
  for (int step = 0; step < nsteps; ++step) {
    transpose_to_lds(pb, pv, c, g);
    if (wave < 2) transpose_to_lds(qb[wave], qv, qc, qg);
    __syncthreads();
    if (step + 1 < nsteps) load(step + 1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8 af[4];
#pragma unroll
      for (int ib = 0; ib < 4; ++ib)
        af[ib] = *reinterpret_cast<const bf16x8*>(pb + tsw(wave * 64 + ib * 16 + r, 4 * kk + q) * 16);
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        if (jb >= nj) continue;
        const bf16x8 bh = *reinterpret_cast<const bf16x8*>(qb[0] + tsw(jb * 16 + r, 4 * kk + q) * 16);
        const bf16x8 bl = *reinterpret_cast<const bf16x8*>(qb[1] + tsw(jb * 16 + r, 4 * kk + q) * 16);
#pragma unroll
        for (int ib = 0; ib < 4; ++ib) {
          acc[ib][jb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[ib], bh, acc[ib][jb], 0, 0, 0);
          acc[ib][jb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[ib], bl, acc[ib][jb], 0, 0, 0);
        }
      }
    }
    __syncthreads();
  }
  // lane (r, q) of block (ib, jb) holds D[i = 64 wave + 16 ib + 4 q + e][j = 16 jb + r]
  float* dst = it.part < 0 ? p.out + static_cast<int64_t>(it.adapter) * p.M * p.rank
                           : p.part + static_cast<int64_t>(it.part) * p.M * p.rank;
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) {
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      const int j = j0 + jb * 16 + r;
      if (j >= p.rank) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t i = i0 + wave * 64 + ib * 16 + 4 * q + e;
        if (i < p.M) dst[TRANSPOSE ? j * p.M + i : i * p.rank + j] = acc[ib][jb][e];
      }
    }
  }
}

// Gradients of adapters with several items: their partial sums in chunk order. Adapters without tokens: zeros.
__global__ __launch_bounds__(256) void routed_reduce_kernel(const float* __restrict__ part, int64_t n,
                                                            const int32_t* __restrict__ off, int chunk,
                                                            float* __restrict__ out) {
  const int a = blockIdx.y;
  const int lo = off[a], hi = off[a + 1];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  if (hi > lo) {
    const int j0 = lo / chunk, j1 = (hi - 1) / chunk;
    if (j0 == j1) return;
    v = part[(2 * static_cast<int64_t>(j0) + 1) * n + i];
    for (int j = j0 + 1; j <= j1; ++j) v += part[2 * static_cast<int64_t>(j) * n + i];
  }
  out[static_cast<int64_t>(a) * n + i] = v;
}

}  // namespace

hipError_t launch_routed_down(const RoutedDown& p, hipStream_t s) {
  if (p.T <= 0) return hipSuccess;
  const unsigned blocks = static_cast<unsigned>((p.T + kRouteBlock - 1) / kRouteBlock);
  const int most = p.rt.n_adapters < kRouteBlock ? (p.rt.n_adapters > 0 ? p.rt.n_adapters : 1) : kRouteBlock;
  const unsigned slots = static_cast<unsigned>(p.T <= 1024 ? most : 1);
  hipLaunchKernelGGL(routed_down_kernel, dim3(blocks, static_cast<unsigned>((p.rt.rank + 63) / 64), slots),
                     dim3(64 * kDownWaves), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_route_plan(const RoutePlan& p, hipStream_t s) {
  hipLaunchKernelGGL(route_plan_kernel, dim3(static_cast<unsigned>(p.n_adapters)), dim3(1024), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_routed_contract(const RoutedContract& p, hipStream_t s) {
  const ContractArgs a{p.P, p.ldp, p.M, p.hi, p.lo, p.ldt, p.rank, p.plan->perm, p.plan->items, p.part, p.out};
  const dim3 grid(static_cast<unsigned>((p.M + kRtI - 1) / kRtI), static_cast<unsigned>(p.plan->n_items),
                  static_cast<unsigned>((p.rank + kRtJ - 1) / kRtJ));
  if (p.transpose) hipLaunchKernelGGL(routed_tn_kernel<true>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(routed_tn_kernel<false>, grid, dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t n = p.M * p.rank;
  hipLaunchKernelGGL(routed_reduce_kernel,
                     dim3(static_cast<unsigned>((n + 255) / 256), static_cast<unsigned>(p.plan->n_adapters)), dim3(256),
                     0, s, p.part, n, p.plan->off, p.plan->chunk, p.out);
  return hipGetLastError();
}

}  // namespace lora
