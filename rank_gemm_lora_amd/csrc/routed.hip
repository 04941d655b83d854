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
#include "lora_mi355x.h"
#include "routed_dev.hpp"
#include "transpose_dev.hpp"

namespace lora {
namespace {

constexpr uint32_t kOutOfRange = 0x80000000u;  // a buffer offset past every range: the load returns zeros

// Rank-wide producer without the ring. Workgroup: one block of 16 tokens, 64 ranks, one slot's share of the
// block's distinct adapters, one part of K; 8 waves split that and add their sums through LDS in wave order.
// Operands go from global memory straight into MFMA fragments (lane (r, q): 8 consecutive k of adapter row r /
// token r), the next 128 k (64 above 32 ranks) in flight during the MFMAs of these; all 16 tokens are
// multiplied, and the rows of the adapter's own tokens are kept. From 17 to 256 tokens the blocks are of the
// tokens sorted by adapter (every workgroup sorts them for itself, counting the tokens before each), which
// leaves a block the fewest adapters. Beside the ring, kBesideSlots workgroups at a time look through blocks a
// stride apart for those that the ring left (down_beside). Bound by the latency of dependent loads (routing, then operands), not by bytes:
// 5.4 us for one token of K 1536, rank 16.
//
// acc[b] += rows 16 b .. of A times the tokens over [k_lo, k_hi), groups of 32 ST k.
template <int NRB, int ST>
__device__ __forceinline__ void down_product(f32x4 (&acc)[4], __amdgpu_buffer_rsrc_t xr, __amdgpu_buffer_rsrc_t ar,
                                             uint32_t x_off, uint32_t a_off, uint32_t lda_b, int64_t k_lo,
                                             int64_t k_hi, int q) {
  struct {
    u32x4 x[ST], a[ST][NRB];
  } f[2];
  auto load = [&](int i, int64_t kg) {
#pragma unroll
    for (int st = 0; st < ST; ++st) {
      const int64_t k = kg + 32 * st + 8 * q;
      const bool in = k < k_hi;
      f[i].x[st] =
          __builtin_amdgcn_raw_buffer_load_b128(xr, in ? x_off + static_cast<uint32_t>(k * 2) : kOutOfRange, 0, 0);
#pragma unroll
      for (int b = 0; b < NRB; ++b)
        f[i].a[st][b] = __builtin_amdgcn_raw_buffer_load_b128(
            ar, in ? a_off + b * 16 * lda_b + static_cast<uint32_t>(k * 2) : kOutOfRange, 0, 0);
    }
  };
  auto mma = [&](int i) {
#pragma unroll
    for (int st = 0; st < ST; ++st)
#pragma unroll
      for (int b = 0; b < NRB; ++b)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f[i].a[st][b]),
                                                         __builtin_bit_cast(bf16x8, f[i].x[st]), acc[b], 0, 0, 0);
  };
  // (loads past k_hi read zeros, so both halves run unconditionally)
  load(0, k_lo);
  for (int64_t kg = k_lo; kg < k_hi; kg += 64 * ST) {
    load(1, kg + 32 * ST);
    mma(0);
    load(0, kg + 64 * ST);
    mma(1);
  }
}

// Up to 256 tokens: adapter, scale and token of each place of the order by adapter (a token's place is the
// number of tokens before it).
struct SortedTokens {
  int key[kFewMaxT], id[kFewMaxT], token[kFewMaxT];
  float scale[kFewMaxT];
};
// order: the sorted tokens, of which `block` is one (null: blocks are of the tokens as they come). Adapters slot,
// slot + slots, .. of the block; part `part` of K; tell: eid and blk are this workgroup's to write.
// FAT: twice the loads in flight where the adapter has more than 16 ranks (160 registers against 117).
template <bool FAT>
__device__ __forceinline__ void down_block(const RoutedDown& p, int64_t block, f32x4 (&red)[kDownWaves][4][64],
                                           const SortedTokens* order, int q0, int slot, int slots, int part, bool tell) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t t0 = block * kRouteBlock;
  const int rows = static_cast<int>(min<int64_t>(kRouteBlock, p.T - t0));
  int64_t token = t0 + r;
  float s;
  int id;
  if (order != nullptr) {
    token = r < rows ? order->token[t0 + r] : p.T;
    id = r < rows ? order->id[t0 + r] : -1;
    s = r < rows ? order->scale[t0 + r] : 0.f;
  } else {
    id = route(p.rt, token, p.T, s);
  }
  uint32_t todo = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(id >= 0)) & 0xffffu;
  if (tell && wave == 0) {
    const int first = __builtin_amdgcn_readfirstlane(id);
    if (q == 0 && r < rows) p.eid[token] = id;
    const bool same = __builtin_amdgcn_ballot_w64(r < rows && id != first) == 0;
    if (lane == 0) p.blk[block] = same ? first : -2;
  }
  const int shares = kDownWaves * p.parts;
  const int64_t kper = ((p.K + shares - 1) / shares + 31) / 32 * 32;
  const int64_t k_lo = (part * kDownWaves + wave) * kper, k_hi = min<int64_t>(p.K, k_lo + kper);
  const uint32_t ldx_b = static_cast<uint32_t>(p.ldx * 2), lda_b = static_cast<uint32_t>(p.K * 2);
  // (sorted: rows of all of x, at most 256 of 4 MB; a place past the last reads zeros)
  const __amdgpu_buffer_rsrc_t xr = order == nullptr
                                        ? make_rsrc(p.x + t0 * p.ldx, static_cast<uint32_t>(rows) * ldx_b)
                                        : make_rsrc(p.x, static_cast<uint32_t>(p.T) * ldx_b);
  const uint32_t x_off = static_cast<uint32_t>(order == nullptr ? r : token) * ldx_b,
                 a_off = static_cast<uint32_t>(r) * lda_b;
  int nth = 0;
  while (todo != 0) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    todo &= ~static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(id == a));
    if (nth++ % slots != slot) continue;
    const int rank = route_rank(p.rt.ranks, p.rt.rank, a);
    const int rows_a = max(0, min(64, rank - q0));
    const __amdgpu_buffer_rsrc_t ar =
        make_rsrc(p.A + (static_cast<int64_t>(a) * p.rt.rank + q0) * p.K, static_cast<uint32_t>(rows_a) * lda_b);
    f32x4 acc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (rows_a > 32) down_product<4, FAT ? 2 : 1>(acc, xr, ar, x_off, a_off, lda_b, k_lo, k_hi, q);
    else if (rows_a > 16) down_product<2, FAT ? 4 : 2>(acc, xr, ar, x_off, a_off, lda_b, k_lo, k_hi, q);
    else if (rows_a > 0) down_product<1, 4>(acc, xr, ar, x_off, a_off, lda_b, k_lo, k_hi, q);
#pragma unroll
    for (int b = 0; b < 4; ++b) red[wave][b][lane] = acc[b];
    __syncthreads();
    // thread (b, lane): ranks q0 + 16 b + 4 q .. +3 of token t0 + r
    if (wave < 4 && id == a) {
      f32x4 v = red[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kDownWaves; ++w) v += red[w][wave][lane];
      const int64_t at = token * p.ldt + q0 + wave * 16 + 4 * q;
      if (p.parts > 1) {
        *reinterpret_cast<f32x4*>(p.tpart + part * p.T * p.ldt + at) = v;
      } else {
        const float t[4] = {v[0], v[1], v[2], v[3]};
        put_rank_wide<4>(p, at, q0 + wave * 16 + 4 * q, route_live(p.rt.ranks, p.rt.rank, a), t, s);
      }
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void sort_tokens(const RoutedDown& p, SortedTokens& o) {
  static_assert(64 * kDownWaves == 2 * kFewMaxT, "two threads a token");
  const int t = threadIdx.x % kFewMaxT, half = threadIdx.x / kFewMaxT, T = static_cast<int>(p.T);
  float s;
  const uint32_t key = static_cast<uint32_t>(route(p.rt, t, p.T, s));  // (-1, no adapter: last)
  if (half == 0) o.key[t] = static_cast<int>(key);
  __syncthreads();
  // this thread's half of the tokens before t (entries past T hold the last key and come after every token)
  const int mid = (T + 7) / 8 * 4;
  int place = 0;
#pragma unroll 4
  for (int u = half * mid; u < (half == 0 ? mid : T); u += 4) {
    const uint4 k = *reinterpret_cast<const uint4*>(o.key + u);
    place += (k.x < key || (k.x == key && u < t)) + (k.y < key || (k.y == key && u + 1 < t)) +
             (k.z < key || (k.z == key && u + 2 < t)) + (k.w < key || (k.w == key && u + 3 < t));
  }
  if (half == 1) o.id[t] = place;
  __syncthreads();
  if (half == 0) place += o.id[t];
  __syncthreads();
  if (half == 0 && t < T) {
    o.id[place] = static_cast<int>(key);
    o.token[place] = t;
    o.scale[place] = s;
  }
  __syncthreads();
}

// Workgroup (block, 64 ranks from q0, job and share) of the producer; mem: LDS of DownMem.
struct DownMem {
  f32x4 red[kDownWaves][4][64];
  SortedTokens sorted;
};
template <bool FAT>
__device__ __forceinline__ void down_group(const RoutedDowns& ps, DownMem& mem, int block, int group, int z) {
  const int job = z >= ps.z0 ? 1 : 0;
  const RoutedDown& p = ps.d[job];
  const bool tell = group == 0 && z == 0;
  z -= job * ps.z0;
  const int slot = z % ps.slots, part = z / ps.slots;
  const bool sorted = p.order != nullptr;
  if (sorted) {
    sort_tokens(p, mem.sorted);
    if (block == 0 && tell && static_cast<int>(threadIdx.x) < p.T) {
      p.order[threadIdx.x] = mem.sorted.token[threadIdx.x];
      p.order[p.T + threadIdx.x] = mem.sorted.id[threadIdx.x];
    }
  }
  down_block<FAT>(p, block, mem.red, sorted ? &mem.sorted : nullptr, group * 64, slot, ps.slots, part, tell);
}

__global__ __launch_bounds__(64 * kDownWaves) void routed_down_kernel(RoutedDowns ps) {
  __shared__ __attribute__((aligned(16))) DownMem mem;
  down_group<true>(ps, mem, blockIdx.x, blockIdx.y, blockIdx.z);
}

// t of the tokens whose sums are in parts (the ring's splits, or parts without the ring), added in order and
// scaled. 32 threads a token and 64 ranks, kDownWaves * 2 tokens a workgroup.
__device__ __forceinline__ void down_join(const RoutedDown& p, int64_t group) {
  const int n = p.splits > 0 ? p.splits : p.parts;
  if (n <= 1) return;
  const int64_t m = group * (2 * kDownWaves) + (threadIdx.x >> 5);
  if (m >= p.T) return;
  const int q = blockIdx.y * 64 + 2 * (threadIdx.x & 31);
  const int64_t at = m * p.ldt + q;
  f32x2 w[8];  // (all parts' loads before their adds; a part past the last reads the last again, unused)
#pragma unroll
  for (int z = 0; z < 8; ++z) w[z] = *reinterpret_cast<const f32x2*>(p.tpart + min(z, n - 1) * p.T * p.ldt + at);
  const int a = p.eid[m];
  if (a < 0 || (p.splits > 0 && p.ring[m / kRingBlock] < 0)) return;
  float v[2] = {0.f, 0.f}, s;
#pragma unroll
  for (int z = 0; z < 8; ++z)
    if (z < n) {
      v[0] += w[z][0];
      v[1] += w[z][1];
    }
  route(p.rt, m, p.T, s);
  put_rank_wide<2>(p, at, q, route_live(p.rt.ranks, p.rt.rank, a), v, s);
}

// The blocks of 16 that the ring did not take: blocks first, + stride, ..; 64 at a time are looked at, one per lane
// (every wave the same). kBesideSlots workgroups share a block's adapters (2000 tokens of 16 mixed adapters,
// 4096 -> 4096: 155 us a call against 209 with one).
constexpr int kBesideSlots = 4;
__device__ __forceinline__ void down_beside(const RoutedDown& p, f32x4 (&red)[kDownWaves][4][64], int64_t first,
                                            int64_t stride, int slot) {
  const int64_t n = (p.T + kRouteBlock - 1) / kRouteBlock;
  for (int64_t base = first; base < n; base += 64 * stride) {
    const int64_t mine = base + (threadIdx.x & 63) * stride;
    uint64_t left = __builtin_amdgcn_ballot_w64(mine < n && p.ring[mine * kRouteBlock / kRingBlock] < 0);
    while (left != 0) {
      const int i = __builtin_ctzll(left);
      left &= left - 1;
      down_block<true>(p, base + i * stride, red, nullptr, blockIdx.y * 64, slot, kBesideSlots, 0, false);
    }
  }
}

// What the first launch left: with BESIDE the blocks of 16 that the ring did not take (workgroups below `beside`),
// and the sums in parts (the others).
template <bool BESIDE>
__global__ __launch_bounds__(64 * kDownWaves) void routed_rest_kernel(RoutedDowns ps, int beside) {
  const RoutedDown& p = ps.d[blockIdx.z];
  if (static_cast<int>(blockIdx.x) >= beside) {
    down_join(p, blockIdx.x - beside);
    return;
  }
  if constexpr (BESIDE) {
    __shared__ f32x4 red[kDownWaves][4][64];
    down_beside(p, red, blockIdx.x / kBesideSlots, beside / kBesideSlots, blockIdx.x % kBesideSlots);
  }
}

// ---------------------------------------------------------------------------
// Few tokens: y = RN(x.W^T + t~.B^T + b) in two launches. The first forms t~ and, in other workgroups, the base
// product: neither needs the other, and the chain of look-ups and loads behind t~ (5 to 14 us) passes while the
// weight streams. The second adds the base product's parts and each token's adapter.
// (Adapters first and the base product in the same accumulators, after the producer: 64 tokens of 64 adapters,
// 4096 -> 14336, 54.8 us against 42.9; 203 of 32, 1536 -> 8960, 39.0 against 32.6; one token, 1536 -> 1536, 14.8
// against 11.8; only 256 of 64, 4096 -> 14336, 85 against 90.)
//
// Base product: workgroup of 8 waves: 64 outputs x BM tokens, one of S parts of K. Stages of 64 k (128 bytes of
// every row of x and W) go through a ring of D LDS slots filled by buffer_load .. lds, D - 1 of them in flight;
// 16-byte chunk c of row r lies at c ^ ((r / 2) % 8), so that a wave's 16-byte reads spread over the banks. (A
// first form fed the MFMAs straight from memory: 16 rows of 64 bytes an instruction. 64 tokens, 4096 -> 14336,
// took 60 us that way.) Up to 32 tokens four waves take the first half of a stage's k and four the second, each
// a part of its own.
constexpr int kFewN = 64, kFewRow = 128;

template <int BM>
struct FewCfg {
  static constexpr int WAVES = kDownWaves, KH = few_halves(BM);
  static constexpr int XR = BM < 32 ? 32 : BM;  // staged rows of x (one copy instruction a wave at least)
  static constexpr int WAVES_M = KH == 2 ? 1 : 4, WAVES_N = WAVES / KH / WAVES_M;
  static constexpr int TB = BM / WAVES_M / 16, NB = kFewN / WAVES_N / 16;  // 16 x 16 blocks of a wave
  static constexpr int STAGE = (XR + kFewN) * kFewRow;
  static constexpr int LOADERS = KH == 2 ? 4 : 8;  // waves that copy
  static constexpr int LPS = (XR + kFewN) / 8 / LOADERS;  // copy instructions of such a wave and stage (8 rows each)
};

// Element of the adapters' tile: 4 outputs 4 c .. of token row; the groups of 4 XOR-swizzled by row, so that
// the 16 tokens of an access spread over the banks.
__device__ __forceinline__ f32x4* few_delta(char* tile, int row, int c) {
  return reinterpret_cast<f32x4*>(tile) + row * (kFewN / 4) + (c ^ (row & 15));
}

// y of a token at 4 outputs of a tile, from nl on: the sums, the bias and one rounding.
__device__ __forceinline__ void few_store(const RoutedFew& p, f32x4 v, int64_t token, int64_t n0, int rows_n, int nl) {
  if (nl >= rows_n) return;
  if (p.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (nl + e < rows_n) v[e] += bf16_to_f32(p.bias[n0 + nl + e]);
  }
  uint16_t* y = p.y + token * p.ldy + n0 + nl;
  const uint2 o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  if (reinterpret_cast<uintptr_t>(y) % 8 == 0 && nl + 4 <= rows_n) {
    *reinterpret_cast<uint2*>(y) = o;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (nl + e < rows_n) y[e] = static_cast<uint16_t>((e < 2 ? o.x : o.y) >> (16 * (e & 1)));
  }
}

// The adapters of a tile: units part, part + parts, .. of its list, P in flight at a time, 32 ranks of each at a
// time. (Code that runs once costs its fetch: eight units at a time, unrolled, took 1-3 us longer on every small
// call and gained nothing on large ones.)
template <int P>
__device__ __forceinline__ void few_adapters(const RoutedFew& p, char* delta, const int* ids, const int* tok,
                                             const int* units, int n_units, int64_t n0, int rows_n, int part, int parts) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const uint32_t ldb = static_cast<uint32_t>(p.rt.rank * 2), ldt_b = static_cast<uint32_t>(p.ldt * 2);
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(p.hi, static_cast<uint32_t>(p.T) * ldt_b);
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(p.mid, static_cast<uint32_t>(p.T) * ldt_b);
  for (int u0 = part; u0 < n_units; u0 += P * parts) {
    int row[P], rank[P], most = 0;
    bool mine[P];
    uint32_t trow[P];
    __amdgpu_buffer_rsrc_t br[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int at = u0 + u * parts;
      const bool in = at < n_units;
      const int unit = __builtin_amdgcn_readfirstlane(units[in ? at : u0]);  // first row, and the rank above bit 8
      const int first = unit & 255;
      const int a = __builtin_amdgcn_readfirstlane(ids[first]);
      row[u] = (first & ~15) + r;
      mine[u] = in && ids[row[u]] == a;
      rank[u] = in ? unit >> 8 : 0;
      most = max(most, rank[u]);
      trow[u] = static_cast<uint32_t>(tok[row[u]]) * ldt_b;
      br[u] = make_rsrc(static_cast<const bf16_bits*>(p.rt.B) + (static_cast<int64_t>(a) * p.N + n0) * p.rt.rank,
                        static_cast<uint32_t>(rows_n) * ldb);
    }
    for (int c0 = 0; c0 < most; c0 += 32) {
      u32x4 w[P][4], t[P][2];
      const int k = c0 + 8 * q;
#pragma unroll
      for (int u = 0; u < P; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[u][i] = __builtin_amdgcn_raw_buffer_load_b128(
              br[u], k < rank[u] ? static_cast<uint32_t>(16 * i + r) * ldb + k * 2 : kOutOfRange, 0, 0);
        const uint32_t off = mine[u] && k < rank[u] ? trow[u] + k * 2 : kOutOfRange;
        t[u][0] = __builtin_amdgcn_raw_buffer_load_b128(hr, off, 0, 0);
        t[u][1] = __builtin_amdgcn_raw_buffer_load_b128(mr, off, 0, 0);
      }
      // (a unit's rows start at zero and are this wave's alone)
#pragma unroll
      for (int u = 0; u < P; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[u][i]),
                                                        __builtin_bit_cast(bf16x8, t[u][k2]), d, 0, 0, 0);
          if (mine[u]) *few_delta(delta, row[u], 4 * i + q) += d;
        }
    }
  }
}

template <int BM, int D>
__global__ __launch_bounds__(64 * kDownWaves, 4) void routed_few_kernel(RoutedFew p, RoutedDowns ps, int downs, int tt,
                                                                       int S, int per) {
  using C = FewCfg<BM>;
  constexpr int TB = C::TB, NB = C::NB;
  // (one LDS object: with several the compiler waits for every copy in flight before each LDS read, a memory
  // latency a stage. 1 token, 4096 -> 14336, no adapter: 42 us a call, 31 without)
  __shared__ __attribute__((aligned(1024))) char ring[D * C::STAGE];
  static_assert(sizeof(DownMem) <= sizeof(ring), "the producer's LDS");
  if (static_cast<int>(blockIdx.x) < downs) {
    const int blocks = static_cast<int>((p.T + kRouteBlock - 1) / kRouteBlock), groups = (p.rt.rank + 63) / 64;
    const int i = blockIdx.x / blocks;
    down_group<false>(ps, *reinterpret_cast<DownMem*>(ring), blockIdx.x - i * blocks, i % groups, i / groups);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  // the token tiles of one stretch of the weight follow one another on one XCD, in whose L2 it stays
  const int G = gridDim.x - downs, pid = blockIdx.x - downs, xcd = pid % 8;
  const int L = xcd * (G / 8) + min(xcd, G % 8) + pid / 8;
  const int tile = L / S, split = L - tile * S;
  const int tile_n = tile / tt, tile_m = tile - tile_n * tt;
  // (consecutive L: parts of one tile; the token tiles of one stretch of W next)
  const int64_t n0 = static_cast<int64_t>(tile_n) * kFewN, m0 = static_cast<int64_t>(tile_m) * BM;
  const int rows_n = static_cast<int>(min<int64_t>(kFewN, p.N - n0));
  const int rows_m = static_cast<int>(min<int64_t>(BM, p.T - m0));
  const uint32_t ldx_b = static_cast<uint32_t>(p.ldx * 2), ldw_b = static_cast<uint32_t>(p.K * 2);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x + m0 * p.ldx, static_cast<uint32_t>(rows_m) * ldx_b);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.W + n0 * p.K, static_cast<uint32_t>(rows_n) * ldw_b);
  const int kb_lo = split * per * kFewRow, kb_hi = min(static_cast<int>(p.K * 2), kb_lo + per * kFewRow);
  const int ns = (kb_hi - kb_lo + kFewRow - 1) / kFewRow;
  // (tiles start their K loops apart where x stays in an XCD's L2: in step they read the same few memory
  // channels at a time when the weight's rows are a power of two apart)
  const int rot = p.T * p.K <= (1 << 19) ? 5 * tile % ns : 0;
  // this lane's part of each copy instruction (8 rows, x first, then W): its chunk's byte offset in part
  // `split` at stage 0; rows past the tile's are out of the resource's range and read as zeros
  uint32_t from[C::LPS];
  int cb[C::LPS];
#pragma unroll
  for (int it = 0; it < C::LPS; ++it) {
    const int group = it * C::LOADERS + wave;
    const bool is_w = group >= C::XR / 8;
    const int row = (is_w ? group - C::XR / 8 : group) * 8 + (lane >> 3);
    cb[it] = kb_lo + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
    from[it] = row < (is_w ? rows_n : rows_m) ? static_cast<uint32_t>(row) * (is_w ? ldw_b : ldx_b) : kOutOfRange;
  }
  auto issue = [&](int st) {
    if (C::LOADERS < C::WAVES && wave >= C::LOADERS) return;
    char* dst = ring + (st % D) * C::STAGE;
    const int at = st + rot < ns ? st + rot : st + rot - ns;
    const int kb = st < ns ? at * kFewRow : 1 << 30;  // (past the last: nothing)
#pragma unroll
    for (int it = 0; it < C::LPS; ++it) {
      const int group = it * C::LOADERS + wave;
      const bool is_w = group >= C::XR / 8;
      const uint32_t off = cb[it] + kb < kb_hi ? from[it] + static_cast<uint32_t>(cb[it] + kb) : kOutOfRange;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_w ? wr : xr, (lds_void*)(dst + group * 1024), 16, off, 0, 0, 0);
    }
  };
#pragma unroll
  for (int st = 0; st < D - 1; ++st) issue(st);

  // lane (r, q) of block (i, j): outputs wn0 + 16 i + 4 q .. +3 of token wm0 + 16 j + r
  const int half = wave / (C::WAVES / C::KH), w = wave % (C::WAVES / C::KH);
  const int wm0 = (w % C::WAVES_M) * (TB * 16), wn0 = (w / C::WAVES_M) * (NB * 16);
  f32x4 acc[NB][TB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint32_t chunk = static_cast<uint32_t>((q ^ ((r >> 1) & 7)) * 16);
  const uint32_t xo = static_cast<uint32_t>((wm0 + r) * kFewRow) + chunk;
  const uint32_t wo = static_cast<uint32_t>((C::XR + wn0 + r) * kFewRow) + chunk;
  for (int st = 0; st < ns; ++st) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vmem((D - 2) * C::LPS));
    lds_barrier();  // stage st landed for every wave; all are done with the slot of stage st - 1
    issue(st + D - 1);
    const char* sp = ring + (st % D) * C::STAGE;
#pragma unroll
    for (int k = 0; k < 2 / C::KH; ++k) {
      const uint32_t kk = static_cast<uint32_t>(C::KH == 2 ? half : k) * 64u;
      bf16x8 wf[NB], xf[TB];
#pragma unroll
      for (int i = 0; i < NB; ++i) wf[i] = *reinterpret_cast<const bf16x8*>(sp + ((wo ^ kk) + i * 16 * kFewRow));
#pragma unroll
      for (int j = 0; j < TB; ++j) xf[j] = *reinterpret_cast<const bf16x8*>(sp + ((xo ^ kk) + j * 16 * kFewRow));
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i], xf[j], acc[i][j], 0, 0, 0);
    }
  }
  wait_vmem();  // (copies past the end)

  float* mine = p.part + ((static_cast<int64_t>(tile_n) * S + split) * C::KH + half) * p.T * kFewN;
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int row = wm0 + 16 * j + r;
      if (row < rows_m) *reinterpret_cast<f32x4*>(mine + (m0 + row) * kFewN + wn0 + 16 * i + 4 * q) = acc[i][j];
    }
}

// Workgroup: 64 outputs x FB tokens (places of the sorted order, where there is one). Each adapter of each 16
// tokens (a unit) is one wave's, its product over the 64 outputs formed apart and the rows of the adapter's own
// tokens put into an LDS tile, so nothing of one adapter meets another's tokens. The parts of the base product
// are added in order, then the adapter's sum and the bias; the loads of the first of them are in flight meanwhile.
// 16 tokens have up to 16 parts and few workgroups: two units and eight parts in flight; more tokens have few parts
// and workgroups to fill the card, whose registers count: one unit and four parts (203 tokens of 32 adapters,
// 1536 -> 8960, a call: 32.6 -> 30.0 us; with 16 tokens that way 25.0 -> 26.3, 8960 -> 1536).
template <int FB>
__global__ __launch_bounds__(FB * 16) void few_finish_kernel(RoutedFew p, int parts) {
  __shared__ __attribute__((aligned(16))) char delta[FB * kFewN * 4];
  // adapter and token of each row, first row and rank of each unit
  __shared__ int ids[FB], tok[FB], units[FB], n_units;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kFewN, m0 = static_cast<int64_t>(blockIdx.y) * FB;
  const int rows_n = static_cast<int>(min<int64_t>(kFewN, p.N - n0));
  const int rows_m = static_cast<int>(min<int64_t>(FB, p.T - m0));
  const bool sorted = p.order != nullptr;
  const int row = tid >> 4, c = tid & 15;  // this thread's token and 4 outputs
  const int64_t place = m0 + min(row, rows_m - 1), token = sorted ? p.order[place] : place;
  if (tid < FB) {
    tok[tid] = tid >= rows_m ? 0 : (sorted ? p.order[m0 + tid] : static_cast<int>(m0) + tid);
    ids[tid] = tid >= rows_m ? -1 : (sorted ? p.order[p.T + m0 + tid] : p.rt.eid[m0 + tid]);
  }
  *few_delta(delta, row, c) = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* base = p.part + (static_cast<int64_t>(blockIdx.x) * parts * p.T + token) * kFewN + 4 * c;
  constexpr int FW = FB == 16 ? 8 : 4;
  f32x4 w[FW];  // (a part past the last reads the last again, unused)
#pragma unroll
  for (int k = 0; k < FW; ++k) w[k] = *reinterpret_cast<const f32x4*>(base + min(k, parts - 1) * p.T * kFewN);
  lds_barrier();
  // units: where an adapter shows first in a block of 16 (in adapter order: where it changes)
  if (wave == 0) {
    bool start = lane < FB && ids[lane % FB] >= 0;
    for (int e = 1; e < (sorted ? 2 : 16); ++e)
      start = start && !(lane % 16 >= e && ids[max(lane % FB - e, 0)] == ids[lane % FB]);
    const uint64_t m = __builtin_amdgcn_ballot_w64(start);
    if (start) {
      const int a = ids[lane];
      const int rank = p.rt.ranks != nullptr ? (min(p.rt.ranks[a], p.rt.rank) + 7) & ~7 : p.rt.rank;
      units[__popcll(m & ((1ull << lane) - 1))] = lane | rank << 8;
    }
    if (lane == 0) n_units = __popcll(m);
  }
  lds_barrier();
  few_adapters<FB == 16 ? 2 : 1>(p, delta, ids, tok, units, __builtin_amdgcn_readfirstlane(n_units), n0, rows_n, wave, FB / 4);
  lds_barrier();
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < FW; ++k)
    if (k < parts) v += w[k];
  for (int k = FW; k < parts; ++k) v += *reinterpret_cast<const f32x4*>(base + k * p.T * kFewN);
  if (row < rows_m) few_store(p, v + *few_delta(delta, row, c), token, n0, rows_n, 4 * c);
}

// ---------------------------------------------------------------------------
// What the backward's other launches need first: the transposed operands and the plan of the contractions.
//
// The plan, tokens sorted by adapter: workgroup a finds its adapter's tokens. The 16 waves take consecutive
// stretches of the tokens, LOADS of 64 in flight; a first pass counts the tokens of every adapter before it
// (one LDS atomic for each adapter among 64 tokens; integers, so their order does not show), from which follow its
// place among tokens and items, and its own by wave; a second writes them, in token order. LOADS 1: before the
// producer, from the routing itself; 8: from eid.
template <int LOADS>
__device__ __forceinline__ void route_plan(const RoutePlan& p, int a, int* counts, int (&sums)[5][16],
                                           int (&mine)[16]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t per = ((p.T + 15) / 16 + 63) / 64 * 64;
  const int64_t lo = wave * per, hi = min<int64_t>(p.T, lo + per);
  for (int i = threadIdx.x; i < p.n_adapters; i += 1024) counts[i] = 0;
  __syncthreads();
  int nm = 0;
  for (int64_t t = lo; t < hi; t += 64 * LOADS) {
    int id[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      float scale;
      const int64_t at = t + 64 * k + lane;
      if constexpr (LOADS == 1) id[k] = route(p.rt, at, hi, scale);
      else id[k] = at < hi ? p.eid[at] : -1;
    }
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      uint64_t todo = __builtin_amdgcn_ballot_w64(id[k] >= 0 && id[k] < a);
      while (todo != 0) {
        const int b = __builtin_amdgcn_readlane(id[k], __builtin_ctzll(todo));
        const uint64_t m = __builtin_amdgcn_ballot_w64(id[k] == b);
        todo &= ~m;
        if (lane == 0) atomicAdd(&counts[b], __popcll(m));
      }
      nm += __popcll(__builtin_amdgcn_ballot_w64(id[k] == a));
    }
  }
  if (lane == 0) mine[wave] = nm;
  __syncthreads();
  // of the adapters before a: tokens, and for each table items and slots of partial sums
  int v[5] = {0, 0, 0, 0, 0};
  for (int i = threadIdx.x; i < a; i += 1024) {
    v[0] += counts[i];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = max(1, (counts[i] + p.table[h].chunk - 1) / p.table[h].chunk);
      v[1 + 2 * h] += k;
      v[2 + 2 * h] += k > 1 ? k : 0;
    }
  }
#pragma unroll
  for (int k = 0; k < 5; ++k) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v[k] += __shfl_xor(v[k], d);
    if (lane == 0) sums[k][wave] = v[k];
  }
  __syncthreads();
  int before[5] = {0, 0, 0, 0, 0}, count = 0, at = 0;
#pragma unroll 2
  for (int w = 0; w < 16; ++w) {
#pragma unroll
    for (int k = 0; k < 5; ++k) before[k] += sums[k][w];
    if (w < wave) at += mine[w];
    count += mine[w];
  }
  const int start = before[0];
  at += start;
  for (int64_t t = lo; t < hi; t += 64 * LOADS) {
    int id[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      float scale;
      const int64_t at = t + 64 * k + lane;
      if constexpr (LOADS == 1) id[k] = route(p.rt, at, hi, scale);
      else id[k] = at < hi ? p.eid[at] : -1;
    }
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
      const uint64_t m = __builtin_amdgcn_ballot_w64(id[k] == a);
      if (id[k] == a) p.perm[at + __popcll(m & ((1ull << lane) - 1))] = static_cast<int32_t>(t + 64 * k + lane);
      at += __popcll(m);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const RouteTable& tb = p.table[h];
    const int item = before[1 + 2 * h], slot = before[2 + 2 * h];
    const int k = max(1, (count + tb.chunk - 1) / tb.chunk);
    for (int i = threadIdx.x; i < k; i += 1024) {
      RouteItem it;
      it.adapter = a;
      it.lo = start + static_cast<int>(static_cast<int64_t>(count) * i / k);
      it.hi = start + static_cast<int>(static_cast<int64_t>(count) * (i + 1) / k);
      it.part = k > 1 ? slot + i : -1;
      tb.items[item + i] = it;
    }
    if (threadIdx.x == 0) tb.first[a] = item;
    if (a == p.n_adapters - 1) {
      if (threadIdx.x == 0) tb.first[a + 1] = item + k;
      for (int64_t z = item + k + static_cast<int64_t>(threadIdx.x); z < tb.n_items; z += 1024)
        tb.items[z] = RouteItem{0, 0, 0, -1};
    }
  }
}

struct RoutePrepare {
  RoutePlan plan;
  TransposeStack s[kTransposeStacks];
  int64_t first[kTransposeStacks + 1];  // 64 x 64 tiles [first, next first) are a stack's
  int64_t at;                           // workgroups of the launches before this one
};

// Workgroups below n_adapters (with LOADS): the plan; the others (TRANSPOSE): tiles, TILES of them by 256 threads
// each.
template <bool TRANSPOSE, int LOADS>
__global__ __launch_bounds__(LOADS > 0 ? 1024 : 256, LOADS == 8 ? 4 : 8) void route_prepare_kernel(RoutePrepare p) {
  constexpr int TILES = LOADS > 0 ? 4 : 1;
  __shared__ __attribute__((aligned(16))) union {
    bf16_bits tile[TILES][64][72];
    int counts[LOADS > 0 ? LORA_MAX_POOL : 1];
  } u;
  if constexpr (LOADS > 0) {
    __shared__ int sums[5][16], mine[16];
    if (!TRANSPOSE || p.at + blockIdx.x < p.plan.n_adapters) {
      route_plan<LOADS>(p.plan, blockIdx.x, u.counts, sums, mine);
      return;
    }
  }
  const int part = threadIdx.x >> 8;
  const int64_t b = (p.at + blockIdx.x - p.plan.n_adapters) * TILES + part;
  int k = 0;
#pragma unroll
  for (int i = 1; i < kTransposeStacks; ++i) k = b >= p.first[i] ? i : k;
  const TransposeStack& s = p.s[k];
  const int64_t tr = (s.R + 63) / 64, tc = (s.C + 63) / 64, at = b - p.first[k];
  const int64_t slot = at / (tr * tc), rest = at - slot * (tr * tc);
  // (past the last tile: no rows, nothing read or written)
  const bool in = b < p.first[kTransposeStacks];
  transpose_tile16(s.src + (in ? slot : 0) * s.R * s.C, s.C, in ? s.R : 0, in ? s.C : 0,
                   s.dst + (in ? slot : 0) * s.R * s.C, in ? s.R : 0, in ? s.C : 0, rest % tr * 64, rest / tr * 64,
                   u.tile[part], threadIdx.x & 255);
}

// ---------------------------------------------------------------------------
// Contraction over an adapter's tokens: grid (256 columns of P, item, 64 ranks), tokens in steps of 64
// gathered through perm. Both operands are token-major and are transposed on the way to LDS (a thread
// turns 8 tokens x 8 columns in registers); lane (r, q) of the MFMA then reads 8 consecutive tokens of
// one column. The rank-wide operand is hi + mid + lo, all multiplied into the same fp32 sum: the gradients
// see it in fp32 (hi + lo alone left them at 2-3e-6 of their norm, against 0.3-1.2e-6 this way).
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

__global__ __launch_bounds__(256, 2) void routed_tn_kernel(RoutedContracts ps) {
  __shared__ __attribute__((aligned(256))) char pb[kRtI * kRtT * 2];
  __shared__ __attribute__((aligned(256))) char qb[3][kRtJ * kRtT * 2];
  __shared__ int32_t tok[kRouteMaxChunk];
  const int job = static_cast<int>(blockIdx.x) >= ps.tiles0 ? 1 : 0;
  const RoutedContract& p = ps.c[job];
  if (blockIdx.y >= p.table.n_items) return;
  const RouteItem it = p.table.items[blockIdx.y];
  const int cnt = it.hi - it.lo;
  if (cnt <= 0) return;
  const int rank = ps.rank;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x - job * ps.tiles0) * kRtI;
  const int j0 = blockIdx.z * kRtJ;
  const int nj = (min(kRtJ, rank - j0) + 15) / 16;
  for (int i = threadIdx.x; i < cnt; i += 256) tok[i] = ps.perm[it.lo + i];
  __syncthreads();
  const int nsteps = (cnt + kRtT - 1) / kRtT;
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;  // P: columns i0 + 8 c .. +7, tokens 8 g .. +7 of the step
  const bool pcol = i0 + 8 * c < p.M;
  const bf16_bits* pcolp = p.P + i0 + 8 * c;
  const int qc = threadIdx.x & 7, qg = (threadIdx.x >> 3) & 7;  // waves 0, 1, 2: hi, mid, lo
  const bf16_bits* qcolp = p.q[min(wave, 2)] + j0 + 8 * qc;
  u32x4 pv[8], qv[8];
  auto load = [&](int step) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = step * kRtT + 8 * g + e;
      pv[e] = u32x4{0u, 0u, 0u, 0u};
      if (pcol && i < cnt) pv[e] = *reinterpret_cast<const u32x4*>(pcolp + tok[i] * p.ldp);
    }
    if (wave < 3) {
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
    if (wave < 3) transpose_to_lds(qb[wave], qv, qc, qg);
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
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const bf16x8 b = *reinterpret_cast<const bf16x8*>(qb[k] + tsw(jb * 16 + r, 4 * kk + q) * 16);
#pragma unroll
          for (int ib = 0; ib < 4; ++ib)
            acc[ib][jb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[ib], b, acc[ib][jb], 0, 0, 0);
        }
      }
    }
    __syncthreads();
  }
  // lane (r, q) of block (ib, jb) holds D[i = 64 wave + 16 ib + 4 q + e][j = 16 jb + r]
  float* dst = it.part < 0 ? p.out + static_cast<int64_t>(it.adapter) * p.M * rank
                           : p.part + static_cast<int64_t>(it.part) * p.M * rank;
  const bool quads = reinterpret_cast<uintptr_t>(dst) % 16 == 0;
  // (zeros from the adapter's rank on: there q's zeros may have met an infinite or NaN P)
  const int live = ps.ranks != nullptr ? min(ps.ranks[it.adapter], rank) : rank;
#pragma unroll
  for (int jb = 0; jb < 4; ++jb)
    if (j0 + jb * 16 + r >= live)
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) acc[ib][jb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ib = 0; ib < 4; ++ib) {
#pragma unroll
    for (int jb = 0; jb < 4; ++jb) {
      const int j = j0 + jb * 16 + r;
      if (j >= rank) continue;
      const int64_t i = i0 + wave * 64 + ib * 16 + 4 * q;
      if (i >= p.M) continue;  // (M is a multiple of 8: all four or none)
      if (p.transpose && quads) {
        *reinterpret_cast<f32x4*>(dst + j * p.M + i) = acc[ib][jb];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[p.transpose ? j * p.M + i + e : (i + e) * rank + j] = acc[ib][jb][e];
      }
    }
  }
}

// Gradients of adapters with several items: their partial sums in order. Adapters without tokens: zeros. Four
// elements a thread.
__global__ __launch_bounds__(256) void routed_reduce_kernel(RoutedContracts ps) {
  const RoutedContract& p = ps.c[blockIdx.z];
  const int64_t n = p.M * ps.rank;
  const int a = blockIdx.y;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;  // (n is a multiple of 64)
  if (i >= n) return;
  const int lo = p.table.first[a], k = p.table.first[a + 1] - lo;
  const RouteItem it = p.table.items[lo];
  if (k == 1 && it.hi > it.lo) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (k > 1) {
    const float* src = p.part + it.part * n + i;
    for (int z = 0; z < k; ++z) v += *reinterpret_cast<const f32x4*>(src + z * n);
  }
  float* dst = p.out + static_cast<int64_t>(a) * n + i;
  if (reinterpret_cast<uintptr_t>(dst) % 16 == 0) {
    *reinterpret_cast<f32x4*>(dst) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) dst[e] = v[e];
  }
}

}  // namespace

// The producer without the ring: slots and z0 of p, returns the workgroups of a block and 64 ranks. Slots for
// blocks of twice the mean while the workgroups stay below 96 and pass beside others (203 tokens of 32 adapters,
// 1536 -> 8960: 31.9 us against 34.4 with one more than the mean; 256 of 16 in five parts, 8960 -> 1536: 43.1
// against 41.7).
static unsigned down_shares(RoutedDowns& p) {
  const RoutedDown& d = p.d[0];
  const int64_t units = (d.T + kRouteBlock - 1) / kRouteBlock * ((d.rt.rank + 63) / 64);
  const int64_t parts = d.parts + (p.n > 1 ? p.d[1].parts : 0);
  p.slots = down_slots(d.T, d.rt.n_adapters, d.order != nullptr, 2);
  if (units * p.slots * parts > 96) p.slots = down_slots(d.T, d.rt.n_adapters, d.order != nullptr, 1);
  p.z0 = p.slots * d.parts;
  return static_cast<unsigned>(p.slots * parts);
}

// What the first launch of a producer leaves.
static hipError_t launch_rest(const RoutedDowns& p, hipStream_t s) {
  const RoutedDown& d = p.d[0];
  const unsigned blocks = static_cast<unsigned>((d.T + kRouteBlock - 1) / kRouteBlock);
  const unsigned groups = static_cast<unsigned>((d.rt.rank + 63) / 64), jobs = static_cast<unsigned>(p.n);
  bool join = false;
  for (int i = 0; i < p.n; ++i) join = join || p.d[i].splits > 1 || (p.d[i].splits == 0 && p.d[i].parts > 1);
  // (up to kRingAdapters adapters every block is the ring's)
  const unsigned beside =
      d.splits > 0 && d.rt.n_adapters > kRingAdapters ? kBesideSlots * (blocks < 128 ? blocks : 128) : 0;
  const unsigned joins = join ? static_cast<unsigned>((d.T + 2 * kDownWaves - 1) / (2 * kDownWaves)) : 0;
  // (one launch for both where it is short: 4977 tokens 7.2 us against 5.4 + 4.7; the registers of the blocks slow
  // many joins down: 18871 tokens, both products, 26 us against 15.4 + 4.8)
  const bool apart = d.T > 8192;
  hipError_t e = hipSuccess;
  if (beside > 0) {
    const unsigned x = beside + (apart ? 0 : joins);
    hipLaunchKernelGGL(routed_rest_kernel<true>, dim3(x, groups, jobs), dim3(64 * kDownWaves), 0, s, p,
                       static_cast<int>(beside));
    e = hipGetLastError();
  }
  if (e == hipSuccess && joins > 0 && (apart || beside == 0)) {
    hipLaunchKernelGGL(routed_rest_kernel<false>, dim3(joins, groups, jobs), dim3(64 * kDownWaves), 0, s, p, 0);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_routed_down(RoutedDowns p, hipStream_t s) {
  const RoutedDown& d = p.d[0];
  if (d.T <= 0) return hipSuccess;
  hipError_t e = hipSuccess;
  if (d.splits == 0) {
    const dim3 grid(static_cast<unsigned>((d.T + kRouteBlock - 1) / kRouteBlock),
                    static_cast<unsigned>((d.rt.rank + 63) / 64), down_shares(p));
    hipLaunchKernelGGL(routed_down_kernel, grid, dim3(64 * kDownWaves), 0, s, p);
    e = hipGetLastError();
  } else {
    e = launch_routed_ring(p, s);
  }
  return e != hipSuccess ? e : launch_rest(p, s);
}

namespace {
template <int BM, int D>
hipError_t few(const RoutedFew& p, RoutedDowns downs, const FewPlan& f, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((p.T + kRouteBlock - 1) / kRouteBlock);
  const unsigned first = blocks * static_cast<unsigned>((p.rt.rank + 63) / 64) * down_shares(downs);
  hipLaunchKernelGGL((routed_few_kernel<BM, D>), dim3(first + static_cast<unsigned>(f.tiles * f.splits)),
                     dim3(64 * kDownWaves), 0, s, p, downs, static_cast<int>(first), f.token_tiles, f.splits, f.stages);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = launch_rest(downs, s);
  if (e != hipSuccess) return e;
  const unsigned x = static_cast<unsigned>(f.tiles / f.token_tiles);
  const unsigned y = static_cast<unsigned>((p.T + 31) / 32);
  if (BM == 16) hipLaunchKernelGGL(few_finish_kernel<16>, dim3(x), dim3(256), 0, s, p, f.parts);
  else hipLaunchKernelGGL(few_finish_kernel<32>, dim3(x, y), dim3(512), 0, s, p, f.parts);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_routed_few(const RoutedFew& p, const RoutedDowns& downs, hipStream_t s) {
  const FewPlan f = few_plan(p.T, p.K, p.N);
  switch (f.bm) {
    case 16: return few<16, 6>(p, downs, f, s);
    case 32: return few<32, 6>(p, downs, f, s);
    case 64: return few<64, 4>(p, downs, f, s);
    default: return few<128, 3>(p, downs, f, s);
  }
}

hipError_t launch_route_prepare(const RoutePlan& plan, const TransposeStack* stacks, int n, hipStream_t s) {
  RoutePrepare p;
  p.plan = plan;
  int64_t tiles = 0;
  for (int i = 0; i < kTransposeStacks; ++i) {
    p.s[i] = i < n ? stacks[i] : TransposeStack{nullptr, nullptr, 64, 64, 0};
    p.first[i] = i < n ? tiles : (int64_t(1) << 62);
    if (i < n) tiles += stacks[i].slots * ((stacks[i].R + 63) / 64) * ((stacks[i].C + 63) / 64);
  }
  p.first[kTransposeStacks] = tiles;
  const int per = plan.n_adapters > 0 ? 4 : 1;  // (transposes alone, 27 MB: 20.5 us one to a workgroup, 25 four)
  const int64_t blocks = plan.n_adapters + (tiles + per - 1) / per;
  // (a launch has fewer than 2^32 threads: the copies of a pool of 2^24 tiles and more take several)
  const int64_t most = (int64_t(1) << 31) / (256 * per);
  for (p.at = 0; p.at < blocks; p.at += most) {
    const int64_t left = blocks - p.at;
    const dim3 grid(static_cast<unsigned>(left < most ? left : most)), block(static_cast<unsigned>(256 * per));
    if (plan.n_adapters == 0) hipLaunchKernelGGL((route_prepare_kernel<true, 0>), grid, block, 0, s, p);
    else if (plan.eid == nullptr) hipLaunchKernelGGL((route_prepare_kernel<true, 1>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((route_prepare_kernel<false, 8>), grid, block, 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_routed_contract(RoutedContracts p, hipStream_t s) {
  int64_t tiles = 0, items = 0, n = 0;
  for (int i = 0; i < p.n; ++i) {
    if (i == 1) p.tiles0 = static_cast<int>(tiles);
    tiles += (p.c[i].M + kRtI - 1) / kRtI;
    items = p.c[i].table.n_items > items ? p.c[i].table.n_items : items;
    n = p.c[i].M * p.rank > n ? p.c[i].M * p.rank : n;
  }
  if (p.n == 1) p.tiles0 = static_cast<int>(tiles);
  hipLaunchKernelGGL(routed_tn_kernel, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(items),
                                            static_cast<unsigned>((p.rank + kRtJ - 1) / kRtJ)), dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(routed_reduce_kernel, dim3(static_cast<unsigned>((n / 4 + 255) / 256),
                                                static_cast<unsigned>(p.n_adapters), static_cast<unsigned>(p.n)),
                     dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace lora
