// C-ABI of the routed linear layer (tokens take their adapters from a pool): argument validation,
// workspace layout and the order of the launches. Every check runs before any launch.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstring>

#include "backward.hpp"
#include "checks.hpp"
#include "lora_mi355x.h"
#include "routed.hpp"

namespace {

using lora::aligned;
using lora::Elt;
using lora::kMaxRowBytes;
using lora::LinearProblem;
using lora::overlaps;
using lora::round_up;
using lora::Span;
using lora::span2d;

struct Take {  // regions of a workspace, each 256-byte aligned
  size_t off = 0;
  size_t operator()(size_t n) {
    const size_t o = off;
    off = round_up(off + n);
    return o;
  }
};

// Partial sums of the few-token kernel for T tokens, K inputs and N outputs.
size_t few_bytes(int64_t T, int64_t K, int64_t N) {
  return lora::few_path(T, N) ? lora::few_part_bytes(lora::few_plan(T, K, N), T) : 0;
}

// How the rank-wide product of K inputs is shared: the ring, or parts. N: outputs of the base product of the
// few-token kernel beside which it runs, K0 its inputs (0: none).
int parts_of(int64_t T, int64_t K, int64_t n, int64_t R, int64_t K0, int64_t N) {
  return K0 > 0 && lora::few_path(T, N) ? lora::down_parts_beside(K, K0, N, R)
                                        : lora::down_parts(T, K, R, static_cast<int>(n));
}
size_t join_bytes(int64_t T, int64_t K, int64_t n, int64_t R, int64_t K0, int64_t N) {
  return std::max(lora::ring_bytes(T, K, lora::rank_pad(R)), lora::part_bytes(parts_of(T, K, n, R, K0, N), T, R));
}
void plan_down(lora::RoutedDown& d, int64_t K0, int64_t N) {
  lora::ring_plan(d.T, d.K, &d.splits, &d.ks);
  d.parts = parts_of(d.T, d.K, d.rt.n_adapters, d.rt.rank, K0, N);
}

struct FwdLayout {
  size_t t[3] = {0, 0, 0}, eid = 0, blk = 0, ring = 0, part = 0, few = 0, order = 0, total = 0;
};

FwdLayout fwd_layout(int64_t T, int64_t K, int64_t N, int64_t n, int64_t R) {
  FwdLayout L;
  const int64_t rp = lora::rank_pad(R);
  Take take;
  L.few = take(few_bytes(T, K, N));
  for (size_t& o : L.t) o = take(static_cast<size_t>(T) * rp * 2);  // (the third place is the gradients': not written)
  L.eid = take(static_cast<size_t>(T) * 4);
  L.blk = take(static_cast<size_t>((T + lora::kRouteBlock - 1) / lora::kRouteBlock) * 4);
  if (lora::sorts_tokens(T)) L.order = take(static_cast<size_t>(T) * 8);
  L.ring = take(static_cast<size_t>(lora::ring_blocks(T)) * 4);
  L.part = take(join_bytes(T, K, n, R, K, N));
  L.total = take.off;
  return L;
}

struct BwdLayout {
  size_t wt = 0, bt = 0, at = 0, u[3] = {0, 0, 0}, t[3] = {0, 0, 0}, upart = 0, tpart = 0, eid = 0, blk = 0;
  size_t ring = 0, perm = 0, part[2] = {0, 0}, few = 0, order = 0, total = 0;
  struct {
    size_t first = 0, items = 0;
    int32_t chunk = 0;
    int64_t n_items = 0;
  } table[2];  // dA, dB
};

BwdLayout bwd_layout(int64_t T, int64_t K, int64_t N, int64_t n, int64_t R, bool want_dx) {
  BwdLayout L;
  Take take;
  const int64_t rp = lora::rank_pad(R);
  if (want_dx) {
    L.few = take(few_bytes(T, N, K));
    L.wt = take(static_cast<size_t>(K) * N * 2);
    L.at = take(static_cast<size_t>(n) * K * R * 2);
  }
  L.bt = take(static_cast<size_t>(n) * N * R * 2);
  const size_t tb = static_cast<size_t>(T) * rp * 2;
  for (size_t& o : L.u) o = take(tb);
  for (size_t& o : L.t) o = take(tb);
  // (dx: a layer of N inputs and K outputs)
  L.upart = take(join_bytes(T, N, n, R, want_dx ? N : 0, K));
  L.tpart = take(join_bytes(T, K, n, R, want_dx ? N : 0, K));
  L.eid = take(static_cast<size_t>(T) * 4);
  L.blk = take(static_cast<size_t>((T + lora::kRouteBlock - 1) / lora::kRouteBlock) * 4);
  if (lora::sorts_tokens(T)) L.order = take(static_cast<size_t>(T) * 8);
  L.ring = take(static_cast<size_t>(lora::ring_blocks(T)) * 4);
  L.perm = take(static_cast<size_t>(T) * 4);
  for (int h = 0; h < 2; ++h) {
    auto& tb = L.table[h];
    const int64_t M = h == 0 ? K : N;
    tb.chunk = lora::route_chunk(T, (M + lora::kRtI - 1) / lora::kRtI * ((R + lora::kRtJ - 1) / lora::kRtJ));
    tb.n_items = lora::route_items(T, n, tb.chunk);
    tb.first = take(static_cast<size_t>(n + 1) * 4);
    tb.items = take(static_cast<size_t>(tb.n_items) * sizeof(lora::RouteItem));
    L.part[h] = take(static_cast<size_t>(lora::route_parts(T, tb.chunk)) * M * R * 4);
  }
  L.total = take.off;
  return L;
}

// (a launch has at most 2^32 threads; and items of a contraction, n_adapters + T / 4096 + 1 with so many tokens,
// stay below the 65535 of a grid's y)
constexpr int64_t kMaxTokens = int64_t(1) << 26;
static_assert(LORA_MAX_POOL + kMaxTokens / lora::kRouteMaxChunk + 1 < 65535, "items of a contraction");

bool in_limits(int64_t T, int64_t K, int64_t N, int64_t n, int64_t R) {
  return T < kMaxTokens && K <= kMaxRowBytes / 4 && N <= kMaxRowBytes / 4 && n <= LORA_MAX_POOL && R <= LORA_MAX_RANK;
}

// Checks of the pool and the routing that both directions share.
int check_pool(const lora_pool* pool, const int32_t* token_adapter, const float* token_scale, int64_t T, int64_t K,
               int64_t N) {
  if (pool == nullptr) return LORA_ERR_NULL_PTR;
  if (pool->n_adapters < 0 || pool->rank < 1 || pool->reserved != 0) return LORA_ERR_SHAPE;
  if (!in_limits(T, K, N, pool->n_adapters, pool->rank)) return LORA_ERR_UNSUPPORTED;
  if (pool->n_adapters > 0) {
    if (pool->A == nullptr || pool->B == nullptr || pool->scales == nullptr) return LORA_ERR_NULL_PTR;
    if (T > 0 && token_adapter == nullptr) return LORA_ERR_NULL_PTR;
  }
  if (pool->rank % 8 != 0 || !aligned(pool->A, 16) || !aligned(pool->B, 16) || !aligned(pool->scales, 4) ||
      !aligned(pool->ranks, 4) || !aligned(token_adapter, 4) || !aligned(token_scale, 4))
    return LORA_ERR_ALIGN;
  return LORA_OK;
}

lora::Routing routing(const lora_pool* pool, const int32_t* token_adapter, const float* token_scale) {
  lora::Routing rt;
  rt.token_adapter = token_adapter;
  rt.token_scale = token_scale;
  rt.scales = pool->scales;
  rt.ranks = pool->ranks;
  rt.n_adapters = pool->n_adapters;
  rt.rank = pool->rank;
  return rt;
}

// Everything a routed call reads that depends on the pool and the routing.
void pool_spans(const lora_pool* pool, const int32_t* token_adapter, const float* token_scale, int64_t T, int64_t K,
                int64_t N, Span (&s)[6]) {
  const int64_t n = pool->n_adapters, R = pool->rank;
  s[0] = span2d(pool->A, 1, n * R * K, n * R * K, 2);
  s[1] = span2d(pool->B, 1, n * R * N, n * R * N, 2);
  s[2] = span2d(pool->scales, 1, n, n, 4);
  s[3] = span2d(pool->ranks, 1, n, n, 4);
  s[4] = n > 0 ? span2d(token_adapter, 1, T, T, 4) : Span{};
  s[5] = n > 0 ? span2d(token_scale, 1, T, T, 4) : Span{};
}

// The rank-wide products and the base product with the adapters of the first of them; B [n, N, rank].
hipError_t launch_layer(const void* x, int64_t T, int64_t K, int64_t ldx, const void* W, int64_t N, const void* bias,
                        void* y, int64_t ldy, const lora::RoutedDowns& downs, const void* B, const lora_pool* pool,
                        void* part, hipStream_t s) {
  const lora::RoutedDown& d = downs.d[0];
  lora::RoutedGemm rt;
  rt.B = B; rt.mid = d.mid; rt.eid = d.eid; rt.blk = d.blk; rt.ranks = pool->ranks; rt.rank = pool->rank;
  if (lora::few_path(T, N)) {
    lora::RoutedFew f;
    f.x = static_cast<const uint16_t*>(x); f.ldx = ldx;
    f.W = static_cast<const uint16_t*>(W);
    f.bias = static_cast<const uint16_t*>(bias);
    f.y = static_cast<uint16_t*>(y); f.ldy = ldy;
    f.T = T; f.K = K; f.N = N;
    f.hi = d.hi; f.mid = d.mid; f.ldt = d.ldt;
    f.rt = rt;
    f.part = static_cast<float*>(part); f.order = d.order;
    return lora::launch_routed_few(f, downs, s);
  }
  const hipError_t e = lora::launch_routed_down(downs, s);
  if (e != hipSuccess) return e;
  LinearProblem p;
  std::memset(&p, 0, sizeof(p));
  p.x = x; p.ldx = ldx; p.W = W; p.bias = bias; p.y = y; p.ldy = ldy; p.T = T; p.N = N; p.K = K;
  p.act = Elt::BF16; p.adapter = Elt::BF16;
  p.work = d.hi; p.ldt = d.ldt;
  p.routed = true;
  p.rt = rt;
  return lora::launch_routed_gemm(p, s);
}

}  // namespace

extern "C" {

int lora_linear_routed_fwd(const void* x, int64_t T, int64_t K, int64_t ldx, const void* W, int64_t N,
                           const void* bias, const lora_pool* pool, const int32_t* token_adapter,
                           const float* token_scale, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (T < 0 || K < 1 || N < 1 || ldx < K || ldy < N) return LORA_ERR_SHAPE;
  if (ldx > kMaxRowBytes / 2 || ldy > kMaxRowBytes / 2) return LORA_ERR_UNSUPPORTED;
  if (W == nullptr || (T > 0 && (x == nullptr || y == nullptr))) return LORA_ERR_NULL_PTR;
  int st = check_pool(pool, token_adapter, token_scale, T, K, N);
  if (st != LORA_OK) return st;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(y, 2) || !aligned(bias, 2) || !aligned(workspace, 16) ||
      K % 8 != 0 || ldx % 8 != 0)
    return LORA_ERR_ALIGN;
  if (T == 0) return LORA_OK;
  const FwdLayout L = fwd_layout(T, K, N, pool->n_adapters, pool->rank);
  if (workspace == nullptr || workspace_bytes < L.total) return LORA_ERR_WORKSPACE;
  Span in[6];
  pool_spans(pool, token_adapter, token_scale, T, K, N, in);
  const Span sy = span2d(y, T, ldy, N, 2);
  const Span sw{reinterpret_cast<uintptr_t>(workspace), reinterpret_cast<uintptr_t>(workspace) + L.total};
  const Span base[3] = {span2d(x, T, ldx, K, 2), span2d(W, N, K, K, 2), span2d(bias, 1, N, N, 2)};
  if (overlaps(sy, sw)) return LORA_ERR_OVERLAP;
  for (const Span& s : base)
    if (overlaps(sy, s) || overlaps(sw, s)) return LORA_ERR_OVERLAP;
  for (const Span& s : in)
    if (overlaps(sy, s) || overlaps(sw, s)) return LORA_ERR_OVERLAP;

  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  lora::RoutedDown d;
  std::memset(&d, 0, sizeof(d));
  d.x = static_cast<const uint16_t*>(x); d.ldx = ldx; d.T = T; d.K = K;
  d.A = static_cast<const uint16_t*>(pool->A);
  d.rt = routing(pool, token_adapter, token_scale);
  d.hi = reinterpret_cast<uint16_t*>(ws + L.t[0]); d.ldt = lora::rank_pad(pool->rank);
  if (lora::sorts_tokens(T)) d.order = reinterpret_cast<int32_t*>(ws + L.order);
  d.mid = reinterpret_cast<uint16_t*>(ws + L.t[1]);
  d.lo = reinterpret_cast<uint16_t*>(ws + L.t[2]);
  d.terms = 2;
  d.eid = reinterpret_cast<int32_t*>(ws + L.eid);
  d.blk = reinterpret_cast<int32_t*>(ws + L.blk);
  plan_down(d, K, N);
  d.ring = reinterpret_cast<int32_t*>(ws + L.ring);
  d.tpart = reinterpret_cast<float*>(ws + L.part);
  const lora::RoutedDowns downs{{d, d}, 1, 0, 0};
  return launch_layer(x, T, K, ldx, W, N, bias, y, ldy, downs, pool->B, pool, ws + L.few, s) == hipSuccess
             ? LORA_OK : LORA_ERR_HIP;
}

size_t lora_linear_routed_workspace_size(int64_t T, int64_t K, int64_t N, int32_t n_adapters, int32_t rank) {
  if (T <= 0 || K <= 0 || N <= 0 || n_adapters < 0 || rank < 1 || !in_limits(T, K, N, n_adapters, rank)) return 0;
  return fwd_layout(T, K, N, n_adapters, rank).total;
}

int lora_linear_routed_bwd(const void* x, int64_t T, int64_t K, int64_t ldx, const void* W, int64_t N,
                           const lora_pool* pool, const int32_t* token_adapter, const float* token_scale,
                           const void* dy, int64_t lddy, void* dx, int64_t lddx, float* dA, float* dB,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || K < 1 || N < 1 || ldx < K || lddy < N || (dx != nullptr && lddx < K)) return LORA_ERR_SHAPE;
  if (ldx > kMaxRowBytes / 2 || lddy > kMaxRowBytes / 2 || (dx != nullptr && lddx > kMaxRowBytes / 2))
    return LORA_ERR_UNSUPPORTED;
  if ((dx != nullptr && W == nullptr) || (T > 0 && (x == nullptr || dy == nullptr))) return LORA_ERR_NULL_PTR;
  int st = check_pool(pool, token_adapter, token_scale, T, K, N);
  if (st != LORA_OK) return st;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(dy, 16) || !aligned(dx, 2) || !aligned(dA, 4) ||
      !aligned(dB, 4) || !aligned(workspace, 16) || K % 8 != 0 || N % 8 != 0 || ldx % 8 != 0 || lddy % 8 != 0)
    return LORA_ERR_ALIGN;
  const int64_t n = pool->n_adapters, R = pool->rank;
  const BwdLayout L = T > 0 ? bwd_layout(T, K, N, n, R, dx != nullptr) : BwdLayout{};
  if (L.total > 0 && (workspace == nullptr || workspace_bytes < L.total)) return LORA_ERR_WORKSPACE;
  Span in[6];
  pool_spans(pool, token_adapter, token_scale, T, K, N, in);
  const Span sw = L.total ? Span{reinterpret_cast<uintptr_t>(workspace),
                                 reinterpret_cast<uintptr_t>(workspace) + L.total} : Span{};
  const Span outs[4] = {span2d(dx, T, lddx, K, 2), span2d(dA, 1, n * R * K, n * R * K, 4),
                        span2d(dB, 1, n * R * N, n * R * N, 4), sw};
  const Span base[3] = {span2d(x, T, ldx, K, 2), span2d(W, N, K, K, 2), span2d(dy, T, lddy, N, 2)};
  for (int i = 0; i < 4; ++i) {
    for (const Span& s : base)
      if (overlaps(outs[i], s)) return LORA_ERR_OVERLAP;
    for (const Span& s : in)
      if (overlaps(outs[i], s)) return LORA_ERR_OVERLAP;
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return LORA_ERR_OVERLAP;
  }

  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool grads = n > 0 && (dA != nullptr || dB != nullptr);
  if (T == 0) {  // an empty batch: zero gradients
    hipError_t e = hipSuccess;
    if (dA != nullptr) e = lora::zero_fill(dA, n * R * K, s);
    if (e == hipSuccess && dB != nullptr) e = lora::zero_fill(dB, n * R * N, s);
    return e == hipSuccess ? LORA_OK : LORA_ERR_HIP;
  }
  if (dx == nullptr && !grads) return LORA_OK;
  char* ws = static_cast<char*>(workspace);
  auto at16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(ws + off); };
  auto at32 = [&](size_t off) { return reinterpret_cast<int32_t*>(ws + off); };
  const int64_t rp = lora::rank_pad(R);
  // the forward's operand layouts for the input dy: B^T [R, N] and A^T [K, R] of every slot, W^T [K, N]
  lora::TransposeStack stacks[3];
  int n_stacks = 0;
  if (n > 0 && (dx != nullptr || dA != nullptr))
    stacks[n_stacks++] = lora::TransposeStack{static_cast<const uint16_t*>(pool->B), at16(L.bt), N, R, n};
  if (n > 0 && dx != nullptr)
    stacks[n_stacks++] = lora::TransposeStack{static_cast<const uint16_t*>(pool->A), at16(L.at), R, K, n};
  if (dx != nullptr) stacks[n_stacks++] = lora::TransposeStack{static_cast<const uint16_t*>(W), at16(L.wt), N, K, 1};
  lora::RoutePlan plan;
  plan.rt = routing(pool, token_adapter, token_scale);
  const bool plan_first = T <= lora::kPlanFirstT;
  plan.eid = plan_first ? nullptr : at32(L.eid);
  plan.T = T; plan.n_adapters = grads && plan_first ? static_cast<int32_t>(n) : 0; plan.perm = at32(L.perm);
  for (int h = 0; h < 2; ++h)
    plan.table[h] = lora::RouteTable{L.table[h].chunk, at32(L.table[h].first),
                                     reinterpret_cast<lora::RouteItem*>(ws + L.table[h].items), L.table[h].n_items};
  if (lora::launch_route_prepare(plan, stacks, n_stacks, s) != hipSuccess) return LORA_ERR_HIP;
  // u over dy and B^T, t over x and A
  lora::RoutedDown du, dt;
  std::memset(&du, 0, sizeof(du));
  du.T = T;
  du.rt = routing(pool, token_adapter, token_scale);
  du.ldt = rp; du.terms = 3;
  du.eid = at32(L.eid); du.blk = at32(L.blk);
  if (lora::sorts_tokens(T)) du.order = at32(L.order);
  du.ring = reinterpret_cast<int32_t*>(ws + L.ring);
  dt = du;
  du.x = static_cast<const uint16_t*>(dy); du.ldx = lddy; du.K = N;
  du.A = at16(L.bt);
  du.hi = at16(L.u[0]); du.mid = at16(L.u[1]); du.lo = at16(L.u[2]);
  du.tpart = reinterpret_cast<float*>(ws + L.upart);
  dt.x = static_cast<const uint16_t*>(x); dt.ldx = ldx; dt.K = K;
  dt.A = static_cast<const uint16_t*>(pool->A);
  dt.hi = at16(L.t[0]); dt.mid = at16(L.t[1]); dt.lo = at16(L.t[2]);
  dt.tpart = reinterpret_cast<float*>(ws + L.tpart);
  plan_down(du, dx != nullptr ? N : 0, K);
  plan_down(dt, dx != nullptr ? N : 0, K);
  const bool want_u = dx != nullptr || dA != nullptr, want_t = dB != nullptr && n > 0;
  lora::RoutedDowns downs{{want_u ? du : dt, dt}, want_u && want_t ? 2 : 1, 0, 0};
  const hipError_t e = dx != nullptr ? launch_layer(dy, T, N, lddy, at16(L.wt), K, nullptr, dx, lddx, downs, at16(L.at),
                                                    pool, ws + L.few, s)
                                     : lora::launch_routed_down(downs, s);
  if (e != hipSuccess) return LORA_ERR_HIP;
  if (!grads) return LORA_OK;
  plan.n_adapters = static_cast<int32_t>(n);
  if (!plan_first && lora::launch_route_prepare(plan, nullptr, 0, s) != hipSuccess) return LORA_ERR_HIP;
  lora::RoutedContracts c;
  std::memset(&c, 0, sizeof(c));
  c.rank = static_cast<int32_t>(R); c.ranks = pool->ranks; c.n_adapters = plan.n_adapters; c.perm = plan.perm;
  if (dA != nullptr)
    c.c[c.n++] = lora::RoutedContract{static_cast<const uint16_t*>(x), ldx, K, {du.hi, du.mid, du.lo}, rp, plan.table[0],
                                      reinterpret_cast<float*>(ws + L.part[0]), dA, true};
  if (dB != nullptr)
    c.c[c.n++] = lora::RoutedContract{static_cast<const uint16_t*>(dy), lddy, N, {dt.hi, dt.mid, dt.lo}, rp, plan.table[1],
                                      reinterpret_cast<float*>(ws + L.part[1]), dB, false};
  return lora::launch_routed_contract(c, s) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

size_t lora_linear_routed_bwd_workspace_size(int64_t T, int64_t K, int64_t N, int32_t n_adapters, int32_t rank,
                                             int32_t want_dx) {
  if (T <= 0 || K <= 0 || N <= 0 || n_adapters < 0 || rank < 1 || !in_limits(T, K, N, n_adapters, rank)) return 0;
  return bwd_layout(T, K, N, n_adapters, rank, want_dx != 0).total;
}

}  // extern "C"
