// C-ABI of a fine-tuning step's operators: argument validation, workspace layout and the order of the launches. Every
// check runs before any launch.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "backward.hpp"
#include "checks.hpp"
#include "lora_mi355x.h"
#include "loss.hpp"
#include "step.hpp"

namespace {

using lora::aligned;
using lora::Contract;
using lora::Drop;
using lora::kMaxRowBytes;
using lora::overlaps;
using lora::RankProduct;
using lora::RingArgs;
using lora::round_up;
using lora::Span;
using lora::span2d;

// (a launch has at most 2^32 threads, one for 4 elements of the rank-wide rows, of which 2048 ranks have 4096)
constexpr int64_t kMaxTokens = int64_t(1) << 21;

struct Take {  // regions of a workspace, each 256-byte aligned
  size_t off = 0;
  size_t operator()(size_t n) {
    const size_t o = off;
    off = round_up(off + n);
    return o;
  }
};

// One adapter of a call: its rank is 0 where it is absent or its combined scale is +-0.
struct Side {
  const void *A, *B;
  int64_t given, rank;
  float scale;
};

int make_side(Side& s, const void* A, const void* B, int32_t rank, double alpha, double strength, double request_scale) {
  s = Side{A, B, 0, 0, 0.f};
  if ((A == nullptr) != (B == nullptr)) return LORA_ERR_NULL_PTR;
  if (!std::isfinite(alpha)) return LORA_ERR_NONFINITE;
  if (A == nullptr) return LORA_OK;
  if (rank < 1) return LORA_ERR_SHAPE;
  if (rank > LORA_MAX_RANK) return LORA_ERR_UNSUPPORTED;
  if (rank % 8 != 0) return LORA_ERR_ALIGN;
  const double v = (alpha / static_cast<double>(rank)) * strength * request_scale;
  if (std::fabs(v) > FLT_MAX) return LORA_ERR_NONFINITE;
  s.given = rank;
  s.rank = v == 0.0 ? 0 : rank;
  s.scale = static_cast<float>(v);
  return LORA_OK;
}

// Sizes that every call of T tokens, K inputs and N outputs keeps to (row strides: two more of its tensors').
int check_sizes(int64_t T, int64_t K, int64_t N, int64_t ld0, int64_t ld1) {
  if (T >= kMaxTokens || K > kMaxRowBytes / 4 || N > kMaxRowBytes / 4 || ld0 > kMaxRowBytes / 2 || ld1 > kMaxRowBytes / 2)
    return LORA_ERR_UNSUPPORTED;
  // (a launch has at most 2^32 threads, one for 16 elements of [T, N] in the widest)
  if (T * std::max(K, N) >= int64_t(1) << 35) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

// Whether a size query is for sizes that a call takes (others have no workspace: 0).
bool known_sizes(int64_t T, int64_t K, int64_t N, int32_t r0, int32_t r1) {
  return T > 0 && K > 0 && N > 0 && r0 >= 0 && r1 >= 0 && r0 <= LORA_MAX_RANK && r1 <= LORA_MAX_RANK &&
         check_sizes(T, K, N, 0, 0) == LORA_OK;
}

// No output overlaps an input, the workspace or another output.
template <int NO, int NI>
bool clash(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (const Span& in : ins)
      if (overlaps(outs[i], in)) return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

Span bytes_at(const void* p, size_t n) {
  return n ? Span{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + n} : Span{};
}

const uint16_t* bf(const void* p) { return static_cast<const uint16_t*>(p); }
uint16_t* bf(void* p) { return static_cast<uint16_t*>(p); }

size_t tt_bytes(int64_t T, int64_t R) { return R > 0 ? static_cast<size_t>(T) * lora::pair_ld(R) * 2 : 0; }

int64_t stages(int64_t K0, int64_t K1, int64_t R) {
  return (R > 0 ? lora::pair_ld(R) / 64 : 0) + (K0 + 63) / 64 + (K1 + 63) / 64;
}

hipError_t zero_grad(void* g, int64_t n, int32_t dtype, hipStream_t s) {
  if (g == nullptr || n == 0) return hipSuccess;
  // (bf16: pairs; n is a multiple of 8 and the buffer 4-byte aligned)
  return lora::zero_fill(static_cast<float*>(g), dtype == LORA_F32 ? n : n / 2, s);
}

// ------------------------------------------------------------------------------------------- dropout

struct DropLayout {
  size_t tt = 0, ut = 0, part = 0, part2 = 0, total = 0;
};
// one layout for both directions (the forward uses a part of it)
DropLayout drop_layout(int64_t T, int64_t K, int64_t N, int64_t R, bool backward) {
  DropLayout L;
  Take take;
  L.tt = take(tt_bytes(T, R));
  // (an inactive adapter has no extension: fewer stages, other parts)
  size_t part = std::max(lora::rank_part_bytes(T, K, R, false),
                         std::max(lora::ring_part_bytes(T, N, stages(K, 0, R)), lora::ring_part_bytes(T, N, stages(K, 0, 0))));
  if (backward) {
    L.ut = take(tt_bytes(T, R));
    L.part2 = take(lora::rank_part_bytes(T, N, R, true));
    part = std::max(part, std::max(lora::ring_part_bytes(T, K, stages(N, 0, R)), lora::ring_part_bytes(T, K, stages(N, 0, 0))));
    const int64_t ta = lora::contract_tiles(K, R), tb = lora::contract_tiles(N, R);
    part = std::max(part, std::max(lora::contract_part_bytes(T, ta, K * R), lora::contract_part_bytes(T, tb, N * R)));
    part = std::max(part, lora::contract_part_bytes(T, ta + tb, (K + N) * R));
  }
  L.part = take(part);
  L.total = take.off;
  return L;
}

int make_drop(Drop& d, double p, uint64_t seed, uint64_t offset, const uint64_t* rng) {
  if (!std::isfinite(p)) return LORA_ERR_NONFINITE;
  const double thr = std::nearbyint(p * 65536.0);
  if (p < 0.0 || thr > 65535.0) return LORA_ERR_UNSUPPORTED;
  if (!aligned(rng, 8)) return LORA_ERR_ALIGN;
  d.thr = static_cast<uint32_t>(thr);
  d.seed = seed;
  d.offset = offset;
  d.rng = rng;
  return LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_linear_dropout_workspace_size(int64_t T, int64_t K, int64_t N, int32_t rank) {
  if (!known_sizes(T, K, N, rank, 0) || rank == 0) return 0;
  return drop_layout(T, K, N, rank, false).total;
}

size_t lora_linear_dropout_bwd_workspace_size(int64_t T, int64_t K, int64_t N, int32_t rank) {
  if (!known_sizes(T, K, N, rank, 0) || rank == 0) return 0;
  return drop_layout(T, K, N, rank, true).total;
}

int lora_linear_dropout_fwd(const void* x, int64_t T, int64_t K, int64_t ldx, const void* W, int64_t N, const void* bias,
                            const void* A, const void* B, int32_t rank, double alpha, double strength,
                            double request_scale, double p, uint64_t seed, uint64_t offset, const uint64_t* rng, void* y,
                            int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || K < 1 || N < 1 || ldx < K || ldy < N) return LORA_ERR_SHAPE;
  if (int e = check_sizes(T, K, N, ldx, ldy)) return e;
  if (!std::isfinite(strength) || !std::isfinite(request_scale)) return LORA_ERR_NONFINITE;
  Drop drop;
  if (int e = make_drop(drop, p, seed, offset, rng)) return e;
  Side a;
  const double keep = 1.0 - static_cast<double>(drop.thr) / 65536.0;
  if (int e = make_side(a, A, B, rank, alpha, strength, request_scale / keep)) return e;
  if (A == nullptr || W == nullptr || (T > 0 && (x == nullptr || y == nullptr))) return LORA_ERR_NULL_PTR;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(workspace, 16) ||
      !aligned(y, 2) || !aligned(bias, 2) || K % 8 != 0 || ldx % 8 != 0)
    return LORA_ERR_ALIGN;
  const DropLayout L = T > 0 ? drop_layout(T, K, N, a.given, false) : DropLayout{};
  if (L.total > 0 && (workspace == nullptr || workspace_bytes < L.total)) return LORA_ERR_WORKSPACE;
  const Span wsp = bytes_at(workspace, L.total);
  const Span outs[2] = {span2d(y, T, ldy, N, 2), wsp};
  const Span ins[6] = {span2d(x, T, ldx, K, 2), span2d(W, N, K, K, 2), span2d(bias, 1, N, N, 2),
                       span2d(A, rank, K, K, 2), span2d(B, N, rank, rank, 2), span2d(rng, 1, 2, 2, 8)};
  if (clash(outs, ins)) return LORA_ERR_OVERLAP;
  if (T == 0) return LORA_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  RingArgs g;
  std::memset(&g, 0, sizeof(g));
  if (a.rank > 0) {
    RankProduct r;
    std::memset(&r, 0, sizeof(r));
    r.x = bf(x); r.ldx = ldx; r.A[0] = bf(A); r.rank[0] = rank; r.scale[0] = a.scale; r.T = T; r.K = K; r.drop = drop;
    r.part = reinterpret_cast<float*>(ws + L.part);
    r.tt = reinterpret_cast<uint16_t*>(ws + L.tt);
    if (lora::launch_rank_products(&r, nullptr, st) != hipSuccess) return LORA_ERR_HIP;
    g.tt = r.tt; g.ldt = lora::pair_ld(rank); g.E[0] = bf(B); g.re[0] = rank;
  }
  g.x[0] = bf(x); g.ldx = ldx; g.W[0] = bf(W); g.K[0] = K; g.n_seg = 1; g.bias[0] = bf(bias); g.T = T; g.N = N;
  g.y = bf(y); g.ldy = ldy; g.part = reinterpret_cast<float*>(ws + L.part);
  return lora::launch_ring(g, false, st) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

int lora_linear_dropout_bwd(const void* x, int64_t T, int64_t K, int64_t ldx, const void* W, int64_t N, const void* A,
                            const void* B, int32_t rank, double alpha, double strength, double request_scale, double p,
                            uint64_t seed, uint64_t offset, const uint64_t* rng, const void* dy, int64_t lddy, void* dx,
                            int64_t lddx, void* dA, void* dB, int32_t grad_dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (grad_dtype != LORA_F32 && grad_dtype != LORA_BF16) return LORA_ERR_DTYPE;
  if (T < 0 || K < 1 || N < 1 || ldx < K || lddy < N || (dx != nullptr && lddx < K)) return LORA_ERR_SHAPE;
  if (int e = check_sizes(T, K, N, ldx, lddy)) return e;
  if (dx != nullptr && lddx > kMaxRowBytes / 2) return LORA_ERR_UNSUPPORTED;
  if (!std::isfinite(strength) || !std::isfinite(request_scale)) return LORA_ERR_NONFINITE;
  Drop drop;
  if (int e = make_drop(drop, p, seed, offset, rng)) return e;
  Side a;
  const double keep = 1.0 - static_cast<double>(drop.thr) / 65536.0;
  if (int e = make_side(a, A, B, rank, alpha, strength, request_scale / keep)) return e;
  if (A == nullptr || (dx != nullptr && W == nullptr) || (T > 0 && (x == nullptr || dy == nullptr)))
    return LORA_ERR_NULL_PTR;
  const int eg = grad_dtype == LORA_F32 ? 4 : 2;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(dy, 16) ||
      !aligned(workspace, 16) || !aligned(dx, 2) || !aligned(dA, 4) || !aligned(dB, 4) || K % 8 != 0 || N % 8 != 0 ||
      ldx % 8 != 0 || lddy % 8 != 0)
    return LORA_ERR_ALIGN;
  const DropLayout L = T > 0 ? drop_layout(T, K, N, a.given, true) : DropLayout{};
  if (L.total > 0 && (workspace == nullptr || workspace_bytes < L.total)) return LORA_ERR_WORKSPACE;
  const Span wsp = bytes_at(workspace, L.total);
  const Span outs[4] = {span2d(dx, T, lddx, K, 2), span2d(dA, 1, rank * K, rank * K, eg),
                        span2d(dB, 1, N * rank, N * rank, eg), wsp};
  const Span ins[6] = {span2d(x, T, ldx, K, 2), span2d(W, N, K, K, 2), span2d(dy, T, lddy, N, 2),
                       span2d(A, rank, K, K, 2), span2d(B, N, rank, rank, 2), span2d(rng, 1, 2, 2, 8)};
  if (clash(outs, ins)) return LORA_ERR_OVERLAP;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (T == 0 || a.rank == 0) {
    if (zero_grad(dA, static_cast<int64_t>(rank) * K, grad_dtype, st) != hipSuccess ||
        zero_grad(dB, N * static_cast<int64_t>(rank), grad_dtype, st) != hipSuccess)
      return LORA_ERR_HIP;
    if (T == 0) return LORA_OK;
  }
  char* ws = static_cast<char*>(workspace);
  float* part = reinterpret_cast<float*>(ws + L.part);
  const int64_t ldt = lora::pair_ld(rank);
  RankProduct u;
  std::memset(&u, 0, sizeof(u));
  u.rank[0] = rank; u.scale[0] = a.scale; u.T = T;
  RankProduct t = u;
  // u = s dy B, and t = s x' A^T as the forward forms it
  u.x = bf(dy); u.ldx = lddy; u.A[0] = bf(B); u.K = N; u.part = reinterpret_cast<float*>(ws + L.part2);
  u.tt = reinterpret_cast<uint16_t*>(ws + L.ut);
  t.x = bf(x); t.ldx = ldx; t.A[0] = bf(A); t.K = K; t.drop = drop; t.part = part;
  t.tt = reinterpret_cast<uint16_t*>(ws + L.tt);
  const bool need_u = a.rank > 0 && (dx != nullptr || dA != nullptr), need_t = a.rank > 0 && dB != nullptr;
  if ((need_u || need_t) &&
      lora::launch_rank_products(need_t ? &t : nullptr, need_u ? &u : nullptr, st) != hipSuccess)
    return LORA_ERR_HIP;
  if (dx != nullptr) {
    RingArgs g;
    std::memset(&g, 0, sizeof(g));
    if (a.rank > 0) {
      g.tt = u.tt; g.ldt = ldt; g.E[0] = bf(A); g.re[0] = rank;
      g.drop = drop;
    }
    g.x[0] = bf(dy); g.ldx = lddy; g.W[0] = bf(W); g.K[0] = N; g.n_seg = 1; g.T = T; g.N = K;
    g.y = bf(dx); g.ldy = lddx; g.part = part;
    if (lora::launch_ring(g, true, st) != hipSuccess) return LORA_ERR_HIP;
  }
  if (a.rank == 0 || (dA == nullptr && dB == nullptr)) return LORA_OK;
  Contract c;
  std::memset(&c, 0, sizeof(c));
  c.T = T; c.out_bf16 = grad_dtype == LORA_BF16; c.part = part; c.drop = drop; c.halves = 1;
  if (dA != nullptr)  // u^T x'
    c.task[c.n_tasks++] = lora::ContractTask{bf(x), ldx, K, u.tt, ldt, rank, 0, rank, true, true, {dA, nullptr}, rank, 0};
  if (dB != nullptr)  // dy^T t
    c.task[c.n_tasks++] = lora::ContractTask{bf(dy), lddy, N, t.tt, ldt, rank, 0, rank, false, false, {dB, nullptr}, rank, 0};
  return lora::launch_contract(c, st) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"

// ------------------------------------------------------------------------------------------- gated feed-forward

namespace {

struct GatedLayout {
  size_t tt = 0, vt = 0, dg = 0, du = 0, saved = 0, part = 0, total = 0;
};

// (partial sums of the rank-wide product, then of the GEMM's cut tiles)
size_t gated_fwd_part(int64_t T, int64_t K, int64_t F, int64_t R) {
  return std::max(R > 0 ? lora::rank_part_bytes(T, K, R, false) : 0, lora::ring_part_bytes(T, 2 * F, stages(K, 0, R)));
}

GatedLayout gated_fwd_layout(int64_t T, int64_t K, int64_t F, int64_t rg, int64_t ru) {
  GatedLayout L;
  Take take;
  L.tt = take(tt_bytes(T, rg + ru));
  size_t part = 0;
  for (int i = 0; i < 4; ++i) {  // both adapters, or either of them inactive
    const int64_t R = (i & 1 ? 0 : rg) + (i & 2 ? 0 : ru);
    part = std::max(part, gated_fwd_part(T, K, F, R));
    if (lora::gated_few(T, K, F)) part = std::max(part, lora::few_part_bytes(T, K, F, R));
  }
  L.part = take(part);
  L.total = take.off;
  return L;
}

// What the forward keeps for the backward: the blocks of g and u, then the rank-wide rows.
size_t saved_tt_at(int64_t T, int64_t F) { return round_up(lora::gated_saved_bytes(T, F)); }
size_t saved_bytes(int64_t T, int64_t F, int64_t R) { return saved_tt_at(T, F) + round_up(tt_bytes(T, R)); }

GatedLayout gated_bwd_layout(int64_t T, int64_t K, int64_t F, int64_t rg, int64_t ru) {
  GatedLayout L;
  Take take;
  const int64_t R = rg + ru;
  const int64_t rows = lora::term_rows(T);
  L.dg = take(static_cast<size_t>(rows) * F * 2);
  L.du = take(static_cast<size_t>(rows) * F * 2);
  L.vt = take(tt_bytes(rows, R));
  size_t part = gated_fwd_layout(T, K, F, rg, ru).total;
  for (int i = 0; i < 4; ++i) {  // both adapters, or either of them inactive
    const int64_t a = i & 1 ? 0 : rg, b = i & 2 ? 0 : ru;
    if (a + b > 0) {
      part = std::max(part, lora::grad_part_bytes(T, F, a + b));
      const size_t halves = T <= lora::kTerms ? 2 : 1;
      const int64_t ta = lora::contract_tiles(K, a + b), tb = lora::contract_tiles(F, a) + lora::contract_tiles(F, b);
      part = std::max(part, lora::contract_part_bytes(T, ta, K * (a + b)));
      part = std::max(part, halves * lora::contract_part_bytes(T, tb, F * (a + b)));
      part = std::max(part, halves * lora::contract_part_bytes(T, ta + tb, (K + F) * (a + b)));
    }
    const int64_t ns = stages(F, F, a + b);
    part = std::max(part, T <= lora::kTerms ? lora::terms_part_bytes(K, ns) : lora::ring_part_bytes(T, K, ns));
  }
  L.part = take(part);
  L.saved = take(saved_bytes(T, F, R));  // (last: not used where the forward's is given)
  L.total = take.off;
  return L;
}

int check_gated(const lora_gated_layer* l, int64_t T, int64_t K, int64_t F, int32_t act, double strength,
                double request_scale, Side (&s)[2]) {
  if (l == nullptr) return LORA_ERR_NULL_PTR;
  if (act != LORA_ACT_SILU && act != LORA_ACT_GELU && act != LORA_ACT_GELU_TANH) return LORA_ERR_UNSUPPORTED;
  if (!std::isfinite(strength) || !std::isfinite(request_scale)) return LORA_ERR_NONFINITE;
  if (int e = make_side(s[0], l->A_gate, l->B_gate, l->rank_gate, l->alpha_gate, strength, request_scale)) return e;
  if (int e = make_side(s[1], l->A_up, l->B_up, l->rank_up, l->alpha_up, strength, request_scale)) return e;
  if (l->W_gate == nullptr || l->W_up == nullptr) return LORA_ERR_NULL_PTR;
  for (const void* p : {l->W_gate, l->W_up, l->A_gate, l->B_gate, l->A_up, l->B_up})
    if (!aligned(p, 16)) return LORA_ERR_ALIGN;
  if (!aligned(l->b_gate, 2) || !aligned(l->b_up, 2) || K % 8 != 0) return LORA_ERR_ALIGN;
  return LORA_OK;
}

void gated_spans(const lora_gated_layer* l, int64_t K, int64_t F, const Side (&s)[2], Span* out) {
  out[0] = span2d(l->W_gate, F, K, K, 2);
  out[1] = span2d(l->W_up, F, K, K, 2);
  out[2] = span2d(l->b_gate, 1, F, F, 2);
  out[3] = span2d(l->b_up, 1, F, F, 2);
  out[4] = span2d(l->A_gate, s[0].given, K, K, 2);
  out[5] = span2d(l->B_gate, F, s[0].given, s[0].given, 2);
  out[6] = span2d(l->A_up, s[1].given, K, K, 2);
  out[7] = span2d(l->B_up, F, s[1].given, s[1].given, 2);
}

hipError_t gated_forward(const void* x, int64_t T, int64_t K, int64_t ldx, const lora_gated_layer* l, const Side (&s)[2],
                         int64_t F, int32_t act, void* h, int64_t ldh, float* saved, uint16_t* tt, float* part,
                         hipStream_t st) {
  if (saved == nullptr && lora::gated_few(T, K, F)) {
    lora::GatedFew f;
    std::memset(&f, 0, sizeof(f));
    f.x = bf(x); f.ldx = ldx; f.W[0] = bf(l->W_gate); f.W[1] = bf(l->W_up); f.bias[0] = bf(l->b_gate);
    f.bias[1] = bf(l->b_up); f.T = T; f.K = K; f.F = F; f.h = bf(h); f.ldh = ldh; f.act = act; f.part = part;
    for (int i = 0; i < 2; ++i) {
      f.A[i] = bf(s[i].A); f.B[i] = bf(s[i].B); f.rank[i] = static_cast<int>(s[i].rank); f.scale[i] = s[i].scale;
    }
    return lora::launch_gated_few(f, st);
  }
  RingArgs g;
  std::memset(&g, 0, sizeof(g));
  const int64_t R = s[0].rank + s[1].rank;
  if (R > 0) {
    RankProduct r;
    std::memset(&r, 0, sizeof(r));
    r.x = bf(x); r.ldx = ldx; r.T = T; r.K = K; r.part = part; r.tt = tt;
    for (int i = 0; i < 2; ++i) {
      r.A[i] = bf(s[i].A); r.rank[i] = static_cast<int>(s[i].rank); r.scale[i] = s[i].scale;
      g.E[i] = bf(s[i].B); g.re[i] = static_cast<int>(s[i].rank);
    }
    const hipError_t e = lora::launch_rank_products(&r, nullptr, st);
    if (e != hipSuccess) return e;
    g.tt = tt; g.ldt = lora::pair_ld(R);
  }
  g.x[0] = bf(x); g.ldx = ldx; g.W[0] = bf(l->W_gate); g.W[1] = bf(l->W_up); g.K[0] = K; g.n_seg = 1;
  g.bias[0] = bf(l->b_gate); g.bias[1] = bf(l->b_up); g.T = T; g.N = F; g.y = bf(h); g.ldy = ldh; g.act = act;
  g.saved = saved; g.part = part;
  return lora::launch_gated(g, st);
}

}  // namespace

extern "C" {

size_t lora_gated_workspace_size(int64_t T, int64_t K, int64_t F, int32_t rank_gate, int32_t rank_up) {
  if (!known_sizes(T, K, F, rank_gate, rank_up)) return 0;
  return gated_fwd_layout(T, K, F, rank_gate, rank_up).total;
}

size_t lora_gated_saved_size(int64_t T, int64_t F, int32_t rank_gate, int32_t rank_up) {
  if (!known_sizes(T, 1, F, rank_gate, rank_up)) return 0;
  return saved_bytes(T, F, rank_gate + rank_up);
}

size_t lora_gated_bwd_workspace_size(int64_t T, int64_t K, int64_t F, int32_t rank_gate, int32_t rank_up) {
  if (!known_sizes(T, K, F, rank_gate, rank_up)) return 0;
  return gated_bwd_layout(T, K, F, rank_gate, rank_up).total;
}

int lora_gated_fwd(const void* x, int64_t T, int64_t K, int64_t ldx, const lora_gated_layer* layer, int64_t F,
                   int32_t act, double strength, double request_scale, void* h, int64_t ldh, void* saved,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || K < 1 || F < 1 || ldx < K || ldh < F) return LORA_ERR_SHAPE;
  if (int e = check_sizes(T, K, F, ldx, ldh)) return e;
  Side s[2];
  if (int e = check_gated(layer, T, K, F, act, strength, request_scale, s)) return e;
  if (T > 0 && (x == nullptr || h == nullptr)) return LORA_ERR_NULL_PTR;
  if (!aligned(x, 16) || !aligned(h, 2) || !aligned(workspace, 16) || !aligned(saved, 16) || ldx % 8 != 0)
    return LORA_ERR_ALIGN;
  const GatedLayout L = T > 0 ? gated_fwd_layout(T, K, F, s[0].given, s[1].given) : GatedLayout{};
  if (L.total > 0 && (workspace == nullptr || workspace_bytes < L.total)) return LORA_ERR_WORKSPACE;
  const Span outs[3] = {span2d(h, T, ldh, F, 2), bytes_at(workspace, L.total),
                        saved != nullptr && T > 0 ? bytes_at(saved, saved_bytes(T, F, s[0].given + s[1].given)) : Span{}};
  Span ins[9];
  gated_spans(layer, K, F, s, ins);
  ins[8] = span2d(x, T, ldx, K, 2);
  if (clash(outs, ins)) return LORA_ERR_OVERLAP;
  if (T == 0) return LORA_OK;
  char* ws = static_cast<char*>(workspace);
  char* keep = static_cast<char*>(saved);
  uint16_t* tt = reinterpret_cast<uint16_t*>(saved != nullptr ? keep + saved_tt_at(T, F) : ws + L.tt);
  return gated_forward(x, T, K, ldx, layer, s, F, act, h, ldh, static_cast<float*>(saved), tt,
                       reinterpret_cast<float*>(ws + L.part), static_cast<hipStream_t>(stream)) == hipSuccess
             ? LORA_OK
             : LORA_ERR_HIP;
}

int lora_gated_bwd(const void* x, int64_t T, int64_t K, int64_t ldx, const lora_gated_layer* layer, int64_t F,
                   int32_t act, double strength, double request_scale, const void* dh, int64_t lddh, const void* saved,
                   void* dx, int64_t lddx, void* dA_gate, void* dB_gate, void* dA_up, void* dB_up, int32_t grad_dtype,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (grad_dtype != LORA_F32 && grad_dtype != LORA_BF16) return LORA_ERR_DTYPE;
  if (T < 0 || K < 1 || F < 1 || ldx < K || lddh < F || (dx != nullptr && lddx < K)) return LORA_ERR_SHAPE;
  if (int e = check_sizes(T, K, F, ldx, lddh)) return e;
  if (dx != nullptr && lddx > kMaxRowBytes / 2) return LORA_ERR_UNSUPPORTED;
  Side s[2];
  if (int e = check_gated(layer, T, K, F, act, strength, request_scale, s)) return e;
  if (T > 0 && (x == nullptr || dh == nullptr)) return LORA_ERR_NULL_PTR;
  void* grads[2][2] = {{dA_gate, dB_gate}, {dA_up, dB_up}};
  for (int i = 0; i < 2; ++i)
    if (s[i].given == 0 && (grads[i][0] != nullptr || grads[i][1] != nullptr)) return LORA_ERR_NULL_PTR;
  if (!aligned(x, 16) || !aligned(dh, 16) || !aligned(workspace, 16) || !aligned(saved, 16) || !aligned(dx, 2) ||
      !aligned(dA_gate, 4) || !aligned(dB_gate, 4) || !aligned(dA_up, 4) || !aligned(dB_up, 4) || ldx % 8 != 0 ||
      lddh % 8 != 0 || F % 8 != 0)
    return LORA_ERR_ALIGN;
  const GatedLayout L = T > 0 ? gated_bwd_layout(T, K, F, s[0].given, s[1].given) : GatedLayout{};
  const size_t need = saved != nullptr ? L.saved : L.total;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return LORA_ERR_WORKSPACE;
  const int eg = grad_dtype == LORA_F32 ? 4 : 2;
  Span outs[6] = {span2d(dx, T, lddx, K, 2), bytes_at(workspace, need)};
  for (int i = 0; i < 2; ++i) {
    const int64_t na = s[i].given * K, nb = s[i].given * F;
    outs[2 + 2 * i] = span2d(grads[i][0], 1, na, na, eg);
    outs[3 + 2 * i] = span2d(grads[i][1], 1, nb, nb, eg);
  }
  Span ins[11];
  gated_spans(layer, K, F, s, ins);
  ins[8] = span2d(x, T, ldx, K, 2);
  ins[9] = span2d(dh, T, lddh, F, 2);
  ins[10] = saved != nullptr && T > 0 ? bytes_at(saved, saved_bytes(T, F, s[0].given + s[1].given)) : Span{};
  if (clash(outs, ins)) return LORA_ERR_OVERLAP;
  hipStream_t st = static_cast<hipStream_t>(stream);
  for (int i = 0; i < 2; ++i)
    if ((T == 0 || s[i].rank == 0) && (zero_grad(grads[i][0], s[i].given * K, grad_dtype, st) != hipSuccess ||
                                       zero_grad(grads[i][1], s[i].given * F, grad_dtype, st) != hipSuccess))
      return LORA_ERR_HIP;
  if (T == 0) return LORA_OK;
  char* ws = static_cast<char*>(workspace);
  float* part = reinterpret_cast<float*>(ws + L.part);
  const char* keep = saved != nullptr ? static_cast<const char*>(saved) : ws + L.saved;
  if (saved == nullptr) {  // g, u and the rank-wide rows once more
    const hipError_t e = gated_forward(x, T, K, ldx, layer, s, F, act, nullptr, F, reinterpret_cast<float*>(ws + L.saved),
                                       reinterpret_cast<uint16_t*>(ws + L.saved + saved_tt_at(T, F)), part, st);
    if (e != hipSuccess) return LORA_ERR_HIP;
  }
  auto* dg = reinterpret_cast<uint16_t*>(ws + L.dg);
  auto* du = reinterpret_cast<uint16_t*>(ws + L.du);
  const int64_t R = s[0].rank + s[1].rank, ldt = lora::pair_ld(R);
  auto* vt = reinterpret_cast<uint16_t*>(ws + L.vt);
  const bool want_a = dA_gate != nullptr || dA_up != nullptr, want_b = dB_gate != nullptr || dB_up != nullptr;
  RankProduct v;  // v = s d B of each projection
  std::memset(&v, 0, sizeof(v));
  v.T = T; v.K = F; v.part = part; v.tt = vt;
  for (int i = 0; i < 2; ++i) {
    v.A[i] = bf(s[i].B); v.rank[i] = static_cast<int>(s[i].rank); v.scale[i] = s[i].scale;
  }
  if (lora::launch_gated_grad(reinterpret_cast<const float*>(keep), bf(dh), lddh, T, F, act, dg, du,
                              R > 0 && (dx != nullptr || want_a) ? &v : nullptr, st) != hipSuccess)
    return LORA_ERR_HIP;
  const int terms = T <= lora::kTerms ? lora::kTerms : 0;
  if (dx != nullptr) {
    RingArgs g;
    std::memset(&g, 0, sizeof(g));
    if (R > 0) {
      g.tt = vt; g.ldt = ldt;
      for (int i = 0; i < 2; ++i) {
        g.E[i] = bf(s[i].A); g.re[i] = static_cast<int>(s[i].rank);
      }
    }
    g.x[0] = dg; g.x[1] = du; g.ldx = F; g.W[0] = bf(layer->W_gate); g.W[1] = bf(layer->W_up); g.K[0] = g.K[1] = F;
    g.n_seg = 2; g.T = T; g.N = K; g.y = bf(dx); g.ldy = lddx; g.part = part; g.terms = terms;
    if (lora::launch_ring(g, true, st) != hipSuccess) return LORA_ERR_HIP;
  }
  if (R == 0) return LORA_OK;
  if (!want_a && !want_b) return LORA_OK;
  Contract c;
  std::memset(&c, 0, sizeof(c));
  c.T = T; c.out_bf16 = grad_dtype == LORA_BF16; c.part = part; c.halves = want_b && terms > 0 ? 2 : 1;
  const int r0 = static_cast<int>(s[0].rank), r1 = static_cast<int>(s[1].rank), rr = r0 + r1;
  if (want_a)  // v^T x, both projections' rows in one pass over x
    c.task[c.n_tasks++] = lora::ContractTask{bf(x), ldx, K, vt, ldt, rr, 0, rr, true, false,
                                             {r0 > 0 ? dA_gate : nullptr, r1 > 0 ? dA_up : nullptr}, r0, 0};
  const auto* tt = reinterpret_cast<const uint16_t*>(keep + saved_tt_at(T, F));
  if (want_b && r0 > 0)  // d^T t of each projection
    c.task[c.n_tasks++] = lora::ContractTask{dg, F, F, tt, ldt, rr, 0, r0, false, false, {dB_gate, nullptr}, r0, terms};
  if (want_b && r1 > 0)
    c.task[c.n_tasks++] = lora::ContractTask{du, F, F, tt, ldt, rr, r0, r1, false, false, {dB_up, nullptr}, r1, terms};
  return lora::launch_contract(c, st) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"

// ------------------------------------------------------------------------------------------- vocabulary loss

namespace {

struct LossLayout {
  size_t ref = 0, sum = 0, tok[5] = {0, 0, 0, 0, 0}, share = 0, shift = 0, part = 0, total = 0;
  int64_t piece = 0;
};

LossLayout loss_layout(int64_t T, int64_t K, int64_t V, bool grad) {
  LossLayout L;
  Take take;
  const size_t blocks = static_cast<size_t>(lora::loss_blocks(V)) * T * 4;
  L.ref = take(blocks);
  L.sum = take(blocks);
  for (size_t& o : L.tok) o = take(static_cast<size_t>(T) * 4);
  if (grad) {
    L.piece = lora::loss_piece(T, V);
    L.share = take(static_cast<size_t>(T) * L.piece * 2);
    L.shift = take(static_cast<size_t>(lora::loss_blocks(L.piece)) * lora::shift_ld(T));
    L.part = take(lora::loss_part_bytes(T, K, V));
  }
  L.total = take.off;
  return L;
}

constexpr int64_t kMaxVocab = int64_t(1) << 24;
// (launches of at most 2^32 threads: one for 4 elements of dh, and 256 for 128 x 128 logits)
bool known_loss(int64_t T, int64_t K, int64_t V) {
  return V <= kMaxVocab && T * V < int64_t(1) << 37 && T * K < int64_t(1) << 34;
}

}  // namespace

extern "C" {

size_t lora_cross_entropy_workspace_size(int64_t T, int64_t K, int64_t V, int32_t want_grad) {
  if (!known_sizes(T, K, 1, 0, 0) || V <= 0 || !known_loss(T, K, V)) return 0;
  return loss_layout(T, K, V, want_grad != 0).total;
}

int lora_cross_entropy(const void* h, int64_t T, int64_t K, int64_t ldh, const void* W, int64_t V, const int64_t* target,
                       const float* dloss, float* loss, float* lse, void* dh, int64_t lddh, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (T < 0 || K < 1 || V < 1 || ldh < K || (dh != nullptr && lddh < K)) return LORA_ERR_SHAPE;
  if (int e = check_sizes(T, K, 1, ldh, dh != nullptr ? lddh : 0)) return e;
  if (!known_loss(T, K, V)) return LORA_ERR_UNSUPPORTED;
  if (W == nullptr || (T > 0 && (h == nullptr || target == nullptr))) return LORA_ERR_NULL_PTR;
  if (!aligned(h, 16) || !aligned(W, 16) || !aligned(workspace, 16) || !aligned(target, 8) || !aligned(dloss, 4) ||
      !aligned(loss, 4) || !aligned(lse, 4) || !aligned(dh, 2) || K % 8 != 0 || ldh % 8 != 0)
    return LORA_ERR_ALIGN;
  const LossLayout L = T > 0 ? loss_layout(T, K, V, dh != nullptr) : LossLayout{};
  if (L.total > 0 && (workspace == nullptr || workspace_bytes < L.total)) return LORA_ERR_WORKSPACE;
  const Span outs[4] = {span2d(loss, 1, T, T, 4), span2d(lse, 1, T, T, 4), span2d(dh, T, lddh, K, 2),
                        bytes_at(workspace, L.total)};
  const Span ins[4] = {span2d(h, T, ldh, K, 2), span2d(W, V, K, K, 2), span2d(target, 1, T, T, 8),
                       span2d(dloss, 1, T, T, 4)};
  if (clash(outs, ins)) return LORA_ERR_OVERLAP;
  if (T == 0 || (loss == nullptr && lse == nullptr && dh == nullptr)) return LORA_OK;
  char* ws = static_cast<char*>(workspace);
  lora::VocabLoss p;
  std::memset(&p, 0, sizeof(p));
  p.h = bf(h); p.ldh = ldh; p.W = bf(W); p.target = target; p.dloss = dloss; p.T = T; p.K = K; p.V = V;
  p.loss = loss; p.lse = lse; p.dh = bf(dh); p.lddh = lddh;
  p.ref = reinterpret_cast<float*>(ws + L.ref);
  p.sum = reinterpret_cast<float*>(ws + L.sum);
  float** tok[5] = {&p.tlogit, &p.top, &p.fade, &p.rest, &p.scale};
  for (int i = 0; i < 5; ++i) *tok[i] = reinterpret_cast<float*>(ws + L.tok[i]);
  p.share = reinterpret_cast<uint16_t*>(ws + L.share);
  p.piece = L.piece;
  p.shift = reinterpret_cast<uint8_t*>(ws + L.shift);
  p.part = reinterpret_cast<float*>(ws + L.part);
  return lora::launch_vocab_loss(p, static_cast<hipStream_t>(stream)) == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"
