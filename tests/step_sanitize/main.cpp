// The host code of a fine-tuning step's operators under AddressSanitizer and UndefinedBehaviorSanitizer: linked with host
// stand-ins for the kernel launchers, which check that every workspace region handed to a kernel lies inside the caller's
// buffer (of exactly the size that the query names) and that regions that are in use together do not overlap, and driven
// with random shapes. No GPU code runs.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <utility>
#include <vector>

#include "backward.hpp"
#include "lora_mi355x.h"
#include "loss.hpp"
#include "step.hpp"

namespace {
uintptr_t ws_lo, ws_hi, sv_lo, sv_hi;  // the workspace; what a forward keeps
int failures = 0, launches = 0;
std::vector<std::pair<uintptr_t, uintptr_t>> live;  // regions that must stay as they are until the call's end

void fail(const char* what) {
  std::printf("FAILED: %s\n", what);
  ++failures;
}

// Written by a launch (keep: read by a later one).
void writes(const void* p, size_t n, const char* what, bool keep) {
  if (n == 0) return;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + n;
  if (!((lo >= ws_lo && hi <= ws_hi) || (lo >= sv_lo && hi <= sv_hi)) || lo % 16 != 0) fail(what);
  for (auto& r : live)
    if (lo < r.second && r.first < hi) fail(what);
  if (keep) live.emplace_back(lo, hi);
}

void reads(const void* p, size_t n, const char* what) {  // something that a launch of this call left, or the caller's
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + n;
  if (lo >= ws_lo && lo < ws_hi) {
    for (auto& r : live)
      if (lo >= r.first && hi <= r.second) return;
    fail(what);
  } else if (lo >= sv_lo && lo < sv_hi && hi > sv_hi) {
    fail(what);
  }
}

size_t rows(int64_t T, int64_t ld, int e) { return static_cast<size_t>(T) * static_cast<size_t>(ld) * e; }
}  // namespace

namespace lora {
hipError_t zero_fill(float*, int64_t, hipStream_t) { return hipSuccess; }

hipError_t launch_rank_products(const RankProduct* nt, const RankProduct* nn, hipStream_t) {
  ++launches;
  size_t mark = live.size();
  for (int i = 0; i < 2; ++i) {
    const RankProduct* p = i ? nn : nt;
    if (p == nullptr) continue;
    const int64_t R = p->rank[0] + p->rank[1];
    if (R < 8 || (i && p->rank[1] != 0)) fail("rank");
    for (int s = 0; s < 2; ++s)
      if (p->rank[s] > 0 && p->A[s] == nullptr) fail("an adapter that is not there");
    // (the partial sums of both are in use together, and the results)
    writes(p->part, rank_part_bytes(p->T, p->K, R, i == 1), "partial sums", true);
    writes(p->tt, rows(p->T, pair_ld(R), 2), "rank-wide rows", true);
  }
  std::vector<std::pair<uintptr_t, uintptr_t>> stay(live.begin(), live.begin() + mark);
  for (size_t i = mark; i < live.size(); ++i)
    for (const RankProduct* p : {nt, nn})
      if (p != nullptr && live[i].first == reinterpret_cast<uintptr_t>(p->tt)) stay.push_back(live[i]);
  live = stay;
  return hipSuccess;
}

static void check_ring(const RingArgs& p, int64_t columns) {
  ++launches;
  if (p.tt != nullptr) reads(p.tt, rows(p.T + p.terms, p.ldt, 2), "rank-wide rows of a GEMM");
  if (p.tt != nullptr && p.ldt != pair_ld(p.re[0] + p.re[1])) fail("their stride");
  if (p.terms != 0 && (p.terms != kTerms || p.T > kTerms || p.n_seg != 2)) fail("second terms");
  writes(p.part, p.terms ? terms_part_bytes(columns, ring_stages(p)) : ring_part_bytes(p.T, columns, ring_stages(p)),
         "parts of tiles", false);
  const RingPlan r = p.terms ? terms_plan(columns, ring_stages(p)) : ring_plan(p.T, columns, ring_stages(p));
  if (r.S < 1 || static_cast<int64_t>(r.S - 1) * r.ks >= ring_stages(p)) fail("parts of a plan");
  if (r.full < 0 || r.full > r.tiles || static_cast<int64_t>(r.S) * r.ks < ring_stages(p)) fail("plan");
}
hipError_t launch_ring(const RingArgs& p, bool, hipStream_t) {
  for (int i = 0; i < p.n_seg; ++i)
    if (p.n_seg == 2) reads(p.x[i], rows(p.T + p.terms, p.ldx, 2), "segments");
  check_ring(p, p.N);
  return hipSuccess;
}
hipError_t launch_gated(const RingArgs& p, hipStream_t) {
  check_ring(p, 2 * p.N);
  if (p.saved != nullptr) writes(p.saved, gated_saved_bytes(p.T, p.N), "what the forward keeps", true);
  return hipSuccess;
}
hipError_t launch_gated_few(const GatedFew& p, hipStream_t) {
  ++launches;
  if (p.T > 128 || !gated_few(p.T, p.K, p.F)) fail("few tokens");
  writes(p.part, few_part_bytes(p.T, p.K, p.F, p.rank[0] + p.rank[1]), "sums of few tokens", false);
  return hipSuccess;
}
hipError_t launch_gated_grad(const float* saved, const uint16_t*, int64_t, int64_t T, int64_t F, int, uint16_t* dg,
                             uint16_t* du, const RankProduct* v, hipStream_t) {
  ++launches;
  reads(saved, gated_saved_bytes(T, F), "kept by the forward");
  writes(dg, rows(term_rows(T), F, 2), "dg", true);
  writes(du, rows(term_rows(T), F, 2), "du", true);
  int S, per;
  grad_plan(T, F, &S, &per);
  if (S < 1 || S > 32 || static_cast<int64_t>(S - 1) * per >= (F + 63) / 64 || static_cast<int64_t>(S) * per < (F + 63) / 64)
    fail("plan of the gradient");
  if (v != nullptr) {
    const int64_t R = v->rank[0] + v->rank[1];
    if (R < 8 || v->T != T || v->K != F) fail("product");
    writes(v->part, grad_part_bytes(T, F, R), "its partial sums", false);
    writes(v->tt, rows(term_rows(T), pair_ld(R), 2), "its rows", true);
  }
  return hipSuccess;
}
hipError_t launch_contract(const Contract& p, hipStream_t) {
  ++launches;
  int64_t tiles = 0, elements = 0;
  for (int i = 0; i < p.n_tasks; ++i) {
    const ContractTask& k = p.task[i];
    tiles += contract_tiles(k.M, k.J);
    elements += k.M * k.J;
    reads(k.tt, rows(p.T, k.ldt, 2), "rank-wide rows of a contraction");
    reads(k.P, rows(p.T + k.terms - 1, k.ldp, 2) + k.M * 2, "the other side of a contraction");
    if (k.terms != 0 && p.halves != 2) fail("halves of a contraction");
    if (k.q_col + k.J > k.R || 2 * k.R > k.ldt || k.M % 8 != 0 || k.J % 8 != 0) fail("columns of a contraction");
  }
  if (p.n_tasks < 1 || p.n_tasks > kMaxContract) fail("tasks");
  if (p.halves < 1 || p.halves > 2) fail("halves");
  writes(p.part, p.halves * contract_part_bytes(p.T, tiles, elements), "sums of a contraction", false);
  return hipSuccess;
}
hipError_t launch_vocab_loss(const VocabLoss& p, hipStream_t) {
  ++launches;
  writes(p.ref, rows(loss_blocks(p.V), p.T, 4), "powers of two", true);
  writes(p.sum, rows(loss_blocks(p.V), p.T, 4), "block sums", true);
  for (float* t : {p.tlogit, p.top, p.fade, p.rest, p.scale}) writes(t, rows(p.T, 1, 4), "a token's numbers", true);
  if (p.dh != nullptr) {
    if (p.piece < 1 || p.piece % 256 != 0) fail("piece");
    writes(p.share, rows(p.T, p.piece, 2), "shares", true);
    writes(p.shift, rows(loss_blocks(p.piece), shift_ld(p.T), 1), "shifts", true);
    writes(p.part, loss_part_bytes(p.T, p.K, p.V), "parts of dh", true);
  }
  return hipSuccess;
}
}  // namespace lora

namespace {
std::mt19937_64 rng(20250);
int64_t pick(int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(rng() % static_cast<uint64_t>(hi - lo + 1)); }
int64_t size_of(int64_t top) { return pick(0, 3) == 0 ? pick(1, top) : pick(1, top > 300 ? 300 : top); }
int32_t rank_of() { return static_cast<int32_t>(8 * (pick(0, 3) == 0 ? pick(1, 128) : pick(1, 12))); }

constexpr uintptr_t kBase = uintptr_t(1) << 44;
const void* in(int i) { return reinterpret_cast<const void*>(kBase * (i + 1)); }
void* out(int i) { return reinterpret_cast<void*>(kBase * (i + 1)); }

void room(size_t ws, size_t saved) {
  ws_lo = kBase * 100;
  ws_hi = ws_lo + ws;
  sv_lo = kBase * 120;
  sv_hi = sv_lo + saved;
  live.clear();
}
void ok(int code, const char* what) {
  if (code != LORA_OK) {
    std::printf("%s: code %d\n", what, code);
    fail(what);
  }
}
}  // namespace

int main() {
  for (int n = 0; n < 6000; ++n) {
    const int64_t T = size_of(40000), K = 8 * size_of(2500), N = 8 * size_of(2500);
    const int32_t r = rank_of();
    const double strength = pick(0, 9) == 0 ? 0.0 : 1.0, p = pick(0, 2) * 0.1;
    size_t need = lora_linear_dropout_workspace_size(T, K, N, r);
    room(need, 0);
    ok(lora_linear_dropout_fwd(in(0), T, K, K, in(1), N, nullptr, in(2), in(3), r, 1.0, strength, 1.0, p, 1, 2, nullptr,
                               out(4), N, reinterpret_cast<void*>(ws_lo), need, nullptr),
       "dropout forward");
    need = lora_linear_dropout_bwd_workspace_size(T, K, N, r);
    room(need, 0);
    ok(lora_linear_dropout_bwd(in(0), T, K, K, in(1), N, in(2), in(3), r, 1.0, strength, 1.0, p, 1, 2, nullptr, in(4), N,
                               pick(0, 1) ? out(5) : nullptr, K, pick(0, 1) ? out(6) : nullptr,
                               pick(0, 1) ? out(7) : nullptr, pick(0, 1) ? LORA_F32 : LORA_BF16,
                               reinterpret_cast<void*>(ws_lo), need, nullptr),
       "dropout backward");

    lora_gated_layer l;
    std::memset(&l, 0, sizeof(l));
    l.W_gate = in(1);
    l.W_up = in(2);
    if (pick(0, 3) != 0) l.A_gate = in(3), l.B_gate = in(4), l.rank_gate = rank_of(), l.alpha_gate = pick(0, 4) ? 2.0 : 0.0;
    if (pick(0, 3) != 0) l.A_up = in(5), l.B_up = in(6), l.rank_up = rank_of(), l.alpha_up = pick(0, 4) ? 2.0 : 0.0;
    const int64_t F = pick(0, 1) ? N : size_of(20000);
    const int act = static_cast<int>(pick(0, 2));
    for (int64_t t : {T, pick(1, 64)}) {
      need = lora_gated_workspace_size(t, K, F, l.rank_gate, l.rank_up);
      const size_t sv = lora_gated_saved_size(t, F, l.rank_gate, l.rank_up);
      const bool keep = pick(0, 1) != 0;
      room(need, sv);
      ok(lora_gated_fwd(in(0), t, K, K, &l, F, act, strength, 1.0, out(8), F, keep ? reinterpret_cast<void*>(sv_lo) : nullptr,
                        reinterpret_cast<void*>(ws_lo), need, nullptr),
         "gated forward");
      need = lora_gated_bwd_workspace_size(t, K, N, l.rank_gate, l.rank_up);
      const size_t sn = lora_gated_saved_size(t, N, l.rank_gate, l.rank_up);
      room(need, sn);
      const int want = static_cast<int>(pick(0, 31));
      ok(lora_gated_bwd(in(0), t, K, K, &l, N, act, strength, 1.0, in(8), N,
                        keep ? reinterpret_cast<const void*>(sv_lo) : nullptr, want & 1 ? out(9) : nullptr, K,
                        want & 2 && l.A_gate ? out(10) : nullptr, want & 4 && l.A_gate ? out(11) : nullptr,
                        want & 8 && l.A_up ? out(12) : nullptr, want & 16 && l.A_up ? out(13) : nullptr, LORA_F32,
                        reinterpret_cast<void*>(ws_lo), need, nullptr),
         "gated backward");
    }
    const int64_t V = size_of(300000);
    for (int grad = 0; grad < 2; ++grad) {
      need = lora_cross_entropy_workspace_size(T, K, V, grad);
      room(need, 0);
      ok(lora_cross_entropy(in(0), T, K, K, in(1), V, static_cast<const int64_t*>(in(2)), nullptr,
                            static_cast<float*>(out(3)), static_cast<float*>(out(4)), grad ? out(5) : nullptr, K,
                            reinterpret_cast<void*>(ws_lo), need, nullptr),
         "loss");
    }
  }
  std::printf("%d launches, %d failures\n", launches, failures);
  return failures != 0;
}
