// The routed linear layer's and the AdamW step's host code under AddressSanitizer and
// UndefinedBehaviorSanitizer: linked with host stand-ins for the kernel launchers, which check that every
// workspace region handed to a kernel lies inside the caller's buffer (sized by the documented query) and that
// regions written by one launch do not overlap, and driven with random shapes. No GPU code runs.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <utility>
#include <vector>

#include "adamw.hpp"
#include "backward.hpp"
#include "lora_mi355x.h"
#include "routed.hpp"

namespace {
uintptr_t ws_lo, ws_hi;
int failures = 0, launches = 0;
std::vector<std::pair<uintptr_t, uintptr_t>> live;  // regions that must stay intact until the call's end

void fail(const char* what) {
  std::printf("FAILED: %s\n", what);
  ++failures;
}

void inside(const void* p, size_t n, const char* what, bool keep = false) {
  if (n == 0) return;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + n;
  if (lo < ws_lo || hi > ws_hi || lo % 16 != 0) fail(what);
  if (keep) {
    for (auto& r : live)
      if (lo < r.second && r.first < hi) fail(what);
    live.emplace_back(lo, hi);
  }
}
}  // namespace

namespace lora {
hipError_t zero_fill(float*, int64_t, hipStream_t) { return hipSuccess; }
static void check_downs(const RoutedDowns& p) {
  if (p.n < 1 || p.n > 2) fail("producer count");
  for (int i = 0; i < p.n; ++i) {
    const RoutedDown& d = p.d[i];
    const size_t t = static_cast<size_t>(d.T) * d.ldt * 2;
    inside(d.hi, t, "hi", true);
    if (d.mid != nullptr) inside(d.mid, t, "mid", true), inside(d.lo, t, "lo", true);
    const int joins = d.splits > 0 ? d.splits : d.parts;
    if (joins < 1 || joins > 8) fail("parts");
    if (joins > 1) inside(d.tpart, static_cast<size_t>(joins) * d.T * d.ldt * 4, "partial sums", true);
    const int64_t nk = (d.K * 2 + 127) / 128;
    if (d.splits > 0 && (static_cast<int64_t>(d.splits) * d.ks < nk || static_cast<int64_t>(d.splits - 1) * d.ks >= nk))
      fail("split of K");
    if (i > 0) continue;
    inside(d.eid, static_cast<size_t>(d.T) * 4, "eid", true);
    inside(d.blk, static_cast<size_t>((d.T + 15) / 16) * 4, "blk", true);
    if (d.splits > 0) inside(d.ring, static_cast<size_t>(ring_blocks(d.T)) * 4, "ring", true);
    if (d.order != nullptr) inside(d.order, static_cast<size_t>(d.T) * 8, "order", true);
    if (sorts_tokens(d.T) != (d.order != nullptr)) fail("order given where it is used");
  }
}
hipError_t launch_routed_down(RoutedDowns p, hipStream_t) {
  ++launches;
  check_downs(p);
  return hipSuccess;
}
hipError_t launch_routed_few(const RoutedFew& p, const RoutedDowns& downs, hipStream_t) {
  ++launches;
  check_downs(downs);
  for (int i = 0; i < downs.n; ++i)
    if (downs.d[i].splits != 0) fail("a producer beside the base product has no ring");
  const FewPlan f = few_plan(p.T, p.K, p.N);
  const int64_t nk = (p.K + 63) / 64;
  if (static_cast<int64_t>(f.splits) * f.stages < nk || static_cast<int64_t>(f.splits - 1) * f.stages >= nk) fail("parts of K");
  inside(p.part, few_part_bytes(f, p.T), "partial sums of the base product", true);
  if (p.mid == nullptr) fail("mid");
  return hipSuccess;
}
hipError_t launch_routed_gemm(const LinearProblem& p, hipStream_t) {
  ++launches;
  if (!p.routed || p.n_groups != 0) fail("gemm problem");
  return hipSuccess;
}
hipError_t launch_route_prepare(const RoutePlan& p, const TransposeStack* s, int n, hipStream_t) {
  ++launches;
  if (n < 0 || n > kTransposeStacks) fail("transpose count");
  for (int i = 0; i < n; ++i) inside(s[i].dst, static_cast<size_t>(s[i].slots) * s[i].R * s[i].C * 2, "transposed copy", true);
  if (p.n_adapters == 0) return hipSuccess;
  inside(p.perm, static_cast<size_t>(p.T) * 4, "perm", true);
  for (const RouteTable& t : p.table) {
    if (t.chunk < 64 || t.chunk > kRouteMaxChunk) fail("chunk");
    inside(t.first, static_cast<size_t>(p.n_adapters + 1) * 4, "first", true);
    inside(t.items, static_cast<size_t>(t.n_items) * sizeof(RouteItem), "items", true);
    // the most items and slots that any division of the tokens among the adapters can need
    std::mt19937 g(static_cast<unsigned>(p.T * 31 + p.n_adapters));
    for (int k = 0; k < 20; ++k) {
      int64_t left = p.T, items = 0, slots = 0;
      for (int a = 0; a < p.n_adapters; ++a) {
        int64_t n = a + 1 == p.n_adapters ? left : static_cast<int64_t>(g() % static_cast<uint64_t>(left + 1));
        if (k % 2) n = std::min<int64_t>(left, t.chunk + 1);
        left -= n;
        const int64_t it = n > 0 ? (n + t.chunk - 1) / t.chunk : 1;
        items += it;
        slots += it > 1 ? it : 0;
      }
      if (items > t.n_items) fail("items exceed their table");
      if (slots > route_parts(p.T, t.chunk)) fail("slots exceed the partial sums");
    }
  }
  return hipSuccess;
}
hipError_t launch_routed_contract(RoutedContracts p, hipStream_t) {
  ++launches;
  for (int i = 0; i < p.n; ++i) {
    const RoutedContract& c = p.c[i];
    inside(c.part, static_cast<size_t>(c.M) * p.rank * 4, "gradient partial sums", true);
    for (const uint16_t* q : c.q) inside(q, 16, "rank-wide operand");
  }
  return hipSuccess;
}
hipError_t launch_adam_upload(const AdamTensor* t, int n, int first, int32_t chunk, void* table, int32_t n_tensors, hipStream_t) {
  ++launches;
  if (n < 1 || n > kAdamUpload || first < 0 || first + n > n_tensors) fail("upload");
  for (int i = 0; i < n; ++i) {
    const int64_t b = (t[i].t.n + chunk - 1) / chunk;
    inside(static_cast<char*>(table) + static_cast<size_t>(first + i) * sizeof(AdamTensor) / 16 * 16, sizeof(AdamTensor), "table");
    if (b > 0) {
      const char* lo = static_cast<char*>(table) + adam_table_shares(n_tensors) + t[i].first_block * sizeof(AdamShare);
      const uintptr_t l = reinterpret_cast<uintptr_t>(lo);
      if (l < ws_lo || l + b * sizeof(AdamShare) > ws_hi) fail("shares");
    }
  }
  return hipSuccess;
}
hipError_t launch_adam_step(const lora_adamw_plan_t&, const AdamConst&, hipStream_t) { ++launches; return hipSuccess; }
}  // namespace lora

int main() {
  std::mt19937_64 g(7);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + static_cast<int64_t>(g() % static_cast<uint64_t>(hi - lo + 1)); };
  auto dev = [](int i) { return reinterpret_cast<void*>(uintptr_t(0x100000000000) * (i + 1)); };  // never read
  const uintptr_t ws = 0x7e0000000000;
  for (int k = 0; k < 4000; ++k) {
    const int64_t T = k % 3 ? pick(1, 300) : pick(1, 60000), K = 8 * pick(1, k % 2 ? 64 : 2000), N = 8 * pick(1, k % 2 ? 64 : 2000);
    const int64_t n = pick(0, k % 5 ? 40 : 8192), R = 8 * pick(1, 128);
    const lora_pool pool{dev(0), dev(1), static_cast<float*>(dev(2)), nullptr, static_cast<int32_t>(n), static_cast<int32_t>(R), 0};
    size_t need = lora_linear_routed_workspace_size(T, K, N, static_cast<int32_t>(n), static_cast<int32_t>(R));
    ws_lo = ws, ws_hi = ws + need;
    live.clear();
    auto* w = reinterpret_cast<void*>(ws);
    auto* ids = static_cast<int32_t*>(dev(3));
    int st = lora_linear_routed_fwd(dev(4), T, K, K, dev(5), N, nullptr, &pool, ids, nullptr, dev(6), N, w, need, nullptr);
    if (st != LORA_OK) fail("forward status");
    if (lora_linear_routed_fwd(dev(4), T, K, K, dev(5), N, nullptr, &pool, ids, nullptr, dev(6), N, w, need - 1, nullptr) !=
        LORA_ERR_WORKSPACE)
      fail("short forward workspace");
    const bool want = k % 4 != 0;
    need = lora_linear_routed_bwd_workspace_size(T, K, N, static_cast<int32_t>(n), static_cast<int32_t>(R), want);
    ws_lo = ws, ws_hi = ws + need;
    live.clear();
    st = lora_linear_routed_bwd(dev(4), T, K, K, dev(5), N, &pool, ids, nullptr, dev(7), N, want ? dev(6) : nullptr, K,
                                k % 7 ? static_cast<float*>(dev(8)) : nullptr, k % 11 ? static_cast<float*>(dev(9)) : nullptr,
                                w, need, nullptr);
    if (st != LORA_OK) fail("backward status");
  }
  for (int k = 0; k < 500; ++k) {
    std::vector<lora_adamw_tensor> ts;
    const int n = static_cast<int>(pick(1, 200));
    const bool eight = k % 2;
    uintptr_t at = 0x100000000000;
    auto take = [&](int64_t bytes) {
      const uintptr_t p = at;
      at += (bytes + 31) / 16 * 16;
      return reinterpret_cast<void*>(p);
    };
    for (int i = 0; i < n; ++i) {
      lora_adamw_tensor t;
      std::memset(&t, 0, sizeof(t));
      t.n = pick(0, 20) == 0 ? 0 : pick(1, k % 5 ? 5000 : 400000);
      t.param = take(t.n * 2);
      t.master = i % 3 ? static_cast<float*>(take(t.n * 4)) : nullptr;
      t.grad = take(t.n * 4);
      t.m = take(t.n * (eight ? 1 : 4));
      t.v = take(t.n * (eight ? 1 : 4));
      if (eight) t.m_scale = static_cast<float*>(take((t.n + 255) / 256 * 4)), t.v_scale = static_cast<float*>(take((t.n + 255) / 256 * 4));
      ts.push_back(t);
    }
    const size_t need = lora_adamw_table_size(ts.data(), n);
    ws_lo = ws, ws_hi = ws + need;
    lora_adamw_plan_t plan;
    if (lora_adamw_plan(ts.data(), n, LORA_BF16, LORA_F32, eight ? 8 : 32, reinterpret_cast<void*>(ws), need, &plan, nullptr) != LORA_OK)
      fail("plan status");
    if (lora_adamw_plan(ts.data(), n, LORA_BF16, LORA_F32, eight ? 8 : 32, reinterpret_cast<void*>(ws), need - 1, &plan, nullptr) !=
        LORA_ERR_WORKSPACE)
      fail("short table");
    if (lora_adamw_step(&plan, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1, nullptr, 1.0, nullptr) != LORA_OK) fail("step status");
    if (ts[0].n > 0) {
      ts[0].m = ts[0].param;
      if (lora_adamw_plan(ts.data(), n, LORA_BF16, LORA_F32, eight ? 8 : 32, reinterpret_cast<void*>(ws), need, &plan, nullptr) !=
          LORA_ERR_OVERLAP)
        fail("overlap");
    }
  }
  std::printf("%d launches, %d failures\n", launches, failures);
  return failures != 0;
}
