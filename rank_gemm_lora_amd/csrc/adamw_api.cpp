// C-ABI of the AdamW step over many tensors: argument validation, the device table and the constants.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <vector>

#include "adamw.hpp"
#include "checks.hpp"

namespace {

using lora::aligned;
using lora::Span;

int esz(int d) { return d == LORA_BF16 ? 2 : 4; }

Span span(const void* p, int64_t n, int64_t esize) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  Span s;
  if (p != nullptr && n > 0) s.lo = lo, s.hi = lo + static_cast<uintptr_t>(n * esize);
  return s;
}

constexpr int64_t kMaxElements = int64_t(1) << 36;  // (workgroups of 256: a launch has at most 2^32 threads)

int64_t total_of(const lora_adamw_tensor* t, int32_t n) {
  int64_t total = 0;
  for (int32_t i = 0; i < n && total <= kMaxElements; ++i) total += std::clamp<int64_t>(t[i].n, 0, kMaxElements + 1);
  return total;
}

int64_t blocks_of(const lora_adamw_tensor* t, int32_t n, int32_t chunk) {
  int64_t b = 0;
  for (int32_t i = 0; i < n; ++i) b += (std::max<int64_t>(0, t[i].n) + chunk - 1) / chunk;
  return b;
}

size_t table_bytes_of(const lora_adamw_tensor* t, int32_t n) {
  return lora::adam_table_shares(n) +
         static_cast<size_t>(blocks_of(t, n, lora::adam_chunk(total_of(t, n)))) * sizeof(lora::AdamShare);
}

}  // namespace

extern "C" {

size_t lora_adamw_table_size(const lora_adamw_tensor* tensors, int32_t n_tensors) {
  if (n_tensors <= 0 || tensors == nullptr || total_of(tensors, n_tensors) > kMaxElements) return 0;
  return table_bytes_of(tensors, n_tensors);
}

int lora_adamw_plan(const lora_adamw_tensor* tensors, int32_t n_tensors, int32_t param_dtype, int32_t grad_dtype,
                    int32_t state_bits, void* table, size_t table_bytes, lora_adamw_plan_t* plan, void* stream) {
  if (plan == nullptr) return LORA_ERR_NULL_PTR;
  if ((param_dtype != LORA_F32 && param_dtype != LORA_BF16) || (grad_dtype != LORA_F32 && grad_dtype != LORA_BF16))
    return LORA_ERR_DTYPE;
  if (state_bits != 32 && state_bits != 8) return LORA_ERR_UNSUPPORTED;
  if (n_tensors < 0) return LORA_ERR_SHAPE;
  if (n_tensors > 0 && tensors == nullptr) return LORA_ERR_NULL_PTR;
  const bool eight = state_bits == 8;
  const int ep = esz(param_dtype), eg = esz(grad_dtype), em = eight ? 1 : 4;
  int64_t total = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const lora_adamw_tensor& t = tensors[i];
    if (t.n < 0) return LORA_ERR_SHAPE;
    if (t.n > kMaxElements || (total += t.n) > kMaxElements) return LORA_ERR_UNSUPPORTED;
    if (t.master != nullptr && param_dtype != LORA_BF16) return LORA_ERR_DTYPE;  // an fp32 parameter is its own master
    if (t.n == 0) continue;
    if (t.param == nullptr || t.grad == nullptr || t.m == nullptr || t.v == nullptr) return LORA_ERR_NULL_PTR;
    if (eight != (t.m_scale != nullptr) || eight != (t.v_scale != nullptr)) return LORA_ERR_NULL_PTR;
    if (!aligned(t.param, ep) || !aligned(t.master, 4) || !aligned(t.grad, eg) || !aligned(t.m, em) ||
        !aligned(t.v, em) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
      return LORA_ERR_ALIGN;
  }
  if (!aligned(table, 16)) return LORA_ERR_ALIGN;
  const int32_t chunk = lora::adam_chunk(total);
  const int64_t blocks = blocks_of(tensors, n_tensors, chunk);
  if (blocks > lora::kAdamMaxBlocks) return LORA_ERR_UNSUPPORTED;
  const size_t need = n_tensors > 0 ? table_bytes_of(tensors, n_tensors) : 0;
  if (need > 0 && (table == nullptr || table_bytes < need)) return LORA_ERR_WORKSPACE;

  // what is written must not overlap anything else: spans in order, each against the furthest end so far
  struct Use {
    Span s;
    bool written;
  };
  std::vector<Use> uses;
  try {
    uses.reserve(static_cast<size_t>(n_tensors) * 7 + 1);
  } catch (...) {
    return LORA_ERR_UNSUPPORTED;
  }
  auto use = [&](const Span& s, bool written) {
    if (!s.empty()) uses.push_back(Use{s, written});
  };
  use(span(table, static_cast<int64_t>(need), 1), true);
  for (int32_t i = 0; i < n_tensors; ++i) {
    const lora_adamw_tensor& t = tensors[i];
    const int64_t nb = (t.n + lora::kAdamBlock - 1) / lora::kAdamBlock;
    use(span(t.param, t.n, ep), true);
    use(span(t.master, t.n, 4), true);
    use(span(t.grad, t.n, eg), false);
    use(span(t.m, t.n, em), true);
    use(span(t.v, t.n, em), true);
    use(span(t.m_scale, nb, 4), true);
    use(span(t.v_scale, nb, 4), true);
  }
  std::sort(uses.begin(), uses.end(), [](const Use& a, const Use& b) { return a.s.lo < b.s.lo; });
  uintptr_t end_written = 0, end_any = 0;
  for (const Use& u : uses) {
    if (u.s.lo < end_written || (u.written && u.s.lo < end_any)) return LORA_ERR_OVERLAP;
    end_any = std::max(end_any, u.s.hi);
    if (u.written) end_written = std::max(end_written, u.s.hi);
  }

  hipStream_t s = static_cast<hipStream_t>(stream);
  lora::AdamTensor batch[lora::kAdamUpload];
  int64_t first_block = 0;
  for (int32_t i = 0; i < n_tensors; i += lora::kAdamUpload) {
    const int n = std::min<int32_t>(lora::kAdamUpload, n_tensors - i);
    for (int k = 0; k < n; ++k) {
      const lora_adamw_tensor& t = tensors[i + k];
      batch[k].t = t;
      batch[k].first_block = first_block;
      const uintptr_t am = eight ? 8 : 16;
      batch[k].vec = aligned(t.param, 16) && aligned(t.master, 16) && aligned(t.grad, 16) && aligned(t.m, am) &&
                     aligned(t.v, am);
      batch[k].pad = 0;
      first_block += (t.n + chunk - 1) / chunk;
    }
    if (lora::launch_adam_upload(batch, n, i, chunk, table, n_tensors, s) != hipSuccess) return LORA_ERR_HIP;
  }
  *plan = lora_adamw_plan_t{table, blocks, n_tensors, chunk, param_dtype, grad_dtype, state_bits, 0};
  return LORA_OK;
}

int lora_adamw_step(const lora_adamw_plan_t* plan, double lr, double beta1, double beta2, double eps,
                    double weight_decay, int64_t step, const double* lr_step, double grad_scale, void* stream) {
  if (plan == nullptr) return LORA_ERR_NULL_PTR;
  if (plan->reserved != 0 || plan->n_blocks < 0 || plan->n_blocks > lora::kAdamMaxBlocks || plan->n_tensors < 0)
    return LORA_ERR_SHAPE;
  if (plan->n_blocks > 0 && plan->table == nullptr) return LORA_ERR_NULL_PTR;
  if ((plan->param_dtype != LORA_F32 && plan->param_dtype != LORA_BF16) ||
      (plan->grad_dtype != LORA_F32 && plan->grad_dtype != LORA_BF16))
    return LORA_ERR_DTYPE;
  if ((plan->state_bits != 32 && plan->state_bits != 8) || (plan->chunk != 2048 && plan->chunk != 8192))
    return LORA_ERR_UNSUPPORTED;
  if (!aligned(lr_step, 8)) return LORA_ERR_ALIGN;
  for (const double v : {beta1, beta2, eps, weight_decay, grad_scale})
    if (!std::isfinite(v)) return LORA_ERR_NONFINITE;
  if (lr_step == nullptr && !std::isfinite(lr)) return LORA_ERR_NONFINITE;
  if (std::fabs(grad_scale) > FLT_MAX || (lr_step == nullptr && std::fabs(lr) > FLT_MAX)) return LORA_ERR_NONFINITE;
  if (beta1 < 0 || beta1 >= 1 || beta2 < 0 || beta2 >= 1 || eps < 0 || weight_decay < 0 ||
      (lr_step == nullptr && (lr < 0 || step < 1)))
    return LORA_ERR_UNSUPPORTED;
  if (plan->n_blocks == 0) return LORA_OK;
  lora::AdamConst c;
  c.b1 = static_cast<float>(beta1); c.c1 = static_cast<float>(1.0 - beta1);
  c.b2 = static_cast<float>(beta2); c.c2 = static_cast<float>(1.0 - beta2);
  c.eps = static_cast<float>(eps); c.grad_scale = static_cast<float>(grad_scale);
  c.beta1 = beta1; c.beta2 = beta2; c.wd = weight_decay; c.lr_step = lr_step;
  c.decay = c.size = c.root = 0.f;
  if (lr_step == nullptr) {
    const double k = static_cast<double>(step);
    c.decay = static_cast<float>(1.0 - lr * weight_decay);
    c.size = static_cast<float>(lr / (1.0 - std::pow(beta1, k)));
    c.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, k)));
  }
  const hipError_t e = lora::launch_adam_step(*plan, c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // extern "C"
