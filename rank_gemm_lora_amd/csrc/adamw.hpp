// Internal interface of the AdamW step over many tensors (adamw.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "lora_mi355x.h"

namespace lora {

constexpr int kAdamBlock = 256;  // elements per scale of an 8-bit moment

// One tensor in the device table.
struct AdamTensor {
  lora_adamw_tensor t;
  int64_t first_block;  // its first workgroup
  int32_t vec;          // every buffer aligned for vector accesses
  int32_t pad;
};
// A workgroup's share: elements [chunk . plan.chunk, + plan.chunk) of a tensor.
struct AdamShare {
  int32_t tensor, chunk;
};

// Elements per workgroup. Large totals take 8192 (the look-up of the share and of its tensor is paid once
// per 8192 elements), small ones 2048, so that a single layer's tensors still spread over many compute units.
inline int32_t adam_chunk(int64_t total) { return total >= (int64_t(1) << 22) ? 8192 : 2048; }
constexpr int64_t kAdamMaxBlocks = (int64_t(1) << 24) - 1;  // of 256 threads: a launch has fewer than 2^32
inline size_t adam_table_shares(int32_t n) { return (static_cast<size_t>(n) * sizeof(AdamTensor) + 255) / 256 * 256; }

// Rounded constants of one step (fp32), or the doubles from which the kernel forms them with the
// learning rate and the step number that it reads from the device.
struct AdamConst {
  float b1, c1, b2, c2;  // beta1, 1 - beta1, beta2, 1 - beta2
  float decay, size, root, eps;  // 1 - lr wd, lr / (1 - beta1^k), 1 / sqrt(1 - beta2^k), eps
  float grad_scale;
  double beta1, beta2, wd;
  const double* lr_step;  // device {lr, step}, or null
};

// Writes n <= kAdamUpload tensors, the first of them number `first`, and their shares to the table.
constexpr int kAdamUpload = 40;
hipError_t launch_adam_upload(const AdamTensor* t, int n, int first, int32_t chunk, void* table, int32_t n_tensors,
                              hipStream_t s);
hipError_t launch_adam_step(const lora_adamw_plan_t& p, const AdamConst& c, hipStream_t s);

}  // namespace lora
