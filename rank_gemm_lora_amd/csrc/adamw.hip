// One AdamW step over many tensors (the adapters' A and B of every layer) in one launch:
//
//   g = grad_scale . grad
//   m = b1 . m + g . (1 - b1),  v = b2 . v + (g . g) . (1 - b2)
//   p = p . (1 - lr wd) - (m / (sqrt(v) . 1 / sqrt(1 - b2^k) + eps)) . lr / (1 - b1^k)
//
// every operation in fp32, rounded once, in this order (built with floating-point contraction off).
// Moments in 8 bits: m and sqrt(v) as e4m3 with one fp32 scale per 256 elements, scale = largest
// magnitude . RN(1 / 448); a value x is stored as RN_e4m3(x . (448 . RN(1 / largest))). The root is stored rather
// than v, whose range is the square of what 8 bits hold. A positive root never becomes zero (it takes
// the smallest e4m3, 2^-9): rounded down to zero it would leave eps alone under the update. The step
// itself uses the new moments before they are rounded.
//
// HBM-bound: an element moves 30 bytes (fp32 moments and gradient, fp32 master, bf16 copy), 18 with
// 8-bit moments. A thread takes 8 consecutive elements at a time, so that every access is 16 bytes (8
// for codes), and 32 threads share one scale.
#include "adamw.hpp"

#include "common.hpp"

namespace lora {
namespace {

struct Upload {
  AdamTensor t[kAdamUpload];
};
static_assert(sizeof(Upload) + 64 <= 4096, "kernel argument size");

__global__ __launch_bounds__(256) void adam_upload_kernel(Upload u, int first, int32_t chunk,
                                                          AdamTensor* __restrict__ table,
                                                          AdamShare* __restrict__ shares) {
  const AdamTensor& t = u.t[blockIdx.x];
  const int id = first + static_cast<int>(blockIdx.x);
  if (threadIdx.x == 0) table[id] = t;
  const int64_t n = (t.t.n + chunk - 1) / chunk;
  for (int64_t i = threadIdx.x; i < n; i += 256) shares[t.first_block + i] = AdamShare{id, static_cast<int32_t>(i)};
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(float (&d)[8], const T* p, int cnt) {
  if constexpr (VEC) {
    if (cnt == 8) {
      if constexpr (sizeof(T) == 4) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = a[e], d[4 + e] = b[e];
      } else {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 4) d[e] = e < cnt ? p[e] : 0.f;
    else d[e] = e < cnt ? bf16_to_f32(p[e]) : 0.f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float (&s)[8], int cnt) {
  if constexpr (VEC) {
    if (cnt == 8) {
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4*>(p) = f32x4{s[0], s[1], s[2], s[3]};
        *reinterpret_cast<f32x4*>(p + 4) = f32x4{s[4], s[5], s[6], s[7]};
      } else {
        *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]),
                                             pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7])};
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (e >= cnt) continue;
    if constexpr (sizeof(T) == 4) p[e] = s[e];
    else p[e] = f32_to_bf16_rne(s[e]);
  }
}

// Eight e4m3 codes as one 8-byte word.
template <bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int cnt) {
  if constexpr (VEC) {
    if (cnt == 8) return *reinterpret_cast<const uint2*>(p);
  }
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) w[e >> 2] |= static_cast<uint32_t>(p[e]) << (8 * (e & 3));
  return uint2{w[0], w[1]};
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 w, int cnt) {
  if constexpr (VEC) {
    if (cnt == 8) {
      *reinterpret_cast<uint2*>(p) = w;
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < cnt) p[e] = static_cast<uint8_t>((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
}

__device__ __forceinline__ void decode8(float (&d)[8], uint2 w, float scale) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true);
  d[0] = a[0] * scale; d[1] = a[1] * scale; d[2] = b[0] * scale; d[3] = b[1] * scale;
  d[4] = c[0] * scale; d[5] = c[1] * scale; d[6] = e[0] * scale; d[7] = e[1] * scale;
}

// The codes of 8 values and, in every lane, the scale of their block of 256 (32 threads). A NaN among
// them makes the block's scale NaN. A block whose largest magnitude is below 2^-100 holds zeros (448
// over it, and its scale, would leave the fp32 range).
template <bool POSITIVE>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float& scale) {
  uint32_t top = 0;  // magnitudes compare as integers, NaN above all
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
  for (int s = 1; s < 32; s *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), s)));
  const float t = __uint_as_float(top);
  const bool some = !(t < 0x1p-100f);
  // (products with reciprocals, as the constants of the step are: true divisions here put a code in 10^7 on the
  // other side of a tie from what tensor libraries write for the same division by a number)
  scale = some ? t * (1.f / 448.f) : 0.f;
  const float inv = some ? (1.f / t) * 448.f : 0.f;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = x[e] * inv;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  uint32_t w[2] = {static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
  if constexpr (POSITIVE) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (y[e] > 0.f && ((w[e >> 2] >> (8 * (e & 3))) & 0xffu) == 0) w[e >> 2] |= 1u << (8 * (e & 3));
  }
  return uint2{w[0], w[1]};
}

template <typename TP, typename TG, bool EIGHT, bool VEC>
__device__ __forceinline__ void adam_share(const lora_adamw_tensor& t, int64_t lo, int64_t hi, const AdamConst& c) {
  for (int64_t base = lo; base < hi; base += 2048) {
    // (all 32 threads of a scale block take part in its maximum, those behind the end with zeros)
    const int64_t i = base + threadIdx.x * 8;
    const int cnt = static_cast<int>(max<int64_t>(0, min<int64_t>(8, hi - i)));
    const int64_t at = cnt > 0 ? i : lo;
    float g[8], m[8], r[8], p[8];
    load8<TG, VEC>(g, static_cast<const TG*>(t.grad) + at, cnt);
    if constexpr (EIGHT) {
      const int64_t blk = at / kAdamBlock;
      const uint2 cm = load_codes<VEC>(static_cast<const uint8_t*>(t.m) + at, cnt);
      const uint2 cv = load_codes<VEC>(static_cast<const uint8_t*>(t.v) + at, cnt);
      decode8(m, cm, t.m_scale[blk]);
      decode8(r, cv, t.v_scale[blk]);
    } else {
      load8<float, VEC>(m, static_cast<const float*>(t.m) + at, cnt);
      load8<float, VEC>(r, static_cast<const float*>(t.v) + at, cnt);
    }
    if (t.master != nullptr) load8<float, VEC>(p, t.master + at, cnt);
    else load8<TP, VEC>(p, static_cast<const TP*>(t.param) + at, cnt);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c.grad_scale != 1.f) g[e] *= c.grad_scale;
      m[e] = m[e] * c.b1 + g[e] * c.c1;
      v[e] = (EIGHT ? r[e] * r[e] : r[e]) * c.b2 + (g[e] * g[e]) * c.c2;
      r[e] = sqrtf(v[e]);
      p[e] = p[e] * c.decay - (m[e] / (r[e] * c.root + c.eps)) * c.size;
    }
    if constexpr (EIGHT) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e >= cnt) m[e] = 0.f, r[e] = 0.f;
      float sm, sv;
      const uint2 cm = encode8<false>(m, sm), cv = encode8<true>(r, sv);
      if (cnt > 0) {
        store_codes<VEC>(static_cast<uint8_t*>(t.m) + at, cm, cnt);
        store_codes<VEC>(static_cast<uint8_t*>(t.v) + at, cv, cnt);
        if (at % kAdamBlock == 0) {
          t.m_scale[at / kAdamBlock] = sm;
          t.v_scale[at / kAdamBlock] = sv;
        }
      }
    } else {
      store8<float, VEC>(static_cast<float*>(t.m) + at, m, cnt);
      store8<float, VEC>(static_cast<float*>(t.v) + at, v, cnt);
    }
    if (t.master != nullptr) store8<float, VEC>(t.master + at, p, cnt);
    store8<TP, VEC>(static_cast<TP*>(t.param) + at, p, cnt);
  }
}

template <typename TP, typename TG, bool EIGHT>
__global__ __launch_bounds__(256) void adam_kernel(const AdamTensor* __restrict__ table,
                                                   const AdamShare* __restrict__ shares, int32_t chunk, AdamConst c) {
  if (c.lr_step != nullptr) {  // the learning rate and the step number of a captured step
    __shared__ float f[3];
    if (threadIdx.x == 0) {
      const double lr = c.lr_step[0], k = c.lr_step[1];
      f[0] = static_cast<float>(1.0 - lr * c.wd);
      f[1] = static_cast<float>(lr / (1.0 - pow(c.beta1, k)));
      f[2] = static_cast<float>(1.0 / sqrt(1.0 - pow(c.beta2, k)));
    }
    __syncthreads();
    c.decay = f[0];
    c.size = f[1];
    c.root = f[2];
  }
  const AdamShare sh = shares[blockIdx.x];
  const AdamTensor& a = table[sh.tensor];
  const lora_adamw_tensor t = a.t;
  const int64_t lo = static_cast<int64_t>(sh.chunk) * chunk, hi = min<int64_t>(t.n, lo + chunk);
  if (a.vec) adam_share<TP, TG, EIGHT, true>(t, lo, hi, c);
  else adam_share<TP, TG, EIGHT, false>(t, lo, hi, c);
}

}  // namespace

hipError_t launch_adam_upload(const AdamTensor* t, int n, int first, int32_t chunk, void* table, int32_t n_tensors,
                              hipStream_t s) {
  Upload u;
  for (int i = 0; i < n; ++i) u.t[i] = t[i];
  for (int i = n; i < kAdamUpload; ++i) u.t[i] = AdamTensor{};
  hipLaunchKernelGGL(adam_upload_kernel, dim3(static_cast<unsigned>(n)), dim3(256), 0, s, u, first, chunk,
                     static_cast<AdamTensor*>(table),
                     reinterpret_cast<AdamShare*>(static_cast<char*>(table) + adam_table_shares(n_tensors)));
  return hipGetLastError();
}

hipError_t launch_adam_step(const lora_adamw_plan_t& p, const AdamConst& c, hipStream_t s) {
  const auto* table = static_cast<const AdamTensor*>(p.table);
  const auto* shares =
      reinterpret_cast<const AdamShare*>(static_cast<const char*>(p.table) + adam_table_shares(p.n_tensors));
  const dim3 grid(static_cast<unsigned>(p.n_blocks)), block(256);
  const bool p32 = p.param_dtype == LORA_F32, g32 = p.grad_dtype == LORA_F32, eight = p.state_bits == 8;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, table, shares, p.chunk, c);
    return hipGetLastError();
  };
  if (p32) {
    if (g32) return eight ? go(adam_kernel<float, float, true>) : go(adam_kernel<float, float, false>);
    return eight ? go(adam_kernel<float, bf16_bits, true>) : go(adam_kernel<float, bf16_bits, false>);
  }
  if (g32) return eight ? go(adam_kernel<bf16_bits, float, true>) : go(adam_kernel<bf16_bits, float, false>);
  return eight ? go(adam_kernel<bf16_bits, bf16_bits, true>) : go(adam_kernel<bf16_bits, bf16_bits, false>);
}

}  // namespace lora
