// Argument checks shared by the C-ABI entry points (host code only).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace lora {

struct Span {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
  bool empty() const { return lo == hi; }
};

inline Span span2d(const void* p, int64_t rows, int64_t ld, int64_t cols, int esize) {
  Span s;
  if (p == nullptr || rows <= 0 || cols <= 0) return s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + static_cast<uintptr_t>(((rows - 1) * ld + cols) * esize);
  return s;
}

inline bool overlaps(const Span& a, const Span& b) {
  return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned(const void* p, uintptr_t a) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % a == 0; }

// The staging kernels address one tile of rows with 32-bit byte offsets.
constexpr int64_t kMaxRowBytes = int64_t(1) << 22;

constexpr size_t kWsAlign = 256;
inline size_t round_up(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }

}  // namespace lora
