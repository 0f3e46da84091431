// Argument checks shared by the host-side entry points (dispatch*.cpp).
#pragma once

#include <stdint.h>

namespace fp4w {

// Element counts (M * K, N * K, M * N, N * scale_cols) are capped at 2^60, so
// every byte count derived from them (at most 4 bytes per element) stays
// below 2^63.
constexpr int64_t kMaxElems = int64_t(1) << 60;

inline bool mul_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// [lo, lo + bytes) and [lo2, lo2 + bytes2) overlap?
inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  if (a == nullptr || b == nullptr || abytes <= 0 || bbytes <= 0) return false;
  uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace fp4w
