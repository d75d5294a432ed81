// Argument checks shared by the C entry points.
#pragma once

#include <cstddef>
#include <cstdint>

#include "ssscan.h"

namespace ssscan {

inline int elem_bytes(ss_dtype io) { return io == SS_BF16 ? 2 : 4; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

struct Range {
  const char* name;
  uintptr_t lo, hi;   // [lo, hi)
};

inline Range rng(const char* name, const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{name, lo, p ? lo + (uintptr_t)bytes : lo};
}

inline bool overlap(const Range& a, const Range& b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

constexpr int64_t kMaxDim = int64_t(1) << 40;

}  // namespace ssscan
