// Argument checks shared by the C entry points.
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>

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

// Elements from the first to one past the last value under these strides, or -1
// where that overflows.
inline int64_t span_of(int64_t batch, int64_t seqlen, int heads, int n, const int64_t* st) {
  if (heads == 0 || seqlen == 0) return 0;
  __int128 last = n;
  last += (__int128)(batch - 1) * st[0] + (__int128)(seqlen - 1) * st[1] + (__int128)(heads - 1) * st[2];
  return last > ((__int128)1 << 58) ? -1 : (int64_t)last;
}

// Whether runs of n values, one for each index of D dimensions, are disjoint: by stride,
// ascending, each dimension has to step over all that the ones before it reach.
template <int D>
bool distinct(int64_t n, int64_t (&size)[D], int64_t (&stride)[D]) {
  for (int i = 0; i < D; ++i)
    for (int j = i + 1; j < D; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(size[i], size[j]);
      }
  int64_t reach = n;
  for (int i = 0; i < D; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < reach) return false;
    reach += stride[i] * (size[i] - 1);
  }
  return true;
}

// Whether two strided gradients, each without shared addresses and the second's first value `apart` after
// the first's, share none: with the same batch and token strides, either all heads of the one lie behind
// those of the other in each token's columns, or their heads alternate under one head stride.
inline bool columns_of_one(int64_t batch, int64_t seqlen, int n, int heads_a, const int64_t* sa, int heads_b,
                           const int64_t* sb, int64_t apart) {
  if ((batch > 1 && sa[0] != sb[0]) || (seqlen > 1 && sa[1] != sb[1])) return false;
  const int64_t ea = (heads_a - 1) * sa[2] + n, eb = (heads_b - 1) * sb[2] + n;
  if (apart >= 0 ? apart >= ea : -apart >= eb) {
    const int64_t lo = apart < 0 ? apart : 0, hi = apart + eb > ea ? apart + eb : ea;
    int64_t size[] = {batch, seqlen}, stride[] = {sa[0], sa[1]};
    if (distinct(hi - lo, size, stride)) return true;
  }
  if (heads_a > 1 && heads_b > 1 && sa[2] != sb[2]) return false;
  int64_t size[] = {batch, seqlen, heads_a > heads_b ? heads_a : heads_b, 2};
  int64_t stride[] = {sa[0], sa[1], heads_a > 1 ? sa[2] : sb[2], apart < 0 ? -apart : apart};
  return distinct(n, size, stride);
}

}  // namespace ssscan
