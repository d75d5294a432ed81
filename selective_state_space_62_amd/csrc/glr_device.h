// Device code shared by the gated linear recurrence's kernels (gfx950).
#pragma once

#include "device_common.h"
#include "glr.h"
#include "internal.h"

namespace ssscan {
namespace glr {

using namespace dev;

constexpr int kConvex = 0, kNormalised = 1;
constexpr int kV = 8;             // tokens per lane and tile
constexpr float kTiny = 1.17549435e-38f;

// kV consecutive elements of a row as they are in memory.
template <typename IO>
struct Raw {
  static constexpr int kWords = kV * (int)sizeof(typename IO::T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ float operator[](int j) const { return span_elem<IO>(w, j); }
};

// A lane's tokens as one or two 16-byte accesses, for a lane whose tokens are all inside
// the row; the lane at its end goes element by element.  A tile's loads stand together
// in one branch for the first and one for the second: with a branch for each of them
// the compiler waited for a load before it sent the next (2.8B-shaped bf16 layer with
// both gates, forward 177 -> 153 us), and with one for the wave as a whole a wave that
// holds a row's end went element by element (40960 rows of 1000 bf16 tokens, normalised,
// input gate, forward 124 -> 85 us, backward 274 -> 150).  Rows of
// odd length start at any element, and gfx950 takes vector accesses at any address, so
// the type promises the compiler no more than its elements' alignment.
template <typename IO>
struct __attribute__((packed, aligned(sizeof(typename IO::T)))) Words {
  uint32_t w[Raw<IO>::kWords];
};

template <typename IO>
__device__ __forceinline__ Raw<IO> load_whole(const typename IO::T* __restrict__ p) {
  Raw<IO> o;
  const Words<IO> v = *reinterpret_cast<const Words<IO>*>(p);
#pragma unroll
  for (int k = 0; k < Raw<IO>::kWords; ++k) o.w[k] = v.w[k];
  return o;
}

// The first `valid` elements; the others read as `pad`, the bits of two bf16 or of one
// fp32 value.
template <typename IO>
__device__ __forceinline__ Raw<IO> load_part(const typename IO::T* __restrict__ p, int valid, uint32_t pad = 0u) {
  Raw<IO> o;
#pragma unroll
  for (int k = 0; k < Raw<IO>::kWords; ++k) o.w[k] = pad;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    if (j < valid) {
      if constexpr (IO::kPerSpan == 4) o.w[j] = __float_as_uint(p[j]);
      else o.w[j >> 1] = j & 1 ? (o.w[j >> 1] & 0xffffu) | (uint32_t)p[j] << 16 : (o.w[j >> 1] & 0xffff0000u) | p[j];
    }
  }
  return o;
}

// The r of tokens past a row's end: an infinite gate, which keeps the state exactly
// (a = 1, m = 0), so that nothing after the load asks where the row ends.
template <typename IO, int KIND>
constexpr uint32_t gate_pad() {
  constexpr uint32_t kSign = KIND == 0 ? 0u : 0x80000000u;
  return IO::kPerSpan == 4 ? 0x7f800000u | kSign : 0x7f807f80u | kSign | kSign >> 16;
}

template <typename IO>
__device__ __forceinline__ void store_whole(typename IO::T* __restrict__ p, const float (&v)[kV]) {
  Words<IO> o;
  if constexpr (IO::kPerSpan == 4) {
#pragma unroll
    for (int j = 0; j < kV; ++j) o.w[j] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kV; j += 2) o.w[j >> 1] = pack_bf16x2(v[j], v[j + 1]);
  }
  *reinterpret_cast<Words<IO>*>(p) = o;
}

template <typename IO>
__device__ __forceinline__ void store_part(typename IO::T* __restrict__ p, int valid, const float (&v)[kV]) {
#pragma unroll
  for (int j = 0; j < kV; ++j)
    if (j < valid) store_one<IO>(p, j, v[j]);
}

// How many of a lane's kV tokens are inside the row, when its wave's tokens start `left`
// before the row's end.
__device__ __forceinline__ int lane_tokens(int64_t left, int lane) {
  const int n = (int)(left < 64 * kV ? left : 64 * kV) - lane * kV;
  return n < 0 ? 0 : n > kV ? kV : n;
}

// What a row's tokens share: the biases times -log2(e), and of the decay
//   convex:     c0 = f, c1 = 1 - f
//   normalised: c0 = -l log2(e), c1 = 2 l, with l = decay_scale softplus(decay)
struct RowConst {
  float rb, ib, c0, c1;
};

template <int KIND>
__device__ __forceinline__ RowConst make_const(float r_bias, float i_bias, float decay, float decay_scale) {
  RowConst c;
  // an infinite bias is held to 2^126: the gate's infinity at the tokens past the end
  // decides (a NaN stays one)
  const float rb = -kLog2e * r_bias;
  c.rb = fabsf(rb) > 0x1p126f ? copysignf(0x1p126f, rb) : rb;
  c.ib = -kLog2e * i_bias;
  if constexpr (KIND == kConvex) {
    c.c0 = decay;
    c.c1 = 1.0f - decay;
  } else {
    // an infinite rate is held to 2^126 (a NaN stays one): a closed gate's 0 times it is 0, so
    // that padding and the tokens past the end keep the state, and an open gate still
    // forgets it all
    const float l = __builtin_elementwise_minimum(decay_scale * softplus_dt(decay, 0.0f), 0x1p126f);
    c.c0 = -kLog2e * l;
    c.c1 = 2.0f * l;
  }
  return c;
}

template <int KIND>
__device__ __forceinline__ RowConst row_const(const GlrArgs& p, int64_t d) {
  return make_const<KIND>(p.r_bias ? p.r_bias[d] : 0.0f, p.i_bias ? p.i_bias[d] : 0.0f, p.decay ? p.decay[d] : 0.0f,
                          p.decay_scale);
}

// sigmoid(v + bias), given nb = -log2(e) bias; e receives exp(-(v + bias)).
__device__ __forceinline__ float sigmoid_e(float v, float nb, float& e) {
  e = __builtin_amdgcn_exp2f(fmaf(v, -kLog2e, nb));
  return __builtin_amdgcn_rcpf(1.0f + e);   // 0 where e overflowed
}

// The same with e held to 2^126, for a gate whose 1 - s is wanted too: e s.  It is
// never below 2^-126, so a gate of -inf passes that much instead of nothing.  The
// minimum of a NaN is a NaN (one v_minimum3; fminf's would be 126, and the gate a number).
__device__ __forceinline__ float sigmoid_both(float v, float nb, float& minus) {
  const float e = __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(fmaf(v, -kLog2e, nb), 126.0f));
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  minus = e * s;
  return s;
}

// 1 - s of the first sigmoid without cancellation: e s where s is the larger
// half.  e s is never formed from an overflowed e (the comparison selects 1 - s).
__device__ __forceinline__ float one_minus(float s, float e) { return e > 1.0f ? 1.0f - s : e * s; }

// 1 - a^2 of the normalised kind, with w = 2 l s and a = e^(-w/2).  1 - a a loses
// digits as a nears 1 (the usual case: decays of 0.9 to 0.999), so below w = 1/8 it
// is the Taylor polynomial of 1 - e^-w, whose first dropped term is w^5/720, 4.3e-8
// relative there; above, a is at most 0.94 and within one step, 2^-24, which moves a^2 by
// 1.1e-7, 9.5e-7 of 1 - a^2 and half as much of its root.
__device__ __forceinline__ float one_minus_sq(float w, float a) {
  float t = fmaf(w, 1.0f / 120.0f, -1.0f / 24.0f);
  t = fmaf(t, w, 1.0f / 6.0f);
  t = fmaf(t, w, -0.5f);
  t = fmaf(t, w, 1.0f) * w;
  return w < 0.125f ? t : fmaf(-a, a, 1.0f);
}

// One token's decay a and input weight m.
template <int KIND>
__device__ __forceinline__ void gate(float r, const RowConst& c, float& a, float& m) {
  float e;
  const float s = sigmoid_e(r, c.rb, e);
  if constexpr (KIND == kConvex) {
    a = fmaf(c.c1, s, c.c0);
    m = c.c1 * one_minus(s, e);
  } else {
    a = __builtin_amdgcn_exp2f(c.c0 * s);
    const float q = one_minus_sq(c.c1 * s, a);
    m = q * __builtin_amdgcn_rsqf(fmaxf(q, kTiny));   // sqrt(q); 0 at 0
  }
}

// --- scans over the wave's 64 lanes of maps h -> A h + B -----------------------
// In each step a lane joins its piece with the one `k` lanes away, or with the
// identity where there is none (update_dpp keeps `old` for a missing source).

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float old, float v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xf, false);
}

template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ void join(float& A, float& B) {
  const float a = dpp<CTRL, ROWS>(1.0f, A), b = dpp<CTRL, ROWS>(0.0f, B);
  B = fmaf(A, b, B);
  A *= a;
}

// Lane l gets the composition of lanes 0 .. l, lane 0's applied first.
__device__ __forceinline__ void scan_up(float& A, float& B) {
  join<0x111>(A, B);        // row_shr:1, 2, 4, 8 within rows of 16 lanes
  join<0x112>(A, B);
  join<0x114>(A, B);
  join<0x118>(A, B);
  join<0x142, 0xa>(A, B);   // row_bcast:15 into rows 1 and 3
  join<0x143, 0xc>(A, B);   // row_bcast:31 into rows 2 and 3
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// Lane l gets the composition of lanes l .. 63, lane 63's applied first.  There is
// no broadcast towards lower rows, so the rows' totals go through scalars.
__device__ __forceinline__ void scan_down(float& A, float& B, int lane) {
  join<0x101>(A, B);        // row_shl:1, 2, 4, 8
  join<0x102>(A, B);
  join<0x104>(A, B);
  join<0x108>(A, B);
  const float a3 = lane_value(A, 48), b3 = lane_value(B, 48);
  const float a2 = lane_value(A, 32), b2 = lane_value(B, 32);
  const float a1 = lane_value(A, 16), b1 = lane_value(B, 16);
  const float a23 = a2 * a3, b23 = fmaf(a2, b3, b2);
  const float a123 = a1 * a23, b123 = fmaf(a1, b23, b1);
  const int row = lane >> 4;
  const float a = row == 0 ? a123 : row == 1 ? a23 : row == 2 ? a3 : 1.0f;
  const float b = row == 0 ? b123 : row == 1 ? b23 : row == 2 ? b3 : 0.0f;
  B = fmaf(A, b, B);
  A *= a;
}

// The compositions of the lanes before (after) a lane's own, from those above.
__device__ __forceinline__ float shift_up(float old, float v) { return dpp<0x138>(old, v); }     // wave_shr:1
__device__ __forceinline__ float shift_down(float old, float v) { return dpp<0x130>(old, v); }   // wave_shl:1

// --- the same over groups of S lanes, a power of 2 up to 32: a short row each -------
// `l` is the lane's place in its group.

template <int K>
__device__ __forceinline__ void join_up(float& A, float& B, int l) {
  float a, b;
  if constexpr (K < 16) {
    a = dpp<0x110 + K>(1.0f, A);
    b = dpp<0x110 + K>(0.0f, B);
  } else {
    a = dpp<0x142, 0xa>(1.0f, A);
    b = dpp<0x142, 0xa>(0.0f, B);
  }
  if (K < 16 && l < K) {
    a = 1.0f;
    b = 0.0f;
  }
  B = fmaf(A, b, B);
  A *= a;
}

__device__ __forceinline__ void group_scan_up(float& A, float& B, int l, int S) {
  if (S > 1) join_up<1>(A, B, l);
  if (S > 2) join_up<2>(A, B, l);
  if (S > 4) join_up<4>(A, B, l);
  if (S > 8) join_up<8>(A, B, l);
  if (S > 16) join_up<16>(A, B, l);
}

template <int K>
__device__ __forceinline__ void join_down(float& A, float& B, int l, int S) {
  float a = dpp<0x100 + K>(1.0f, A), b = dpp<0x100 + K>(0.0f, B);
  if (l + K >= S) {
    a = 1.0f;
    b = 0.0f;
  }
  B = fmaf(A, b, B);
  A *= a;
}

__device__ __forceinline__ void group_scan_down(float& A, float& B, int l, int S, int lane) {
  if (S > 1) join_down<1>(A, B, l, S);
  if (S > 2) join_down<2>(A, B, l, S);
  if (S > 4) join_down<4>(A, B, l, S);
  if (S > 8) join_down<8>(A, B, l, S);
  if (S > 16) {   // the first 16 lanes with the total of the second
    const float a1 = lane_value(A, 16), b1 = lane_value(B, 16), a3 = lane_value(A, 48), b3 = lane_value(B, 48);
    const float a = l >= 16 ? 1.0f : lane < 32 ? a1 : a3;
    const float b = l >= 16 ? 0.0f : lane < 32 ? b1 : b3;
    B = fmaf(A, b, B);
    A *= a;
  }
}

// Rows of up to 256 tokens take the smallest group that holds them.
inline int group_of(int64_t seqlen) {
  int s = 1;
  while (s * kV < seqlen) s <<= 1;
  return s;
}

// Sum over the wave's lanes in a fixed order, in lane 63.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111>(0.0f, v);
  v += dpp<0x112>(0.0f, v);
  v += dpp<0x114>(0.0f, v);
  v += dpp<0x118>(0.0f, v);
  v += dpp<0x142, 0xa>(0.0f, v);
  v += dpp<0x143, 0xc>(0.0f, v);
  return v;
}

// --- joining the tiles of a split row ---------------------------------------------
// Each tile is a workgroup.  Workgroups take their row's tiles in order (a counter
// for each row), publish their tile's map as soon as they have it, and join the maps
// of the tiles before theirs: those of their group of 32 tiles, onto the state
// entering the group, which the last tile of the group before has published.  A
// workgroup waits only for ones that took their tile earlier and so already run, and
// no map waits for anything: every wait ends.  What is joined does not depend on
// timing, so neither does the result.  A slot is one 64-bit word, written and read
// whole past the caches that are not shared, and never 0 once written.  A call that
// shares its workspace with one that runs at the same time, which is not allowed,
// could find its slots cleared: a wait gives up after seconds and enters NaN.
constexpr int kMostPolls = 1 << 22;   // of about a microsecond each

struct Chain {
  uint64_t* map;      // (rows, tiles)
  uint64_t* state;    // (rows, groups): the state entering each group
  uint32_t* counter;  // (rows), 8 bytes apart
  __device__ __forceinline__ Chain(const GlrArgs& p, int64_t tiles) {
    const int64_t groups = (tiles + kGlrGroup - 1) / kGlrGroup;
    map = (uint64_t*)p.chain;
    state = map + p.rows * tiles;
    counter = (uint32_t*)(state + p.rows * groups);
  }
};

__device__ __forceinline__ uint64_t pack_map(float A, float B) {
  const uint64_t v = (uint64_t)__float_as_uint(A) << 32 | __float_as_uint(B);
  return v ? v : uint64_t(1) << 63;   // A = -0 for 0
}

__device__ __forceinline__ void publish(uint64_t* slot, uint64_t v) {
  __hip_atomic_store(slot, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// For one wave: publishes tile n's map (A, B) of row `row` and returns the state
// entering the tile; `first` is the one entering the row.
__device__ __forceinline__ float chain_enter(const Chain& ch, int64_t row, int64_t n, int64_t tiles, float first, float A,
                                             float B, int lane) {
  const int64_t group = n / kGlrGroup, groups = (tiles + kGlrGroup - 1) / kGlrGroup;
  const int before = (int)(n - group * kGlrGroup);   // tiles of the group before this one
  uint64_t* map = ch.map + row * tiles + group * kGlrGroup;
  if (lane == 0) publish(map + before, pack_map(A, B));
  const bool reads = lane < before || (lane == kGlrGroup && group > 0);
  uint64_t* slot = lane == kGlrGroup ? ch.state + row * groups + group : map + lane;
  uint64_t v = 0;
  for (int polls = 0;; ++polls) {
    if (reads && v == 0) v = __hip_atomic_load(slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__ballot(reads && v == 0) == 0) break;
    if (polls == kMostPolls) {
      first = __builtin_nanf("");
      v = pack_map(first, first);
      break;
    }
    __builtin_amdgcn_s_sleep(1);
  }
  const float enter = group > 0 ? lane_value(__uint_as_float((uint32_t)v), kGlrGroup) : first;
  float a = lane < before ? __uint_as_float((uint32_t)(v >> 32)) : 1.0f;
  float b = lane < before ? __uint_as_float((uint32_t)v) : 0.0f;
  scan_up(a, b);
  const float h = fmaf(lane_value(a, 63), enter, lane_value(b, 63));
  if (before == kGlrGroup - 1 && n + 1 < tiles && lane == 0)
    publish(ch.state + row * groups + group + 1, pack_map(0.0f, fmaf(A, h, B)));
  return h;
}

// --- launch shape ---------------------------------------------------------------
// Workgroups of 256 threads hold 4 / W rows of W waves; a grid dimension's
// threads are 32-bit, so large launches use two dimensions.
inline bool grid_of(int64_t blocks, dim3* g) {
  constexpr int64_t kX = int64_t(1) << 22;
  if (blocks <= kX) {
    *g = dim3((unsigned)blocks);
    return true;
  }
  const int64_t y = (blocks + kX - 1) / kX;
  if (y > 65535) return false;
  *g = dim3((unsigned)kX, (unsigned)y);
  return true;
}

__device__ __forceinline__ int64_t block_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// OP<io, kind, has i, has z>::go(a, s) for the call's form.
template <template <typename, int, bool, bool> class OP, typename IO, int KIND>
hipError_t by_gates(const GlrArgs& a, hipStream_t s) {
  if (a.i) return a.z ? OP<IO, KIND, true, true>::go(a, s) : OP<IO, KIND, true, false>::go(a, s);
  return a.z ? OP<IO, KIND, false, true>::go(a, s) : OP<IO, KIND, false, false>::go(a, s);
}

template <template <typename, int, bool, bool> class OP>
hipError_t by_form(const GlrArgs& a, hipStream_t s) {
  if (a.io == kIoBf16)
    return a.kind == kConvex ? by_gates<OP, BF16, kConvex>(a, s) : by_gates<OP, BF16, kNormalised>(a, s);
  return a.kind == kConvex ? by_gates<OP, F32, kConvex>(a, s) : by_gates<OP, F32, kNormalised>(a, s);
}

}  // namespace glr
}  // namespace ssscan
