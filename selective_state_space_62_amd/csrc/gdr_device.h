// Device code shared by the chunked kernels of the gated delta rule (gfx950).
//
// Products run on the matrix cores in fp16 planes: a value x scaled by a power of 2 s is hi = fp16(x s) and
// lo = fp16(x s - hi), 22 bits together, and a product of two such operands is hi hi + hi lo + lo hi in fp32, within
// about 2^-22 of the sizes of its terms: fp32 results at 3 of the 16 times that an fp32 matrix instruction costs.  A
// bf16 input is one plane, exact to 2^-17 of its row's largest value and within 2^-25 of it below.  Scales keep a tile's largest
// value near 2^13 (rows of keys and queries: in [1, 2)), so what an fp16 exponent cannot hold is below 2^-38 of it.
//
// Tiles are 32x32x16.  A result's lane holds column l & 31 and rows (r & 3) + 8 (r >> 2) + 4 (l >> 5): for 16 rows
// these are the 8 values that the same lane gives an operand whose summed index is that row, if the other operand
// lists its 16 in the order 0-3 8-11 | 4-7 12-15.  So results feed the next product from registers, and everything
// that stands in LDS or memory stands in that order: one block of 64 lanes times 8 values for 32 rows by 16 columns.
#pragma once

#include "device_common.h"
#include "gdr.h"
#include "internal.h"

namespace ssscan {
namespace gdr {

using namespace dev;

constexpr int kC = kGdrChunk;            // tokens of a chunk: two tiles

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float acc16 __attribute__((ext_vector_type(16)));

// An operand block in LDS is 64 x 16 bytes; blocks are 32 bytes further apart than that, so that a row's blocks start in
// different banks when they are written.
constexpr int kBlock = 1024 + 32;

struct Planes {
  h8 hi, lo;
};

template <typename IO>
constexpr int planes_of() { return IO::kPerSpan == 4 ? 2 : 1; }

// acc += A B for operands of NA and NB planes.
template <int NA, int NB>
__device__ __forceinline__ acc16 mm(const Planes& a, const Planes& b, acc16 acc) {
  if constexpr (NB == 2) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.hi, b.lo, acc, 0, 0, 0);
  if constexpr (NA == 2) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.lo, b.hi, acc, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a.hi, b.hi, acc, 0, 0, 0);
}

// Values 8 half .. 8 half + 7 of a result tile as an operand, scaled.
__device__ __forceinline__ Planes split(const acc16& v, int half, float s) {
  Planes p;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = v[8 * half + j];
    p.hi[j] = (_Float16)(x * s);
    p.lo[j] = (_Float16)fmaf(x, s, -(float)p.hi[j]);
  }
  return p;
}

__device__ __forceinline__ acc16 zero16() {
  acc16 z;
#pragma unroll
  for (int j = 0; j < 16; ++j) z[j] = 0.0f;
  return z;
}

// Row (of 32) of register r in a result tile.
__device__ __forceinline__ int tile_row(int r, int lane) { return (r & 3) + 8 * (r >> 2) + 4 * (lane >> 5); }

// Largest |value| over the wave, NaN left out.
__device__ __forceinline__ float wave_max(float v) {
  // quad permutes, mirrors of 8 and of 16 lanes, then exchanges across rows
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0xB1, 0xf, 0xf, false));
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0x4E, 0xf, 0xf, false));
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0x141, 0xf, 0xf, false));
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0x140, 0xf, 0xf, false));
  v = fmaxf(v, __shfl_xor(v, 16));
  v = fmaxf(v, __shfl_xor(v, 32));
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

__device__ __forceinline__ float max_of(const acc16& v, float m) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) m = fmaxf(fmaxf(m, fabsf(v[j])), fabsf(v[j + 1]));
  return m;
}

// 2^e, e held to what a float's exponent is.
__device__ __forceinline__ float pow2(int e) {
  e = e < -126 ? -126 : e > 127 ? 127 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Exponent of a largest |value|: floor(log2 m), -127 for zero and what is below normal numbers, 128 for an infinity.
__device__ __forceinline__ int exponent(float m) { return (int)(__float_as_uint(m) >> 23) - 127; }

// The scale 2^e that takes a largest |value| m to [2^13, 2^14), e at most `most`.  With an infinity among the values it is NaN:
// what stands beside it could not be held, and is not lost silently.
struct Scale {
  int e;
  float f;
};

__device__ __forceinline__ Scale scale_of(float m, int most) {
  Scale s;
  s.e = m == 0.0f ? 0 : 13 - exponent(m);
  s.e = s.e < most ? s.e : most;
  s.f = exponent(m) == 128 ? __builtin_nanf("") : pow2(s.e);
  return s;
}

// The scale that takes a row whose largest |value| is m to [1, 2); 1 for a row of zeros or with an infinity (which then stays one).
__device__ __forceinline__ float row_scale(float m) {
  const int e = exponent(m);
  return m == 0.0f || e == 128 ? 1.0f : pow2(-e);
}

__device__ __forceinline__ float quad_max(float m) {
  m = fmaxf(m, __builtin_amdgcn_update_dpp(0.0f, m, 0xB1, 0xf, 0xf, false));
  return fmaxf(m, __builtin_amdgcn_update_dpp(0.0f, m, 0x4E, 0xf, 0xf, false));
}

// 8 consecutive values at any element alignment, as they stand in memory.
template <typename IO>
struct __attribute__((packed, aligned(sizeof(typename IO::T)))) Raw8 {
  uint32_t w[8 * sizeof(typename IO::T) / 4];
};

// Values at .. at + 7 of a row of n, zeros from n on.
template <typename IO>
__device__ __forceinline__ Raw8<IO> load_raw8(const typename IO::T* __restrict__ row, int at, int n) {
  if (at + 8 <= n) return *reinterpret_cast<const Raw8<IO>*>(row + at);
  Raw8<IO> r;
#pragma unroll
  for (int j = 0; j < (int)(sizeof(r.w) / 4); ++j) r.w[j] = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (at + j < n) {
      if constexpr (IO::kPerSpan == 4) r.w[j] = __float_as_uint(row[at + j]);
      else r.w[j >> 1] |= (uint32_t)row[at + j] << ((j & 1) * 16);
    }
  return r;
}

template <typename IO>
__device__ __forceinline__ float raw_value(const Raw8<IO>& r, int j) {
  if constexpr (IO::kPerSpan == 4) return __uint_as_float(r.w[j]);
  else return (j & 1) ? __uint_as_float(r.w[j >> 1] & 0xffff0000u) : __uint_as_float(r.w[j >> 1] << 16);
}

template <typename IO>
__device__ __forceinline__ void load8(const typename IO::T* __restrict__ row, int at, int n, float (&x)[8]) {
  const Raw8<IO> r = load_raw8<IO>(row, at, n);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = raw_value<IO>(r, j);
}

// Run c (8 values, of index 8 c on) of row `row` (0..63) into the operand blocks of a chunk's rows: tiles of 32 rows,
// of each `steps` blocks.  Values 0-3 and 4-7 are of the two halves of the lanes.
template <typename IO>
__device__ __forceinline__ void store_operand_rows(char* hi, char* lo, int row, int c, int steps, const float (&x)[8], float s) {
  char* p = hi + ((row >> 5) * steps + (c >> 1)) * kBlock + (row & 31) * 16 + (c & 1) * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    h4 v, w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = (_Float16)(x[4 * h + j] * s);
      if constexpr (planes_of<IO>() == 2) w[j] = (_Float16)fmaf(x[4 * h + j], s, -(float)v[j]);
    }
    *reinterpret_cast<h4*>(p + 512 * h) = v;
    if constexpr (planes_of<IO>() == 2) *reinterpret_cast<h4*>(p + (lo - hi) + 512 * h) = w;
  }
}

// The vectors that belong to a chunk of a head, kC floats each, as the preparation leaves them.  c_j scales column j of
// the inverse T, s_j row j of k, gam_j the sum of log decays up to j (over log 2), gam_C the whole chunk's.
enum Vec {
  kVecF1,      // beta_j / c_j
  kVecF2,      // beta_j 2^gam_j / (c_j s_j)
  kVecEnd,     // 2^(gam_C - gam_j) / s_j
  kVecHi,      // gam_j = hi + lo
  kVecLo,
  kVecRel,     // log2 of s_j over the chunk's smallest
  kVecInto,    // 2^gam_j
  kVecS,       // s_j
  kVecGrow,    // whole number p_i >= 0 with gam_i - gam_j - rel_j <= p_i for every j <= i: 0 where no gate grows
  kVecBeta,    // beta_j
  kVecs
};

// The inverse's operand blocks: tiles (0, 0), (1, 0), (1, 1), of each two steps of 16, of each two planes.
constexpr int kTBlocks = 3 * 2 * 2;
constexpr int64_t kTHalfs = kTBlocks * 512;      // fp16 values of one chunk's

}  // namespace gdr
}  // namespace ssscan
