// Device code shared by the chunked kernels of the gated delta rule (gfx950).
//
// Products run on the matrix cores in fp16 planes: a value x scaled by a power of 2 s is hi = fp16(x s) and
// lo = fp16(x s - hi), 22 bits together, and a product of two such operands is hi hi + hi lo + lo hi in fp32, within
// about 2^-22 of the sizes of its terms: fp32 results at 3 of the 16 times that an fp32 matrix instruction costs.  A
// bf16 input is one plane.  Scales keep a tile's (of keys and queries a row's, of T a column's) largest value near 2^13, so that
// what an fp16 cannot hold, 2^-25, is below 2^-37 of it: a chunk's later tokens may be as much smaller as decays make them.  A tile is
// a wave's 32 columns of all keys or of 64 tokens: what is 2^-24 of the largest in it keeps 14 bits.
//
// Tiles are 32x32x16.  A result's lane holds column l & 31 and rows (r & 3) + 8 (r >> 2) + 4 (l >> 5): for 16 rows
// these are the 8 values that the same lane gives an operand whose summed index is that row, if the other operand
// lists its 16 in the order 0-3 8-11 | 4-7 12-15.  So results feed the next product from registers, and everything
// that stands in LDS or memory stands in that order: one block of 64 lanes times 8 values for 32 rows by 16 columns.
#pragma once

#include <type_traits>

#include "device_common.h"
#include "gdr.h"
#include "internal.h"

namespace ssscan {
namespace gdr {

using namespace dev;

constexpr int kC = kGdrChunk;            // tokens of a chunk: two tiles

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
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

// 16 inner elements of a 16x16 product in fp32: lane l holds row (column) l & 15, inner elements 4 (l >> 4) + 0..3.  The result's
// lane has column l & 15 and rows 4 (l >> 4) + 0..3, so that it is the right operand of the next product as it is.
__device__ __forceinline__ f4 mm16(f4 x, f4 y, f4 acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], acc, 0, 0, 0);
  return acc;
}

// The value as a register has it.  What is split right after a product goes through here: the product would else be rounded to fp16
// at once, while its difference from that fp16 is formed of the product rounded to fp32, and now and then the two planes are a whole
// step of the first apart.  (A product with a power of 2 rounds nothing.)
__device__ __forceinline__ float held(float v) {
  asm("" : "+v"(v));
  return v;
}

// Values 8 half .. 8 half + 7 of a result tile as an operand of two planes, times s, a power of 2 (so that it rounds nothing).
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

// The operand block of this lane in LDS, in N planes (of which lo is `apart` bytes behind hi).
template <int N>
__device__ __forceinline__ Planes operand(const char* p, int lane, int apart) {
  Planes o;
  o.hi = *reinterpret_cast<const h8*>(p + lane * 16);
  if constexpr (N == 2) o.lo = *reinterpret_cast<const h8*>(p + apart + lane * 16);
  return o;
}

// Nothing is moved over this line: the steps of a product keep their loads one step ahead, and no more of them, in registers.
__device__ __forceinline__ void step_end() { __builtin_amdgcn_sched_barrier(0); }

// Row (of 32) of register r in a result tile.
__device__ __forceinline__ int tile_row(int r, int lane) { return (r & 3) + 8 * (r >> 2) + 4 * (lane >> 5); }

// A vector's values of a lane's 16 rows in a result tile.
__device__ __forceinline__ acc16 rows_of(const float* v, int lane) {
  acc16 o;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float4 x = *reinterpret_cast<const float4*>(v + 8 * g + 4 * (lane >> 5));
    o[4 * g] = x.x; o[4 * g + 1] = x.y; o[4 * g + 2] = x.z; o[4 * g + 3] = x.w;
  }
  return o;
}

// Largest of nonnegative values over the wave, NaN left out, in a scalar register: quad permutes and mirrors of 8 and of
// 16 lanes, then the four rows' (as integers, which order nonnegative floats as they are).
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0xB1, 0xf, 0xf, false));
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0x4E, 0xf, 0xf, false));
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0x141, 0xf, 0xf, false));
  v = fmaxf(v, __builtin_amdgcn_update_dpp(0.0f, v, 0x140, 0xf, 0xf, false));
  const int i = __float_as_int(v);
  const int a = __builtin_amdgcn_readlane(i, 0), b = __builtin_amdgcn_readlane(i, 16);
  const int c = __builtin_amdgcn_readlane(i, 32), d = __builtin_amdgcn_readlane(i, 48);
  return __int_as_float(max(max(a, b), max(c, d)));
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

// x 2^e, where e may be the sum of several scales' exponents: too small a power leaves zero, where pow2 would hold it at 2^-126.
__device__ __forceinline__ float times_pow2(float x, int e) { return __builtin_amdgcn_ldexpf(x, e); }

// The largest exponent of a scale whose inverse is a normal number too.
constexpr int kMostE = 126;

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

// The scale that takes a row whose largest |value| is m to [2^12, 2^13); 2^kZeroRow, larger than any row's that counts, for a row of
// zeros, and 1 with an infinity (which then stays one).
constexpr int kZeroRow = 100;

__device__ __forceinline__ float row_scale(float m) {
  const int e = exponent(m);
  return m == 0.0f ? pow2(kZeroRow) : e == 128 ? 1.0f : pow2(12 - e < kZeroRow ? 12 - e : kZeroRow);
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

// Rows of a chunk as a buffer: what lies behind the last token reads as zero, and a row is a 32-bit offset away (the host sees
// to it that 64 rows stay below 2^31 bytes).
template <typename IO>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rows(const typename IO::T* base, int64_t stride, int valid, int n) {
  return make_rsrc(base, ((valid - 1) * stride + n) * (int64_t)sizeof(typename IO::T));
}

constexpr uint32_t kNowhere = 0x80000000u;    // an offset behind every such buffer

// Values at .. at + 7 of the row at byte offset voff + soff, zeros from n on.  WHOLE: n is a multiple of 8 and rows are aligned
// to 4 bytes.
template <typename IO, bool WHOLE>
__device__ __forceinline__ Raw8<IO> buf_load8(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, int at, int n) {
  constexpr int kSize = sizeof(typename IO::T);
  Raw8<IO> o;
  if constexpr (WHOLE) {
    const uint32_t off = at < n ? voff + at * kSize : kNowhere;
#pragma unroll
    for (int w = 0; w < (int)sizeof(o) / 4; w += 4) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off + w * 4, soff, 0);
      o.w[w] = v[0]; o.w[w + 1] = v[1]; o.w[w + 2] = v[2]; o.w[w + 3] = v[3];
    }
    return o;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t off = at + j < n ? voff + (at + j) * kSize : kNowhere;
    if constexpr (kSize == 4) {
      o.w[j] = __builtin_amdgcn_raw_buffer_load_b32(r, off, soff, 0);
    } else {
      const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, soff, 0);
      o.w[j >> 1] = j & 1 ? o.w[j >> 1] | v << 16 : v;
    }
  }
  return o;
}

// Four consecutive values as they stand in memory.
template <typename IO>
struct Raw4 {
  uint32_t w[sizeof(typename IO::T)];

  __device__ __forceinline__ float value(int j) const {
    if constexpr (IO::kPerSpan == 4) return __uint_as_float(w[j]);
    else return (j & 1) ? __uint_as_float(w[j >> 1] & 0xffff0000u) : __uint_as_float(w[j >> 1] << 16);
  }
};

// Values at .. at + 3 of a row, as buf_load8.
template <typename IO, bool WHOLE>
__device__ __forceinline__ Raw4<IO> buf_load4(__amdgpu_buffer_rsrc_t r, uint32_t voff, int at, int n) {
  constexpr int kSize = sizeof(typename IO::T);
  Raw4<IO> o;
  if constexpr (WHOLE) {
    const uint32_t off = at < n ? voff + at * kSize : kNowhere;
    if constexpr (kSize == 4) {
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
      o.w[0] = v[0]; o.w[1] = v[1]; o.w[2] = v[2]; o.w[3] = v[3];
    } else {
      const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
      o.w[0] = v[0]; o.w[1] = v[1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t off = at + j < n ? voff + (at + j) * kSize : kNowhere;
      if constexpr (kSize == 4) {
        o.w[j] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
      } else {
        const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
        o.w[j >> 1] = j & 1 ? o.w[j >> 1] | v << 16 : v;
      }
    }
  }
  return o;
}

// The value again, in a scalar register that nothing formed from it leaves the loop around: products with it are formed where they
// are used instead of being kept.
__device__ __forceinline__ uint32_t here(uint32_t v) {
  asm volatile("" : "+s"(v));
  return v;
}

// The same for a lane's value.
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// 16 bytes of every lane's own from memory to LDS, to the wave's place there plus 16 times the lane, past the registers.  They stand
// in LDS for the workgroup after loads_stand and a barrier.
__device__ __forceinline__ void load_to_lds(const void* from, void* wave_place) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                   (__attribute__((address_space(3))) void*)wave_place, 16, 0, 0);
}

__device__ __forceinline__ void loads_stand() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Values 8 c .. 8 c + 7 of tokens 4 g .. 4 g + 3 (as x[token][value], with a scale each) into the blocks of the transposed rows:
// tiles of 32 values, of each four steps of 16 tokens.
template <typename IO>
__device__ __forceinline__ void store_operand_turned(char* hi, char* lo, int g, int c, const float (&x)[4][8], const float (&s)[4]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    char* p = hi + ((c >> 2) * 4 + (g >> 2)) * kBlock + (8 * (c & 3) + j + 32 * (g & 1)) * 16 + (g >> 1 & 1) * 8;
    h4 v, w;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v[t] = (_Float16)(x[t][j] * s[t]);
      if constexpr (planes_of<IO>() == 2) w[t] = (_Float16)fmaf(x[t][j], s[t], -(float)v[t]);
    }
    *reinterpret_cast<h4*>(p) = v;
    if constexpr (planes_of<IO>() == 2) *reinterpret_cast<h4*>(p + (lo - hi)) = w;
  }
}

typedef __bf16 b8 __attribute__((ext_vector_type(8)));

// A 32x32 tile as it is loaded, a lane a row and runs of 8 columns, into a result tile, by a product with the identity in bf16: an
// fp32 value is the sum of three bf16 exactly.  Lane l brings columns 16 (l >> 5) + 8 s .. + 7 for s = 0, 1.
template <typename IO>
__device__ __forceinline__ acc16 turn(const Raw8<IO> (&x)[2], int lane) {
  acc16 acc = zero16();
  const int off = (lane & 31) - 16 * (lane >> 5);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    b8 one;
#pragma unroll
    for (int j = 0; j < 8; ++j) one[j] = (__bf16)(off == 8 * s + j ? 1.0f : 0.0f);
    if constexpr (IO::kPerSpan == 8) {
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, x[s]), one, acc, 0, 0, 0);
    } else {
      b8 p[3];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = __uint_as_float(x[s].w[j]);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          p[n][j] = (__bf16)v;
          v -= (float)p[n][j];
        }
      }
#pragma unroll
      for (int n = 2; n >= 0; --n) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(p[n], one, acc, 0, 0, 0);
    }
  }
  return acc;
}

// The identity as an operand whose summed index is in the order of a result's rows, step s of the tile.
__device__ __forceinline__ h8 identity(int s, int lane) {
  const int n = lane & 31, at = (n >> 4) == s && ((n >> 2) & 1) == (lane >> 5) ? ((n >> 3) & 1) * 4 + (n & 3) : -1;
  h8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = (_Float16)(at == j ? 1.0f : 0.0f);
  return o;
}

// A result tile that has been split (both steps), back as fp32 and transposed: a lane has a row of the tile and 16 of its columns,
// runs of four at 8 g + 4 (lane >> 5).
__device__ __forceinline__ acc16 transposed(const Planes& p0, const Planes& p1, int lane) {
  const h8 e0 = identity(0, lane), e1 = identity(1, lane);
  acc16 acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(p0.hi, e0, zero16(), 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(p1.hi, e1, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(p0.lo, e0, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(p1.lo, e1, acc, 0, 0, 0);
  return acc;
}

// Rows of ldv columns in fp32 stand in memory as operands too: for 32 rows by 16 columns 2 x 64 x 16 bytes, of which a lane has its
// first four values in the first half, its others in the second, so that every access is of whole lines.  The values of such a
// lane after transposed are those of steps col0 / 16 and the next.
__device__ __forceinline__ int64_t block_of(int tile, int step, int64_t ldv) { return ((int64_t)tile * (ldv / 16) + step) * 512; }

__device__ __forceinline__ void store_blocks(float* rows, int tile, int col0, int64_t ldv, int lane, const acc16& v, float f) {
  float* p = rows + block_of(tile, col0 / 16, ldv) + lane * 4;
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<float4*>(p + 256 * g) = make_float4(v[4 * g] * f, v[4 * g + 1] * f, v[4 * g + 2] * f, v[4 * g + 3] * f);
}

// Runs of four of such a lane's columns at `at`, times f, to the row of n at byte offset voff in the I/O type; what lies behind the
// buffer is not written.  WHOLE: n is a multiple of 8 and the tensor is 16-byte aligned.
template <typename IO, bool WHOLE>
__device__ __forceinline__ void store_runs(__amdgpu_buffer_rsrc_t rows, uint32_t voff, int at, int n, const acc16& v, float f) {
  constexpr int kSize = sizeof(typename IO::T);
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int c = at + 8 * g;
    const float x[4] = {v[4 * g] * f, v[4 * g + 1] * f, v[4 * g + 2] * f, v[4 * g + 3] * f};
    if constexpr (WHOLE) {
      const uint32_t off = c < n ? voff + c * kSize : kNowhere;
      if constexpr (kSize == 4) {
        const u4 w = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
        __builtin_amdgcn_raw_buffer_store_b128(w, rows, off, 0, 0);
      } else {
        const u2 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
        __builtin_amdgcn_raw_buffer_store_b64(w, rows, off, 0, 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t off = c + j < n ? voff + (c + j) * kSize : kNowhere;
        if constexpr (kSize == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[j]), rows, off, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16x2(x[j], x[j]), rows, off, 0, 0);
      }
    }
  }
}

// The same, times 1, by address and without knowing n.
template <typename IO>
__device__ __forceinline__ void store_runs(typename IO::T* row, int at, int n, const acc16& v) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int c = at + 8 * g;
    const float x[4] = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
    if (n % 4 == 0) {                                      // the tensor is 16-byte aligned: runs of four are too
      if (c < n) {
        if constexpr (IO::kPerSpan == 4) *reinterpret_cast<float4*>(row + c) = make_float4(x[0], x[1], x[2], x[3]);
        else *reinterpret_cast<uint2*>(row + c) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < n) store_one<IO>(row, c + j, x[j]);
    }
  }
}

template <typename IO>
__device__ __forceinline__ float raw_value(const Raw8<IO>& r, int j) {
  if constexpr (IO::kPerSpan == 4) return __uint_as_float(r.w[j]);
  else return (j & 1) ? __uint_as_float(r.w[j >> 1] & 0xffff0000u) : __uint_as_float(r.w[j >> 1] << 16);
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

// f with dk as the kernels pad it, and whether whole runs of 8 values can be loaded.
template <typename F>
hipError_t by_keys(int dk, bool whole, F f) {
  using std::integral_constant;
  auto g = [&](auto kp) {
    if (whole) f(kp, integral_constant<bool, true>());
    else f(kp, integral_constant<bool, false>());
  };
  if (dk <= 32) g(integral_constant<int, 32>());
  else if (dk <= 64) g(integral_constant<int, 64>());
  else if (dk <= 96) g(integral_constant<int, 96>());
  else g(integral_constant<int, 128>());
  return hipGetLastError();
}

// The vectors that belong to a chunk of a head, kC floats each, as the preparation leaves them.  c_j scales column j of the
// inverse T, s_j row j of k, z_i row i of q (powers of 2); gam_j is the sum of log decays up to j (over log 2), gam_C the
// whole chunk's; s the smallest s_j.  p_i is a whole number: what the gates let the state grow up to token i since it was smallest, less
// half of what it has decayed till then (16 at most).  T, P, U and their like are kept balanced by it, rows times 2^-p_i,
// columns times 2^p_j, U and R as 2^-p_i U_i (their gradients times 2^p_i), so that growth costs no digits, and neither does a decay
// of 2^-32 within the chunk, whether a token's value or the old state is the larger.  The operand P holds
// q_i.k_j s z_i 2^(gam_i - gam_j - p_i + p_j - kPShift).
enum Vec {
  kVecF1,      // beta_j 2^-p_j / c_j
  kVecF2,      // beta_j 2^(gam_j - p_j) / (c_j s_j)
  kVecEnd,     // 2^(gam_C - gam_j + p_j) / s_j
  kVecInto,    // 2^gam_j
  kVecS,       // s_j
  kVecZ,       // z_i
  kVecOut,     // scale 2^(p_i + kPShift) / (z_i s)
  kVecQ,       // scale 2^gam_i / z_i
  kVecJoin,    // kVecQ / kVecOut
  kVecGrow = kVecJoin,   // backward: p_j
  kVecC,       // 1 / c_j
  kVecWhole,   // gam_j - p_j as a whole number and the rest
  kVecRest,
  kVecs
};
static_assert(kVecs * kC * 4 == 3 * 1024, "three waves load the vectors");

// P in an fp16 plane: rows of q and k are of up to 2^7 values below 2^13, so that q_i.k_j is up to 2^33, and the balance adds a factor
// below 2^2.  With low the smallest sum so far, which only falls, and half what is let decay of it (between 0 and 16), gam - p is
// gam - ceil(gam - low), in (low - 1, low], plus floor(half).  From j to a later i low falls by some d >= 0 and half rises by
// d / 2 at most, its whole part by less than d / 2 + 1: gam - p rises by less than 1 - d + d / 2 + 1 <= 2.  So P stays below 2^15.
constexpr int kPShift = 20;

// 2^(whole + rest) of a difference of two such numbers: what an fp32 exponent of that size would lose stays in the rest.
__device__ __forceinline__ float exp2_of(float whole, float rest) {
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(rest), (int)whole);
}

// The operand blocks of a triangular matrix of a chunk: tiles (0, 0), (1, 0), (1, 1), of each two steps of 16; two planes.
constexpr int kTriBlocks = 3 * 2;
constexpr int kTriBytes = kTriBlocks * 1024;     // of a plane

}  // namespace gdr
}  // namespace ssscan
