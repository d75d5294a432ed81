// Device code shared by the kernels of the norm and rotation of queries and keys (gfx950).
#pragma once

#include "device_common.h"
#include "internal.h"
#include "qk_norm_rot.h"

namespace ssscan {
namespace qk {

using namespace dev;

// cos and sin of pos * freq (radians).  The angle in turns is formed and reduced
// to an eighth of a turn in fp64 (an fp32 product is off by radians at positions
// of millions); the rest is a Taylor polynomial on |x| <= pi/4, whose first dropped
// terms are below 2e-9 (sin) and 3e-8 (cos).
__device__ __forceinline__ void angle(double pos, double freq, float& c, float& s) {
  const double turns = pos * (freq * 0.15915494309189533577);
  const double f = turns - __builtin_rint(turns);
  const double q = __builtin_rint(4.0 * f);
  const float x = (float)(f - 0.25 * q) * 6.28318530717958647693f;
  const float x2 = x * x;
  float ps = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  ps = fmaf(ps, x2, 1.0f / 120.0f);
  ps = fmaf(ps, x2, -1.0f / 6.0f);
  ps = fmaf(ps * x2, x, x);
  float pc = fmaf(x2, 1.0f / 40320.0f, -1.0f / 720.0f);
  pc = fmaf(pc, x2, 1.0f / 24.0f);
  pc = fmaf(pc, x2, -0.5f);
  pc = fmaf(pc, x2, 1.0f);
  const int k = (int)q & 3;
  const float cs = k & 1 ? ps : pc, sn = k & 1 ? pc : ps;
  c = k == 1 || k == 2 ? -cs : cs;
  s = k >= 2 ? -sn : sn;
}

__device__ __forceinline__ float wave_total(float v) {
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) v += __shfl_xor(v, k);
  return v;
}

// 1 / sqrt(mean + eps), for the sum of n squares (the hardware's root is within one step).
__device__ __forceinline__ float inv_norm(float sum, const QkArgs& a) {
  return __builtin_amdgcn_rsqf(fmaf(sum, a.inv_n, a.eps));
}

__device__ __forceinline__ double position(const QkArgs& a, int64_t tok, int64_t t) {
  return (double)(a.positions ? a.positions[tok] : a.pos0 + t);
}

// K consecutive elements at any element alignment.
template <typename IO, int K>
struct __attribute__((packed, aligned(sizeof(typename IO::T)))) Run {
  typename IO::T v[K];
};

template <typename IO, int K>
__device__ __forceinline__ void load_run(const typename IO::T* __restrict__ p, float (&x)[K]) {
  const Run<IO, K> r = *reinterpret_cast<const Run<IO, K>*>(p);
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if constexpr (IO::kPerSpan == 4) x[j] = r.v[j];
    else x[j] = bf16_bits_to_float(r.v[j]);
  }
}

template <typename IO, int K>
__device__ __forceinline__ void store_run(typename IO::T* __restrict__ p, const float (&x)[K]) {
  Run<IO, K> r;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if constexpr (IO::kPerSpan == 4) r.v[j] = x[j];
    else r.v[j] = (uint16_t)float_to_bf16_bits(x[j]);
  }
  *reinterpret_cast<Run<IO, K>*>(p) = r;
}

}  // namespace qk
}  // namespace ssscan
