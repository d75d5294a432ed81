// Norm and position rotation of queries and keys into feature-major outputs (gfx950):
// the scan's C and B from a projection's rows.
//
// A lane takes one token: its head_dim values (at most 16) are one or two vector
// loads, the sums stay in the lane, the angles are formed once for both sides and
// all heads, and value j of 64 tokens is one run of the output.
#include "qk_device.h"

namespace ssscan {
namespace {

using namespace qk;

// How a vector lies in registers: pair p is values 2p and 2p + 1 of the input
// (kAdjacent: interleaved, or nothing rotated), p and p + N/2 (kHalves: all of it
// rotated), or p and p + half up to half and 2p and 2p + 1 from there (kPartial,
// whose element addresses depend on half, so it loads one by one).
enum Order { kAdjacent, kHalves, kPartial };

template <int N, int ORDER>
__device__ __forceinline__ int place(int p, int h, int half) {
  if constexpr (ORDER == kAdjacent) return 2 * p + h;
  else if constexpr (ORDER == kHalves) return p + h * (N / 2);
  else return p < half ? p + h * half : 2 * p + h;
}

// x[2 p + h] = value h of pair p.
template <typename IO, int N, int ORDER>
__device__ __forceinline__ void load_pairs(const typename IO::T* __restrict__ in, int half, float (&x)[N]) {
  if constexpr (N == 1) {
    x[0] = load_one<IO>(in, 0);
  } else if constexpr (ORDER == kPartial) {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = load_one<IO>(in, place<N, ORDER>(k >> 1, k & 1, half));
  } else {
    float v[N];
    load_run<IO, N>(in, v);
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = v[place<N, ORDER>(k >> 1, k & 1, half)];
  }
}

template <typename IO, int N, int ORDER>
__device__ __forceinline__ void store_pairs(typename IO::T* __restrict__ out, int half, const float (&x)[N]) {
  if constexpr (N == 1) {
    store_one<IO>(out, 0, x[0]);
  } else if constexpr (ORDER == kPartial) {
#pragma unroll
    for (int k = 0; k < N; ++k) store_one<IO>(out, place<N, ORDER>(k >> 1, k & 1, half), x[k]);
  } else {
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[place<N, ORDER>(k >> 1, k & 1, half)] = x[k];
    store_run<IO, N>(out, v);
  }
}

template <int N, int ORDER>
__device__ __forceinline__ void load_weight(const float* __restrict__ w, int half, float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = w ? w[N == 1 ? 0 : place<N, ORDER>(k >> 1, k & 1, half)] : 1.0f;
}

template <int N>
__device__ __forceinline__ void angles(const QkArgs& a, double pos, float (&c)[N / 2 + 1], float (&s)[N / 2 + 1]) {
#pragma unroll
  for (int p = 0; p < N / 2; ++p) {
    c[p] = 1.0f;
    s[p] = 0.0f;
    if (p < a.half) angle(pos, a.inv_freq[p], c[p], s[p]);
  }
}

template <typename IO, int N, int ORDER>
__global__ __launch_bounds__(64) void qk_cols_fwd_kernel(QkArgs a) {
  using T = typename IO::T;
  const int64_t tokens = a.batch * a.seqlen;
  for (int64_t tok = (int64_t)blockIdx.x * 64 + threadIdx.x; tok < tokens; tok += (int64_t)gridDim.x * 64) {
    const int64_t b = tok / a.seqlen, t = tok - b * a.seqlen;
    float c[N / 2 + 1], sn[N / 2 + 1];
    angles<N>(a, position(a, tok, t), c, sn);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkSide& sd = a.side[side];
      float w[N];
      load_weight<N, ORDER>(sd.w, a.half, w);
      for (int h = 0; h < sd.heads; ++h) {
        float x[N];
        load_pairs<IO, N, ORDER>((const T*)sd.in + b * sd.stride[0] + t * sd.stride[1] + h * sd.stride[2], a.half, x);
        float sq = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) sq = fmaf(x[k], x[k], sq);
        const float rho = inv_norm(sq, a);
        T* out = (T*)sd.out + (b * sd.heads + h) * N * a.seqlen + t;
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = x[k] * rho * w[k];
#pragma unroll
        for (int p = 0; p < N / 2; ++p) {
          if (p >= a.half) continue;
          const float r = x[2 * p] * c[p] - x[2 * p + 1] * sn[p];
          x[2 * p + 1] = fmaf(x[2 * p + 1], c[p], x[2 * p] * sn[p]);
          x[2 * p] = r;
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
          store_one<IO>(out, (N == 1 ? 0 : place<N, ORDER>(k >> 1, k & 1, a.half)) * a.seqlen, x[k]);
      }
    }
  }
}

// With n = rho w v and o the rotated n: dn is the gradient of o rotated back, and
// with p = w dn, dv = rho p - rho^3 v mean(p v), dw = sum of dn rho v.
template <typename IO, int N, int ORDER>
__global__ __launch_bounds__(64) void qk_cols_bwd_kernel(QkArgs a) {
  using T = typename IO::T;
  const int64_t tokens = a.batch * a.seqlen;
  float dw[2][N] = {};
  for (int64_t tok = (int64_t)blockIdx.x * 64 + threadIdx.x; tok < tokens; tok += (int64_t)gridDim.x * 64) {
    const int64_t b = tok / a.seqlen, t = tok - b * a.seqlen;
    float c[N / 2 + 1], sn[N / 2 + 1];
    angles<N>(a, position(a, tok, t), c, sn);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkSide& sd = a.side[side];
      float w[N];
      load_weight<N, ORDER>(sd.w, a.half, w);
      for (int h = 0; h < sd.heads; ++h) {
        float x[N], d[N];
        load_pairs<IO, N, ORDER>((const T*)sd.in + b * sd.stride[0] + t * sd.stride[1] + h * sd.stride[2], a.half, x);
        const T* dout = (const T*)sd.dout + (b * sd.heads + h) * N * a.seqlen + t;
#pragma unroll
        for (int k = 0; k < N; ++k)
          d[k] = load_one<IO>(dout, (N == 1 ? 0 : place<N, ORDER>(k >> 1, k & 1, a.half)) * a.seqlen);
#pragma unroll
        for (int p = 0; p < N / 2; ++p) {
          if (p >= a.half) continue;
          const float r = fmaf(d[2 * p], c[p], d[2 * p + 1] * sn[p]);
          d[2 * p + 1] = d[2 * p + 1] * c[p] - d[2 * p] * sn[p];
          d[2 * p] = r;
        }
        float sq = 0.0f, pv = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          sq = fmaf(x[k], x[k], sq);
          pv = fmaf(d[k] * w[k], x[k], pv);
        }
        const float rho = inv_norm(sq, a), back = rho * rho * (pv / (float)N);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          dw[side][k] = fmaf(d[k], rho * x[k], dw[side][k]);
          x[k] = rho * (d[k] * w[k] - x[k] * back);
        }
        store_pairs<IO, N, ORDER>((T*)sd.din + b * sd.dstride[0] + t * sd.dstride[1] + h * sd.dstride[2], a.half, x);
      }
    }
  }
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (!a.side[side].dw) continue;
    float* part = a.part + (a.part_row[side] + blockIdx.x) * N;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float v = dw[side][k];
#pragma unroll
      for (int step = 1; step < 64; step <<= 1) v += __shfl_xor(v, step);
      if (threadIdx.x == 0) part[N == 1 ? 0 : place<N, ORDER>(k >> 1, k & 1, a.half)] = v;
    }
  }
}

template <typename IO, int N, int ORDER>
void launch(const QkArgs& a, bool back, unsigned blocks, hipStream_t s) {
  if (back) hipLaunchKernelGGL((qk_cols_bwd_kernel<IO, N, ORDER>), dim3(blocks), dim3(64), 0, s, a);
  else hipLaunchKernelGGL((qk_cols_fwd_kernel<IO, N, ORDER>), dim3(blocks), dim3(64), 0, s, a);
}

template <typename IO, int N>
void by_order(const QkArgs& a, bool back, unsigned blocks, hipStream_t s) {
  if constexpr (N <= 2) {   // one pair at most: every order is the same
    launch<IO, N, kAdjacent>(a, back, blocks, s);
  } else {
    if (a.interleaved || a.half == 0) launch<IO, N, kAdjacent>(a, back, blocks, s);
    else if (2 * a.half == N) launch<IO, N, kHalves>(a, back, blocks, s);
    else launch<IO, N, kPartial>(a, back, blocks, s);
  }
}

template <typename IO>
hipError_t by_dim(const QkArgs& a, bool back, unsigned blocks, hipStream_t s) {
  switch (a.n) {
    case 1: by_order<IO, 1>(a, back, blocks, s); break;
    case 2: by_order<IO, 2>(a, back, blocks, s); break;
    case 4: by_order<IO, 4>(a, back, blocks, s); break;
    case 8: by_order<IO, 8>(a, back, blocks, s); break;
    case 16: by_order<IO, 16>(a, back, blocks, s); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t go(const QkArgs& a, bool back, int64_t most, hipStream_t s) {
  int64_t blocks = (a.batch * a.seqlen + 63) / 64;
  if (blocks > most) blocks = most;
  return a.io == kIoBf16 ? by_dim<BF16>(a, back, (unsigned)blocks, s) : by_dim<F32>(a, back, (unsigned)blocks, s);
}

}  // namespace

hipError_t launch_qk_cols(const QkArgs& a, hipStream_t s) { return go(a, false, 1 << 20, s); }

hipError_t launch_qk_cols_bwd(QkArgs& a, const QkBwdPlan& p, hipStream_t s) {
  int64_t blocks = (a.batch * a.seqlen + 63) / 64;
  if (blocks > p.token_blocks) blocks = p.token_blocks;
  for (int i = 0; i < 2; ++i) a.part_rows[i] = a.side[i].heads ? blocks : 0;
  a.part_row[1] = a.part_rows[0];
  return go(a, true, blocks, s);
}

}  // namespace ssscan
