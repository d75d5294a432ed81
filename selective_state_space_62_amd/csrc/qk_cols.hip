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

// How a vector's pairs lie in it: 2p and 2p + 1 (HALF 0: interleaved, or nothing
// rotated), or p and p + HALF up to HALF and 2p and 2p + 1 from there.  A constant, so
// that pairs are picked from vector loads by register (612000 tokens cut from rows of 192
// values, half of 16 rotated, whole call: bf16 28 us, element by element 51; fp32 40 and 62).
template <int N, int HALF>
__device__ __forceinline__ constexpr int place(int k) {   // of value k % 2 of pair k / 2
  return N == 1 ? 0 : k / 2 < HALF ? k / 2 + k % 2 * HALF : k;
}

// x[2 p + h] = value h of pair p.
template <typename IO, int N, int HALF>
__device__ __forceinline__ void load_pairs(const typename IO::T* __restrict__ in, float (&x)[N]) {
  float v[N];
  load_run<IO, N>(in, v);
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = v[place<N, HALF>(k)];
}

template <typename IO, int N, int HALF>
__device__ __forceinline__ void store_pairs(typename IO::T* __restrict__ out, const float (&x)[N]) {
  float v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) v[place<N, HALF>(k)] = x[k];
  store_run<IO, N>(out, v);
}

template <int N, int HALF>
__device__ __forceinline__ void load_weight(const float* __restrict__ w, float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = w ? w[place<N, HALF>(k)] : 1.0f;
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

// The lane's token of a turn of blockDim.x; past the last one, the last one again.
struct Token {
  int64_t tok, b, t;
  bool act;
  __device__ __forceinline__ Token(const QkArgs& a, int64_t turn) {
    const int64_t tokens = a.batch * a.seqlen;
    tok = turn * blockDim.x + threadIdx.x;
    act = tok < tokens;
    tok = act ? tok : tokens - 1;
    b = tok / a.seqlen;
    t = tok - b * a.seqlen;
  }
};

// The norm, weight and rotation of one vector.
template <int N>
__device__ __forceinline__ void forward(const QkArgs& a, const float (&w)[N], const float (&c)[N / 2 + 1],
                                        const float (&sn)[N / 2 + 1], float (&x)[N]) {
  float sq = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) sq = fmaf(x[k], x[k], sq);
  const float rho = inv_norm(sq, a);
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = x[k] * rho * w[k];
#pragma unroll
  for (int p = 0; p < N / 2; ++p) {
    if (p >= a.half) continue;
    const float r = x[2 * p] * c[p] - x[2 * p + 1] * sn[p];
    x[2 * p + 1] = fmaf(x[2 * p + 1], c[p], x[2 * p] * sn[p]);
    x[2 * p] = r;
  }
}

// Both sides' loads are out before the angles are formed: the rows' 64 bytes of B and C
// are the wait (a million bf16 tokens, half of 16 values rotated, interleaved, whole call:
// one side after the other 52.4, ahead 45.7, with the registers for six waves to a SIMD
// 43.5 us; a copy of the same 64 bytes of each 320-byte row 32 us).  Turning tiles in LDS for 16-byte stores took 54 us, for 16-byte pieces
// of a row to neighbouring lanes 77 us, 4-byte stores of two tokens 51 us.
template <typename IO, int N, int HALF>
__global__ __launch_bounds__(64, N == 16 && IO::kPerSpan == 4 ? 5 : 6) void qk_cols_fwd_kernel(QkArgs a, int64_t turns) {
  using T = typename IO::T;
  const int heads = a.side[0].heads + a.side[1].heads;
  for (int64_t turn = blockIdx.x; turn < turns; turn += gridDim.x) {
    const Token tk(a, turn);
    // the token's vectors, queries first; one is loaded ahead
    auto fetch = [&](int item, float (&x)[N]) {
      const int side = item >= a.side[0].heads, h = item - (side ? a.side[0].heads : 0);
      const QkSide& sd = a.side[side];
      load_pairs<IO, N, HALF>((const T*)sd.in + tk.b * sd.stride[0] + tk.t * sd.stride[1] + h * sd.stride[2], x);
    };
    float x[N], next[N];
    fetch(0, x);
    if (heads > 1) fetch(1, next);
    float c[N / 2 + 1], sn[N / 2 + 1];
    angles<N>(a, position(a, tk.tok, tk.t), c, sn);
    for (int item = 0; item < heads; ++item) {
      const int side = item >= a.side[0].heads, h = item - (side ? a.side[0].heads : 0);
      const QkSide& sd = a.side[side];
      float w[N];
      load_weight<N, HALF>(sd.w, w);
      forward<N>(a, w, c, sn, x);
      T* out = (T*)sd.out + (tk.b * sd.heads + h) * N * a.seqlen;
      if (tk.act) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          store_one<IO>(out, place<N, HALF>(k) * a.seqlen + tk.t, x[k]);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = next[k];
      if (item + 2 < heads) fetch(item + 2, next);
    }
  }
}

// With n = rho w v and o the rotated n: dn is the gradient of o rotated back, and
// with p = w dn, dv = rho p - rho^3 v mean(p v), dw = sum of dn rho v.
template <typename IO, int N, int HALF>
__global__ __launch_bounds__(256) void qk_cols_bwd_kernel(QkArgs a, int64_t turns) {
  using T = typename IO::T;
  __shared__ float s_dw[2][4][N];
  float dw[2][N] = {};
  for (int64_t turn = blockIdx.x; turn < turns; turn += gridDim.x) {
    const Token tk(a, turn);
    float c[N / 2 + 1], sn[N / 2 + 1];
    angles<N>(a, position(a, tk.tok, tk.t), c, sn);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkSide& sd = a.side[side];
      float w[N];
      load_weight<N, HALF>(sd.w, w);
      for (int h = 0; h < sd.heads; ++h) {
        float x[N], d[N];
        load_pairs<IO, N, HALF>((const T*)sd.in + tk.b * sd.stride[0] + tk.t * sd.stride[1] + h * sd.stride[2], x);
        const T* dout = (const T*)sd.dout + (tk.b * sd.heads + h) * N * a.seqlen;
#pragma unroll
        for (int k = 0; k < N; ++k)
          d[k] = load_one<IO>(dout, place<N, HALF>(k) * a.seqlen + tk.t);
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
        const float rho = inv_norm(sq, a), back = rho * rho * (pv * (1.0f / N));
        if (tk.act) {
#pragma unroll
          for (int k = 0; k < N; ++k) {
            dw[side][k] = fmaf(d[k], rho * x[k], dw[side][k]);
            x[k] = rho * (d[k] * w[k] - x[k] * back);
          }
          store_pairs<IO, N, HALF>((T*)sd.din + tk.b * sd.dstride[0] + tk.t * sd.dstride[1] + h * sd.dstride[2], x);
        }
      }
    }
  }
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (!a.side[side].dw) continue;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float v = wave_total(dw[side][k]);
      if ((threadIdx.x & 63) == 0) s_dw[side][wave][place<N, HALF>(k)] = v;
    }
  }
  __syncthreads();
  const int side = threadIdx.x / N, j = threadIdx.x % N;
  if (side < 2 && a.side[side].dw) {
    float v = s_dw[side][0][j];
    for (int k = 1; k < (int)blockDim.x / 64; ++k) v += s_dw[side][k][j];
    a.part[(a.part_row[side] + blockIdx.x) * N + j] = v;
  }
}

struct ColsShape {
  int64_t turns;   // of a workgroup's threads, a token each
  unsigned blocks, threads;
};

template <typename IO, int N, int HALF>
void launch(const QkArgs& a, bool back, const ColsShape& sh, hipStream_t s) {
  if (back) hipLaunchKernelGGL((qk_cols_bwd_kernel<IO, N, HALF>), dim3(sh.blocks), dim3(sh.threads), 0, s, a, sh.turns);
  else hipLaunchKernelGGL((qk_cols_fwd_kernel<IO, N, HALF>), dim3(sh.blocks), dim3(64), 0, s, a, sh.turns);
}

// The kernel for this half: HALF down to 1 where pairs lie apart, or 0.
template <typename IO, int N, int HALF = N / 2>
void by_half(const QkArgs& a, bool back, const ColsShape& sh, hipStream_t s) {
  if constexpr (N >= 4 && HALF > 0) {   // one pair at most lies as adjacent ones do
    if (!a.interleaved && a.half == HALF) launch<IO, N, HALF>(a, back, sh, s);
    else by_half<IO, N, HALF - 1>(a, back, sh, s);
  } else {
    launch<IO, N, 0>(a, back, sh, s);
  }
}

template <typename IO>
hipError_t by_dim(const QkArgs& a, bool back, const ColsShape& sh, hipStream_t s) {
  switch (a.n) {
    case 1: by_half<IO, 1>(a, back, sh, s); break;
    case 2: by_half<IO, 2>(a, back, sh, s); break;
    case 4: by_half<IO, 4>(a, back, sh, s); break;
    case 8: by_half<IO, 8>(a, back, sh, s); break;
    case 16: by_half<IO, 16>(a, back, sh, s); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

ColsShape shape_of(const QkArgs& a, unsigned threads, int64_t most) {
  ColsShape sh;
  sh.threads = threads;
  sh.turns = (a.batch * a.seqlen + threads - 1) / threads;
  sh.blocks = (unsigned)(sh.turns < most ? sh.turns : most);
  return sh;
}

hipError_t go(const QkArgs& a, bool back, const ColsShape& sh, hipStream_t s) {
  return a.io == kIoBf16 ? by_dim<BF16>(a, back, sh, s) : by_dim<F32>(a, back, sh, s);
}

}  // namespace

hipError_t launch_qk_cols(const QkArgs& a, hipStream_t s) { return go(a, false, shape_of(a, 64, 1 << 20), s); }

hipError_t launch_qk_cols_bwd(QkArgs& a, const QkBwdPlan& p, hipStream_t s) {
  int64_t most = 1 << 20;
  for (int i = 0; i < 2; ++i)
    if (a.side[i].heads && p.blocks[i] < most) most = p.blocks[i];
  // the workgroups are few, each with a row of sums: four waves each where the tokens fill
  // them (whole call, one wave -> four: 320860 tokens, half of 16 values rotated, bf16 42.8 ->
  // 36.9 us, fp32 43.5 -> 48.2; a million, all rotated, bf16 167 -> 123, fp32 147 -> 131)
  const ColsShape sh = shape_of(a, a.batch * a.seqlen >= 256 * most ? 256 : 64, most);
  for (int i = 0; i < 2; ++i) a.part_rows[i] = a.side[i].heads ? (int64_t)sh.blocks : 0;
  a.part_row[1] = a.part_rows[0];
  return go(a, true, sh, s);
}

}  // namespace ssscan
