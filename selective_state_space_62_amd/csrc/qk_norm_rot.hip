// Norm and position rotation of queries and keys: dispatch, the backward's sums, and
// the kernels for token-major heads of any shape (gfx950).
//
// Here a wave takes one vector (the values of one head at one token) at a time; a
// lane holds pairs of values that a rotation mixes, so that after the sum of squares
// no value crosses lanes.  It loads element by element, for shapes whose pairs do
// not come in runs of two or more (an odd head_dim, an odd number of rotated pairs).
#include "qk_device.h"

namespace ssscan {
namespace {

using namespace qk;

constexpr int kSlots = 2;   // pairs per lane: head_dim <= 256

// The places of pair p's two values; the second is -1 for a last single value.
__device__ __forceinline__ void places(const QkArgs& a, int p, int& j1, int& j2) {
  if (p < a.half) {
    j1 = a.interleaved ? 2 * p : p;
    j2 = a.interleaved ? 2 * p + 1 : p + a.half;
  } else {
    j1 = 2 * p;
    j2 = j1 + 1 < a.n ? j1 + 1 : -1;
  }
}

struct Vec {
  int64_t b, t, tok;
  int h;
};

__device__ __forceinline__ Vec vec_of(const QkArgs& a, int64_t v, int heads) {
  Vec o;
  o.tok = v / heads;
  o.h = (int)(v - o.tok * heads);
  o.b = o.tok / a.seqlen;
  o.t = o.tok - o.b * a.seqlen;
  return o;
}

template <typename IO>
__global__ __launch_bounds__(256) void qk_fwd_kernel(QkArgs a) {
  using T = typename IO::T;
  const QkSide& sd = a.side[blockIdx.z];
  const int lane = threadIdx.x & 63;
  const int64_t vectors = a.batch * a.seqlen * sd.heads;
  const int64_t waves = (int64_t)gridDim.x * 4;
  const int pairs = a.half + (a.n - 2 * a.half + 1) / 2;
  for (int64_t v = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); v < vectors; v += waves) {
    const Vec o = vec_of(a, v, sd.heads);
    const T* in = (const T*)sd.in + o.b * sd.stride[0] + o.t * sd.stride[1] + o.h * sd.stride[2];
    T* out = (T*)sd.out + (o.tok * sd.heads + o.h) * a.n;
    float x[kSlots][2];
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const int p = lane + 64 * k;
      int j1, j2;
      places(a, p, j1, j2);
      x[k][0] = p < pairs ? load_one<IO>(in, j1) : 0.0f;
      x[k][1] = p < pairs && j2 >= 0 ? load_one<IO>(in, j2) : 0.0f;
      sq = fmaf(x[k][0], x[k][0], sq);
      sq = fmaf(x[k][1], x[k][1], sq);
    }
    const float rho = inv_norm(wave_total(sq), a);
    const double pos = position(a, o.tok, o.t);
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const int p = lane + 64 * k;
      if (p >= pairs) continue;
      int j1, j2;
      places(a, p, j1, j2);
      float n1 = x[k][0] * rho * (sd.w ? sd.w[j1] : 1.0f);
      float n2 = j2 >= 0 ? x[k][1] * rho * (sd.w ? sd.w[j2] : 1.0f) : 0.0f;
      if (p < a.half) {
        float c, s;
        angle(pos, a.inv_freq[p], c, s);
        const float r1 = n1 * c - n2 * s;
        n2 = fmaf(n2, c, n1 * s);
        n1 = r1;
      }
      store_one<IO>(out, j1, n1);
      if (j2 >= 0) store_one<IO>(out, j2, n2);
    }
  }
}

// With n = rho w v and o the rotated n: dn is the gradient of o rotated back, and
// with p = w dn, dv = rho p - rho^3 v mean(p v), dw = sum of dn rho v.
template <typename IO>
__global__ __launch_bounds__(256) void qk_bwd_kernel(QkArgs a) {
  using T = typename IO::T;
  __shared__ float s_dw[4][256];
  const QkSide& sd = a.side[blockIdx.z];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t vectors = a.batch * a.seqlen * sd.heads;
  if ((int64_t)blockIdx.x >= a.part_rows[blockIdx.z]) return;
  const int64_t waves = a.part_rows[blockIdx.z] * 4;
  const int pairs = a.half + (a.n - 2 * a.half + 1) / 2;
  float dw[kSlots][2] = {};
  for (int64_t v = (int64_t)blockIdx.x * 4 + wave; v < vectors; v += waves) {
    const Vec o = vec_of(a, v, sd.heads);
    const T* in = (const T*)sd.in + o.b * sd.stride[0] + o.t * sd.stride[1] + o.h * sd.stride[2];
    T* din = (T*)sd.din + o.b * sd.dstride[0] + o.t * sd.dstride[1] + o.h * sd.dstride[2];
    const T* dout = (const T*)sd.dout + (o.tok * sd.heads + o.h) * a.n;
    const double pos = position(a, o.tok, o.t);
    float x[kSlots][2], d[kSlots][2], pw[kSlots][2];
    float sq = 0.0f, pv = 0.0f;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const int p = lane + 64 * k;
      int j1, j2;
      places(a, p, j1, j2);
      const bool one = p < pairs, two = one && j2 >= 0;
      x[k][0] = one ? load_one<IO>(in, j1) : 0.0f;
      x[k][1] = two ? load_one<IO>(in, j2) : 0.0f;
      float d1 = one ? load_one<IO>(dout, j1) : 0.0f;
      float d2 = two ? load_one<IO>(dout, j2) : 0.0f;
      if (p < a.half) {
        float c, s;
        angle(pos, a.inv_freq[p], c, s);
        const float r1 = fmaf(d1, c, d2 * s);
        d2 = d2 * c - d1 * s;
        d1 = r1;
      }
      d[k][0] = d1;
      d[k][1] = d2;
      pw[k][0] = one && sd.w ? d1 * sd.w[j1] : d1;
      pw[k][1] = two && sd.w ? d2 * sd.w[j2] : d2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sq = fmaf(x[k][h], x[k][h], sq);
        pv = fmaf(pw[k][h], x[k][h], pv);
      }
    }
    const float rho = inv_norm(wave_total(sq), a);
    const float back = rho * rho * (wave_total(pv) * a.inv_n);
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const int p = lane + 64 * k;
      int j1, j2;
      places(a, p, j1, j2);
#pragma unroll
      for (int h = 0; h < 2; ++h) dw[k][h] = fmaf(d[k][h], rho * x[k][h], dw[k][h]);
      if (p < pairs) store_one<IO>(din, j1, rho * (pw[k][0] - x[k][0] * back));
      if (p < pairs && j2 >= 0) store_one<IO>(din, j2, rho * (pw[k][1] - x[k][1] * back));
    }
  }
  if (!sd.dw) return;
#pragma unroll
  for (int k = 0; k < kSlots; ++k) {
    const int p = lane + 64 * k;
    int j1, j2;
    places(a, p, j1, j2);
    if (p < pairs) s_dw[wave][j1] = dw[k][0];
    if (p < pairs && j2 >= 0) s_dw[wave][j2] = dw[k][1];
  }
  __syncthreads();
  const int j = threadIdx.x;
  if (j < a.n)
    a.part[(a.part_row[blockIdx.z] + blockIdx.x) * a.n + j] = (s_dw[0][j] + s_dw[1][j]) + (s_dw[2][j] + s_dw[3][j]);
}

// dw[j] of a side: its rows of partial sums in a fixed order, 64 runs of them summed
// by 64 threads and then joined.
__global__ __launch_bounds__(1024) void qk_reduce_kernel(QkArgs a) {
  __shared__ float s_sum[64][16];
  const QkSide& sd = a.side[blockIdx.z];
  if (!sd.dw) return;
  const int col = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int j = (int)blockIdx.x * 16 + col;
  float v = 0.0f;
  if (j < a.n) {
    const float* in = a.part + a.part_row[blockIdx.z] * a.n + j;
#pragma unroll 4
    for (int64_t b = run; b < a.part_rows[blockIdx.z]; b += 64) v += in[b * a.n];
  }
  s_sum[run][col] = v;
  __syncthreads();
  if (run == 0 && j < a.n) {
    for (int k = 1; k < 64; ++k) v += s_sum[k][col];
    sd.dw[j] = v;
  }
}

}  // namespace

// About 1024 rows of partial sums, shared by the sides as their heads are: four workgroups
// to a CU, which is what the registers of the kernel for runs allow (25 fp32 heads of 80 at 8188
// tokens counted from pos0, whole call: 1024 rows 46, 2048 50, 4096 53 us).  Twice as many for the short
// heads of the feature-major kernel, which needs less of both.
QkBwdPlan qk_bwd_plan(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int n) {
  QkBwdPlan p;
  const int64_t heads = (int64_t)heads_q + heads_k, tokens = batch * seqlen;
  for (int i = 0; i < 2; ++i) {
    const int64_t h = i ? heads_k : heads_q, most = (n <= 16 ? 2048 : 1024) * h / heads;
    p.blocks[i] = h == 0 ? 0 : most < 1 ? 1 : most < tokens ? most : tokens;
  }
  return p;
}

hipError_t launch_qk_norm_rot(const QkArgs& a, hipStream_t s) {
  if (a.feature_major) return launch_qk_cols(a, s);
  if (qk_rows_take(a)) return launch_qk_rows(a, s);
  const int hmax = a.side[0].heads > a.side[1].heads ? a.side[0].heads : a.side[1].heads;
  int64_t blocks = (a.batch * a.seqlen * hmax + 3) / 4;
  if (blocks > 8192) blocks = 8192;
  const dim3 g((unsigned)blocks, 1, 2);
  if (a.io == kIoBf16) hipLaunchKernelGGL((qk_fwd_kernel<BF16>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((qk_fwd_kernel<F32>), g, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_qk_norm_rot_bwd(QkArgs a, hipStream_t s) {
  const QkBwdPlan p = qk_bwd_plan(a.batch, a.seqlen, a.side[0].heads, a.side[1].heads, a.n);
  hipError_t e;
  if (a.feature_major) {
    e = launch_qk_cols_bwd(a, p, s);
  } else if (qk_rows_take(a)) {
    e = launch_qk_rows_bwd(a, p, s);
  } else {
    for (int i = 0; i < 2; ++i) a.part_rows[i] = p.blocks[i];
    a.part_row[1] = a.part_rows[0];
    const dim3 g((unsigned)(p.blocks[0] > p.blocks[1] ? p.blocks[0] : p.blocks[1]), 1, 2);
    if (a.io == kIoBf16) hipLaunchKernelGGL((qk_bwd_kernel<BF16>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((qk_bwd_kernel<F32>), g, dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  if (e != hipSuccess || (!a.side[0].dw && !a.side[1].dw)) return e;
  hipLaunchKernelGGL(qk_reduce_kernel, dim3((unsigned)((a.n + 15) / 16), 1, 2), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssscan
