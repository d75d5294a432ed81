// Gated linear recurrence, backward pass (gfx950).
//
// With w_t = dy_t silu(z_t) and G_t = a_t g_t, the adjoint that token t hands to
// the state before it, g_t = w_t + G_(t+1): the same kind of recurrence from the
// other end, with the same decays.  A tile of a row is loaded once; the wave scans
// the forward maps upwards (the states, from the state entering the tile) and the
// adjoint's maps downwards, both exchanged between the row's waves in one step.
// Tiles run from the row's end to its start; the state entering each comes from
// the stored ones.
#include "glr_device.h"

namespace ssscan {
namespace glr {
namespace {

template <typename IO, int KIND, bool HI, bool HZ, int W>
__global__ __launch_bounds__(256) void glr_bwd_kernel(GlrArgs p) {
  using T = typename IO::T;
  constexpr int R = 4 / W;
  constexpr int64_t kTile = W * 64 * kV;
  __shared__ float s_tot[2][4][3];
  __shared__ float s_sum[4][3];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % W;
  const int64_t first = block_index() * R;
  if (first >= p.rows) return;
  const bool act = first + wave / W < p.rows;
  const int64_t row = act ? first + wave / W : p.rows - 1;   // a padding wave repeats a row and stores nothing
  const int64_t d = row % p.dim;
  const RowConst c = row_const<KIND>(p, d);
  const int64_t base = row * p.seqlen;
  const int64_t tiles = (p.seqlen + kTile - 1) / kTile;
  float G = p.dh_final ? p.dh_final[row] : 0.0f;   // the adjoint entering the tile from its end
  float sum_d = 0.0f, sum_r = 0.0f, sum_i = 0.0f;
  for (int64_t n = tiles - 1; n >= 0; --n) {
    float hc = n > 0 ? p.ckpt[row * tiles + n] : p.h0 ? p.h0[row] : 0.0f;
    const int64_t t = n * kTile + (part * 64 + lane) * kV;
    const int valid = (int)(p.seqlen - t < kV ? (p.seqlen - t > 0 ? p.seqlen - t : 0) : kV);
    const Raw<IO> xv = load_raw<IO>((const T*)p.x + base + t, valid);
    const Raw<IO> rv = load_raw<IO>((const T*)p.r + base + t, valid);
    const Raw<IO> yv = load_raw<IO>((const T*)p.dy + base + t, valid);
    Raw<IO> iv, zv;
    if constexpr (HI) iv = load_raw<IO>((const T*)p.i + base + t, valid);
    if constexpr (HZ) zv = load_raw<IO>((const T*)p.z + base + t, valid);
    float a[kV], m[kV], ix[kV], w[kV];
    float A = 1.0f, B = 0.0f, D = 0.0f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      gate<KIND>(rv[j], c, a[j], m[j]);
      ix[j] = xv[j];
      if constexpr (HI) {
        float e;
        ix[j] *= sigmoid_e(iv[j], c.ib, e);
      }
      w[j] = yv[j];
      if constexpr (HZ) w[j] *= silu(zv[j]);
      if (j >= valid) {
        a[j] = 1.0f;
        m[j] = 0.0f;
      }
      A *= a[j];
      B = fmaf(a[j], B, m[j] * ix[j]);
    }
#pragma unroll
    for (int j = kV - 1; j >= 0; --j) D = a[j] * (w[j] + D);
    float Ad = A;
    scan_up(A, B);
    scan_down(Ad, D, lane);
    const float At = lane_value(A, 63), Bt = lane_value(B, 63), Dt = lane_value(D, 0);
    float h_enter = hc, g_enter = G;
    if constexpr (W == 1) {
      G = fmaf(At, G, Dt);
    } else {
      float(&tot)[4][3] = s_tot[n & 1];
      if (lane == 0) {
        tot[wave][0] = At;
        tot[wave][1] = Bt;
        tot[wave][2] = Dt;
      }
      __syncthreads();   // the other parity's totals are read before the next barrier only
#pragma unroll
      for (int k = 0; k < W; ++k) {
        if (k == part) h_enter = hc;
        hc = fmaf(tot[wave - part + k][0], hc, tot[wave - part + k][1]);
      }
#pragma unroll
      for (int k = W - 1; k >= 0; --k) {
        if (k == part) g_enter = G;
        G = fmaf(tot[wave - part + k][0], G, tot[wave - part + k][2]);
      }
    }
    float h = fmaf(shift_up(1.0f, A), h_enter, shift_up(0.0f, B));
    float g_in = fmaf(shift_down(1.0f, Ad), g_enter, shift_down(0.0f, D));
    float before[kV], dz[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      before[j] = h;
      h = fmaf(a[j], h, m[j] * ix[j]);
      if constexpr (HZ) {
        float e;
        const float zj = zv[j], s = sigmoid_e(zj, 0.0f, e);
        dz[j] = yv[j] * h * (s * fmaf(zj, one_minus(s, e), 1.0f));
      }
    }
    float dx[kV], dr[kV], di[kV];
#pragma unroll
    for (int j = kV - 1; j >= 0; --j) {
      const float g = w[j] + g_in;
      g_in = a[j] * g;
      float e;
      const float s = sigmoid_e(rv[j], c.rb, e), oms = one_minus(s, e);
      float dd;   // the token's part of ddecay (normalised: over its common factor)
      if constexpr (KIND == kConvex) {
        const float da = g * (before[j] - ix[j]);
        dr[j] = da * m[j] * s;
        dd = da * oms;
      } else {
        const float ls = 0.5f * c.c1 * s;
        const float q = one_minus_sq(c.c1 * s, a[j]);
        const float k = ls * __builtin_amdgcn_rsqf(fmaxf(q, kTiny));   // 0 where ls is 0
        dd = g * a[j] * fmaf(a[j] * k, ix[j], -ls * before[j]);
        dr[j] = dd * oms;
      }
      const float gm = g * m[j];
      if constexpr (HI) {
        float ei;
        const float iota = sigmoid_e(iv[j], c.ib, ei);
        dx[j] = gm * iota;
        di[j] = gm * ix[j] * one_minus(iota, ei);
      } else {
        dx[j] = gm;
        di[j] = 0.0f;
      }
      if (j < valid) {
        sum_d += dd;
        sum_r += dr[j];
        sum_i += di[j];
      }
    }
    if (act) {
      store_raw<IO>((T*)p.dx + base + t, valid, dx);
      store_raw<IO>((T*)p.dr + base + t, valid, dr);
      if constexpr (HI) store_raw<IO>((T*)p.di + base + t, valid, di);
      if constexpr (HZ) store_raw<IO>((T*)p.dz + base + t, valid, dz);
    }
  }
  if (p.dh0 && act && part == 0 && lane == 0) p.dh0[row] = G;
  if (!p.sums) return;
  float sums[3] = {wave_sum(sum_d), wave_sum(sum_r), wave_sum(sum_i)};
  if constexpr (KIND == kNormalised) {
    // dl/ddecay / l = sigmoid(decay) / softplus(decay), which nears 1 for very negative
    // decays, where both may underflow to 0
    float e;
    const float v = p.decay[d], sp = softplus_dt(v, 0.0f), sg = sigmoid_e(v, 0.0f, e);
    sums[0] *= sp > 0.0f ? sg / sp : 1.0f;
  }
  if (lane == 63) {
#pragma unroll
    for (int k = 0; k < 3; ++k) s_sum[wave][k] = sums[k];
  }
  __syncthreads();
  if (part == 0 && act && lane < 3) {
    float v = s_sum[wave][lane];
    for (int k = 1; k < W; ++k) v += s_sum[wave + k][lane];
    p.sums[lane * p.rows + row] = v;
  }
}

__global__ __launch_bounds__(256) void glr_reduce_kernel(int64_t batch, int64_t dim, const float* __restrict__ sums,
                                                         float* ddecay, float* dr_bias, float* di_bias) {
  float* out = blockIdx.y == 0 ? ddecay : blockIdx.y == 1 ? dr_bias : di_bias;
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (!out || d >= dim) return;
  const float* in = sums + (int64_t)blockIdx.y * batch * dim + d;
  float v = 0.0f;
  for (int64_t b = 0; b < batch; ++b) v += in[b * dim];
  out[d] = v;
}

template <typename IO, int KIND, bool HI, bool HZ>
struct Bwd {
  static hipError_t go(const GlrArgs& a, hipStream_t s) {
    const int w = waves_for(a.seqlen);
    dim3 g;
    if (!grid_of((a.rows + 4 / w - 1) / (4 / w), &g)) return hipErrorInvalidValue;
    if (w == 1) hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, 1>), g, dim3(256), 0, s, a);
    else if (w == 2) hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, 2>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, 4>), g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
};

}  // namespace
}  // namespace glr

hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s) { return glr::by_form<glr::Bwd>(a, s); }

hipError_t launch_glr_reduce(int64_t batch, int64_t dim, const float* sums, float* ddecay, float* dr_bias,
                             float* di_bias, hipStream_t s) {
  hipLaunchKernelGGL(glr::glr_reduce_kernel, dim3((unsigned)((dim + 255) / 256), 3), dim3(256), 0, s, batch, dim, sums,
                     ddecay, dr_bias, di_bias);
  return hipGetLastError();
}

}  // namespace ssscan
