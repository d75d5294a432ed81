// Gated linear recurrence, forward pass and single-token step (gfx950).
//
// h_t = a_t h_(t-1) + u_t composes: tokens s .. t act as one map h -> A h + B.  A
// lane composes its 8 consecutive tokens, the wave scans the 64 lanes' maps with
// DPP, the waves of a row exchange their totals through LDS, and every lane
// replays its tokens from its true entering state.  So each element is read and
// written once, and a row's tokens are consecutive in memory for the wave.
#include "glr_device.h"

namespace ssscan {
namespace glr {
namespace {

// W waves share a row, which is taken in tiles of W * 512 tokens.
template <typename IO, int KIND, bool HI, bool HZ, int W>
__global__ __launch_bounds__(256) void glr_fwd_kernel(GlrArgs p) {
  using T = typename IO::T;
  constexpr int R = 4 / W;
  constexpr int64_t kTile = W * 64 * kV;
  __shared__ float s_tot[2][4][2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % W;
  const int64_t first = block_index() * R;
  if (first >= p.rows) return;
  const bool act = first + wave / W < p.rows;
  const int64_t row = act ? first + wave / W : p.rows - 1;   // a padding wave repeats a row and stores nothing
  const RowConst c = row_const<KIND>(p, row % p.dim);
  const int64_t base = row * p.seqlen;
  const int64_t ncheck = (p.seqlen + kGlrCkptTokens - 1) / kGlrCkptTokens;
  float carry = p.h0 ? p.h0[row] : 0.0f;
  for (int64_t t0 = 0, n = 0; t0 < p.seqlen; t0 += kTile, ++n) {
    if (p.ckpt && act && t0 % kGlrCkptTokens == 0 && part == 0 && lane == 0)
      p.ckpt[row * ncheck + t0 / kGlrCkptTokens] = carry;
    const int64_t t = t0 + (part * 64 + lane) * kV;
    const int valid = (int)(p.seqlen - t < kV ? (p.seqlen - t > 0 ? p.seqlen - t : 0) : kV);
    const Raw<IO> xv = load_raw<IO>((const T*)p.x + base + t, valid);
    const Raw<IO> rv = load_raw<IO>((const T*)p.r + base + t, valid);
    Raw<IO> iv, zv;
    if constexpr (HI) iv = load_raw<IO>((const T*)p.i + base + t, valid);
    if constexpr (HZ) zv = load_raw<IO>((const T*)p.z + base + t, valid);
    float a[kV], u[kV];
    float A = 1.0f, B = 0.0f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      float m;
      gate<KIND>(rv[j], c, a[j], m);
      u[j] = m * xv[j];
      if constexpr (HI) {
        float e;
        u[j] *= sigmoid_e(iv[j], c.ib, e);
      }
      if (j >= valid) {
        a[j] = 1.0f;
        u[j] = 0.0f;
      }
      A *= a[j];
      B = fmaf(a[j], B, u[j]);
    }
    scan_up(A, B);
    float h = fmaf(shift_up(1.0f, A), carry, shift_up(0.0f, B));
    const float At = lane_value(A, 63), Bt = lane_value(B, 63);
    if constexpr (W == 1) {
      carry = fmaf(At, carry, Bt);
    } else {
      float(&tot)[4][2] = s_tot[n & 1];
      if (lane == 0) {
        tot[wave][0] = At;
        tot[wave][1] = Bt;
      }
      __syncthreads();   // the other parity's totals are read before the next barrier only
      float enter = carry;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        if (k == part) enter = carry;
        carry = fmaf(tot[wave - part + k][0], carry, tot[wave - part + k][1]);
      }
      h = fmaf(shift_up(1.0f, A), enter, shift_up(0.0f, B));
    }
    if (p.y) {
      float y[kV];
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        h = fmaf(a[j], h, u[j]);
        y[j] = h;
        if constexpr (HZ) y[j] *= silu(zv[j]);
      }
      if (act) store_raw<IO>((T*)p.y + base + t, valid, y);
    }
  }
  if (p.h_final && act && part == 0 && lane == 0) p.h_final[row] = carry;
}

template <typename IO, int KIND, bool HI, bool HZ>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrArgs p) {
  using T = typename IO::T;
  for (int64_t ch = block_index() * 256 + threadIdx.x; ch < p.rows; ch += (int64_t)gridDim.x * gridDim.y * 256) {
    const RowConst c = row_const<KIND>(p, ch % p.dim);
    float a, m;
    gate<KIND>(load_one<IO>((const T*)p.r, ch), c, a, m);
    float u = m * load_one<IO>((const T*)p.x, ch);
    if constexpr (HI) {
      float e;
      u *= sigmoid_e(load_one<IO>((const T*)p.i, ch), c.ib, e);
    }
    const float h = fmaf(a, p.h0[ch], u);
    p.h_final[ch] = h;
    float y = h;
    if constexpr (HZ) y *= silu(load_one<IO>((const T*)p.z, ch));
    store_one<IO>((T*)p.y, ch, y);
  }
}

template <typename IO, int KIND, bool HI, bool HZ>
struct Fwd {
  static hipError_t go(const GlrArgs& a, hipStream_t s) {
    const int w = waves_for(a.seqlen);
    dim3 g;
    if (!grid_of((a.rows + 4 / w - 1) / (4 / w), &g)) return hipErrorInvalidValue;
    if (w == 1) hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 1>), g, dim3(256), 0, s, a);
    else if (w == 2) hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 2>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 4>), g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
};

template <typename IO, int KIND, bool HI, bool HZ>
struct Step {
  static hipError_t go(const GlrArgs& a, hipStream_t s) {
    dim3 g;
    if (!grid_of((a.rows + 255) / 256, &g)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((glr_step_kernel<IO, KIND, HI, HZ>), g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
};

}  // namespace
}  // namespace glr

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) { return glr::by_form<glr::Fwd>(a, s); }
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t s) { return glr::by_form<glr::Step>(a, s); }

}  // namespace ssscan
