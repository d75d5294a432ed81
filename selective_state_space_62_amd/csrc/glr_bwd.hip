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

// A lane's tokens of one tile: operands, gates, and after load() the compositions
// over the wave's lanes of the forward maps up to its own (A, B) and of the adjoint's
// maps from its own on (Ad, D).
template <typename IO, int KIND, bool HI, bool HZ>
struct BwdTile {
  using T = typename IO::T;
  Raw<IO> x, r, i, z, dy;
  int valid;
  float a[kV], m[kV], ix[kV], w[kV];
  float A, B, Ad, D;

  __device__ __forceinline__ void load(const GlrArgs& p, const RowConst& c, int64_t base, int64_t t, int lane) {
    valid = lane_tokens(p.seqlen, t);
    x = load_raw<IO>((const T*)p.x + base + t, valid);
    r = load_raw<IO>((const T*)p.r + base + t, valid);
    dy = load_raw<IO>((const T*)p.dy + base + t, valid);
    if constexpr (HI) i = load_raw<IO>((const T*)p.i + base + t, valid);
    if constexpr (HZ) z = load_raw<IO>((const T*)p.z + base + t, valid);
    A = 1.0f;
    B = D = 0.0f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      gate<KIND>(r[j], c, a[j], m[j]);
      ix[j] = x[j];
      if constexpr (HI) {
        float e;
        ix[j] *= sigmoid_e(i[j], c.ib, e);
      }
      w[j] = dy[j];
      if constexpr (HZ) w[j] *= silu(z[j]);
      if (j >= valid) {
        a[j] = 1.0f;
        m[j] = 0.0f;
      }
      A *= a[j];
      B = fmaf(a[j], B, m[j] * ix[j]);
    }
#pragma unroll
    for (int j = kV - 1; j >= 0; --j) D = a[j] * (w[j] + D);
    Ad = A;
    scan_up(A, B);
    scan_down(Ad, D, lane);
  }

  // Writes the lane's gradients, from the state and the adjoint entering its wave's
  // tokens, and adds its parts of the sums over tokens.
  __device__ __forceinline__ void finish(const GlrArgs& p, const RowConst& c, int64_t at, bool act, float h_enter,
                                         float g_enter, float& sum_d, float& sum_r, float& sum_i) const {
    float h = fmaf(shift_up(1.0f, A), h_enter, shift_up(0.0f, B));
    float g_in = fmaf(shift_down(1.0f, Ad), g_enter, shift_down(0.0f, D));
    float before[kV], dz[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      before[j] = h;
      h = fmaf(a[j], h, m[j] * ix[j]);
      if constexpr (HZ) {
        float e;
        const float zj = z[j], s = sigmoid_e(zj, 0.0f, e);
        dz[j] = dy[j] * h * (s * fmaf(zj, one_minus(s, e), 1.0f));
      }
    }
    float dx[kV], dr[kV], di[kV];
#pragma unroll
    for (int j = kV - 1; j >= 0; --j) {
      const float g = w[j] + g_in;
      g_in = a[j] * g;
      float e;
      const float s = sigmoid_e(r[j], c.rb, e), oms = one_minus(s, e);
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
        const float iota = sigmoid_e(i[j], c.ib, ei);
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
    if (!act) return;
    store_raw<IO>((T*)p.dx + at, valid, dx);
    store_raw<IO>((T*)p.dr + at, valid, dr);
    if constexpr (HI) store_raw<IO>((T*)p.di + at, valid, di);
    if constexpr (HZ) store_raw<IO>((T*)p.dz + at, valid, dz);
  }
};

// The sums of a row's piece over the waves that share it, to element `at` of each third of p.sums.
template <int KIND, int WAVES>
__device__ __forceinline__ void store_sums(const GlrArgs& p, int64_t d, int64_t at, int64_t third, int wave, int part,
                                           int parts, int lane, bool act, float sum_d, float sum_r, float sum_i) {
  __shared__ float s_sum[WAVES][3];
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
    for (int k = 1; k < parts; ++k) v += s_sum[wave + k][lane];
    p.sums[lane * third + at] = v;
  }
}

template <typename IO, int KIND, bool HI, bool HZ, int W>
__global__ __launch_bounds__(W > 4 ? W * 64 : 256) void glr_bwd_kernel(GlrArgs p) {
  constexpr int R = W > 4 ? 1 : 4 / W;
  constexpr int64_t kTile = W * 64 * kV;
  __shared__ float s_tot[2][R * W][3];
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
    float hc = n > 0 ? p.ckpt[row * glr_tiles(p.seqlen) + n * (kTile / kGlrCkptTokens)] : p.h0 ? p.h0[row] : 0.0f;
    const int64_t t = n * kTile + (part * 64 + lane) * kV;
    BwdTile<IO, KIND, HI, HZ> in;
    in.load(p, c, base, t, lane);
    const float At = lane_value(in.A, 63), Bt = lane_value(in.B, 63), Dt = lane_value(in.D, 0);
    float h_enter = hc, g_enter = G;
    if constexpr (W == 1) {
      G = fmaf(At, G, Dt);
    } else {
      float(&tot)[R * W][3] = s_tot[n & 1];
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
    in.finish(p, c, base + t, act, h_enter, g_enter, sum_d, sum_r, sum_i);
  }
  if (p.dh0 && act && part == 0 && lane == 0) p.dh0[row] = G;
  if (p.sums) store_sums<KIND, R * W>(p, d, row, p.rows, wave, part, W, lane, act, sum_d, sum_r, sum_i);
}

// Split rows: a workgroup takes one tile of 2048 tokens; the adjoint's chain counts
// the tiles from the row's end.
template <typename IO, int KIND, bool HI, bool HZ>
__global__ __launch_bounds__(256) void glr_bwd_split_kernel(GlrArgs p) {
  __shared__ float s_tot[4][3];
  __shared__ float s_enter;
  __shared__ uint32_t s_tile;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tiles = glr_tiles(p.seqlen);
  const int64_t block = block_index();
  if (block >= p.rows * tiles) return;
  const int64_t row = block % p.rows, d = row % p.dim;
  const Chain chain(p, tiles);
  if (threadIdx.x == 0)
    s_tile = __hip_atomic_fetch_add(chain.counter + 2 * row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const RowConst c = row_const<KIND>(p, d);
  const float last = p.dh_final ? p.dh_final[row] : 0.0f;
  __syncthreads();
  const int64_t back = __builtin_amdgcn_readfirstlane(s_tile), n = tiles - 1 - back;
  if (n < 0) return;   // not without a call that shares the workspace
  const int64_t base = row * p.seqlen, t = n * kGlrCkptTokens + (wave * 64 + lane) * kV;
  float h_enter = n > 0 ? p.ckpt[row * tiles + n] : p.h0 ? p.h0[row] : 0.0f;
  BwdTile<IO, KIND, HI, HZ> in;
  in.load(p, c, base, t, lane);
  const float At = lane_value(in.A, 63), Bt = lane_value(in.B, 63), Dt = lane_value(in.D, 0);
  if (lane == 0) {
    s_tot[wave][0] = At;
    s_tot[wave][1] = Bt;
    s_tot[wave][2] = Dt;
  }
  __syncthreads();
  if (wave == 0) {
    float A = 1.0f, D = 0.0f;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
      D = fmaf(s_tot[k][0], D, s_tot[k][2]);
      A *= s_tot[k][0];
    }
    const float g = chain_enter(chain, row, back, tiles, last, A, D, lane);
    if (lane == 0) {
      s_enter = g;
      if (p.dh0 && n == 0) p.dh0[row] = fmaf(A, g, D);
    }
  }
  __syncthreads();
  float g_enter = s_enter;
  for (int k = 3; k > wave; --k) g_enter = fmaf(s_tot[k][0], g_enter, s_tot[k][2]);
  for (int k = 0; k < wave; ++k) h_enter = fmaf(s_tot[k][0], h_enter, s_tot[k][1]);
  float sum_d = 0.0f, sum_r = 0.0f, sum_i = 0.0f;
  in.finish(p, c, base + t, true, h_enter, g_enter, sum_d, sum_r, sum_i);
  if (p.sums)
    store_sums<KIND, 4>(p, d, row * tiles + n, p.rows * tiles, wave, wave, 4, lane, true, sum_d, sum_r, sum_i);
}

// Rows of one part each: a thread sums a channel's batch rows in order.
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

// Rows of several parts: a wave sums a channel, its lanes every 64th part.
__global__ __launch_bounds__(64) void glr_reduce_parts_kernel(int64_t batch, int64_t dim, int64_t parts,
                                                              const float* __restrict__ sums, float* ddecay,
                                                              float* dr_bias, float* di_bias) {
  float* out = blockIdx.y == 0 ? ddecay : blockIdx.y == 1 ? dr_bias : di_bias;
  if (!out) return;
  const int64_t d = blockIdx.x;
  float v = 0.0f;
  for (int64_t b = 0; b < batch; ++b) {
    const float* in = sums + ((int64_t)blockIdx.y * batch * dim + b * dim + d) * parts;
    for (int64_t k = threadIdx.x; k < parts; k += 64) v += in[k];
  }
  v = wave_sum(v);
  if (threadIdx.x == 63) out[d] = v;
}

template <typename IO, int KIND, bool HI, bool HZ>
struct Bwd {
  static hipError_t go(const GlrArgs& a, hipStream_t s) {
    dim3 g;
    if (a.chain) {
      if (!grid_of(a.rows * glr_tiles(a.seqlen), &g)) return hipErrorInvalidValue;
      hipLaunchKernelGGL((glr_bwd_split_kernel<IO, KIND, HI, HZ>), g, dim3(256), 0, s, a);
      return hipGetLastError();
    }
    // bf16 rows of many tiles take eight waves: 384 rows of 128K tokens 251 -> 208 us, 2048 of 256K 1632 ->
    // 1568 us; in fp32 four are as fast (384 rows of 128K 320, with eight 350 us)
    const int w = a.seqlen <= 64 * kV ? 1 : a.seqlen <= 128 * kV ? 2 : a.io == kIoBf16 && a.seqlen >= (1 << 14) ? 8 : 4;
    if (!grid_of(w > 4 ? a.rows : (a.rows + 4 / w - 1) / (4 / w), &g)) return hipErrorInvalidValue;
    if constexpr (IO::kPerSpan == 8) {
      if (w == 8) {
        hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, 8>), g, dim3(512), 0, s, a);
        return hipGetLastError();
      }
    }
    if (w == 1) hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, 1>), g, dim3(256), 0, s, a);
    else if (w == 2) hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, 2>), g, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, 4>), g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
};

}  // namespace
}  // namespace glr

hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s) { return glr::by_form<glr::Bwd>(a, s); }

hipError_t launch_glr_reduce(int64_t batch, int64_t dim, int64_t parts, const float* sums, float* ddecay,
                             float* dr_bias, float* di_bias, hipStream_t s) {
  if (parts == 1) {
    hipLaunchKernelGGL(glr::glr_reduce_kernel, dim3((unsigned)((dim + 255) / 256), 3), dim3(256), 0, s, batch, dim,
                       sums, ddecay, dr_bias, di_bias);
  } else {
    hipLaunchKernelGGL(glr::glr_reduce_parts_kernel, dim3((unsigned)dim, 3), dim3(64), 0, s, batch, dim, parts, sums,
                       ddecay, dr_bias, di_bias);
  }
  return hipGetLastError();
}

}  // namespace ssscan
