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

// A lane's operands of one tile.
template <typename IO, int KIND, bool HI, bool HZ>
struct BwdRaw {
  using T = typename IO::T;
  Raw<IO> x, r, i, z, dy;
  // `at`: the wave's first element, the same for all lanes
  __device__ __forceinline__ void load(const GlrArgs& p, int64_t at, int64_t left, int lane) {
    const unsigned off = (unsigned)lane * kV;
    const int valid = lane_tokens(left, lane);
    if (valid >= kV) {
      x = load_whole<IO>((const T*)p.x + at + off);
      r = load_whole<IO>((const T*)p.r + at + off);
      dy = load_whole<IO>((const T*)p.dy + at + off);
      if constexpr (HI) i = load_whole<IO>((const T*)p.i + at + off);
      if constexpr (HZ) z = load_whole<IO>((const T*)p.z + at + off);
    } else {
      x = load_part<IO>((const T*)p.x + at + off, valid);
      r = load_part<IO>((const T*)p.r + at + off, valid, gate_pad<IO, KIND>());
      dy = load_part<IO>((const T*)p.dy + at + off, valid);
      if constexpr (HI) i = load_part<IO>((const T*)p.i + at + off, valid);
      if constexpr (HZ) z = load_part<IO>((const T*)p.z + at + off, valid);
    }
  }
};

// What the lane makes of them before it knows the state and the adjoint that enter:
// what each token's gradients are products with, and the compositions of its
// tokens' forward maps (A, B) and adjoint's maps (Ad, D).
template <typename IO, int KIND, bool HI, bool HZ>
struct BwdTile {
  using T = typename IO::T;
  float a[kV], u[kV];       // the forward's maps
  float w[kV];              // dy silu(z)
  float gx[kV], gi[kV];     // dx and di over g
  // convex:     ddecay = g (h - p1) p2,  dr = ddecay p3, with h the state before
  // normalised: ddecay = g (p1 - p2 h),  dr = ddecay p3  (ddecay over its common factor)
  float p1[kV], p2[kV], p3[kV];
  float gz[kV];             // dz over the state after
  float A, B, Ad, D;

  __device__ __forceinline__ void prepare(const BwdRaw<IO, KIND, HI, HZ>& in, const RowConst& c) {
    A = 1.0f;
    B = D = 0.0f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      float e, m;
      const float s = sigmoid_e(in.r[j], c.rb, e), oms = one_minus(s, e);
      float ix = in.x[j], k = 0.0f, ls = 0.0f;
      if constexpr (KIND == kConvex) {
        a[j] = fmaf(c.c1, s, c.c0);
        m = c.c1 * oms;
      } else {
        a[j] = __builtin_amdgcn_exp2f(c.c0 * s);
        const float w2 = c.c1 * s, q = one_minus_sq(w2, a[j]), root = __builtin_amdgcn_rsqf(fmaxf(q, kTiny));
        m = q * root;
        ls = 0.5f * w2;
        k = ls * root;   // 0 where ls is 0
      }
      gx[j] = m;
      if constexpr (HI) {
        float minus;
        const float iota = sigmoid_both(in.i[j], c.ib, minus);
        ix *= iota;
        gx[j] = m * iota;
        gi[j] = m * ix * minus;
      }
      if constexpr (KIND == kConvex) {
        p1[j] = ix;
        p2[j] = oms;
        p3[j] = c.c1 * s;
      } else {
        p1[j] = a[j] * a[j] * k * ix;   // from the left: a 0 takes k, at rates of 2^126 too, before x could overflow it
        p2[j] = a[j] * ls;
        p3[j] = oms;
      }
      u[j] = m * ix;
      w[j] = in.dy[j];
      if constexpr (HZ) {
        float minus;
        const float zj = in.z[j], sz = sigmoid_both(zj, 0.0f, minus), act = zj * sz;
        w[j] = in.dy[j] * act;
        gz[j] = in.dy[j] * fmaf(act, minus, sz);
      }
      A *= a[j];
      B = fmaf(a[j], B, u[j]);
    }
#pragma unroll
    for (int j = kV - 1; j >= 0; --j) D = a[j] * (w[j] + D);
    Ad = A;
  }

  // Over the wave's lanes: up to the lane's own (A, B), from it on (Ad, D).
  __device__ __forceinline__ void scan(int lane) {
    scan_up(A, B);
    scan_down(Ad, D, lane);
  }
  // The state and the adjoint entering the lane's tokens, from those entering the wave's.
  __device__ __forceinline__ float state(float h) const { return fmaf(shift_up(1.0f, A), h, shift_up(0.0f, B)); }
  __device__ __forceinline__ float adjoint(float g) const { return fmaf(shift_down(1.0f, Ad), g, shift_down(0.0f, D)); }

  // Writes the lane's gradients, the wave's (or the group's) first element being `at`,
  // from the state h and the adjoint g_in entering its tokens, and adds its parts of
  // the sums over tokens.
  __device__ __forceinline__ void finish(const GlrArgs& p, int64_t at, int64_t left, int lane, float h, float g_in,
                                         float& sum_d, float& sum_r, float& sum_i) {
    const unsigned off = (unsigned)lane * kV;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      if constexpr (KIND == kConvex) p1[j] = h - p1[j];
      else p1[j] = fmaf(-p2[j], h, p1[j]);
      h = fmaf(a[j], h, u[j]);
      if constexpr (HZ) gz[j] *= h;
    }
#pragma unroll
    for (int j = kV - 1; j >= 0; --j) {
      const float g = w[j] + g_in;
      g_in = a[j] * g;
      const float dd = KIND == kConvex ? g * p1[j] * p2[j] : g * p1[j];
      sum_d += dd;
      p3[j] *= dd;
      sum_r += p3[j];
      gx[j] *= g;
      if constexpr (HI) {
        gi[j] *= g;
        sum_i += gi[j];
      }
    }
    const int valid = lane_tokens(left, lane);
    if (valid >= kV) {
      if constexpr (HZ) store_whole<IO>((T*)p.dz + at + off, gz);
      store_whole<IO>((T*)p.dx + at + off, gx);
      store_whole<IO>((T*)p.dr + at + off, p3);
      if constexpr (HI) store_whole<IO>((T*)p.di + at + off, gi);
    } else {
      if constexpr (HZ) store_part<IO>((T*)p.dz + at + off, valid, gz);
      store_part<IO>((T*)p.dx + at + off, valid, gx);
      store_part<IO>((T*)p.dr + at + off, valid, p3);
      if constexpr (HI) store_part<IO>((T*)p.di + at + off, valid, gi);
    }
  }
};

// What the sums of `dd` over a row are of ddecay: in the normalised kind dl/ddecay / l =
// sigmoid(decay) / softplus(decay), which nears 1 for very negative decays, where both may underflow
// to 0.
template <int KIND>
__device__ __forceinline__ float decay_factor(const GlrArgs& p, int64_t d) {
  if constexpr (KIND == kConvex) return 1.0f;
  float e;
  const float v = p.decay[d], sp = softplus_dt(v, 0.0f), sg = sigmoid_e(v, 0.0f, e);
  return sp > 0.0f ? sg / sp : 1.0f;
}

// The sums of a row's piece over the waves that share it, to element `at` of each third of p.sums.
template <int KIND, int WAVES>
__device__ __forceinline__ void store_sums(const GlrArgs& p, int64_t d, int64_t at, int64_t third, int wave, int part,
                                           int parts, int lane, bool act, float sum_d, float sum_r, float sum_i) {
  __shared__ float s_sum[WAVES][3];
  const float sums[3] = {wave_sum(sum_d), wave_sum(sum_r), wave_sum(sum_i)};
  if (lane == 63) {
#pragma unroll
    for (int k = 0; k < 3; ++k) s_sum[wave][k] = sums[k];
  }
  __syncthreads();
  if (part == 0 && act && lane < 3) {
    float v = s_sum[wave][lane];
    for (int k = 1; k < parts; ++k) v += s_sum[wave + k][lane];
    p.sums[lane * third + at] = lane == 0 ? v * decay_factor<KIND>(p, d) : v;
  }
}

// W waves share a row, in tiles of W * 512 tokens from its end to its start; workgroups
// of four waves hold 4 / W rows.
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
  const int64_t base = row * p.seqlen;
  const int64_t tiles = (p.seqlen + kTile - 1) / kTile;
  const RowConst c = row_const<KIND>(p, d);
  float G = p.dh_final ? p.dh_final[row] : 0.0f;   // the adjoint entering the tile from its end
  float sum_d = 0.0f, sum_r = 0.0f, sum_i = 0.0f;
  for (int64_t n = tiles - 1; n >= 0; --n) {
    const int64_t t = n * kTile + part * 64 * kV;
    float hc = n > 0 ? p.ckpt[row * glr_tiles(p.seqlen) + n * (kTile / kGlrCkptTokens)] : p.h0 ? p.h0[row] : 0.0f;
    BwdTile<IO, KIND, HI, HZ> in;
    {
      BwdRaw<IO, KIND, HI, HZ> raw;
      raw.load(p, base + t, p.seqlen - t, lane);
      in.prepare(raw, c);
    }
    in.scan(lane);
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
    in.finish(p, base + t, act ? p.seqlen - t : 0, lane, in.state(h_enter), in.adjoint(g_enter), sum_d, sum_r, sum_i);
  }
  if (p.dh0 && act && part == 0 && lane == 0) p.dh0[row] = G;
  if (p.sums) store_sums<KIND, R * W>(p, d, row, p.rows, wave, part, W, lane, act, sum_d, sum_r, sum_i);
}

// Short rows: S lanes each, so that a wave holds 64 / S.
template <typename IO, int KIND, bool HI, bool HZ>
__global__ __launch_bounds__(256) void glr_bwd_short_kernel(GlrArgs p, int S) {
  const int lane = threadIdx.x & 63, l = threadIdx.x & (S - 1);
  int64_t row = block_index() * (256 / S) + threadIdx.x / S;
  const bool act = row < p.rows;
  row = act ? row : p.rows - 1;   // padding lanes repeat the last row and store nothing
  const int64_t d = row % p.dim, base = row * p.seqlen;
  const RowConst c = row_const<KIND>(p, d);
  const float first = p.h0 ? p.h0[row] : 0.0f, last = p.dh_final ? p.dh_final[row] : 0.0f;
  BwdTile<IO, KIND, HI, HZ> in;
  {
    BwdRaw<IO, KIND, HI, HZ> raw;
    raw.load(p, base, p.seqlen, l);
    in.prepare(raw, c);
  }
  group_scan_up(in.A, in.B, l, S);
  group_scan_down(in.Ad, in.D, l, S, lane);
  const float h = in.state(first), g = in.adjoint(last);
  float sum_d = 0.0f, sum_r = 0.0f, sum_i = 0.0f;
  in.finish(p, base, act ? p.seqlen : 0, l, l == 0 ? first : h, l == S - 1 ? last : g, sum_d, sum_r, sum_i);
  if (act && p.dh0 && l == 0) p.dh0[row] = fmaf(in.Ad, last, in.D);
  if (!p.sums) return;
  sum_d = group_sum(sum_d, S) * decay_factor<KIND>(p, d);
  sum_r = group_sum(sum_r, S);
  sum_i = group_sum(sum_i, S);
  if (act && l == 0) {
    p.sums[row] = sum_d;
    p.sums[p.rows + row] = sum_r;
    p.sums[2 * p.rows + row] = sum_i;
  }
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
  const int64_t base = row * p.seqlen, t = n * kGlrCkptTokens + wave * 64 * kV;
  float h_enter = n > 0 ? p.ckpt[row * tiles + n] : p.h0 ? p.h0[row] : 0.0f;
  BwdTile<IO, KIND, HI, HZ> in;
  {
    BwdRaw<IO, KIND, HI, HZ> raw;
    raw.load(p, base + t, p.seqlen - t, lane);
    in.prepare(raw, c);
  }
  in.scan(lane);
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
  in.finish(p, base + t, p.seqlen - t, lane, in.state(h_enter), in.adjoint(g_enter), sum_d, sum_r, sum_i);
  if (p.sums)
    store_sums<KIND, 4>(p, d, row * tiles + n, p.rows * tiles, wave, wave, 4, lane, true, sum_d, sum_r, sum_i);
}

// Rows of one part each: 32 threads sum a channel's batch rows, every 32nd each, and are
// joined in order.
constexpr int64_t kReduceBlocks = int64_t(1) << 20;   // a grid axis holds fewer than 2^32 threads

__global__ __launch_bounds__(1024) void glr_reduce_kernel(int64_t batch, int64_t dim, const float* __restrict__ sums,
                                                          float* ddecay, float* dr_bias, float* di_bias) {
  __shared__ float s_sum[32][32];
  float* out = blockIdx.y == 0 ? ddecay : blockIdx.y == 1 ? dr_bias : di_bias;
  if (!out) return;
  const int col = threadIdx.x & 31, run = threadIdx.x >> 5;
  for (int64_t first = (int64_t)blockIdx.x * 32; first < dim; first += (int64_t)gridDim.x * 32) {
    const int64_t d = first + col;
    float v = 0.0f;
    if (d < dim) {
      const float* in = sums + (int64_t)blockIdx.y * batch * dim + d;
#pragma unroll 4
      for (int64_t b = run; b < batch; b += 32) v += in[b * dim];
    }
    s_sum[run][col] = v;
    __syncthreads();
    if (run == 0 && d < dim) {
      const int runs = batch < 32 ? (int)batch : 32;
      for (int k = 1; k < runs; ++k) v += s_sum[k][col];
      out[d] = v;
    }
    __syncthreads();
  }
}

// Rows of several parts: a workgroup sums a channel, a thread every 256th part of all its batch rows.
__global__ __launch_bounds__(256) void glr_reduce_parts_kernel(int64_t batch, int64_t dim, int64_t parts,
                                                               const float* __restrict__ sums, float* ddecay,
                                                               float* dr_bias, float* di_bias) {
  __shared__ float s_sum[4];
  float* out = blockIdx.y == 0 ? ddecay : blockIdx.y == 1 ? dr_bias : di_bias;
  if (!out) return;
  const int64_t d = blockIdx.x;
  const float* in = sums + ((int64_t)blockIdx.y * batch * dim + d) * parts;
  float v = 0.0f;
#pragma unroll 4
  for (int64_t e = threadIdx.x; e < batch * parts; e += 256) {
    const int64_t b = e / parts;
    v += in[b * dim * parts + (e - b * parts)];
  }
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 63) s_sum[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) out[d] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

template <typename IO, int KIND, bool HI, bool HZ>
struct Bwd {
  template <int W>
  static hipError_t rows(const GlrArgs& a, hipStream_t s) {
    constexpr int kThreads = W > 4 ? W * 64 : 256, R = W > 4 ? 1 : 4 / W;
    dim3 g;
    if (!grid_of((a.rows + R - 1) / R, &g)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((glr_bwd_kernel<IO, KIND, HI, HZ, W>), g, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  static hipError_t go(const GlrArgs& a, hipStream_t s) {
    if (a.chain) {
      dim3 g;
      if (!grid_of(a.rows * glr_tiles(a.seqlen), &g)) return hipErrorInvalidValue;
      hipLaunchKernelGGL((glr_bwd_split_kernel<IO, KIND, HI, HZ>), g, dim3(256), 0, s, a);
      return hipGetLastError();
    }
    if (a.seqlen <= 32 * kV) {
      const int S = group_of(a.seqlen);
      dim3 g;
      if (!grid_of((a.rows + 256 / S - 1) / (256 / S), &g)) return hipErrorInvalidValue;
      hipLaunchKernelGGL((glr_bwd_short_kernel<IO, KIND, HI, HZ>), g, dim3(256), 0, s, a, S);
      return hipGetLastError();
    }
    if (a.seqlen <= 64 * kV) return rows<1>(a, s);
    if (a.seqlen <= 128 * kV) return rows<2>(a, s);
    // bf16 rows of many tiles take eight waves.  Whole calls from stored states, four -> eight, normalised
    // with an input gate: 384 rows of 128K tokens 204 -> 180 us, 1536 of 32K 154 -> 145, 2048 of 256K 1573 ->
    // 1514; 384 of 128K convex without gates 149 -> 120, but with both gates 234 -> 257.  In fp32 four are as
    // fast (384 rows of 128K with an input gate 292, with eight 305 us)
    if constexpr (IO::kPerSpan == 8)
      if (a.seqlen >= (1 << 14)) return rows<8>(a, s);
    return rows<4>(a, s);
  }
};

}  // namespace
}  // namespace glr

hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s) { return glr::by_form<glr::Bwd>(a, s); }

hipError_t launch_glr_reduce(int64_t batch, int64_t dim, int64_t parts, const float* sums, float* ddecay,
                             float* dr_bias, float* di_bias, hipStream_t s) {
  if (parts == 1) {
    const int64_t blocks = (dim + 31) / 32;
    const dim3 g((unsigned)(blocks < glr::kReduceBlocks ? blocks : glr::kReduceBlocks), 3);
    hipLaunchKernelGGL(glr::glr_reduce_kernel, g, dim3(1024), 0, s, batch, dim, sums, ddecay, dr_bias, di_bias);
  } else {
    hipLaunchKernelGGL(glr::glr_reduce_parts_kernel, dim3((unsigned)dim, 3), dim3(256), 0, s, batch, dim, parts, sums,
                       ddecay, dr_bias, di_bias);
  }
  return hipGetLastError();
}

}  // namespace ssscan
