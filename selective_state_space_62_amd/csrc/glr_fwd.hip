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

// A lane's operands of one tile.  `at` is the wave's first element, the same for all
// lanes, so that every access is a scalar base and one 32-bit lane offset.
template <typename IO, int KIND, bool HI, bool HZ>
struct FwdTile {
  Raw<IO> x, r, i, z;
  __device__ __forceinline__ void load(const GlrArgs& p, int64_t at, int64_t left, int lane) {
    using T = typename IO::T;
    const unsigned off = (unsigned)lane * kV;
    const int valid = lane_tokens(left, lane);
    if (valid >= kV) {
      x = load_whole<IO>((const T*)p.x + at + off);
      r = load_whole<IO>((const T*)p.r + at + off);
      if constexpr (HI) i = load_whole<IO>((const T*)p.i + at + off);
      if constexpr (HZ) z = load_whole<IO>((const T*)p.z + at + off);
    } else {
      x = load_part<IO>((const T*)p.x + at + off, valid);
      r = load_part<IO>((const T*)p.r + at + off, valid, gate_pad<IO, KIND>());
      if constexpr (HI) i = load_part<IO>((const T*)p.i + at + off, valid);
      if constexpr (HZ) z = load_part<IO>((const T*)p.z + at + off, valid);
    }
  }
};

// The decays and inputs of a lane's tokens, and their composition.
template <int KIND, bool HI, typename TILE>
__device__ __forceinline__ void lane_maps(const TILE& in, const RowConst& c, float (&a)[kV], float (&u)[kV], float& A,
                                          float& B) {
  A = 1.0f;
  B = 0.0f;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    float m;
    gate<KIND>(in.r[j], c, a[j], m);
    u[j] = m * in.x[j];
    if constexpr (HI) {
      float e;
      u[j] *= sigmoid_e(in.i[j], c.ib, e);
    }
    A *= a[j];
    B = fmaf(a[j], B, u[j]);
  }
}

// The lane's outputs, from the state entering it.
template <typename IO, bool HZ, typename TILE>
__device__ __forceinline__ void replay(const TILE& in, const float (&a)[kV], const float (&u)[kV], float h, int64_t left, int lane,
                                       typename IO::T* __restrict__ out) {
  float y[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    h = fmaf(a[j], h, u[j]);
    y[j] = h;
    if constexpr (HZ) y[j] *= silu(in.z[j]);
  }
  out += (unsigned)lane * kV;
  const int valid = lane_tokens(left, lane);
  if (valid >= kV) store_whole<IO>(out, y);
  else store_part<IO>(out, valid, y);
}

// W waves share a row, which is taken in tiles of W * 512 tokens; workgroups of four
// waves hold 4 / W rows.  With MORE tiles than one, the next one's operands are loaded
// while a tile is worked on (96 fp32 rows of 300001 tokens, a workgroup to each, normalised,
// input gate, 260 -> 190 us); without, the registers for it would only cost waves (2.8B-shaped
// bf16 layer with both gates, one tile to a row, 156 -> 161 us).
template <typename IO, int KIND, bool HI, bool HZ, int W, bool MORE>
__global__ __launch_bounds__(W > 4 ? W * 64 : 256) void glr_fwd_kernel(GlrArgs p) {
  using T = typename IO::T;
  constexpr int R = W > 4 ? 1 : 4 / W;
  constexpr int64_t kTile = W * 64 * kV;
  __shared__ float s_tot[2][R * W][2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % W;
  const int64_t first = block_index() * R;
  if (first >= p.rows) return;
  const bool act = first + wave / W < p.rows;
  const int64_t row = act ? first + wave / W : p.rows - 1;   // a padding wave repeats a row and stores nothing
  const RowConst c = row_const<KIND>(p, row % p.dim);
  const int64_t base = row * p.seqlen;
  const int64_t mine = part * 64 * kV;
  float carry = p.h0 ? p.h0[row] : 0.0f;
  FwdTile<IO, KIND, HI, HZ> next;
  next.load(p, base + mine, p.seqlen - mine, lane);
  for (int64_t t0 = 0, n = 0; MORE ? t0 < p.seqlen : n == 0; t0 += kTile, ++n) {
    const FwdTile<IO, KIND, HI, HZ> in = next;
    const int64_t t = t0 + mine;
    if constexpr (MORE)
      if (t0 + kTile < p.seqlen) next.load(p, base + t + kTile, p.seqlen - t - kTile, lane);
    float a[kV], u[kV], A, B;
    lane_maps<KIND, HI>(in, c, a, u, A, B);
    scan_up(A, B);
    const float At = lane_value(A, 63), Bt = lane_value(B, 63);
    float enter = carry;   // the state entering the wave's tokens
    if constexpr (W == 1) {
      carry = fmaf(At, carry, Bt);
    } else {
      float(&tot)[R * W][2] = s_tot[n & 1];
      if (lane == 0) {
        tot[wave][0] = At;
        tot[wave][1] = Bt;
      }
      __syncthreads();   // the other parity's totals are read before the next barrier only
#pragma unroll
      for (int k = 0; k < W; ++k) {
        if (k == part) enter = carry;
        carry = fmaf(tot[wave - part + k][0], carry, tot[wave - part + k][1]);
      }
    }
    if (p.ckpt && act && lane == 0 && t % kGlrCkptTokens == 0 && t < p.seqlen)
      p.ckpt[row * glr_tiles(p.seqlen) + t / kGlrCkptTokens] = enter;
    const float h = fmaf(shift_up(1.0f, A), enter, shift_up(0.0f, B));
    if (p.y && act) replay<IO, HZ>(in, a, u, h, p.seqlen - t, lane, (T*)p.y + (base + t));
  }
  if (p.h_final && act && part == 0 && lane == 0) p.h_final[row] = carry;
}

// Short rows: S lanes each, so that a wave holds 64 / S.
template <typename IO, int KIND, bool HI, bool HZ>
__global__ __launch_bounds__(256) void glr_fwd_short_kernel(GlrArgs p, int S) {
  using T = typename IO::T;
  const int l = threadIdx.x & (S - 1);
  int64_t row = block_index() * (256 / S) + threadIdx.x / S;
  const bool act = row < p.rows;
  row = act ? row : p.rows - 1;   // padding lanes repeat the last row and store nothing
  const RowConst c = row_const<KIND>(p, row % p.dim);
  const float first = p.h0 ? p.h0[row] : 0.0f;
  const int64_t base = row * p.seqlen;
  FwdTile<IO, KIND, HI, HZ> in;
  in.load(p, base, p.seqlen, l);
  float a[kV], u[kV], A, B;
  lane_maps<KIND, HI>(in, c, a, u, A, B);
  group_scan_up(A, B, l, S);
  const float Ab = shift_up(1.0f, A), Bb = shift_up(0.0f, B);
  const float h = l == 0 ? first : fmaf(Ab, first, Bb);
  if (p.y) replay<IO, HZ>(in, a, u, h, act ? p.seqlen : 0, l, (T*)p.y + base);
  if (act && p.ckpt && l == 0) p.ckpt[row] = first;
  if (act && p.h_final && l == S - 1) p.h_final[row] = fmaf(A, first, B);
}

// Split rows: a workgroup takes SEG pieces of 2048 tokens each, whose loads are in flight together.
// It waits for its ticket, its loads and the tiles before it in turn, so the bytes in flight are the
// rate: 64 bf16 rows of a million tokens without gates, SEG 1, 2, 3, 4: 149, 109, 101, 95 us; 4 of four
// million with both 122, 77, 65, 65; 96 fp32 rows of 300001 with an input gate, convex, 120, 110, 107, 106.
// Rows of fewer pieces, whose tiles all run at once, wait longer for each: 240 bf16 rows of 31949 tokens with
// an input gate 22, 23, 26, 22; 36 of 155719 with both 29, 26, 24, 25 us.
template <typename IO, int KIND, bool HI, bool HZ, int SEG>
__global__ __launch_bounds__(256) void glr_fwd_split_kernel(GlrArgs p) {
  using T = typename IO::T;
  __shared__ float s_tot[SEG * 4][2];
  __shared__ float s_enter;
  __shared__ uint32_t s_tile;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t pieces = glr_tiles(p.seqlen), tiles = (pieces + SEG - 1) / SEG;
  const int64_t block = block_index();
  if (block >= p.rows * tiles) return;
  const int64_t row = block % p.rows;
  const Chain chain(p, tiles);
  if (threadIdx.x == 0)
    s_tile = __hip_atomic_fetch_add(chain.counter + 2 * row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const RowConst c = row_const<KIND>(p, row % p.dim);
  const float first = p.h0 ? p.h0[row] : 0.0f;
  __syncthreads();
  const int64_t n = __builtin_amdgcn_readfirstlane(s_tile);
  if (n >= tiles) return;   // not without a call that shares the workspace
  const int64_t base = row * p.seqlen, t = n * SEG * kGlrCkptTokens + wave * 64 * kV;
  FwdTile<IO, KIND, HI, HZ> in[SEG];
#pragma unroll
  for (int s = 0; s < SEG; ++s) in[s].load(p, base + t + s * kGlrCkptTokens, p.seqlen - t - s * kGlrCkptTokens, lane);
  float a[SEG][kV], u[SEG][kV], A[SEG], B[SEG];
#pragma unroll
  for (int s = 0; s < SEG; ++s) {
    lane_maps<KIND, HI>(in[s], c, a[s], u[s], A[s], B[s]);
    scan_up(A[s], B[s]);
    if (lane == 63) {
      s_tot[s * 4 + wave][0] = A[s];
      s_tot[s * 4 + wave][1] = B[s];
    }
  }
  __syncthreads();
  if (wave == 0) {
    float At = 1.0f, Bt = 0.0f;
#pragma unroll
    for (int k = 0; k < SEG * 4; ++k) {
      Bt = fmaf(s_tot[k][0], Bt, s_tot[k][1]);
      At *= s_tot[k][0];
    }
    const float h = chain_enter(chain, row, n, tiles, first, At, Bt, lane);
    if (lane == 0) {
      s_enter = h;
      if (p.h_final && n == tiles - 1) p.h_final[row] = fmaf(At, h, Bt);
    }
  }
  __syncthreads();
  float enter = s_enter;
#pragma unroll
  for (int s = 0; s < SEG; ++s) {
    if (p.ckpt && threadIdx.x == 0 && n * SEG + s < pieces) p.ckpt[row * pieces + n * SEG + s] = enter;
    float mine = enter;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k == wave) mine = enter;
      enter = fmaf(s_tot[s * 4 + k][0], enter, s_tot[s * 4 + k][1]);
    }
    const float h = fmaf(shift_up(1.0f, A[s]), mine, shift_up(0.0f, B[s]));
    const int64_t at = t + s * kGlrCkptTokens;
    if (p.y) replay<IO, HZ>(in[s], a[s], u[s], h, p.seqlen - at, lane, (T*)p.y + (base + at));
  }
}

// One token.  A lane takes two neighbouring channels of two batch rows, so that it forms
// the channels' constants once and has all its loads in flight together; the last of an odd
// number of channels goes by itself.  256 x 5120 bf16, normalised, both gates: 6.8 us (one channel of one row 8.0, of
// four rows 6.7, four channels of two rows 7.4; a loop over rows, which held the loads back behind the
// constants, 10.7); 4096 x 5120: 68 us, 5.5 TB/s (one channel of four rows 76, four of one row 70).
constexpr int kStepC = 2, kStepB = 2;
static_assert(kGlrStepDim == ((int64_t(1) << 24) - 1) * 64 * kStepC, "64 lanes side by side");

template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Few {
  T v[kStepC];
};

template <typename T, bool WHOLE>
__device__ __forceinline__ Few<T> load_few(const T* __restrict__ p, int valid) {
  if constexpr (WHOLE) return *reinterpret_cast<const Few<T>*>(p);
  Few<T> o = {};
#pragma unroll
  for (int j = 0; j < kStepC; ++j)
    if (j < valid) o.v[j] = p[j];
  return o;
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void store_few(T* __restrict__ p, int valid, const Few<T>& o) {
  if constexpr (WHOLE) {
    *reinterpret_cast<Few<T>*>(p) = o;
    return;
  }
#pragma unroll
  for (int j = 0; j < kStepC; ++j)
    if (j < valid) p[j] = o.v[j];
}

template <typename IO>
__device__ __forceinline__ float value(typename IO::T v) {
  if constexpr (IO::kPerSpan == 4) return v;
  else return bf16_bits_to_float(v);
}

template <typename IO, int KIND, bool HI, bool HZ, bool WHOLE>
__device__ __forceinline__ void step(const GlrArgs& p, int64_t batch, int64_t b, int64_t d, int valid) {
  using T = typename IO::T;
  Few<T> x[kStepB], r[kStepB], i[kStepB], z[kStepB];
  Few<float> h[kStepB];
#pragma unroll
  for (int k = 0; k < kStepB; ++k) {
    const int64_t at = (b + k < batch ? b + k : b) * p.dim + d;
    r[k] = load_few<T, WHOLE>((const T*)p.r + at, valid);
    x[k] = load_few<T, WHOLE>((const T*)p.x + at, valid);
    if constexpr (HI) i[k] = load_few<T, WHOLE>((const T*)p.i + at, valid);
    if constexpr (HZ) z[k] = load_few<T, WHOLE>((const T*)p.z + at, valid);
    h[k] = load_few<float, WHOLE>(p.h0 + at, valid);
  }
  Few<float> rb = {}, ib = {}, dc = {};
  if (p.r_bias) rb = load_few<float, WHOLE>(p.r_bias + d, valid);
  if (p.i_bias) ib = load_few<float, WHOLE>(p.i_bias + d, valid);
  if (p.decay) dc = load_few<float, WHOLE>(p.decay + d, valid);
  RowConst c[kStepC];
#pragma unroll
  for (int j = 0; j < kStepC; ++j) c[j] = make_const<KIND>(rb.v[j], ib.v[j], dc.v[j], p.decay_scale);
#pragma unroll
  for (int k = 0; k < kStepB; ++k) {
    if (b + k >= batch) break;
    const int64_t at = (b + k) * p.dim + d;
    Few<T> y;
#pragma unroll
    for (int j = 0; j < kStepC; ++j) {
      float a, m;
      gate<KIND>(value<IO>(r[k].v[j]), c[j], a, m);
      float u = m * value<IO>(x[k].v[j]);
      if constexpr (HI) {
        float e;
        u *= sigmoid_e(value<IO>(i[k].v[j]), c[j].ib, e);
      }
      h[k].v[j] = fmaf(a, h[k].v[j], u);
      float o = h[k].v[j];
      if constexpr (HZ) o *= silu(value<IO>(z[k].v[j]));
      if constexpr (IO::kPerSpan == 4) y.v[j] = o;
      else y.v[j] = (uint16_t)float_to_bf16_bits(o);
    }
    store_few<float, WHOLE>(p.h_final + at, valid, h[k]);
    store_few<T, WHOLE>((T*)p.y + at, valid, y);
  }
}

template <typename IO, int KIND, bool HI, bool HZ>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrArgs p, int64_t batch) {
  const int64_t d = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * kStepC;
  const int64_t b = (((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 4 + (threadIdx.x >> 6)) * kStepB;
  if (d >= p.dim || b >= batch) return;
  if (p.dim - d >= kStepC) step<IO, KIND, HI, HZ, true>(p, batch, b, d, kStepC);
  else step<IO, KIND, HI, HZ, false>(p, batch, b, d, (int)(p.dim - d));
}

// A row's waves.  Rows of up to 512 or 1024 tokens fit one or two.  bf16 rows of many
// tiles take eight or sixteen: a tile of four waves is 4 KB of each tensor, which the loads of one
// tile ahead do not keep the memory busy with.  Whole calls of four, eight and sixteen, normalised with an
// input gate: 384 rows of 128K tokens 117, 112, 114 us, 1536 of 32K 86, 86, 92, 2048 of 256K 883, 876, 833;
// 384 of 128K with both gates 129, 118, 122, convex without 76, 64, 67.  In fp32 four are as fast (384 rows
// of 128K with an input gate 165, 169, 178).
int waves_for(const GlrArgs& a) {
  if (a.seqlen <= 128 * kV) return a.seqlen <= 64 * kV ? 1 : 2;
  if (a.io != kIoBf16 || a.seqlen < (1 << 14)) return 4;
  return a.seqlen < (1 << 17) ? 8 : 16;
}

template <typename IO, int KIND, bool HI, bool HZ>
struct Fwd {
  template <int SEG>
  static hipError_t split(const GlrArgs& a, hipStream_t s) {
    dim3 g;
    if (!grid_of(a.rows * ((glr_tiles(a.seqlen) + SEG - 1) / SEG), &g)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((glr_fwd_split_kernel<IO, KIND, HI, HZ, SEG>), g, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  static hipError_t go(const GlrArgs& a, hipStream_t s) {
    if (a.chain) {
      const int64_t pieces = glr_tiles(a.seqlen);   // figures: the kernel's comment
      return pieces >= 128 ? split<4>(a, s) : pieces >= 64 ? split<2>(a, s) : split<1>(a, s);
    }
    dim3 g;
    if (a.seqlen <= 32 * kV) {
      const int S = group_of(a.seqlen);
      if (!grid_of((a.rows + 256 / S - 1) / (256 / S), &g)) return hipErrorInvalidValue;
      hipLaunchKernelGGL((glr_fwd_short_kernel<IO, KIND, HI, HZ>), g, dim3(256), 0, s, a, S);
      return hipGetLastError();
    }
    const int w = waves_for(a);
    if (!grid_of(w > 4 ? a.rows : (a.rows + 4 / w - 1) / (4 / w), &g)) return hipErrorInvalidValue;
    const bool more = a.seqlen > w * 64 * kV;
    if (w == 1) hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 1, false>), g, dim3(256), 0, s, a);
    else if (w == 2) hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 2, false>), g, dim3(256), 0, s, a);
    else if (!more) hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 4, false>), g, dim3(256), 0, s, a);
    else if (w == 4) hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 4, true>), g, dim3(256), 0, s, a);
    else if constexpr (IO::kPerSpan == 8) {
      if (w == 8) hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 8, true>), g, dim3(512), 0, s, a);
      else hipLaunchKernelGGL((glr_fwd_kernel<IO, KIND, HI, HZ, 16, true>), g, dim3(1024), 0, s, a);
    }
    return hipGetLastError();
  }
};

template <typename IO, int KIND, bool HI, bool HZ>
struct Step {
  static hipError_t go(const GlrArgs& a, hipStream_t s) {
    const int64_t batch = a.rows / a.dim, x = (a.dim + 64 * kStepC - 1) / (64 * kStepC);
    const int64_t groups = (batch + 4 * kStepB - 1) / (4 * kStepB);
    const int64_t y = groups < 65535 ? groups : 65535, z = (groups + y - 1) / y;
    if (a.dim > kGlrStepDim || z > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((glr_step_kernel<IO, KIND, HI, HZ>), dim3((unsigned)x, (unsigned)y, (unsigned)z), dim3(256), 0, s,
                       a, batch);
    return hipGetLastError();
  }
};

}  // namespace
}  // namespace glr

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) { return glr::by_form<glr::Fwd>(a, s); }
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t s) { return glr::by_form<glr::Step>(a, s); }

}  // namespace ssscan
