// The gated delta rule in chunks of 64 tokens, first step: what a chunk has without its state (gdr_device.h has the layouts).
//
// Within a chunk u_i = beta_i (v_i - 2^gam_i S^T k_i - sum over j < i of 2^(gam_i - gam_j) (k_i.k_j) u_j), S being the
// state before the chunk and gam the sums of log decays: (I + A) U = R with A the strict lower triangle of
// beta_i 2^(gam_i - gam_j) k_i.k_j.  This kernel makes T = (I + A)^-1, P, the lower triangle of 2^(gam_i - gam_j) q_i.k_j, and the
// decays' vectors, a workgroup to each chunk of a head.  k.k^T and q.k^T are matrix products; the inverse is by 16x16
// triangles on the diagonal, a lane to a column, and then by twice joining neighbours, T21 = -T22 A21 T11, in fp32: a product's
// result is the next one's operand as it stands.  P's exponentials and stores run beside the triangles' chain.
// The workgroups' chains bound it, not memory (0.32 GB of T, P and vectors, 60 us as a copy): 8 x 40 heads of 2048 tokens by 128 keys
// in bf16 take 163 us (two workgroups on a CU), 222 before the joins were matrix products, the gates' sums went over lanes by DPP and
// P left the chain; with T transposed for the backward 221.
// (A, T and P are formed balanced by the growth p; gdr_device.h says how.)
// Sums of log decays are formed in fp64 and kept as a whole number and the rest: a forgotten state (a decay of -inf, held to -2000
// here) must not cost the decays behind it their digits.
#include "gdr_device.h"

namespace ssscan {
namespace {

using namespace gdr;

constexpr int kThreads = 256;
constexpr int kPitch = 68;               // floats of a row in LDS

// A sum of log decays as a whole number and the rest, at most 1/2.
struct Two {
  float whole, rest;
};

__device__ __forceinline__ Two two(double v) {
  const double w = __builtin_rint(v);
  return {(float)w, (float)(v - w)};
}

__device__ __forceinline__ float exp2_wide(double v) {
  const Two t = two(v);
  return exp2_of(t.whole, t.rest);
}

// Running sums or minima over the wave's lanes: shifts within rows of 16, then the last lane of a row to the rows behind it.
// These moves cost a few cycles each where a shuffle through LDS costs about a hundred.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double from, double none) {
  const int lo = __builtin_amdgcn_update_dpp(__double2loint(none), __double2loint(from), CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(__double2hiint(none), __double2hiint(from), CTRL, ROWS, 0xf, false);
  return __hiloint2double(hi, lo);
}

template <typename Op>
__device__ __forceinline__ double running(double v, double none, Op op) {
  v = op(v, moved<0x111, 0xf>(v, none));
  v = op(v, moved<0x112, 0xf>(v, none));
  v = op(v, moved<0x114, 0xf>(v, none));
  v = op(v, moved<0x118, 0xf>(v, none));
  v = op(v, moved<0x142, 0xa>(v, none));
  return op(v, moved<0x143, 0xc>(v, none));
}

__device__ __forceinline__ double last_of(double v) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), kC - 1), __builtin_amdgcn_readlane(__double2loint(v), kC - 1));
}

template <typename IO, int KP, bool WHOLE, bool BWD>
__global__ __launch_bounds__(kThreads) void gdr_prep_kernel(GdrArgs a) {
  using T = typename IO::T;
  constexpr int NP = planes_of<IO>(), kSteps = KP / 16, kRuns = KP / 32;
  constexpr int kSide = 2 * kSteps * kBlock, kRows = 2 * NP * kSide, kTile = kC * kPitch * 4;
  __shared__ alignas(16) char s_rows[kRows > kTile ? kRows : kTile];      // rows of k, of q; then T
  __shared__ alignas(16) float s_a[kC][kPitch];
  __shared__ alignas(16) float s_whole[3][kC], s_rest[3][kC], s_beta[kC];      // of A's row, of P's row, of a column
  __shared__ float s_scale[2][kC], s_max[4][kC], s_col[kC];
  float(&s_t)[kC][kPitch] = *reinterpret_cast<float(*)[kC][kPitch]>(s_rows);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t bh = blockIdx.x / a.chunks, chunk = blockIdx.x - bh * a.chunks;
  const int64_t b = bh / a.hv;
  const int h = (int)(bh - b * a.hv), hkey = h / (a.hv / a.hk);
  const int64_t first = chunk * kC;
  const int valid = a.seqlen - first < kC ? (int)(a.seqlen - first) : kC;

  // four lanes to a token, each every fourth run of 8 values; k, then q
  {
    const int tok = tid >> 2, sub = tid & 3;
    Raw8<IO> raw[2][kRuns];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int64_t* st = n ? a.qs : a.ks;
      const T* base = static_cast<const T*>(n ? a.q : a.k) + b * st[0] + first * st[1] + hkey * st[2];
      const __amdgpu_buffer_rsrc_t rows = chunk_rows<IO>(base, st[1], valid, a.dk);
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
        raw[n][r] = buf_load8<IO, WHOLE>(rows, tok * (uint32_t)st[1] * sizeof(T), 0, 8 * (sub + 4 * r), a.dk);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float x[kRuns][8], m = 0.0f;
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[r][j] = raw_value<IO>(raw[n][r], j);
          m = fmaxf(m, fabsf(x[r][j]));
        }
      const float s = row_scale(quad_max(m));
      if (sub == 0) s_scale[n][tok] = s;
      char* rows = s_rows + n * NP * kSide;
#pragma unroll
      for (int r = 0; r < kRuns; ++r) store_operand_rows<IO>(rows, rows + (NP - 1) * kSide, tok, sub + 4 * r, kSteps, x[r], s);
    }
  }
  __syncthreads();

  // products: waves 0-2 a tile of A each, waves 1-3 one of P
  const bool of_a = wave < 3, of_p = wave > 0;
  const int ta = wave, tp = wave - 1;
  acc16 A = zero16(), P = zero16();
  {
    const char* ai = s_rows + (ta > 0) * kSteps * kBlock;
    const char* aj = s_rows + (ta > 1) * kSteps * kBlock;
    const char* pi = s_rows + NP * kSide + (tp > 0) * kSteps * kBlock;
    const char* pj = s_rows + (tp > 1) * kSteps * kBlock;
    if (of_a) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        A = mm<NP, NP>(operand<NP>(ai + s * kBlock, lane, kSide), operand<NP>(aj + s * kBlock, lane, kSide), A);
    }
    if (of_p) {                                            // as the forward reads it, P is made transposed
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        P = mm<NP, NP>(operand<NP>((BWD ? pi : pj) + s * kBlock, lane, kSide), operand<NP>((BWD ? pj : pi) + s * kBlock, lane, kSide), P);
    }
  }
  double gam = 0.0, end = 0.0, bal = 0.0;
  float beta = 0.0f, into = 0.0f, sk = 1.0f, sq = 1.0f, grow = 0.0f;
  int least = 0;
  if (wave == 3) {
    const int64_t at = (b * a.seqlen + first + lane) * a.hv + h;
    beta = lane < valid ? a.beta[at] : 0.0f;
    float g = lane < valid && a.g ? a.g[at] : 0.0f;
    g = g < -2000.0f ? -2000.0f : g;                       // a NaN stays one
    gam = (double)g * 1.4426950408889634074;
    gam = running(gam, 0.0, [](double x, double o) { return x + o; });
    end = last_of(gam);
    sk = s_scale[0][lane];
    sq = s_scale[1][lane];
    const int es = exponent(sk);
    const auto less = [](double x, double o) { return o < x ? o : x; };
    const double low = running(gam, HUGE_VAL, less);       // the smallest gam_j up to here
    least = (int)last_of(running((double)es, HUGE_VAL, less));
    least = least == kZeroRow ? 0 : least;
    const double p = ceil(gam - low) - floor(fmin(fmax(-0.5 * low, 0.0), 16.0));
    grow = (float)p;
    bal = gam - p;
    const Two ri = two(bal - (double)es), pi = two(bal + (double)(least - kPShift)), cj = two(bal + (double)es);
    s_whole[0][lane] = ri.whole; s_rest[0][lane] = ri.rest;
    s_whole[1][lane] = pi.whole; s_rest[1][lane] = pi.rest;
    s_whole[2][lane] = cj.whole; s_rest[2][lane] = cj.rest;
    s_beta[lane] = beta;
    into = exp2_wide(gam);
  }
  __syncthreads();
  const int64_t at = blockIdx.x;
  if (of_a) {
    const int i0 = 32 * (ta > 0), j = 32 * (ta > 1) + (lane & 31);
    const float whole = s_whole[2][j], rest = s_rest[2][j];
    const acc16 w = rows_of(s_whole[0] + i0, lane), v = rows_of(s_rest[0] + i0, lane), f = rows_of(s_beta + i0, lane);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = i0 + tile_row(r, lane);
      const float x = f[r] * (A[r] * exp2_of(w[r] - whole, v[r] - rest));
      s_a[i][j] = j < i ? x : 0.0f;
    }
  }
  // above the diagonal T stays zero (the rows of k and q have been read)
  for (int e = tid; e < 32 * 32; e += kThreads) s_t[e >> 5][32 + (e & 31)] = 0.0f;
  __syncthreads();

  // P, while the first wave solves the triangles
  if (of_p) {
    const int i0 = 32 * (tp > 0), j0 = 32 * (tp > 1), c = (BWD ? j0 : i0) + (lane & 31), r0 = BWD ? i0 : j0;
    const float whole = s_whole[BWD ? 2 : 1][c], rest = s_rest[BWD ? 2 : 1][c], sign = BWD ? 1.0f : -1.0f;
    const acc16 w = rows_of(s_whole[BWD ? 1 : 2] + r0, lane), v = rows_of(s_rest[BWD ? 1 : 2] + r0, lane);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = r0 + tile_row(r, lane);
      const float x = held(P[r] * exp2_of(sign * (w[r] - whole), sign * (v[r] - rest)));
      P[r] = (BWD ? c <= row : row <= c) ? x : 0.0f;
    }
    char* out = static_cast<char*>(a.p) + at * (2 * kTriBytes) + tp * 2048 + lane * 16;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Planes p = split(P, s, 1.0f);
      *reinterpret_cast<h8*>(out + s * 1024) = p.hi;
      *reinterpret_cast<h8*>(out + kTriBytes + s * 1024) = p.lo;
    }
  }
  // 16x16 triangles: lane 16 q + c solves column c of triangle q
  if (wave == 0) {
    const int q = lane >> 4, c = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      float v[2] = {x[i], 0.0f};                           // two sums: a row waits half as long for the one before
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const f4 l = *reinterpret_cast<const f4*>(&s_a[16 * q + i][16 * q + j]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (j + k < i) v[k & 1] = fmaf(-l[k], x[j + k], v[k & 1]);
      }
      x[i] = v[0] + v[1];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s_t[16 * q + i][16 * q + c] = x[i];
    // the upper of the off-diagonal 16x16 blocks inside the 32x32 triangles
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(q & 1)) s_t[16 * q + i][16 * q + 16 + c] = 0.0f;
  }
  __syncthreads();
  const int n16 = lane & 15, g4 = 4 * (lane >> 4);
  // 16 -> 32: a wave to a pair
  if (wave < 2) {
    const int o = 32 * wave;
    f4 t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = s_t[o + g4 + i][o + n16];
    const f4 none = {};
    const f4 m = mm16(*reinterpret_cast<const f4*>(&s_a[o + 16 + n16][o + g4]), t, none);
    const f4 r = mm16(*reinterpret_cast<const f4*>(&s_t[o + 16 + n16][o + 16 + g4]), m, none);
#pragma unroll
    for (int i = 0; i < 4; ++i) s_t[o + 16 + g4 + i][o + n16] = -r[i];
  }
  __syncthreads();
  // 32 -> 64: a wave to a 16x16 block; A21 T11 is formed for its 16 columns by each wave of two
  {
    const int i0 = 16 * (wave >> 1), n0 = 16 * (wave & 1);
    f4 m[2] = {}, r = {};
#pragma unroll
    for (int k = 0; k < 32; k += 16) {
      f4 t;
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = s_t[k + g4 + i][n0 + n16];
#pragma unroll
      for (int i = 0; i < 2; ++i) m[i] = mm16(*reinterpret_cast<const f4*>(&s_a[32 + 16 * i + n16][k + g4]), t, m[i]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) r = mm16(*reinterpret_cast<const f4*>(&s_t[32 + i0 + n16][32 + 16 * k + g4]), m[k], r);
#pragma unroll
    for (int i = 0; i < 4; ++i) s_t[32 + i0 + g4 + i][n0 + n16] = -r[i];
  }
  __syncthreads();
  // columns to [2^13, 2^14)
  {
    const int col = tid & 63, part = tid >> 6;
    float m = 0.0f;
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(s_t[16 * part + i][col]));
    s_max[part][col] = m;
  }
  __syncthreads();
  if (wave == 3) {
    const float m = fmaxf(fmaxf(s_max[0][lane], s_max[1][lane]), fmaxf(s_max[2][lane], s_max[3][lane]));
    const int ec = exponent(m) - 13, es = exponent(sk), ez = exponent(sq), p = (int)grow;
    s_col[lane] = pow2(-ec);
    const float inv_c = pow2(ec), inv_s = pow2(-es), inv_z = pow2(-ez), scaled = a.scale * inv_z;
    float* v = a.vecs + at * (kVecs * kC) + lane;
    v[kVecF1 * kC] = beta * pow2(-p) * inv_c;
    v[kVecF2 * kC] = beta * exp2_wide(bal) * inv_c * inv_s;
    v[kVecEnd * kC] = exp2_wide(end - bal) * inv_s;
    v[kVecInto * kC] = into;
    v[kVecS * kC] = sk;
    v[kVecZ * kC] = sq;
    v[kVecOut * kC] = scaled * pow2(p + kPShift - least);
    v[kVecQ * kC] = scaled * into;
    if constexpr (BWD) v[kVecGrow * kC] = grow;
    else v[kVecJoin * kC] = exp2_wide(bal) * pow2(least - kPShift);
    v[kVecC * kC] = inv_c;
    const Two b2 = two(bal);
    v[kVecWhole * kC] = b2.whole;
    v[kVecRest * kC] = b2.rest;
  }
  __syncthreads();
  // tiles as operands: slot (tile, step, lane)
  for (int e = tid; e < kTriBlocks * 64 * (BWD ? 2 : 1); e += kThreads) {
    const int turned = e / (kTriBlocks * 64), slot = e % (kTriBlocks * 64);
    const int tile = slot >> 7, step = (slot >> 6) & 1, l = slot & 63, ti = tile > 0, tj = tile > 1;
    const int row = 32 * (turned ? tj : ti) + (l & 31), j0 = 32 * (turned ? ti : tj) + 16 * step + 4 * (l >> 5);
    Planes p;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = j0 + (j & 3) + 8 * (j >> 2);
      const float x = turned ? s_t[k][row] * s_col[row] : s_t[row][k] * s_col[k];
      p.hi[j] = (_Float16)x;
      p.lo[j] = (_Float16)(x - (float)p.hi[j]);
    }
    char* out = static_cast<char*>(turned ? a.tri_t : a.tri) + at * (2 * kTriBytes) + slot * 16;
    *reinterpret_cast<h8*>(out) = p.hi;
    *reinterpret_cast<h8*>(out + kTriBytes) = p.lo;
  }
}

template <typename IO>
hipError_t launch(const GdrArgs& a, bool backward, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.hv * a.chunks));
  return by_keys(a.dk, a.whole, [&](auto kp, auto whole) {
    if (backward) gdr_prep_kernel<IO, decltype(kp)::value, decltype(whole)::value, true><<<grid, kThreads, 0, s>>>(a);
    else gdr_prep_kernel<IO, decltype(kp)::value, decltype(whole)::value, false><<<grid, kThreads, 0, s>>>(a);
  });
}

}  // namespace

size_t gdr_tri_bytes(int64_t chunk_heads) { return (size_t)chunk_heads * 2 * kTriBytes; }

size_t gdr_vecs_bytes(int64_t chunk_heads) { return (size_t)chunk_heads * kVecs * kC * sizeof(float); }

hipError_t launch_gdr_prep(const GdrArgs& a, bool backward, hipStream_t s) {
  return a.io == kIoBf16 ? launch<BF16>(a, backward, s) : launch<F32>(a, backward, s);
}

}  // namespace ssscan
