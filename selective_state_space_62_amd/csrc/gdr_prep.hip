// The gated delta rule in chunks of 64 tokens, first step: what a chunk has without its state (gdr_device.h has the layouts).
//
// Within a chunk u_i = beta_i (v_i - 2^gam_i S^T k_i - sum over j < i of 2^(gam_i - gam_j) (k_i.k_j) u_j), S being the
// state before the chunk and gam the sums of log decays: (I + A) U = R with A the strict lower triangle of
// beta_i 2^(gam_i - gam_j) k_i.k_j.  This kernel makes T = (I + A)^-1, P, the lower triangle of 2^(gam_i - gam_j) q_i.k_j, and the
// decays' vectors, a workgroup to each chunk of a head.  k.k^T and q.k^T are matrix products; the inverse is by 16x16
// triangles on the diagonal, a lane to a column, and then by twice joining neighbours, T21 = -T22 A21 T11, in fp32.
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

  // products: tasks 0-2 the tiles of A, 3-5 those of P, two to each of the first two waves; then the vectors by the last wave
  acc16 acc[2] = {zero16(), zero16()};
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int task = wave + 4 * n;
    if (task > 5) break;
    const int tile = task % 3, ti = tile > 0, tj = tile > 1;
    const bool of_p = task > 2, turned = of_p && !BWD;     // P as the forward reads it is made transposed
    const char* pi = s_rows + (of_p ? NP * kSide : 0) + ti * kSteps * kBlock;
    const char* pj = s_rows + tj * kSteps * kBlock;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      acc[n] = mm<NP, NP>(operand<NP>((turned ? pj : pi) + s * kBlock, lane, kSide),
                          operand<NP>((turned ? pi : pj) + s * kBlock, lane, kSide), acc[n]);
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
#pragma unroll
    for (int d = 1; d < kC; d <<= 1) {
      const double o = __shfl_up(gam, d);
      if (lane >= d) gam += o;
    }
    end = __shfl(gam, kC - 1);
    sk = s_scale[0][lane];
    sq = s_scale[1][lane];
    const int es = exponent(sk);
    least = es;
    double low = gam;                                      // the smallest gam_j up to here
#pragma unroll
    for (int d = 1; d < kC; d <<= 1) {
      const int o = __shfl_xor(least, d);
      least = o < least ? o : least;
      const double l = __shfl_up(low, d);
      if (lane >= d) low = l < low ? l : low;
    }
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
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int task = wave + 4 * n;
    if (task > 5) break;
    const int tile = task % 3, ti = tile > 0, tj = tile > 1;
    if (task > 2) {
      const int v = !BWD ? 1 : 2, w = 3 - v;               // the vector of a lane's column, of its 16 rows
      const int c = 32 * (BWD ? tj : ti) + (lane & 31), r0 = 32 * (BWD ? ti : tj);
      const float sign = BWD ? -1.0f : 1.0f, whole = s_whole[v][c], rest = s_rest[v][c];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = r0 + tile_row(r, lane);
        const float d = exp2_of(sign * (whole - s_whole[w][row]), sign * (rest - s_rest[w][row]));
        acc[n][r] = (BWD ? c <= row : row <= c) ? acc[n][r] * d : 0.0f;
      }
      constexpr int NO = BWD ? 2 : NP;
      char* out = static_cast<char*>(a.p) + at * (NO * kTriBytes) + tile * 2048 + lane * 16;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Planes p = split<NO>(acc[n], s, 1.0f);
        *reinterpret_cast<h8*>(out + s * 1024) = p.hi;
        if constexpr (NO == 2) *reinterpret_cast<h8*>(out + kTriBytes + s * 1024) = p.lo;
      }
    } else {
      const int j = 32 * tj + (lane & 31);
      const float whole = s_whole[2][j], rest = s_rest[2][j];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int i = 32 * ti + tile_row(r, lane);
        const float d = exp2_of(s_whole[0][i] - whole, s_rest[0][i] - rest);
        s_a[i][j] = j < i ? s_beta[i] * (acc[n][r] * d) : 0.0f;
      }
    }
  }
  // above the diagonal T stays zero (the rows of k and q have been read)
  for (int e = tid; e < 32 * 32; e += kThreads) s_t[e >> 5][32 + (e & 31)] = 0.0f;
  __syncthreads();

  // 16x16 triangles: lane 16 q + c solves column c of triangle q
  if (wave == 0) {
    const int q = lane >> 4, c = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == c ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) v = fmaf(-s_a[16 * q + i][16 * q + j], x[j], v);
      x[i] = v;
      s_t[16 * q + i][16 * q + c] = v;
    }
    // the upper of the off-diagonal 16x16 blocks inside the 32x32 triangles
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(q & 1)) s_t[16 * q + i][16 * q + 16 + c] = 0.0f;
  }
  __syncthreads();
  // 16 -> 32: both pairs at once, 128 threads to a pair, two elements of a row each
  {
    const int p = tid >> 7, e = tid & 127, i = e >> 3, n = (e & 7) * 2, o = 32 * p;
    float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float l = s_a[o + 16 + i][o + k];
      m0 = fmaf(l, s_t[o + k][o + n], m0);
      m1 = fmaf(l, s_t[o + k][o + n + 1], m1);
    }
    s_a[o + i][o + 16 + n] = m0;                           // above A's diagonal there is room
    s_a[o + i][o + 16 + n + 1] = m1;
    __syncthreads();
    m0 = m1 = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float l = s_t[o + 16 + i][o + 16 + k];
      m0 = fmaf(-l, s_a[o + k][o + 16 + n], m0);
      m1 = fmaf(-l, s_a[o + k][o + 16 + n + 1], m1);
    }
    s_t[o + 16 + i][o + n] = m0;
    s_t[o + 16 + i][o + n + 1] = m1;
    __syncthreads();
  }
  // 32 -> 64: four elements of a row to a thread
  {
    const int i = tid >> 3, n = (tid & 7) * 4;
    float m[4] = {};
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      const float l = s_a[32 + i][k];
      const float4 t = *reinterpret_cast<const float4*>(&s_t[k][n]);
      m[0] = fmaf(l, t.x, m[0]); m[1] = fmaf(l, t.y, m[1]); m[2] = fmaf(l, t.z, m[2]); m[3] = fmaf(l, t.w, m[3]);
    }
    *reinterpret_cast<float4*>(&s_a[i][32 + n]) = make_float4(m[0], m[1], m[2], m[3]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = 0.0f;
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      const float l = -s_t[32 + i][32 + k];
      const float4 t = *reinterpret_cast<const float4*>(&s_a[k][32 + n]);
      m[0] = fmaf(l, t.x, m[0]); m[1] = fmaf(l, t.y, m[1]); m[2] = fmaf(l, t.z, m[2]); m[3] = fmaf(l, t.w, m[3]);
    }
    *reinterpret_cast<float4*>(&s_t[32 + i][n]) = make_float4(m[0], m[1], m[2], m[3]);
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

size_t gdr_p_bytes(int64_t chunk_heads, int io, bool backward) {
  return (size_t)chunk_heads * kTriBytes * (backward || io == kIoF32 ? 2 : 1);
}

size_t gdr_vecs_bytes(int64_t chunk_heads) { return (size_t)chunk_heads * kVecs * kC * sizeof(float); }

hipError_t launch_gdr_prep(const GdrArgs& a, bool backward, hipStream_t s) {
  return a.io == kIoBf16 ? launch<BF16>(a, backward, s) : launch<F32>(a, backward, s);
}

}  // namespace ssscan
