// The gated delta rule in chunks of 64 tokens, first step: what a chunk has without its state (gdr_device.h has the layouts).
//
// Within a chunk u_i = beta_i (v_i - 2^gam_i S^T k_i - sum over j < i of 2^(gam_i - gam_j) (k_i.k_j) u_j), S being the
// state before the chunk and gam the sums of log decays: (I + A) U = R with A the strict lower triangle of
// beta_i 2^(gam_i - gam_j) k_i.k_j.  This kernel makes T = (I + A)^-1 and the decays' vectors, a workgroup to each chunk of a
// head.  k.k^T is a matrix product; the inverse is by 16x16 triangles on the diagonal, a lane to a column, and then
// by twice joining neighbours, T21 = -T22 A21 T11, all of it in fp32.
// Sums of log decays are formed in fp64 and kept as two floats: a forgotten state (a decay of -inf, held to -2000 here)
// must not cost the decays behind it their digits.
#include "gdr_device.h"

namespace ssscan {
namespace {

using namespace gdr;

constexpr int kThreads = 256;
constexpr int kPitch = 68;               // floats of a row in LDS

template <typename IO, int KP, bool WHOLE>
__global__ __launch_bounds__(kThreads) void gdr_prep_kernel(GdrArgs a) {
  using T = typename IO::T;
  constexpr int NP = planes_of<IO>(), kSteps = KP / 16, kRuns = KP / 32;
  __shared__ alignas(16) char s_k[NP][2 * kSteps * kBlock];
  __shared__ alignas(16) float s_a[kC][kPitch], s_t[kC][kPitch];
  __shared__ double s_gam[kC];
  __shared__ float s_beta[kC], s_scale[kC], s_max[4][kC], s_col[kC];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t bh = blockIdx.x / a.chunks, chunk = blockIdx.x - bh * a.chunks;
  const int64_t b = bh / a.hv;
  const int h = (int)(bh - b * a.hv), hkey = h / (a.hv / a.hk);
  const int64_t first = chunk * kC;
  const int valid = a.seqlen - first < kC ? (int)(a.seqlen - first) : kC;

  // four lanes to a token, each every fourth run of 8 values
  {
    const int tok = tid >> 2, sub = tid & 3;
    const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + first * a.ks[1] + hkey * a.ks[2];
    const __amdgpu_buffer_rsrc_t kr = chunk_rows<IO>(k, a.ks[1], valid, a.dk);
    Raw8<IO> raw[kRuns];
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
      raw[r] = buf_load8<IO, WHOLE>(kr, tok * (uint32_t)a.ks[1] * sizeof(T), 0, 8 * (sub + 4 * r), a.dk);
    float x[kRuns][8], m = 0.0f;
#pragma unroll
    for (int r = 0; r < kRuns; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[r][j] = raw_value<IO>(raw[r], j);
        m = fmaxf(m, fabsf(x[r][j]));
      }
    m = quad_max(m);
    const float s = row_scale(m);
    if (sub == 0) s_scale[tok] = s;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) store_operand_rows<IO>(s_k[0], NP == 2 ? s_k[NP - 1] : nullptr, tok, sub + 4 * r, kSteps, x[r], s);
  }
  if (tid < kC) {
    const int64_t at = (b * a.seqlen + first + tid) * a.hv + h;
    const float beta = tid < valid ? a.beta[at] : 0.0f;
    float g = tid < valid && a.g ? a.g[at] : 0.0f;
    g = g < -2000.0f ? -2000.0f : g;                       // a NaN stays one
    double gam = (double)g * 1.4426950408889634074;
#pragma unroll
    for (int d = 1; d < kC; d <<= 1) {
      const double o = __shfl_up(gam, d);
      if (lane >= d) gam += o;
    }
    s_gam[tid] = gam;
    s_beta[tid] = beta;
  }
  __syncthreads();

  // A, tile by tile: wave 0 (0, 0), wave 1 (1, 0), wave 2 (1, 1)
  if (wave < 3) {
    const int ti = wave > 0, tj = wave > 1;
    acc16 acc = zero16();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Planes p, q;
      p.hi = *reinterpret_cast<const h8*>(s_k[0] + (ti * kSteps + s) * kBlock + lane * 16);
      q.hi = *reinterpret_cast<const h8*>(s_k[0] + (tj * kSteps + s) * kBlock + lane * 16);
      if constexpr (NP == 2) {
        p.lo = *reinterpret_cast<const h8*>(s_k[1] + (ti * kSteps + s) * kBlock + lane * 16);
        q.lo = *reinterpret_cast<const h8*>(s_k[1] + (tj * kSteps + s) * kBlock + lane * 16);
      }
      acc = mm<NP, NP>(p, q, acc);
    }
    const int j = 32 * tj + (lane & 31);
    const double gj = s_gam[j];
    const float inv_j = 1.0f / s_scale[j];                 // powers of 2
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = 32 * ti + tile_row(r, lane);
      const float d = __builtin_amdgcn_exp2f((float)(s_gam[i] - gj));
      s_a[i][j] = j < i ? s_beta[i] * ((acc[r] * (1.0f / s_scale[i])) * inv_j) * d : 0.0f;
    }
  } else {
    // above the diagonal T stays zero
    for (int e = lane; e < 32 * 32; e += 64) s_t[e >> 5][32 + (e & 31)] = 0.0f;
  }
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
  // columns to [1, 2) or below 1 (the diagonal is 1)
  {
    const int col = tid & 63, part = tid >> 6;
    float m = 0.0f;
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(s_t[16 * part + i][col]));
    s_max[part][col] = m;
  }
  __syncthreads();
  if (tid < kC) {
    const float m = fmaxf(fmaxf(s_max[0][tid], s_max[1][tid]), fmaxf(s_max[2][tid], s_max[3][tid]));
    const float c = pow2(-exponent(m));
    s_col[tid] = c;
    const double gam = s_gam[tid], end = s_gam[kC - 1];
    const float beta = s_beta[tid], s = s_scale[tid], inv_s = 1.0f / s, into = __builtin_amdgcn_exp2f((float)gam);
    const int es = exponent(s);
    int least = es;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_xor(least, d);
      least = o < least ? o : least;
    }
    const float rel = (float)(es - least);
    double low = gam + (double)rel;                        // the smallest gam_j + rel_j up to here
#pragma unroll
    for (int d = 1; d < kC; d <<= 1) {
      const double o = __shfl_up(low, d);
      if (lane >= d) low = o < low ? o : low;
    }
    const double grow = ceil(gam - low);
    const double pi = grow > 0.0 ? grow : 0.0, gi = gam - pi, gj = gam + (double)rel;
    const float hi = (float)gi, hij = (float)gj;
    float* v = a.vecs + ((int64_t)blockIdx.x * kVecs) * kC + tid;
    v[kVecF1 * kC] = beta / c;
    v[kVecF2 * kC] = beta * into / c * inv_s;
    v[kVecEnd * kC] = __builtin_amdgcn_exp2f((float)(end - gam)) * inv_s;
    v[kVecHi * kC] = hi;
    v[kVecLo * kC] = (float)(gi - (double)hi);
    v[kVecHiJ * kC] = hij;
    v[kVecLoJ * kC] = (float)(gj - (double)hij);
    v[kVecRel * kC] = rel;
    v[kVecInto * kC] = into;
    v[kVecS * kC] = s;
    v[kVecGrow * kC] = (float)pi;
  }
  __syncthreads();
  // tiles as operands: slot (tile, step, lane)
  _Float16* out = static_cast<_Float16*>(a.tri) + (int64_t)blockIdx.x * kTHalfs;
  for (int e = tid; e < 3 * 2 * 64; e += kThreads) {
    const int tile = e >> 7, step = (e >> 6) & 1, l = e & 63;
    const int i = 32 * (tile > 0) + (l & 31), j0 = 32 * (tile > 1) + 16 * step + 4 * (l >> 5);
    Planes p;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = j0 + (j & 3) + 8 * (j >> 2);
      const float x = s_t[i][col] * s_col[col];
      p.hi[j] = (_Float16)x;
      p.lo[j] = (_Float16)(x - (float)p.hi[j]);
    }
    *reinterpret_cast<h8*>(out + ((tile * 2 + step) * 2 + 0) * 512 + l * 8) = p.hi;
    *reinterpret_cast<h8*>(out + ((tile * 2 + step) * 2 + 1) * 512 + l * 8) = p.lo;
  }
}

template <typename IO>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.hv * a.chunks));
  return by_keys(a.dk, a.whole, [&](auto kp, auto whole) {
    gdr_prep_kernel<IO, decltype(kp)::value, decltype(whole)::value><<<grid, kThreads, 0, s>>>(a);
  });
}

}  // namespace

size_t gdr_tri_bytes(int64_t batch, int64_t seqlen, int hv) {
  return (size_t)(batch * hv * ((seqlen + kC - 1) / kC)) * kTHalfs * 2;
}

size_t gdr_vecs_bytes(int64_t batch, int64_t seqlen, int hv) {
  return (size_t)(batch * hv * ((seqlen + kC - 1) / kC)) * kVecs * kC * sizeof(float);
}

hipError_t launch_gdr_prep(const GdrArgs& a, hipStream_t s) {
  return a.io == kIoBf16 ? launch<BF16>(a, s) : launch<F32>(a, s);
}

}  // namespace ssscan
