// The gated delta rule backward, in chunks of 64 tokens: the gradients of the states in turn, from the last chunk to the
// first (gdr_device.h has the layouts).
//
// With dS the gradient of the state behind a chunk, D = 2^(gam_C - gam), and T, P, G as in the forward:
//   dU = P^T dO + D K dS,  dR = T^T dU,  dV = beta dR,  dS <- G_C dS + (scale G Q)^T dO - (beta G K)^T dR.
// It is the forward's recurrence with other operands: 32 columns to a wave, everything in registers from one product to the
// next; where there are few heads, in segments as well, with the forward's factors transposed.  dS and dR are stored, transposed by a product with the identity, for the gradients that need no turn.
// 8 x 40 heads of 2048 tokens, 128 by 128, bf16: 640 us, of them about 200 the 1 GB that it writes; the rest, as in the forward, is
// the latency of one product after another.  dO a chunk ahead of its use spills registers: 710.
#include "gdr_device.h"

namespace ssscan {
namespace {

using namespace gdr;

constexpr int kThreads = 256;
constexpr int kCols = 128;               // of a workgroup

// ENDS: nothing but the gradients of the states before segments.
template <typename IO, int KP, bool WHOLE, bool ENDS>
__global__ __launch_bounds__(kThreads, IO::kPerSpan == 8 || KP <= 64 ? 2 : 1) void gdr_chunk_bwd_kernel(GdrArgs a) {
  using T = typename IO::T;
  constexpr int NP = planes_of<IO>(), kSteps = KP / 16, kTiles = KP / 32;
  constexpr int kSide = 2 * kSteps * kBlock, kTurned = kTiles * 4 * kBlock;
  __shared__ alignas(16) char s_k[NP * kSide], s_kt[NP * kTurned], s_qt[NP * kTurned];
  __shared__ alignas(16) char s_t[2 * kTriBytes], s_p[2 * kTriBytes];
  __shared__ alignas(16) float s_vecs[2][kVecs][kC];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t bh = blockIdx.x / a.segments, seg = blockIdx.x - bh * a.segments;
  const int64_t begin = seg * a.per, last = min(begin + a.per, a.chunks) - 1;
  if (ENDS && seg == 0) return;
  const int64_t b = bh / a.hv;
  const int h = (int)(bh - b * a.hv), hkey = h / (a.hv / a.hk);
  const int col0 = blockIdx.y * kCols + 32 * wave;

  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hkey * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hkey * a.ks[2];
  const int64_t ostride = (int64_t)a.hv * a.dv;
  const T* dout = static_cast<const T*>(a.dout) + b * a.seqlen * ostride + (int64_t)h * a.dv;

  T* dv = static_cast<T*>(a.dv_out) + b * a.seqlen * ostride + (int64_t)h * a.dv;

  acc16 st[kTiles];                      // the gradient is st 2^ce
  int ce = 0;
  {
    const int lane = threadIdx.x & 63, col = col0 + (lane & 31);
    const bool first = seg == a.segments - 1 || ENDS;
    const int64_t ld = first ? a.dv : a.ldv;
    const float* from = first ? (seg == a.segments - 1 ? a.dh_final : nullptr) : a.ends;
    if (from) from += first ? bh * a.dk * a.dv : (bh * a.segments + seg + 1) * KP * a.ldv;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * m + tile_row(r, lane);
        st[m][r] = from && row < a.dk && col < a.dv ? from[(uint32_t)(row * ld + col)] : 0.0f;
      }
  }

  // What this thread brings of a chunk: 4 tokens by 8 values of k and of q.
  const uint32_t krow = (uint32_t)a.ks[1] * sizeof(T), qrow = (uint32_t)a.qs[1] * sizeof(T), orow = (uint32_t)ostride * sizeof(T);
  Raw8<IO> rk[4], rq[4];
  float4 rs, rz;
  auto fetch = [&](int64_t chunk) {
    const int tid = anew(threadIdx.x), kg = tid & 15, kc = tid >> 4;
    const int64_t first = chunk * kC;
    const int valid = (int)min(a.seqlen - first, (int64_t)kC);
    const float* vec = a.vecs + (bh * a.chunks + chunk) * (kVecs * kC);
    const __amdgpu_buffer_rsrc_t kr = chunk_rows<IO>(k + first * a.ks[1], a.ks[1], valid, a.dk);
    const __amdgpu_buffer_rsrc_t qr = chunk_rows<IO>(q + first * a.qs[1], a.qs[1], valid, a.dk);
#pragma unroll
    for (int t = 0; t < 4; ++t) rk[t] = buf_load8<IO, WHOLE>(kr, 4 * kg * krow, t * here(krow), 8 * kc, a.dk);
#pragma unroll
    for (int t = 0; t < 4; ++t) rq[t] = buf_load8<IO, WHOLE>(qr, 4 * kg * qrow, t * here(qrow), 8 * kc, a.dk);
    rs = *reinterpret_cast<const float4*>(vec + kVecS * kC + 4 * kg);
    rz = *reinterpret_cast<const float4*>(vec + kVecZ * kC + 4 * kg);
  };
  auto fetch_lds = [&](int64_t chunk) {
    const int off = anew(threadIdx.x) * 16;
    const int64_t at = bh * a.chunks + chunk;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      load_to_lds(static_cast<const char*>(a.tri_t) + at * (2 * kTriBytes) + 4096 * i + off, s_t + 4096 * i + wave * 1024);
      load_to_lds(static_cast<const char*>(a.p) + at * (2 * kTriBytes) + 4096 * i + off, s_p + 4096 * i + wave * 1024);
    }
    if (wave < 3)
      load_to_lds(reinterpret_cast<const char*>(a.vecs) + at * (kVecs * kC * 4) + off,
                  reinterpret_cast<char*>(&s_vecs[chunk & 1][0][0]) + wave * 1024);
  };
  // dO, as it is turned
  Raw8<IO> ro[2][2];
  auto fetch_o = [&](int64_t chunk) {
    const int64_t first = chunk * kC;
    const int lane = anew(threadIdx.x & 63), valid = (int)min(a.seqlen - first, (int64_t)kC);
    const __amdgpu_buffer_rsrc_t rows = chunk_rows<IO>(dout + first * ostride, ostride, valid, a.dv);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        ro[i][s] = buf_load8<IO, WHOLE>(rows, (32 * i + (lane & 31)) * orow, 0, col0 + 16 * (lane >> 5) + 8 * s, a.dv);
  };

  fetch(last);
  fetch_lds(last);
  for (int64_t chunk = last; chunk >= begin; --chunk) {
    const int64_t first = chunk * kC, at = bh * a.chunks + chunk;
    const int valid = (int)min(a.seqlen - first, (int64_t)kC);
    const int tid = anew(threadIdx.x), lane = tid & 63, half = lane >> 5, low = lane & 31;
    const float(&s_vec)[kVecs][kC] = s_vecs[chunk & 1];
    const bool stores = !ENDS && col0 < a.ldv;
    float* const maxima = a.maxima + at * (a.ldv / 32) + col0 / 32;
    fetch_o(chunk);
    __syncthreads();
    {
      const int kg = tid & 15, kc = tid >> 4;
      if (kc < KP / 8) {
        const float s[4] = {rs.x, rs.y, rs.z, rs.w}, z[4] = {rz.x, rz.y, rz.z, rz.w};
        float x[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[t][j] = raw_value<IO>(rk[t], j);
          store_operand_rows<IO>(s_k, s_k + (NP - 1) * kSide, 4 * kg + t, kc, kSteps, x[t], s[t]);
        }
        store_operand_turned<IO>(s_kt, s_kt + (NP - 1) * kTurned, kg, kc, x, s);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[t][j] = raw_value<IO>(rq[t], j);
        store_operand_turned<IO>(s_qt, s_qt + (NP - 1) * kTurned, kg, kc, x, z);
      }
    }
    loads_stand();
    __syncthreads();

    acc16 X[2], D[2], W[2];
    float mS = 0.0f;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) mS = max_of(st[m], mS);
    mS = wave_max(mS);
    const Scale cs = scale_of(mS, kMostE + min(ce, 0));    // (its inverse times 2^ce is a normal number)
    const float back = pow2(ce - cs.e);
    X[0] = X[1] = zero16();
    {
      float* out = a.dstates + at * KP * a.ldv;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        Planes sp[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          sp[s] = split(st[m], s, cs.f);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            X[i] = mm<NP, 2>(operand<NP>(s_k + (i * kSteps + 2 * m + s) * kBlock, lane, kSide), sp[s], X[i]);
        }
        if constexpr (!ENDS) {
          const acc16 t = transposed(sp[0], sp[1], lane);
          if (stores) store_blocks(out, m, col0, a.ldv, lane, t, back);
        }
        step_end();
      }
      if (stores && lane == 0) maxima[kMaxDs * a.max_apart] = mS * pow2(ce);
    }
    D[0] = turn<IO>(ro[0], lane);
    D[1] = turn<IO>(ro[1], lane);
    if (stores) {
      const float m = wave_max(max_of(D[1], max_of(D[0], 0.0f)));
      if (lane == 0) maxima[kMaxDo * a.max_apart] = m;
    }
    // P^T dO: tiles (0, 0), (1, 0), (1, 1) of P are of keys 0, 0, 1
    {
      acc16 y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) y[i][r] = D[i][r] * s_vec[kVecOut][32 * i + tile_row(r, lane)];
      const Scale c = scale_of(wave_max(max_of(y[1], max_of(y[0], 0.0f))), kMostE);
      W[0] = W[1] = zero16();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const Planes p = split(y[s >> 1], s & 1, c.f);
#pragma unroll
        for (int j = 0; j <= s >> 1; ++j)
          W[j] = mm<2, 2>(operand<2>(s_p + ((j + (s >> 1)) * 2 + (s & 1)) * 1024, lane, kTriBytes), p, W[j]);
        step_end();
      }
      const float f = pow2(-c.e);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) W[j][r] = fmaf(W[j][r], f, s_vec[kVecEnd][32 * j + tile_row(r, lane)] * (back * X[j][r]));
    }
    if (chunk > begin) fetch(chunk - 1);
    // dR = T^T dU, over the inverse's columns' scales
    const Scale cu = scale_of(wave_max(max_of(W[1], max_of(W[0], 0.0f))), kMostE);
    X[0] = X[1] = zero16();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const Planes p = split(W[s >> 1], s & 1, cu.f);
#pragma unroll
      for (int j = 0; j <= s >> 1; ++j)
        X[j] = mm<2, 2>(operand<2>(s_t + ((j + (s >> 1)) * 2 + (s & 1)) * 1024, lane, kTriBytes), p, X[j]);
      step_end();
    }
    const float unit = pow2(-cu.e);
    {
      acc16 y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          X[i][r] *= unit;
          y[i][r] = X[i][r] * s_vec[kVecC][32 * i + tile_row(r, lane)];
        }
      const float m = wave_max(max_of(y[1], max_of(y[0], 0.0f)));
      const Scale c = scale_of(m, kMostE);
      if (stores) {
        float* out = a.dr + at * kC * a.ldv;
        const __amdgpu_buffer_rsrc_t rows = chunk_rows<IO>(dv + first * ostride, ostride, valid, a.dv);
        const float f = pow2(-c.e);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tok = 32 * i + low;
          const acc16 t = transposed(split(y[i], 0, c.f), split(y[i], 1, c.f), lane);
          store_blocks(out, i, col0, a.ldv, lane, t, f);
          store_runs<IO, WHOLE>(rows, tok * orow, col0 + 4 * half, a.dv, t, s_vec[kVecF1][tok] / s_vec[kVecC][tok] * f);
        }
        if (lane == 0) maxima[kMaxDr * a.max_apart] = m;
      }
    }
    __syncthreads();                                       // T and P have been read
    if (chunk > begin) fetch_lds(chunk - 1);
    float mE = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * i + tile_row(r, lane);
        X[i][r] *= -s_vec[kVecF2][row];
        D[i][r] *= s_vec[kVecQ][row];
      }
      mE = max_of(D[i], max_of(X[i], mE));
    }
    const float gC = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(s_vec[kVecInto][kC - 1])));
    const int eG = exponent(gC);
    const int room = min(59 - exponent(mS) - eG, kMostE - max(eG, 0)) - ce;
    const Scale ue = scale_of(wave_max(mE), min(room, kMostE));
    const float f = gC * pow2(ce + ue.e);
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) st[m][r] *= f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const Planes xp = split(X[s >> 1], s & 1, ue.f), dp = split(D[s >> 1], s & 1, ue.f);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) {
        st[m] = mm<NP, 2>(operand<NP>(s_kt + (m * 4 + s) * kBlock, lane, kTurned), xp, st[m]);
        st[m] = mm<NP, 2>(operand<NP>(s_qt + (m * 4 + s) * kBlock, lane, kTurned), dp, st[m]);
      }
      step_end();
    }
    ce = -ue.e;
  }
  const int lane = anew(threadIdx.x & 63), col = col0 + (lane & 31);
  const float f = pow2(ce);
  if constexpr (ENDS) {
    float* to = a.ends + (bh * a.segments + seg) * KP * a.ldv;
    if (col < a.ldv) {
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) to[(uint32_t)((32 * m + tile_row(r, lane)) * a.ldv + col)] = st[m][r] * f;
    }
  } else if (a.dh0 && seg == 0 && col < a.dv) {
    float* d = a.dh0 + bh * a.dk * a.dv;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * m + tile_row(r, lane);
        if (row < a.dk) d[(uint32_t)(row * a.dv + col)] = st[m][r] * f;
      }
  }
}

template <typename IO, bool ENDS>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.hv * a.segments), (unsigned)((a.dv + kCols - 1) / kCols));
  return by_keys(a.dk, a.whole, [&](auto kp, auto whole) {
    gdr_chunk_bwd_kernel<IO, decltype(kp)::value, decltype(whole)::value, ENDS><<<grid, kThreads, 0, s>>>(a);
  });
}

template <bool ENDS>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  return a.io == kIoBf16 ? launch<BF16, ENDS>(a, s) : launch<F32, ENDS>(a, s);
}

}  // namespace

hipError_t launch_gdr_chunk_bwd(const GdrArgs& a, hipStream_t s) {
  if (a.segments > 1) {
    hipError_t e = launch<true>(a, s);
    if (e == hipSuccess) e = launch_gdr_join(a, true, s);
    if (e != hipSuccess) return e;
  }
  return launch<false>(a, s);
}

}  // namespace ssscan
