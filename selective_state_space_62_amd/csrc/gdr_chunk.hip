// The gated delta rule in chunks of 64 tokens, second step: the states in turn, and the outputs (gdr_device.h has the layouts).
//
// With S the state before a chunk, T the inverse that the preparation made, G = 2^gam, P_ij = 2^(gam_i - gam_j) q_i.k_j (j <= i):
//   R = beta (V - G K S),  U = T R,  O = scale (G Q S + P U),  S <- G_C S + K^T (2^(gam_C - gam) U).
// A wave holds 32 columns of the state, a workgroup four waves that share the chunk's tiles through LDS; R, U and
// S stay in registers from one product to the next.  The chunks of a head follow one another, so what counts is how long one
// takes: the next chunk's keys, queries and T are loaded while this one is computed.
#include "gdr_device.h"

namespace ssscan {
namespace {

using namespace gdr;

constexpr int kThreads = 256;
constexpr int kCols = 128;               // of a workgroup

template <typename IO, int KP, bool WHOLE>
__global__ __launch_bounds__(kThreads, IO::kPerSpan == 8 || KP <= 64 ? 2 : 1) void gdr_chunk_kernel(GdrArgs a) {
  using T = typename IO::T;
  // What leads to O alone is rounded to bf16 where the I/O is: there one fp16 plane (2^-12) of S, U and P does.
  constexpr int NP = planes_of<IO>(), NO = NP, kSteps = KP / 16, kTiles = KP / 32, kRuns = KP / 32;
  __shared__ alignas(16) char s_k[NP][2 * kSteps * kBlock], s_q[NP][2 * kSteps * kBlock], s_kt[NP][kTiles * 4 * kBlock];
  __shared__ alignas(16) char s_t[kTBlocks * 1024], s_p[NO][kTBlocks * 512];
  __shared__ alignas(16) float s_vecs[2][kVecs][kC], s_qinv[kC];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / a.hv;
  const int h = (int)(bh - b * a.hv), hkey = h / (a.hv / a.hk);
  const int col0 = blockIdx.y * kCols + 32 * wave;

  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hkey * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hkey * a.ks[2];
  const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[2];

  acc16 st[kTiles];                      // the state is st 2^ce
  int ce = 0;
  {
    const int lane = threadIdx.x & 63, col = col0 + (lane & 31);
    const float* h0 = a.h0 + bh * a.dk * a.dv;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * m + tile_row(r, lane);
        st[m][r] = a.h0 && row < a.dk && col < a.dv ? h0[(uint32_t)(row * a.dv + col)] : 0.0f;
      }
  }

  // What this thread brings of a chunk: 4 tokens by 8 values of k, a quarter of a token's runs of q, its share of T and of
  // the vectors, those straight to LDS.
  const uint32_t krow = (uint32_t)a.ks[1] * sizeof(T), qrow = (uint32_t)a.qs[1] * sizeof(T), vrow = (uint32_t)a.vs[1] * sizeof(T);
  Raw8<IO> rk[4], rq[kRuns];
  float4 rs;
  auto fetch = [&](int64_t chunk) {
    const int tid = anew(threadIdx.x), kg = tid & 15, kc = tid >> 4, qtok = tid >> 2, qsub = tid & 3;
    const int64_t first = chunk * kC, at = bh * a.chunks + chunk;
    const int valid = (int)min(a.seqlen - first, (int64_t)kC);
    const float* vec = a.vecs + at * (kVecs * kC);
    const __amdgpu_buffer_rsrc_t kr = chunk_rows<IO>(k + first * a.ks[1], a.ks[1], valid, a.dk);
    const __amdgpu_buffer_rsrc_t qr = chunk_rows<IO>(q + first * a.qs[1], a.qs[1], valid, a.dk);
#pragma unroll
    for (int t = 0; t < 4; ++t) rk[t] = buf_load8<IO, WHOLE>(kr, 4 * kg * krow, t * here(krow), 8 * kc, a.dk);
    rs = *reinterpret_cast<const float4*>(vec + kVecS * kC + 4 * kg);
#pragma unroll
    for (int r = 0; r < kRuns; ++r) rq[r] = buf_load8<IO, WHOLE>(qr, qtok * qrow, 0, 8 * (qsub + 4 * r), a.dk);
    const char* tri = static_cast<const char*>(a.tri) + at * (kTHalfs * 2) + tid * 16;
#pragma unroll
    for (int i = 0; i < 3; ++i) load_to_lds(tri + 4096 * i, s_t + 4096 * i + wave * 1024);
    if (wave < 3) load_to_lds(reinterpret_cast<const char*>(vec) + tid * 16, reinterpret_cast<char*>(&s_vecs[chunk & 1][0][0]) + wave * 1024);
  };
  // V, as it is turned
  Raw8<IO> rvv[2][2];
  auto fetch_v = [&](int64_t chunk) {
    const int64_t first = chunk * kC;
    const int lane = anew(threadIdx.x & 63), valid = (int)min(a.seqlen - first, (int64_t)kC);
    const __amdgpu_buffer_rsrc_t vr = chunk_rows<IO>(v + first * a.vs[1], a.vs[1], valid, a.dv);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        rvv[i][s] = buf_load8<IO, WHOLE>(vr, (32 * i + (lane & 31)) * vrow, 0, col0 + 16 * (lane >> 5) + 8 * s, a.dv);
  };

  fetch(0);
  for (int64_t chunk = 0; chunk < a.chunks; ++chunk) {
    const int64_t first = chunk * kC;
    const int valid = a.seqlen - first < kC ? (int)(a.seqlen - first) : kC;
    const int tid = anew(threadIdx.x), lane = tid & 63, half = lane >> 5, low = lane & 31;
    const int kg = tid & 15, kc = tid >> 4, qtok = tid >> 2, qsub = tid & 3;
    const float(&s_vec)[kVecs][kC] = s_vecs[chunk & 1];
    __syncthreads();
    if (kc < KP / 8) {
      const float s[4] = {rs.x, rs.y, rs.z, rs.w};
      float x[4][8];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[t][j] = raw_value<IO>(rk[t], j);
        store_operand_rows<IO>(s_k[0], s_k[NP - 1], 4 * kg + t, kc, kSteps, x[t], s[t]);
      }
      // transposed: rows are values of k, tokens 4 kg .. 4 kg + 3 a quarter of step kg / 4
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int off = ((kc >> 2) * 4 + (kg >> 2)) * kBlock + (8 * (kc & 3) + j + 32 * (kg & 1)) * 16 + (kg >> 1 & 1) * 8;
        h4 hi, lo;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          hi[t] = (_Float16)(x[t][j] * s[t]);
          if constexpr (NP == 2) lo[t] = (_Float16)fmaf(x[t][j], s[t], -(float)hi[t]);
        }
        *reinterpret_cast<h4*>(s_kt[0] + off) = hi;
        if constexpr (NP == 2) *reinterpret_cast<h4*>(s_kt[NP - 1] + off) = lo;
      }
    }
    {
      float x[kRuns][8], m = 0.0f;
#pragma unroll
      for (int r = 0; r < kRuns; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[r][j] = raw_value<IO>(rq[r], j);
          m = fmaxf(m, fabsf(x[r][j]));
        }
      const float s = row_scale(quad_max(m));
      if (qsub == 0) s_qinv[qtok] = pow2(-exponent(s));
#pragma unroll
      for (int r = 0; r < kRuns; ++r) store_operand_rows<IO>(s_q[0], s_q[NP - 1], qtok, qsub + 4 * r, kSteps, x[r], s);
    }
    loads_stand();
    __syncthreads();
    fetch_v(chunk);
    // P, a tile to a wave, transposed: a lane has a query i and 16 keys j
    if (wave < 3) {
      const int ti = wave > 0, tj = wave > 1;
      acc16 acc = zero16();
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        acc = mm<NP, NP>(operand<NP>(s_k[0] + (tj * kSteps + s) * kBlock, lane, sizeof(s_k[0])),
                         operand<NP>(s_q[0] + (ti * kSteps + s) * kBlock, lane, sizeof(s_q[0])), acc);
      }
      const int i = 32 * ti + low;
      const float hi = s_vec[kVecHi][i], lo = s_vec[kVecLo][i];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int j = 32 * tj + tile_row(r, lane);
        const float e = (hi - s_vec[kVecHiJ][j]) + (lo - s_vec[kVecLoJ][j]);
        acc[r] = j <= i ? acc[r] * __builtin_amdgcn_exp2f(e) : 0.0f;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const Planes p = split<NO>(acc, s, 1.0f);
        *reinterpret_cast<h8*>(s_p[0] + (wave * 2 + s) * 1024 + lane * 16) = p.hi;
        if constexpr (NO == 2) *reinterpret_cast<h8*>(s_p[NO - 1] + (wave * 2 + s) * 1024 + lane * 16) = p.lo;
      }
    }

    acc16 R[2], O[2], U[2];
    Planes sp[kSteps];
    float mS = 0.0f;
    int er = 0, es = 0;
    {
#pragma unroll
      for (int m = 0; m < kTiles; ++m) mS = max_of(st[m], mS);
      mS = wave_max(mS);
      const Scale cs = scale_of(mS, 100);
      es = cs.e;
      R[0] = R[1] = zero16();
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        sp[s] = split(st[s >> 1], s & 1, cs.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) R[i] = mm<NP, 2>(operand<NP>(s_k[0] + (i * kSteps + s) * kBlock, lane, sizeof(s_k[0])), sp[s], R[i]);
        if (s & 1) step_end();
      }
      const float back = pow2(ce - es);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const acc16 V = turn<IO>(rvv[i], lane);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = 32 * i + tile_row(r, lane);
          R[i][r] = s_vec[kVecF1][row] * V[r] - s_vec[kVecF2][row] * (back * R[i][r]);
        }
      }
    }
    {
      const Scale cr = scale_of(wave_max(max_of(R[1], max_of(R[0], 0.0f))), 100);
      er = cr.e;
      U[0] = U[1] = zero16();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const Planes rp = split(R[s >> 1], s & 1, cr.f);
#pragma unroll
        for (int i = s >> 1; i < 2; ++i) {
          const int blk = (i + (s >> 1)) * 2 + (s & 1);    // tiles (0, 0), (1, 0), (1, 1)
          U[i] = mm<2, 2>(operand<2>(s_t + blk * 2048, lane, 1024), rp, U[i]);
        }
        step_end();
      }
    }
    __syncthreads();                                       // P stands
    {
      if (chunk + 1 < a.chunks) fetch(chunk + 1);          // T has been read
      O[0] = O[1] = zero16();
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
#pragma unroll
        for (int i = 0; i < 2; ++i) O[i] = mm<NO, NP>(sp[s], operand<NP>(s_q[0] + (i * kSteps + s) * kBlock, lane, sizeof(s_q[0])), O[i]);
        if (s & 1) step_end();
      }
      const int lsk = exponent(s_vec[kVecS][0]) - (int)s_vec[kVecRel][0];
      const Scale cu = scale_of(wave_max(max_of(U[1], max_of(U[0], 0.0f))), min(20, 40 - (ce - es + er + lsk)));
      const float join = pow2(ce - es + er + lsk + cu.e);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 32 * i + low;
        const float f = s_vec[kVecInto][tok] * pow2(-(int)s_vec[kVecGrow][tok]) * join;
#pragma unroll
        for (int r = 0; r < 16; ++r) O[i][r] *= f;
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const Planes up = split<NO>(U[s >> 1], s & 1, cu.f);
#pragma unroll
        for (int i = s >> 1; i < 2; ++i)
          O[i] = mm<NO, NO>(up, operand<NO>(s_p[0] + ((i + (s >> 1)) * 2 + (s & 1)) * 1024, lane, sizeof(s_p[0])), O[i]);
        step_end();
      }
      float mE = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int r = 0; r < 16; ++r) U[i][r] *= s_vec[kVecEnd][32 * i + tile_row(r, lane)];
        mE = max_of(U[i], mE);
      }
      const float gC = s_vec[kVecInto][kC - 1], kept = mS * gC;
      const int room = kept > 0.0f ? 60 - exponent(kept) - ce - er : 100;
      const Scale ue = scale_of(wave_max(mE), min(room, 100 - er));
      const float f = gC * pow2(ce + er + ue.e);
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) st[m][r] *= f;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const Planes up = split(U[s >> 1], s & 1, ue.f);
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
          st[m] = mm<NP, 2>(operand<NP>(s_kt[0] + (m * 4 + s) * kBlock, lane, sizeof(s_kt[0])), up, st[m]);
        step_end();
      }
      // O, transposed: a lane has a token and runs of four columns
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 32 * i + low;
        if (tok >= valid) continue;
        const float fo = a.scale * s_qinv[tok] * pow2((int)s_vec[kVecGrow][tok] - (er + cu.e + lsk));
        T* o = static_cast<T*>(a.o) + ((b * a.seqlen + first + tok) * a.hv + h) * a.dv;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = col0 + 8 * g + 4 * half;
          if (a.dv % 4 == 0) {                             // o is 16-byte aligned: runs of four are too
            if (c >= a.dv) continue;
            if constexpr (IO::kPerSpan == 4) {
              *reinterpret_cast<float4*>(o + c) = make_float4(O[i][4 * g] * fo, O[i][4 * g + 1] * fo, O[i][4 * g + 2] * fo, O[i][4 * g + 3] * fo);
            } else {
              *reinterpret_cast<uint2*>(o + c) =
                  make_uint2(pack_bf16x2(O[i][4 * g] * fo, O[i][4 * g + 1] * fo), pack_bf16x2(O[i][4 * g + 2] * fo, O[i][4 * g + 3] * fo));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (c + j < a.dv) store_one<IO>(o, c + j, O[i][4 * g + j] * fo);
          }
        }
      }
      ce = -(er + ue.e);
    }
  }
  const int lane = anew(threadIdx.x & 63), col = col0 + (lane & 31);
  if (a.h_final && col < a.dv) {
    const float f = pow2(ce);
    float* hf = a.h_final + bh * a.dk * a.dv;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * m + tile_row(r, lane);
        if (row < a.dk) hf[(uint32_t)(row * a.dv + col)] = st[m][r] * f;
      }
  }
}

template <typename IO>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.hv), (unsigned)((a.dv + kCols - 1) / kCols));
  return by_keys(a.dk, a.whole, [&](auto kp, auto whole) {
    gdr_chunk_kernel<IO, decltype(kp)::value, decltype(whole)::value><<<grid, kThreads, 0, s>>>(a);
  });
}

}  // namespace

hipError_t launch_gdr_chunk(const GdrArgs& a, hipStream_t s) { return a.io == kIoBf16 ? launch<BF16>(a, s) : launch<F32>(a, s); }

}  // namespace ssscan
