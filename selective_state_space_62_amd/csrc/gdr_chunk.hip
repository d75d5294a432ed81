// The gated delta rule in chunks of 64 tokens, second step: the states in turn, and the outputs (gdr_device.h has the layouts).
//
// With S the state before a chunk, T and P as the preparation made them, G = 2^gam:
//   R = beta (V - G K S),  U = T R,  O = scale (G Q S + P U),  S <- G_C S + K^T (2^(gam_C - gam) U).
// A wave holds 32 columns of the state, a workgroup four waves that share the chunk's tiles through LDS; R, U and
// S stay in registers from one product to the next.  The chunks of a head follow one another, so what counts is how long one
// takes: the next chunk's tiles are on their way while this one is computed, those that need no conversion straight
// to LDS, and nothing waits for a value that a workgroup could not form beforehand.
// Where there are too few heads for the GPU, the chunks of one go in segments at the same time: the state behind a segment is a
// product with the state before it and a sum, both made first (Of::kEnds) and put together in turn by a small kernel.
// 8 x 40 heads of 2048 tokens, 128 by 128, bf16: 418 us, 13 us to a chunk with two workgroups on a CU; 4 x 40 heads, one on a CU, 8.5.
// Its matrix instructions alone would take 1.8 us of that (4352 cycles of a SIMD), the other vector instructions 2 (about 1200); the
// rest is the latency of seven products in turn.  (S, U and P in one plane for bf16 outputs took 380, but then those are off by 2^-12
// before they are rounded.)  Loads of V a chunk ahead (more registers) made that 397.
// For the backward the same kernel makes S before every chunk and U (transposed by a product with the identity, as
// operands of the gradients) instead of O: 420 us, of them about 200 the 1 GB that it writes.
#include "gdr_device.h"

namespace ssscan {
namespace {

using namespace gdr;

constexpr int kThreads = 256;
constexpr int kCols = 128;               // of a workgroup

enum class Of {
  kOut,        // O and the last state
  kStates,     // the backward's states and U
  kEnds,       // the states behind segments
};

constexpr int per_cu(bool bf16, int keys) { return bf16 || keys <= 64 ? 2 : 1; }

template <typename IO, int KP, bool WHOLE, Of OF>
__global__ __launch_bounds__(kThreads, per_cu(IO::kPerSpan == 8, KP)) void gdr_chunk_kernel(GdrArgs a) {
  using T = typename IO::T;
  constexpr bool OUT = OF == Of::kOut, STATES = OF == Of::kStates, ENDS = OF == Of::kEnds;
  constexpr int NP = planes_of<IO>(), kSteps = KP / 16, kTiles = KP / 32, kRuns = KP / 32;
  // In bf16 the state's part of O is formed beside K S where keys are many: its planes kept till U stands would spill at 128 (8 x 40 heads
  // of 2048: 557 us, 582 behind U).  Behind U it leaves a third workgroup on a CU at 32 keys, and in fp32, with registers to spare, K S is
  // done sooner (1036 us, 1046 beside).
  constexpr bool kEarly = OUT && NP == 1 && KP > 64;
  constexpr int kSide = 2 * kSteps * kBlock, kTurned = kTiles * 4 * kBlock, kP = OUT ? 2 * kTriBytes : 0;
  __shared__ alignas(16) char s_k[NP * kSide], s_kt[NP * kTurned], s_q[OUT ? NP * kSide : 16];
  __shared__ alignas(16) char s_t[2 * kTriBytes], s_p[OUT ? kP : 16];
  __shared__ alignas(16) float s_vecs[2][kVecs][kC];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t bh = blockIdx.x / a.segments, seg = blockIdx.x - bh * a.segments;
  const int64_t b = bh / a.hv, begin = seg * a.per, stop = min(begin + a.per, a.chunks);
  const int h = (int)(bh - b * a.hv), hkey = h / (a.hv / a.hk);
  // behind the columns of the values, the columns of the segment's factor: what the identity becomes without values
  const int blocks = (a.dv + kCols - 1) / kCols;
  const bool moves = ENDS && (int)blockIdx.y >= blocks;
  const int col0 = ((int)blockIdx.y - (moves ? blocks : 0)) * kCols + 32 * wave, ncols = moves ? 0 : a.dv;
  if (ENDS && (seg == a.segments - 1 || (moves && seg == 0))) return;

  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hkey * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hkey * a.ks[2];
  const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[2];

  const int64_t ostride = (int64_t)a.hv * a.dv;
  T* o = static_cast<T*>(a.o) + b * a.seqlen * ostride + (int64_t)h * a.dv;

  acc16 st[kTiles];                      // the state is st 2^ce, a factor st 2^(ce + moved)
  int ce = 0, moved = 0;
  {
    const int lane = threadIdx.x & 63, col = col0 + (lane & 31);
    const bool first = seg == 0 || ENDS;
    const int64_t ld = first ? a.dv : a.ldv;
    const float* from = first ? (seg == 0 ? a.h0 : nullptr) : a.ends;
    if (from) from += first ? bh * a.dk * a.dv : (bh * a.segments + seg - 1) * KP * a.ldv;
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * m + tile_row(r, lane);
        st[m][r] = moves ? (row == col ? 1.0f : 0.0f) : from && row < a.dk && col < a.dv ? from[(uint32_t)(row * ld + col)] : 0.0f;
      }
  }

  // What this thread brings of a chunk: 4 tokens by 8 values of k, a quarter of a token's runs of q.
  const uint32_t krow = (uint32_t)a.ks[1] * sizeof(T), qrow = (uint32_t)a.qs[1] * sizeof(T), vrow = (uint32_t)a.vs[1] * sizeof(T);
  const uint32_t orow = (uint32_t)ostride * sizeof(T);
  Raw8<IO> rk[4], rq[kRuns];
  float4 rs;
  float rz;
  auto fetch = [&](int64_t chunk) {
    const int tid = anew(threadIdx.x), kg = tid & 15, kc = tid >> 4, qtok = tid >> 2, qsub = tid & 3;
    const int64_t first = chunk * kC;
    const int valid = (int)min(a.seqlen - first, (int64_t)kC);
    const float* vec = a.vecs + (bh * a.chunks + chunk) * (kVecs * kC);
    const __amdgpu_buffer_rsrc_t kr = chunk_rows<IO>(k + first * a.ks[1], a.ks[1], valid, a.dk);
#pragma unroll
    for (int t = 0; t < 4; ++t) rk[t] = buf_load8<IO, WHOLE>(kr, 4 * kg * krow, t * here(krow), 8 * kc, a.dk);
    rs = *reinterpret_cast<const float4*>(vec + kVecS * kC + 4 * kg);
    if constexpr (OUT) {
      const __amdgpu_buffer_rsrc_t qr = chunk_rows<IO>(q + first * a.qs[1], a.qs[1], valid, a.dk);
#pragma unroll
      for (int r = 0; r < kRuns; ++r) rq[r] = buf_load8<IO, WHOLE>(qr, qtok * qrow, 0, 8 * (qsub + 4 * r), a.dk);
      rz = vec[kVecZ * kC + qtok];
    }
  };
  // T, P and the vectors, straight to LDS
  auto fetch_lds = [&](int64_t chunk) {
    const int off = anew(threadIdx.x) * 16;
    const int64_t at = bh * a.chunks + chunk;
    const char* tri = static_cast<const char*>(a.tri) + at * (2 * kTriBytes);
#pragma unroll
    for (int i = 0; i < 3; ++i) load_to_lds(tri + 4096 * i + off, s_t + 4096 * i + wave * 1024);
    if constexpr (OUT) {
      const char* p = static_cast<const char*>(a.p) + at * kP;
#pragma unroll
      for (int i = 0; i < kP / 4096; ++i) load_to_lds(p + 4096 * i + off, s_p + 4096 * i + wave * 1024);
    }
    if (wave < 3)
      load_to_lds(reinterpret_cast<const char*>(a.vecs) + at * (kVecs * kC * 4) + off,
                  reinterpret_cast<char*>(&s_vecs[chunk & 1][0][0]) + wave * 1024);
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
        rvv[i][s] = buf_load8<IO, WHOLE>(vr, (32 * i + (lane & 31)) * vrow, 0, col0 + 16 * (lane >> 5) + 8 * s, ncols);
  };

  fetch(begin);
  fetch_lds(begin);
  for (int64_t chunk = begin; chunk < stop; ++chunk) {
    const int64_t first = chunk * kC;
    const int valid = (int)min(a.seqlen - first, (int64_t)kC);
    const int tid = anew(threadIdx.x), lane = tid & 63, half = lane >> 5, low = lane & 31;
    const float(&s_vec)[kVecs][kC] = s_vecs[chunk & 1];
    fetch_v(chunk);
    __syncthreads();
    {
      const int kg = tid & 15, kc = tid >> 4;
      if (kc < KP / 8) {
        const float s[4] = {rs.x, rs.y, rs.z, rs.w};
        float x[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[t][j] = raw_value<IO>(rk[t], j);
          store_operand_rows<IO>(s_k, s_k + (NP - 1) * kSide, 4 * kg + t, kc, kSteps, x[t], s[t]);
        }
        store_operand_turned<IO>(s_kt, s_kt + (NP - 1) * kTurned, kg, kc, x, s);
      }
    }
    if constexpr (OUT) {
      const int qtok = tid >> 2, qsub = tid & 3;
#pragma unroll
      for (int r = 0; r < kRuns; ++r) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = raw_value<IO>(rq[r], j);
        store_operand_rows<IO>(s_q, s_q + (NP - 1) * kSide, qtok, qsub + 4 * r, kSteps, x, rz);
      }
    }
    loads_stand();
    __syncthreads();

    acc16 R[2], O[2], U[2];
    Planes sp[kSteps];
    float mS = 0.0f;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) mS = max_of(st[m], mS);
    mS = wave_max(mS);
    if (moves) {                                           // a factor goes on from 1: without values only its proportions count
      moved += ce;
      ce = 0;
    }
    const Scale cs = scale_of(mS, kMostE + min(ce, 0));    // (its inverse times 2^ce is a normal number)
    const int es = cs.e;
    const float back = pow2(ce - es);
    R[0] = R[1] = zero16();
    O[0] = O[1] = zero16();
    auto through_q = [&](int s) {
#pragma unroll
      for (int i = 0; i < 2; ++i) O[i] = mm<2, NP>(sp[s], operand<NP>(s_q + (i * kSteps + s) * kBlock, lane, kSide), O[i]);
    };
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      sp[s] = split(st[s >> 1], s & 1, cs.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) R[i] = mm<NP, 2>(operand<NP>(s_k + (i * kSteps + s) * kBlock, lane, kSide), sp[s], R[i]);
      if constexpr (kEarly) through_q(s);
      if (s & 1) step_end();
    }
    if constexpr (STATES) {
      // the state before the chunk, its rows behind dk and columns behind dv zeros
      float* out = a.states + (bh * a.chunks + chunk) * KP * a.ldv;
      if (col0 < a.ldv) {
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const acc16 t = transposed(sp[2 * m], sp[2 * m + 1], lane);
          store_blocks(out, m, col0, a.ldv, lane, t, back);
          step_end();
        }
        if (lane == 0) a.maxima[kMaxS * a.max_apart + (bh * a.chunks + chunk) * (a.ldv / 32) + col0 / 32] = mS * pow2(ce);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const acc16 V = turn<IO>(rvv[i], lane);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * i + tile_row(r, lane);
        R[i][r] = s_vec[kVecF1][row] * V[r] - back * (s_vec[kVecF2][row] * R[i][r]);
      }
    }
    const Scale cr = scale_of(wave_max(max_of(R[1], max_of(R[0], 0.0f))), kMostE);
    const int er = cr.e;
    U[0] = U[1] = zero16();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const Planes rp = split(R[s >> 1], s & 1, cr.f);
#pragma unroll
      for (int i = s >> 1; i < 2; ++i)                     // tiles (0, 0), (1, 0), (1, 1)
        U[i] = mm<2, 2>(operand<2>(s_t + ((i + (s >> 1)) * 2 + (s & 1)) * 1024, lane, kTriBytes), rp, U[i]);
      step_end();
    }
    if (chunk + 1 < stop) fetch(chunk + 1);
    const float mU = wave_max(max_of(U[1], max_of(U[0], 0.0f)));
    if constexpr (STATES) {
      const Scale cu = scale_of(mU, min(20, kMostE - er));
      float* out = a.u + (bh * a.chunks + chunk) * kC * a.ldv;
      if (col0 < a.ldv) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const acc16 t = transposed(split(U[i], 0, cu.f), split(U[i], 1, cu.f), lane);
          store_blocks(out, i, col0, a.ldv, lane, t, pow2(-(er + cu.e)));
        }
        if (lane == 0) a.maxima[kMaxU * a.max_apart + (bh * a.chunks + chunk) * (a.ldv / 32) + col0 / 32] = mU * pow2(-er);
      }
    } else if constexpr (OUT) {
      if constexpr (!kEarly) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          through_q(s);
          if (s & 1) step_end();
        }
      }
      // The state's part, below 2^34, is multiplied into U's units, by 2^40 at most, and stays a float: kVecJoin, which is large where keys
      // are next to nothing, rises by less than 2^2 from the first token on, as P does.  (Of a U of zeros the largest scale that is
      // allowed: the state's part is then all there is.)
      const int eJ = exponent(__int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(s_vec[kVecJoin][0]))));
      const Scale cu = scale_of(fmaxf(mU, 0x1p-126f), min(min(20, kMostE - er), min(40, 87 - eJ) - (ce - es + er)));
      const float join = pow2(ce - es + er + cu.e);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = s_vec[kVecJoin][32 * i + low] * join;
#pragma unroll
        for (int r = 0; r < 16; ++r) O[i][r] *= f;
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const Planes up = split(U[s >> 1], s & 1, cu.f);
#pragma unroll
        for (int i = s >> 1; i < 2; ++i)
          O[i] = mm<2, 2>(up, operand<2>(s_p + ((i + (s >> 1)) * 2 + (s & 1)) * 1024, lane, kTriBytes), O[i]);
        step_end();
      }
      // O, transposed: a lane has a token and runs of four columns
      const __amdgpu_buffer_rsrc_t rows = chunk_rows<IO>(o + first * ostride, ostride, valid, a.dv);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 32 * i + low;
        const float by = s_vec[kVecOut][tok];              // not at once with the power, which may be 2^-126
#pragma unroll
        for (int r = 0; r < 16; ++r) O[i][r] *= by;
        store_runs<IO, WHOLE>(rows, tok * orow, col0 + 4 * half, a.dv, O[i], pow2(-(er + cu.e)));
      }
    }
    __syncthreads();                                       // T and P have been read
    if (chunk + 1 < stop) fetch_lds(chunk + 1);
    float mE = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int r = 0; r < 16; ++r) U[i][r] *= s_vec[kVecEnd][32 * i + tile_row(r, lane)];
      mE = max_of(U[i], mE);
    }
    const float gC = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(s_vec[kVecInto][kC - 1])));
    const int eG = exponent(gC);
    // in units in which the kept state stays below 2^61 and its factor a float
    const int room = min(59 - exponent(mS) - eG, kMostE - max(eG, 0)) - ce - er;
    const Scale ue = scale_of(fmaxf(wave_max(mE), 0x1p-126f), min(room, kMostE - er));
    const float f = gC * pow2(ce + er + ue.e);
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) st[m][r] *= f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const Planes up = split(U[s >> 1], s & 1, ue.f);
#pragma unroll
      for (int m = 0; m < kTiles; ++m) st[m] = mm<NP, 2>(operand<NP>(s_kt + (m * 4 + s) * kBlock, lane, kTurned), up, st[m]);
      step_end();
    }
    ce = -(er + ue.e);
  }
  const int lane = anew(threadIdx.x & 63), col = col0 + (lane & 31);
  float f = pow2(ce);
  if constexpr (ENDS) {
    if (moves) {                                           // largest value to [1, 2)
      float m = 0.0f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) m = max_of(st[t], m);
      m = wave_max(m);
      const int e = exponent(m);
      f = pow2(-e);
      // (zeros meet a state times 0, not one times what they have been)
      if (lane == 0) a.moves_e[(bh * a.segments + seg) * 4 + wave] = m == 0.0f ? -(1 << 20) : moved + ce + e;
    }
    const int64_t ld = moves ? KP : a.ldv;
    float* to = (moves ? a.moves : a.ends) + (bh * a.segments + seg) * KP * ld;
    if (col < ld) {
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) to[(uint32_t)((32 * m + tile_row(r, lane)) * ld + col)] = st[m][r] * f;
    }
  } else if (a.h_final && seg == a.segments - 1 && col < a.dv) {
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

// The segments' ends in turn, end <- move * (the end before it) + end from the second on, or, of gradients, with the transposed
// factors from the last but one to the second: a workgroup has 16 columns of a head, a wave 16 rows of every product, in fp32.  The
// next segment's values are on their way meanwhile: 3 us to a segment (16 heads, 128 by 128, 32 segments: 97 us).
template <int KP, bool BWD>
__global__ __launch_bounds__(KP * 4) void gdr_join_ends_kernel(GdrArgs a) {
  constexpr int kPitch = 20;
  __shared__ alignas(16) float s_end[2][KP][kPitch];
  const int lane = threadIdx.x & 63, n = lane & 15, g4 = 4 * (lane >> 4), i0 = 16 * (threadIdx.x >> 6);
  const int64_t col = 16 * (int64_t)blockIdx.y + n;
  float* ends = a.ends + (int64_t)blockIdx.x * a.segments * KP * a.ldv + (i0 + g4) * a.ldv + col;
  const float* moves = a.moves + (int64_t)blockIdx.x * a.segments * KP * KP + (BWD ? g4 * KP + i0 + n : (i0 + n) * KP + g4);
  const int32_t* moves_e = a.moves_e + (int64_t)blockIdx.x * a.segments * 4;
  f4 m[KP / 16], end, acc;
  int e[KP / 32];
  auto fetch = [&](int64_t seg) {
#pragma unroll
    for (int t = 0; t < KP / 16; ++t) {
      if constexpr (BWD) {
#pragma unroll
        for (int r = 0; r < 4; ++r) m[t][r] = moves[seg * KP * KP + (16 * t + r) * KP];
      } else {
        m[t] = *reinterpret_cast<const f4*>(moves + seg * KP * KP + 16 * t);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) end[r] = ends[seg * KP * a.ldv + r * a.ldv];
#pragma unroll
    for (int t = 0; t < KP / 32; ++t) e[t] = moves_e[seg * 4 + (BWD ? i0 / 32 : t)];
  };
  const int64_t step = BWD ? -1 : 1, stop = BWD ? 0 : a.segments - 1;
  int64_t seg = BWD ? a.segments - 1 : 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r] = ends[seg * KP * a.ldv + r * a.ldv];
  seg += step;
  if (seg != stop) fetch(seg);
  for (; seg != stop; seg += step) {
    float(&s)[KP][kPitch] = s_end[seg & 1];
#pragma unroll
    for (int r = 0; r < 4; ++r) s[i0 + g4 + r][n] = acc[r];
    __syncthreads();                                       // the other buffer is written a barrier after its last use
    f4 now[KP / 16], sum = end, out = {};
    int now_e[KP / 32];
#pragma unroll
    for (int t = 0; t < KP / 16; ++t) now[t] = m[t];
#pragma unroll
    for (int t = 0; t < KP / 32; ++t) now_e[t] = e[t];
    if (seg + step != stop) fetch(seg + step);
#pragma unroll
    for (int t = 0; t < KP / 16; ++t) {
      f4 y;
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = BWD ? s[16 * t + g4 + r][n] : ldexpf(s[16 * t + g4 + r][n], now_e[t >> 1]);
      out = mm16(now[t], y, out);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      acc[r] = (BWD ? ldexpf(out[r], now_e[0]) : out[r]) + sum[r];
      ends[seg * KP * a.ldv + r * a.ldv] = acc[r];
    }
  }
}

template <typename IO, Of OF>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  const int blocks = (a.dv + kCols - 1) / kCols + (OF == Of::kEnds ? (a.dk + kCols - 1) / kCols : 0);
  const dim3 grid((unsigned)(a.batch * a.hv * a.segments), (unsigned)blocks);
  return by_keys(a.dk, a.whole, [&](auto kp, auto whole) {
    gdr_chunk_kernel<IO, decltype(kp)::value, decltype(whole)::value, OF><<<grid, kThreads, 0, s>>>(a);
  });
}

template <Of OF>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  return a.io == kIoBf16 ? launch<BF16, OF>(a, s) : launch<F32, OF>(a, s);
}

}  // namespace

hipError_t launch_gdr_join(const GdrArgs& a, bool backward, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.hv), (unsigned)(a.ldv / 16));
  return by_keys(a.dk, true, [&](auto kp, auto) {
    constexpr int KP = decltype(kp)::value;
    if (backward) gdr_join_ends_kernel<KP, true><<<grid, KP * 4, 0, s>>>(a);
    else gdr_join_ends_kernel<KP, false><<<grid, KP * 4, 0, s>>>(a);
  });
}

hipError_t launch_gdr_chunk(const GdrArgs& a, bool states, hipStream_t s) {
  if (a.segments > 1) {
    hipError_t e = launch<Of::kEnds>(a, s);
    if (e == hipSuccess) e = launch_gdr_join(a, false, s);
    if (e != hipSuccess) return e;
  }
  return states ? launch<Of::kStates>(a, s) : launch<Of::kOut>(a, s);
}

int gdr_chunk_room(int io, int dk) { return 256 * per_cu(io == kIoBf16, dk); }

}  // namespace ssscan
