// The gated delta rule backward, last step: the gradients that need no turn, a workgroup to each chunk of a head
// (gdr_device.h has the layouts).
//
// (U, dR and the triangles come and stay balanced by p; gdr_device.h says how.)
// With S before the chunk, dS behind it, U, dR and dO, D_ij = 2^(gam_i - gam_j), and M_ij = D_ij dR_i.U_j (j < i),
// N_ij = scale D_ij dO_i.U_j (j <= i):
//   dq_i = scale G_i S dO_i + sum_j N_ij k_j
//   X_i  = G_i S dR_i + sum_j M_ij k_j                      (what k_i reads, over -beta_i)
//   Y_j  = D_Cj dS U_j + sum_i N_ij q_i - sum_i beta_i M_ij k_i
//   dk = Y - beta X,  dbeta = dR.v - k.X,
//   dgam_i = q_i.dq_i - beta_i k_i.X_i - k_i.Y_i, at the chunk's last token also sum_j k_j.(D_Cj dS U_j) + G_C <dS, S>,
// and dg the sums of dgam from a token to the chunk's end.  Everything is fp32 in two planes, as dbeta and dg are differences, and the dot
// products and sums that dg is what remains of (64 tokens' parts, each several times as large) are fp64: they were most of its error.
// Rows of dO, U and dR pass LDS 64 columns at a time; a wave reads its own rows of S and dS from memory.  The products run
// transposed, a lane a token, so that gradients are stored in runs.  A triangle is summed over its rows and over its
// columns; its other orientation is a product with the identity.  The chunks depend on nothing of each other: memory's
// latency is hidden by a second workgroup on the CU, which bounds a lane to 128 registers (bf16).
// Value heads that share a key head leave fp32 parts, added in their order afterwards.
// 8 x 40 heads of 2048 tokens, 128 by 128, bf16: 1010 us for 2.6 GB (500 us as a copy): loads that wait for one another, at four waves
// to a SIMD (dg's sums in fp32 took 975).  One workgroup on a CU with all registers took 1352, rows loaded a pass ahead at 128 registers twice as long (spills).
#include "gdr_device.h"

namespace ssscan {
namespace {

using namespace gdr;

constexpr int kThreads = 512;
constexpr int kRowBytes = 2 * 4 * kBlock;                  // 64 rows by 64 columns, of a plane

template <typename IO, int KP, bool WHOLE>
__global__ __launch_bounds__(kThreads, IO::kPerSpan == 8 ? 4 : 2) void gdr_grad_kernel(GdrArgs a) {
  using T = typename IO::T;
  constexpr int NP = planes_of<IO>(), kTiles = KP / 32, kTurned = kTiles * 4 * kBlock;
  constexpr bool kAhead = NP == 2;                         // one workgroup on a CU, with registers to spare
  constexpr int kRegion = (NP + 4) * kRowBytes;            // dO, U, dR; then two triangles at a time, and sums over values of keys
  static_assert(kRegion >= 4 * kTriBytes + 4 * kTiles * kC * 8, "");
  __shared__ alignas(16) char s_kt[NP * kTurned], s_qt[NP * kTurned], s_r[kRegion];
  __shared__ alignas(16) float s_vec[kVecs][kC], s_beta[kC];
  __shared__ float s_mx[8], s_rv[4][kC];
  __shared__ double s_sd[8];
  double(&s_dot)[4][kTiles][kC] = *reinterpret_cast<double(*)[4][kTiles][kC]>(s_r + 4 * kTriBytes);
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, low = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t at = blockIdx.x, bh = at / a.chunks, chunk = at - bh * a.chunks;
  const int64_t b = bh / a.hv;
  const int h = (int)(bh - b * a.hv), hkey = h / (a.hv / a.hk);
  const int64_t first = chunk * kC, ostride = (int64_t)a.hv * a.dv, gate = (b * a.seqlen + first) * a.hv + h;
  const int valid = (int)min(a.seqlen - first, (int64_t)kC), ld = (int)a.ldv;
  const __amdgpu_buffer_rsrc_t qr = chunk_rows<IO>(static_cast<const T*>(a.q) + b * a.qs[0] + first * a.qs[1] + hkey * a.qs[2], a.qs[1], valid, a.dk);
  const __amdgpu_buffer_rsrc_t kr = chunk_rows<IO>(static_cast<const T*>(a.k) + b * a.ks[0] + first * a.ks[1] + hkey * a.ks[2], a.ks[1], valid, a.dk);
  const uint32_t krow = (uint32_t)a.ks[1] * sizeof(T), qrow = (uint32_t)a.qs[1] * sizeof(T);

  // k and q, transposed, each with one scale: threads 0-255 k, the others q
  int ek, eq;
  float most[kMaxKinds] = {};
  {
    const int t = tid & 255, g = t & 15, c = t >> 4;
    Raw8<IO> r[4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
      r[n] = wave < 4 ? buf_load8<IO, WHOLE>(kr, (4 * g + n) * krow, 0, 8 * c, a.dk) : buf_load8<IO, WHOLE>(qr, (4 * g + n) * qrow, 0, 8 * c, a.dk);
    for (int e = lane; e < ld / 32; e += 64)
#pragma unroll
      for (int i = 0; i < kMaxKinds; ++i) most[i] = fmaxf(most[i], a.maxima[i * a.max_apart + at * (ld / 32) + e]);
    for (int e = tid; e < kVecs * kC; e += kThreads) (&s_vec[0][0])[e] = a.vecs[at * (kVecs * kC) + e];
    if (tid < kC) s_beta[tid] = tid < valid ? a.beta[gate + (int64_t)tid * a.hv] : 0.0f;
    float x[4][8], mx = 0.0f;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[n][j] = raw_value<IO>(r[n], j);
        mx = fmaxf(mx, fabsf(x[n][j]));
      }
    mx = wave_max(mx);
    if (lane == 0) s_mx[wave] = mx;
    __syncthreads();
    const Scale sk = scale_of(fmaxf(fmaxf(s_mx[0], s_mx[1]), fmaxf(s_mx[2], s_mx[3])), kMostE);
    const Scale sq = scale_of(fmaxf(fmaxf(s_mx[4], s_mx[5]), fmaxf(s_mx[6], s_mx[7])), kMostE);
    ek = sk.e;
    eq = sq.e;
    const float f = tid < 256 ? sk.f : sq.f, s[4] = {f, f, f, f};
    char* to = tid < 256 ? s_kt : s_qt;
    if (c < KP / 8) store_operand_turned<IO>(to, to + (NP - 1) * kTurned, g, c, x, s);
  }
  const Scale cS = scale_of(wave_max(most[kMaxS]), kMostE), cU = scale_of(wave_max(most[kMaxU]), kMostE);
  const Scale cE = scale_of(wave_max(most[kMaxDs]), kMostE), cD = scale_of(wave_max(most[kMaxDr]), kMostE);
  const Scale cO = scale_of(wave_max(most[kMaxDo]), kMostE);

  // this wave's rows of keys 32 m .. and tokens 32 ti ..; of the triangles N (waves 0-2) and M (4-6) its tile, a lane a row i
  const int m = wave >> 1, ti = wave & 1, tok = 32 * ti + low, tile = wave & 3, i0 = 32 * (tile > 0), j0 = 32 * (tile > 1);
  const bool active = m < kTiles, of_n = wave < 4;
  char* const s_o = s_r;
  char* const s_u = s_r + NP * kRowBytes;
  char* const s_d = s_u + 2 * kRowBytes;
  acc16 Q = zero16(), X = zero16(), Y = zero16(), C = zero16();
  double sd = 0.0;
  float rv = 0.0f;
  {
    const __amdgpu_buffer_rsrc_t orows = chunk_rows<IO>(static_cast<const T*>(a.dout) + (b * a.seqlen + first) * ostride + (int64_t)h * a.dv, ostride, valid, a.dv);
    const __amdgpu_buffer_rsrc_t vrows = chunk_rows<IO>(static_cast<const T*>(a.v) + b * a.vs[0] + first * a.vs[1] + h * a.vs[2], a.vs[1], valid, a.dv);
    const __amdgpu_buffer_rsrc_t urows = make_rsrc(a.u + at * kC * a.ldv, kC * a.ldv * 4), drows = make_rsrc(a.dr + at * kC * a.ldv, kC * a.ldv * 4);
    const __amdgpu_buffer_rsrc_t srows = make_rsrc(a.states + at * KP * a.ldv, KP * a.ldv * 4);
    const __amdgpu_buffer_rsrc_t erows = make_rsrc(a.dstates + at * KP * a.ldv, KP * a.ldv * 4);
    // rows of 64 columns: of dO a thread has 8 columns of one, of U and dR (with v) the operand that its lane is of its wave's block
    const int utile = wave >> 2, ustep = wave & 3;
    Raw8<IO> ro;
    Raw4<IO> rw[2];
    Raw8<F32> ru, rd;
    auto load_rows = [&](int v0) {
      const int ln = anew(lane), c = v0 + 16 * ustep, w = (utile * (ld / 16) + c / 16) * 512 + ln * 4;
      ro = buf_load8<IO, WHOLE>(orows, (8 * wave + (ln >> 3)) * (uint32_t)ostride * sizeof(T), 0, v0 + 8 * (ln & 7), a.dv);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rw[e] = buf_load4<IO, WHOLE>(vrows, (32 * utile + (ln & 31)) * (uint32_t)a.vs[1] * sizeof(T), c + 8 * e + 4 * (ln >> 5), a.dv);
        const auto x = __builtin_amdgcn_raw_buffer_load_b128(urows, c < ld ? w * 4 + 1024 * e : kNowhere, 0, 0);
        const auto y = __builtin_amdgcn_raw_buffer_load_b128(drows, c < ld ? w * 4 + 1024 * e : kNowhere, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ru.w[4 * e + j] = x[j];
          rd.w[4 * e + j] = y[j];
        }
      }
    };
    if constexpr (kAhead) load_rows(0);
    for (int v0 = 0; v0 < ld; v0 += 64) {
      if constexpr (!kAhead) load_rows(v0);
      {
        float o[8];
        Planes u, d;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = raw_value<IO>(ro, j);
          const float x = raw_value<F32>(ru, j), y = raw_value<F32>(rd, j);
          u.hi[j] = (_Float16)(x * cU.f);
          u.lo[j] = (_Float16)fmaf(x, cU.f, -(float)u.hi[j]);
          d.hi[j] = (_Float16)(y * cD.f);
          d.lo[j] = (_Float16)fmaf(y, cD.f, -(float)d.hi[j]);
          rv = fmaf(y, rw[j >> 2].value(j & 3), rv);
        }
        __syncthreads();                                   // the columns before have been read
        store_operand_rows<IO>(s_o, s_o + (NP - 1) * kRowBytes, tid >> 3, tid & 7, 4, o, cO.f);
        *reinterpret_cast<h8*>(s_u + wave * kBlock + lane * 16) = u.hi;
        *reinterpret_cast<h8*>(s_u + kRowBytes + wave * kBlock + lane * 16) = u.lo;
        *reinterpret_cast<h8*>(s_d + wave * kBlock + lane * 16) = d.hi;
        *reinterpret_cast<h8*>(s_d + kRowBytes + wave * kBlock + lane * 16) = d.lo;
      }
      __syncthreads();
      if constexpr (kAhead)
        if (v0 + 64 < ld) load_rows(v0 + 64);
      if (tile < 3) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const Planes u = operand<2>(s_u + ((j0 >> 5) * 4 + s) * kBlock, lane, kRowBytes);
          if (of_n) C = mm<2, NP>(u, operand<NP>(s_o + ((i0 >> 5) * 4 + s) * kBlock, lane, kRowBytes), C);
          else C = mm<2, 2>(u, operand<2>(s_d + ((i0 >> 5) * 4 + s) * kBlock, lane, kRowBytes), C);
        }
      }
      if (active) {
        const uint32_t off = ((m * (ld / 16) + v0 / 16) * 512 + lane * 4) * 4;
        float part = 0.0f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t o = v0 + 16 * s < ld ? off + 2048 * s : kNowhere;
          const auto s0 = __builtin_amdgcn_raw_buffer_load_b128(srows, o, 0, 0), s1 = __builtin_amdgcn_raw_buffer_load_b128(srows, o + 1024, 0, 0);
          const auto d0 = __builtin_amdgcn_raw_buffer_load_b128(erows, o, 0, 0), d1 = __builtin_amdgcn_raw_buffer_load_b128(erows, o + 1024, 0, 0);
          Planes S, E;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float sv = __uint_as_float(j < 4 ? s0[j & 3] : s1[j & 3]), ev = __uint_as_float(j < 4 ? d0[j & 3] : d1[j & 3]);
            part = fmaf(sv, ev, part);
            S.hi[j] = (_Float16)(sv * cS.f);
            S.lo[j] = (_Float16)fmaf(sv, cS.f, -(float)S.hi[j]);
            E.hi[j] = (_Float16)(ev * cE.f);
            E.lo[j] = (_Float16)fmaf(ev, cE.f, -(float)E.hi[j]);
          }
          Q = mm<2, NP>(S, operand<NP>(s_o + (ti * 4 + s) * kBlock, lane, kRowBytes), Q);
          X = mm<2, 2>(S, operand<2>(s_d + (ti * 4 + s) * kBlock, lane, kRowBytes), X);
          Y = mm<2, 2>(E, operand<2>(s_u + (ti * 4 + s) * kBlock, lane, kRowBytes), Y);
        }
        sd += part;
      }
    }
  }

  // the triangles' values; sums over rows of dR.v; <dS, S>
  {
    const float f = times_pow2(of_n ? a.scale : 1.0f, -cU.e - (of_n ? cO.e : cD.e));
    const int i = i0 + low;
    // U comes times 2^-p_j, so N would be times 2^-p_i; of that only growth is left in it.  So that both orientations hold the same
    // values where gates decay: what one of them adds to dg the other takes back (else dg of strong decays is off by 10^-5).
    const float whole = s_vec[kVecWhole][i] + (of_n ? fminf(s_vec[kVecGrow][i], 0.0f) : 0.0f), rest = s_vec[kVecRest][i];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int j = j0 + tile_row(r, lane);
      const float w = C[r] * f * exp2_of(whole - s_vec[kVecWhole][j], rest - s_vec[kVecRest][j]);
      C[r] = j < i || (j == i && of_n) ? w : 0.0f;
    }
  }
  const float mC = wave_max(max_of(C, 0.0f));
  rv += __shfl_xor(rv, 32);
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) sd += __shfl_xor(sd, i);
  if (lane == 0) {
    s_mx[wave] = tile < 3 ? mC : 0.0f;
    s_sd[wave] = active && ti == 0 ? sd : 0.0;
  }
  if (half == 0) s_rv[wave & 3][32 * (wave >> 2) + low] = rv;
  __syncthreads();
  const Scale t0 = scale_of(fmaxf(s_mx[0], fmaxf(s_mx[1], s_mx[2])), kMostE), t1 = scale_of(fmaxf(s_mx[4], fmaxf(s_mx[5], s_mx[6])), kMostE);
  // the other orientation: a lane a column j, rows times what is not yet theirs: 2^p_i of N where p_i > 0, beta_i of M, at most 2^rise
  const int rise_n = (int)wave_max(fmaxf(s_vec[kVecGrow][lane], 0.0f));
  const int rise_m = max(exponent(wave_max(fabsf(s_beta[lane]))) + 1, 0);
  auto write_triangles = [&]() {
    char* out = s_r + tile * 2048 + lane * 16;
    const float f = of_n ? t0.f : t1.f;
    Planes p[2] = {split(C, 0, f), split(C, 1, f)};
    acc16 t = transposed(p[0], p[1], lane);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      *reinterpret_cast<h8*>(out + s * 1024) = p[s].hi;
      *reinterpret_cast<h8*>(out + kTriBytes + s * 1024) = p[s].lo;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = i0 + tile_row(r, lane);
      t[r] = held(t[r] * (of_n ? pow2(max((int)s_vec[kVecGrow][i], 0) - rise_n) : s_beta[i] * pow2(-rise_m)));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const Planes q = split(t, s, 1.0f);
      *reinterpret_cast<h8*>(out + 2 * kTriBytes + s * 1024) = q.hi;
      *reinterpret_cast<h8*>(out + 3 * kTriBytes + s * 1024) = q.lo;
    }
  };
  // sum over tokens of a transposed side (rows 32 m) times a triangle, for this wave's tokens; `lower`: over tokens not after
  // this one, else over those not before it
  auto through = [&](const char* side, bool lower) {
    acc16 acc = zero16();
#pragma unroll
    for (int t = 0; t < 2; ++t) {                          // tile of the summed tokens
      if (lower ? t > ti : t < ti) continue;
#pragma unroll
      for (int s = 0; s < 2; ++s)                          // tiles (0, 0), (1, 0) either way round, (1, 1)
        acc = mm<NP, 2>(operand<NP>(side + (m * 4 + 2 * t + s) * kBlock, lane, kTurned),
                        operand<2>(s_r + (lower ? 0 : 2 * kTriBytes) + ((t + ti) * 2 + s) * 1024, lane, kTriBytes), acc);
    }
    return acc;
  };
  if (of_n && tile < 3) write_triangles();
  __syncthreads();
  Raw4<IO> rq[4], rk[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    rq[g] = buf_load4<IO, WHOLE>(qr, tok * qrow, 32 * m + 8 * g + 4 * half, active ? a.dk : 0);
    rk[g] = buf_load4<IO, WHOLE>(kr, tok * krow, 32 * m + 8 * g + 4 * half, active ? a.dk : 0);
  }
  if (active) {
    const float into = s_vec[kVecInto][tok];
    const float f = times_pow2(a.scale * into, -cS.e - cO.e), fn = times_pow2(1.0f, max((int)s_vec[kVecGrow][tok], 0) - ek - t0.e), fy = times_pow2(1.0f, rise_n - eq - t0.e);
    const float fe = times_pow2(s_vec[kVecEnd][tok] * s_vec[kVecS][tok], -cE.e - cU.e);
    const float fx = times_pow2(exp2_of(s_vec[kVecWhole][tok], s_vec[kVecRest][tok]), -cS.e - cD.e);
    double qdq = 0.0, kend = 0.0;
    const acc16 nk = through(s_kt, true);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      Q[r] = fmaf(Q[r], f, nk[r] * fn);
      qdq = fma((double)rq[r >> 2].value(r & 3), (double)Q[r], qdq);
    }
    const acc16 nq = through(s_qt, false);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float e = Y[r] * fe;
      kend = fma((double)rk[r >> 2].value(r & 3), (double)e, kend);
      Y[r] = fmaf(nq[r], fy, e);
      X[r] *= fx;
    }
    qdq += __shfl_xor(qdq, 32);
    kend += __shfl_xor(kend, 32);
    if (half == 0) {
      s_dot[0][m][tok] = qdq;
      s_dot[3][m][tok] = kend;
    }
    if (tok < valid) {
      if (a.hv > a.hk) {
        store_runs<F32>(a.part_q + (at * kC + tok) * KP + 32 * m + 4 * half, 0, 32, Q);
      } else {
        store_runs<IO>(static_cast<T*>(a.dq) + ((b * a.seqlen + first + tok) * a.hk + hkey) * a.dk, 32 * m + 4 * half, a.dk, Q);
      }
    }
  }
  __syncthreads();
  if (!of_n && tile < 3) write_triangles();
  __syncthreads();
  if (active) {
    const float fm = times_pow2(1.0f, -ek - t1.e), fb = times_pow2(1.0f, rise_m - ek - t1.e), beta = s_beta[tok];
    const acc16 mk = through(s_kt, true), mb = through(s_kt, false);
    double kx = 0.0, ky = 0.0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float kv = rk[r >> 2].value(r & 3), x = fmaf(mk[r], fm, X[r]), y = fmaf(-mb[r], fb, Y[r]);
      kx = fma((double)kv, (double)x, kx);
      ky = fma((double)kv, (double)y, ky);
      Y[r] = fmaf(-beta, x, y);
    }
    kx += __shfl_xor(kx, 32);
    ky += __shfl_xor(ky, 32);
    if (half == 0) {
      s_dot[1][m][tok] = kx;
      s_dot[2][m][tok] = ky;
    }
    if (tok < valid) {
      if (a.hv > a.hk) {
        store_runs<F32>(a.part_k + (at * kC + tok) * KP + 32 * m + 4 * half, 0, 32, Y);
      } else {
        store_runs<IO>(static_cast<T*>(a.dk_out) + ((b * a.seqlen + first + tok) * a.hk + hkey) * a.dk, 32 * m + 4 * half, a.dk, Y);
      }
    }
  }
  __syncthreads();
  if (wave == 0) {
    double d[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < kTiles; ++t) d[i] += s_dot[i][t][lane];
    double end = d[3], all = 0.0;
#pragma unroll
    for (int i = 1; i < kC; i <<= 1) end += __shfl_xor(end, i);
#pragma unroll
    for (int i = 0; i < 8; ++i) all += s_sd[i];
    end += s_vec[kVecInto][kC - 1] * all;
    double dgam = d[0] - s_beta[lane] * d[1] - d[2] + (lane == kC - 1 ? end : 0.0);
#pragma unroll
    for (int i = 1; i < kC; i <<= 1) {
      const double o = __shfl_down(dgam, i);
      if (lane + i < kC) dgam += o;
    }
    if (lane < valid) {
      if (a.dbeta) a.dbeta[gate + (int64_t)lane * a.hv] = (s_rv[0][lane] + s_rv[1][lane] + s_rv[2][lane] + s_rv[3][lane]) * pow2(-(int)s_vec[kVecGrow][lane]) - (float)d[1];
      if (a.dg) a.dg[gate + (int64_t)lane * a.hv] = (float)dgam;
    }
  }
}

// dq (blockIdx.y 0) and dk of key heads with several value heads: their parts' sums, four values a thread.
template <typename IO>
__global__ __launch_bounds__(256) void gdr_join_kernel(GdrArgs a, int kp) {
  using T = typename IO::T;
  const int runs = (a.dk + 3) / 4, group = a.hv / a.hk;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = e / runs;                            // (batch, token, key head)
  const int col = (int)(e - row * runs) * 4;
  if (row >= a.batch * a.seqlen * a.hk) return;
  const int64_t tok = row / a.hk, b = tok / a.seqlen, t = tok - b * a.seqlen;
  const int hkey = (int)(row - tok * a.hk);
  const float* part = blockIdx.y ? a.part_k : a.part_q;
  float x[4] = {};
  for (int n = 0; n < group; ++n) {
    const int64_t at = (b * a.hv + hkey * group + n) * a.chunks + t / kC;
    const float4 p = *reinterpret_cast<const float4*>(part + (at * kC + t % kC) * kp + col);
    x[0] += p.x; x[1] += p.y; x[2] += p.z; x[3] += p.w;
  }
  T* out = static_cast<T*>(blockIdx.y ? a.dk_out : a.dq) + row * a.dk;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col + j < a.dk) store_one<IO>(out, col + j, x[j]);
}

template <typename IO>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.hv * a.chunks));
  const hipError_t e = by_keys(a.dk, a.whole, [&](auto kp, auto whole) {
    gdr_grad_kernel<IO, decltype(kp)::value, decltype(whole)::value><<<grid, kThreads, 0, s>>>(a);
  });
  if (e != hipSuccess || a.hv == a.hk) return e;
  const int64_t threads = a.batch * a.seqlen * a.hk * ((a.dk + 3) / 4);
  gdr_join_kernel<IO><<<dim3((unsigned)((threads + 255) / 256), 2), 256, 0, s>>>(a, (a.dk + 31) / 32 * 32);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_grad(const GdrArgs& a, hipStream_t s) { return a.io == kIoBf16 ? launch<BF16>(a, s) : launch<F32>(a, s); }

}  // namespace ssscan
