// The gated delta rule backward, last step: the gradients that need no turn, a workgroup to each chunk of a key head
// (gdr_device.h has the layouts).
//
// (U, dR and the triangles come and stay balanced by the growth p; gdr_device.h says how.)
// With S before the chunk, dS behind it, U, dR and dO, D_ij = 2^(gam_i - gam_j), and M_ij = D_ij dR_i.U_j (j < i),
// N_ij = scale D_ij dO_i.U_j (j <= i):
//   dq_i = scale G_i S dO_i + sum_j N_ij k_j
//   X_i  = G_i S dR_i + sum_j M_ij k_j                      (what k_i reads, over -beta_i)
//   Y_j  = D_Cj dS U_j + sum_i N_ij q_i - sum_i beta_i M_ij k_i
//   dk = Y - beta X,  dbeta = dR.v - k.X,
//   dgam_i = q_i.dq_i - beta_i k_i.X_i - k_i.Y_i, at the chunk's last token also sum_j k_j.(D_Cj dS U_j) + G_C <dS, S>,
// and dg the sums of dgam from a token to the chunk's end.  Everything is fp32 in two planes, as dbeta and dg are differences.
// Rows of dO, U and dR pass LDS 64 columns at a time; a wave reads its own rows of S and dS from memory, each value once.
// The products run transposed, a lane a token, so that gradients are stored in runs.  The value heads of a key head are
// taken one after the other and summed in registers.
#include "gdr_device.h"

namespace ssscan {
namespace {

using namespace gdr;

constexpr int kThreads = 512;
constexpr int kRowBytes = 2 * 4 * kBlock;                  // 64 rows by 64 columns, of a plane

// SHARED: value heads share key heads.
template <typename IO, int KP, bool WHOLE, bool SHARED>
__global__ __launch_bounds__(kThreads, 2) void gdr_grad_kernel(GdrArgs a) {
  using T = typename IO::T;
  constexpr int NP = planes_of<IO>(), kTiles = KP / 32, kTurned = kTiles * 4 * kBlock;
  constexpr int kRegion = (NP + 4) * kRowBytes;            // dO, U, dR; then two triangles at a time
  static_assert(kRegion >= 4 * kTriBytes, "");
  __shared__ alignas(16) char s_kt[NP * kTurned], s_qt[NP * kTurned], s_r[kRegion];
  __shared__ alignas(16) float s_vec[kVecs][kC], s_beta[kC];
  __shared__ float s_mx[8], s_sd[8], s_rv[kC], s_dot[4][kTiles][kC];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, low = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t bk = blockIdx.x / a.chunks, chunk = blockIdx.x - bk * a.chunks;
  const int64_t b = bk / a.hk;
  const int hkey = (int)(bk - b * a.hk), group = SHARED ? a.hv / a.hk : 1;
  const int64_t first = chunk * kC, ostride = (int64_t)a.hv * a.dv;
  const int valid = (int)min(a.seqlen - first, (int64_t)kC);
  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + first * a.qs[1] + hkey * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + first * a.ks[1] + hkey * a.ks[2];
  const __amdgpu_buffer_rsrc_t qr = chunk_rows<IO>(q, a.qs[1], valid, a.dk), kr = chunk_rows<IO>(k, a.ks[1], valid, a.dk);
  const uint32_t krow = (uint32_t)a.ks[1] * sizeof(T), qrow = (uint32_t)a.qs[1] * sizeof(T);

  // this wave's rows of keys 32 m .. and tokens 32 ti ..; of the triangles its type and tiles
  const int m = wave >> 1, ti = wave & 1, type = wave >> 1, tok = 32 * ti + low;
  const bool active = m < kTiles;

  // What is loaded ahead: this thread's 8 columns of a row of dO, v, U and dR, its wave's rows of S and dS; of 64 columns.
  const uint32_t ld = (uint32_t)a.ldv;
  Raw8<IO> ro, rw;
  Raw8<F32> ru, rd;
  float4 rS[4][2], rE[4][2];
  int64_t at, gate;
  __amdgpu_buffer_rsrc_t orows, vrows, urows, drows, srows, erows;
  auto open_head = [&](int n) {
    const int h = hkey * group + n;
    at = (b * a.hv + h) * a.chunks + chunk;
    gate = (b * a.seqlen + first) * a.hv + h;
    orows = chunk_rows<IO>(static_cast<const T*>(a.dout) + (b * a.seqlen + first) * ostride + (int64_t)h * a.dv, ostride, valid, a.dv);
    vrows = chunk_rows<IO>(static_cast<const T*>(a.v) + b * a.vs[0] + first * a.vs[1] + h * a.vs[2], a.vs[1], valid, a.dv);
    urows = make_rsrc(a.u + at * kC * a.ldv, kC * a.ldv * 4);
    drows = make_rsrc(a.dr + at * kC * a.ldv, kC * a.ldv * 4);
    srows = make_rsrc(a.states + at * KP * a.ldv, KP * a.ldv * 4);
    erows = make_rsrc(a.dstates + at * KP * a.ldv, KP * a.ldv * 4);
  };
  auto load_rows = [&](int v0) {
    const int row = anew(tid) >> 3, col = v0 + 8 * (anew(tid) & 7);
    ro = buf_load8<IO, WHOLE>(orows, row * (uint32_t)ostride * sizeof(T), 0, col, a.dv);
    rw = buf_load8<IO, WHOLE>(vrows, row * (uint32_t)a.vs[1] * sizeof(T), 0, col, a.dv);
    ru = buf_load8<F32, true>(urows, row * ld * 4, 0, col, (int)ld);
    rd = buf_load8<F32, true>(drows, row * ld * 4, 0, col, (int)ld);
  };
  auto load_states = [&](int v0) {
    const uint32_t off = ((32 * m + (anew(lane) & 31)) * ld + v0 + 4 * (anew(lane) >> 5)) * 4;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t o = active && v0 + 16 * s < (int)ld ? off + 64 * s + 32 * e : kNowhere;
        const auto x = __builtin_amdgcn_raw_buffer_load_b128(srows, o, 0, 0);
        const auto y = __builtin_amdgcn_raw_buffer_load_b128(erows, o, 0, 0);
        rS[s][e] = make_float4(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]), __uint_as_float(x[3]));
        rE[s][e] = make_float4(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]), __uint_as_float(y[3]));
      }
  };

  // k and q, transposed, each with one scale: threads 0-255 k, the others q
  int ek, eq;
  {
    const int t = tid & 255, g = t & 15, c = t >> 4;
    Raw8<IO> r[4];
    if (wave < 4) {
#pragma unroll
      for (int n = 0; n < 4; ++n) r[n] = buf_load8<IO, WHOLE>(kr, (4 * g + n) * krow, 0, 8 * c, a.dk);
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n) r[n] = buf_load8<IO, WHOLE>(qr, (4 * g + n) * qrow, 0, 8 * c, a.dk);
    }
    open_head(0);
    load_rows(0);
    load_states(0);
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
    const Scale sk = scale_of(fmaxf(fmaxf(s_mx[0], s_mx[1]), fmaxf(s_mx[2], s_mx[3])), 100);
    const Scale sq = scale_of(fmaxf(fmaxf(s_mx[4], s_mx[5]), fmaxf(s_mx[6], s_mx[7])), 100);
    ek = sk.e;
    eq = sq.e;
    const float f = tid < 256 ? sk.f : sq.f, s[4] = {f, f, f, f};
    char* to = tid < 256 ? s_kt : s_qt;
    if (c < KP / 8) store_operand_turned<IO>(to, to + (NP - 1) * kTurned, g, c, x, s);
  }

  acc16 dQ = zero16(), dK = zero16();
  for (int n = 0; n < group; ++n) {
    if (n > 0) {
      __syncthreads();
      open_head(n);
      load_rows(0);
      load_states(0);
    }
    float most[kMaxKinds] = {};
    for (int64_t e = lane; e < a.ldv / 32; e += 64)
#pragma unroll
      for (int i = 0; i < kMaxKinds; ++i) most[i] = fmaxf(most[i], a.maxima[i * a.max_apart + at * (a.ldv / 32) + e]);
    for (int e = tid; e < kVecs * kC; e += kThreads) (&s_vec[0][0])[e] = a.vecs[at * (kVecs * kC) + e];
    if (tid < kC) s_beta[tid] = tid < valid ? a.beta[gate + (int64_t)tid * a.hv] : 0.0f;
    const Scale cS = scale_of(wave_max(most[kMaxS]), 100), cU = scale_of(wave_max(most[kMaxU]), 100);
    const Scale cE = scale_of(wave_max(most[kMaxDs]), 100), cD = scale_of(wave_max(most[kMaxDr]), 100);
    const Scale cO = scale_of(wave_max(most[kMaxDo]), 100);
    char* const s_o = s_r;
    char* const s_u = s_r + NP * kRowBytes;
    char* const s_d = s_u + 2 * kRowBytes;

    acc16 Q = zero16(), X = zero16(), Y = zero16(), C[2] = {zero16(), zero16()};
    float sd = 0.0f, rv = 0.0f;
    for (int v0 = 0; v0 < (int)ld; v0 += 64) {
      {
        const int row = tid >> 3, run = tid & 7;
        float o[8], u[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = raw_value<IO>(ro, j);
          u[j] = raw_value<F32>(ru, j);
          d[j] = raw_value<F32>(rd, j);
          rv = fmaf(d[j], raw_value<IO>(rw, j), rv);
        }
        if (v0 > 0) __syncthreads();                       // the columns before have been read
        store_operand_rows<IO>(s_o, s_o + (NP - 1) * kRowBytes, row, run, 4, o, cO.f);
        store_operand_rows<F32>(s_u, s_u + kRowBytes, row, run, 4, u, cU.f);
        store_operand_rows<F32>(s_d, s_d + kRowBytes, row, run, 4, d, cD.f);
      }
      __syncthreads();
      if (v0 + 64 < (int)ld) load_rows(v0 + 64);
      // triangles: types 0, 1 of N with a lane a row i, a column j; 2, 3 of M
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tile = (wave & 1) ? 2 : e, i = tile > 0, j = tile > 1;
        if (e && (wave & 1)) break;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const Planes u = operand<2>(s_u + (j * 4 + s) * kBlock, lane, kRowBytes);
          if (type < 2) {
            const Planes o = operand<NP>(s_o + (i * 4 + s) * kBlock, lane, kRowBytes);
            C[e] = type & 1 ? mm<NP, 2>(o, u, C[e]) : mm<2, NP>(u, o, C[e]);
          } else {
            const Planes d = operand<2>(s_d + (i * 4 + s) * kBlock, lane, kRowBytes);
            C[e] = type & 1 ? mm<2, 2>(d, u, C[e]) : mm<2, 2>(u, d, C[e]);
          }
        }
      }
      if (active) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float sv[8] = {rS[s][0].x, rS[s][0].y, rS[s][0].z, rS[s][0].w, rS[s][1].x, rS[s][1].y, rS[s][1].z, rS[s][1].w};
          const float dv[8] = {rE[s][0].x, rE[s][0].y, rE[s][0].z, rE[s][0].w, rE[s][1].x, rE[s][1].y, rE[s][1].z, rE[s][1].w};
          Planes S, E;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sd = fmaf(sv[j], dv[j], sd);
            S.hi[j] = (_Float16)(sv[j] * cS.f);
            S.lo[j] = (_Float16)fmaf(sv[j], cS.f, -(float)S.hi[j]);
            E.hi[j] = (_Float16)(dv[j] * cE.f);
            E.lo[j] = (_Float16)fmaf(dv[j], cE.f, -(float)E.hi[j]);
          }
          Q = mm<2, NP>(S, operand<NP>(s_o + (ti * 4 + s) * kBlock, lane, kRowBytes), Q);
          X = mm<2, 2>(S, operand<2>(s_d + (ti * 4 + s) * kBlock, lane, kRowBytes), X);
          Y = mm<2, 2>(E, operand<2>(s_u + (ti * 4 + s) * kBlock, lane, kRowBytes), Y);
          step_end();
        }
      }
      if (v0 + 64 < (int)ld) load_states(v0 + 64);
    }

    // the triangles' values; their sums over rows of dR.v; <dS, S>
    float mC = 0.0f;
    {
      const float f = type < 2 ? a.scale * pow2(-cU.e) * pow2(-cO.e) : pow2(-cU.e) * pow2(-cD.e);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tile = (wave & 1) ? 2 : e, i0 = 32 * (tile > 0), j0 = 32 * (tile > 1);
        const int col = (type & 1 ? j0 : i0) + low;
        const float whole = s_vec[kVecWhole][col], rest = s_vec[kVecRest][col], sign = type & 1 ? -1.0f : 1.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = (type & 1 ? i0 : j0) + tile_row(r, lane);
          const float d = exp2_of(sign * (whole - s_vec[kVecWhole][row]), sign * (rest - s_vec[kVecRest][row]));
          const int i = type & 1 ? row : col, j = type & 1 ? col : row;
          const float w = C[e][r] * f * d;
          C[e][r] = j < i || (j == i && type < 2) ? (type == 3 ? w * s_beta[row] : type == 1 ? w * pow2((int)s_vec[kVecGrow][row]) : w) : 0.0f;
        }
        if (!(e && (wave & 1))) mC = max_of(C[e], mC);
      }
    }
    mC = wave_max(mC);
    rv = group_sum(rv, 8);
    sd = group_sum(sd, 64);
    if (lane == 0) {
      s_mx[wave] = mC;
      s_sd[wave] = active && ti == 0 ? sd : 0.0f;
    }
    if ((lane & 7) == 0) s_rv[tid >> 3] = rv;
    __syncthreads();
    const Scale t0 = scale_of(fmaxf(s_mx[0], s_mx[1]), 100), t1 = scale_of(fmaxf(s_mx[2], s_mx[3]), 100);
    const Scale t2 = scale_of(fmaxf(s_mx[4], s_mx[5]), 100), t3 = scale_of(fmaxf(s_mx[6], s_mx[7]), 100);
    auto write_triangle = [&]() {
      char* out = s_r + (type & 1) * (2 * kTriBytes) + lane * 16;
      const float f = type == 0 ? t0.f : type == 1 ? t1.f : type == 2 ? t2.f : t3.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (e && (wave & 1)) break;
        const int tile = (wave & 1) ? 2 : e;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const Planes p = split(C[e], s, f);
          *reinterpret_cast<h8*>(out + (tile * 2 + s) * 1024) = p.hi;
          *reinterpret_cast<h8*>(out + kTriBytes + (tile * 2 + s) * 1024) = p.lo;
        }
      }
    };
    // sum over tokens of a transposed side (rows 32 m) times a triangle, for this wave's tokens; `lower`: over tokens not after
    // this one, else over those not before it
    auto through = [&](const char* side, int which, bool lower) {
      acc16 acc = zero16();
#pragma unroll
      for (int t = 0; t < 2; ++t) {                        // tile of the summed tokens
        if (lower ? t > ti : t < ti) continue;
        const int tile = t + ti;                           // (0, 0), (1, 0) either way round, (1, 1)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          acc = mm<NP, 2>(operand<NP>(side + (m * 4 + 2 * t + s) * kBlock, lane, kTurned),
                          operand<2>(s_r + which * (2 * kTriBytes) + (tile * 2 + s) * 1024, lane, kTriBytes), acc);
      }
      return acc;
    };
    if (type < 2) write_triangle();
    __syncthreads();
    float kend = 0.0f, into = s_vec[kVecInto][tok];
    acc16 kv;
    if (active) {
      const acc16 nk = through(s_kt, 0, true), nq = through(s_qt, 1, false);
      const float f = a.scale * into * pow2(-cS.e) * pow2(-cO.e), fn = pow2((int)s_vec[kVecGrow][tok] - ek - t0.e), fy = pow2(-eq - t1.e);
      const float fe = s_vec[kVecEnd][tok] * s_vec[kVecS][tok] * pow2(-cE.e) * pow2(-cU.e);
      const float fx = exp2_of(s_vec[kVecWhole][tok], s_vec[kVecRest][tok]) * pow2(-cS.e) * pow2(-cD.e);
      float qdq = 0.0f;
      acc16 qv;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int at_k = 32 * m + 8 * g + 4 * half;
        float x[4];
        buf_load4<IO, WHOLE>(kr, tok * krow, at_k, a.dk, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[4 * g + j] = x[j];
        buf_load4<IO, WHOLE>(qr, tok * qrow, at_k, a.dk, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) qv[4 * g + j] = x[j];
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float dq = fmaf(Q[r], f, nk[r] * fn);
        qdq = fmaf(qv[r], dq, qdq);
        if constexpr (SHARED) dQ[r] += dq;
        else dQ[r] = dq;
        const float e = Y[r] * fe;
        kend = fmaf(kv[r], e, kend);
        Y[r] = fmaf(nq[r], fy, e);
        X[r] *= fx;
      }
      qdq += __shfl_xor(qdq, 32);
      kend += __shfl_xor(kend, 32);
      if (half == 0) {
        s_dot[0][m][tok] = qdq;
        s_dot[3][m][tok] = kend;
      }
    }
    __syncthreads();
    if (type >= 2) write_triangle();
    __syncthreads();
    if (active) {
      const acc16 mk = through(s_kt, 0, true), mb = through(s_kt, 1, false);
      const float fm = pow2(-ek - t2.e), fb = pow2(-ek - t3.e), beta = s_beta[tok];
      float kx = 0.0f, ky = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float x = fmaf(mk[r], fm, X[r]), y = fmaf(-mb[r], fb, Y[r]);
        kx = fmaf(kv[r], x, kx);
        ky = fmaf(kv[r], y, ky);
        if constexpr (SHARED) dK[r] += fmaf(-beta, x, y);
        else dK[r] = fmaf(-beta, x, y);
      }
      kx += __shfl_xor(kx, 32);
      ky += __shfl_xor(ky, 32);
      if (half == 0) {
        s_dot[1][m][tok] = kx;
        s_dot[2][m][tok] = ky;
      }
    }
    __syncthreads();
    if (wave == 0) {
      float d[4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) d[i] += s_dot[i][t][lane];
      float all = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) all += s_sd[i];
      const float end = group_sum(d[3], 64) + s_vec[kVecInto][kC - 1] * all;
      float dgam = d[0] - s_beta[lane] * d[1] - d[2] + (lane == kC - 1 ? end : 0.0f);
#pragma unroll
      for (int i = 1; i < kC; i <<= 1) {
        const float o = __shfl_down(dgam, i);
        if (lane + i < kC) dgam += o;
      }
      if (lane < valid) {
        if (a.dbeta) a.dbeta[gate + (int64_t)lane * a.hv] = s_rv[lane] * pow2(-(int)s_vec[kVecGrow][lane]) - d[1];
        if (a.dg) a.dg[gate + (int64_t)lane * a.hv] = dgam;
      }
    }
  }
  if (active && tok < valid) {
    const int64_t row = ((b * a.seqlen + first + tok) * a.hk + hkey) * a.dk;
    store_runs<IO>(static_cast<T*>(a.dq) + row, 32 * m + 4 * half, a.dk, dQ, 1.0f);
    store_runs<IO>(static_cast<T*>(a.dk_out) + row, 32 * m + 4 * half, a.dk, dK, 1.0f);
  }
}

template <typename IO>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.batch * a.hk * a.chunks));
  return by_keys(a.dk, a.whole, [&](auto kp, auto whole) {
    if (a.hv > a.hk) gdr_grad_kernel<IO, decltype(kp)::value, decltype(whole)::value, true><<<grid, kThreads, 0, s>>>(a);
    else gdr_grad_kernel<IO, decltype(kp)::value, decltype(whole)::value, false><<<grid, kThreads, 0, s>>>(a);
  });
}

}  // namespace

hipError_t launch_gdr_grad(const GdrArgs& a, hipStream_t s) { return a.io == kIoBf16 ? launch<BF16>(a, s) : launch<F32>(a, s); }

}  // namespace ssscan
