// The gated delta rule token by token (include/ssscan.h): single tokens and short sequences.
//
// With S~ = a S (a = e^g) a token needs S~^T k, then u = beta (v - S~^T k), S = S~ + k u^T and S^T q =
// S~^T q + (q.k) u: both products with the state are of S before the token, so the state is passed once a token
// and q.k is one more sum.  A workgroup holds dk rows by up to 128 columns of the state in registers, a thread
// ROWS rows by VEC columns; sums over rows go over lanes and, through LDS, over the four waves: one barrier a token.
// A single token is bound by the state's read and write: 256 x 40 heads, 128 by 128, in 233 us, 5.8 TB/s.
#include "device_common.h"
#include "gdr.h"
#include "internal.h"

namespace ssscan {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxK = 128;
constexpr int kMaxCols = 128;

template <typename IO, int VEC, int ROWS>
__global__ __launch_bounds__(kThreads, 3) void gdr_recur_kernel(GdrArgs a, int log_groups, int col_blocks) {
  using T = typename IO::T;
  __shared__ alignas(16) float s_qk[2][2][kMaxK];                      // parity; q, k
  __shared__ float s_part[2][kWaves][2][kMaxCols];         // parity, wave; sums with k, with q
  __shared__ float s_dot[2][kWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int groups = 1 << log_groups;                      // of VEC columns
  const int64_t bh = blockIdx.x / col_blocks;
  const int cb = (int)(blockIdx.x - bh * col_blocks);
  const int64_t b = bh / a.hv;
  const int h = (int)(bh - b * a.hv), hkey = h / (a.hv / a.hk);
  const int cg = tid & (groups - 1), row0 = (tid >> log_groups) * ROWS;
  const int col = (cb * groups + cg) * VEC;
  const bool rows = row0 < kMaxK;
  const bool live = col < a.dv;                            // VEC 4: dv is a multiple of 4

  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hkey * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hkey * a.ks[2];
  const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[2];
  const int64_t token0 = b * a.seqlen, state0 = bh * a.dk * a.dv;

  float st[ROWS][VEC];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) st[i][c] = 0.0f;
    if (live && row0 + i < a.dk && a.h0) {
      const float* p = a.h0 + state0 + (uint32_t)((row0 + i) * a.dv + col);
      if constexpr (VEC == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        st[i][0] = w.x; st[i][1] = w.y; st[i][2] = w.z; st[i][3] = w.w;
      } else {
        st[i][0] = *p;
      }
    }
  }

  const int side = tid >> 7, elem = tid & 127;             // this thread's value of q or k
  auto fetch = [&](int64_t t) -> float {
    if (elem >= a.dk) return 0.0f;
    return side ? load_one<IO>(k + t * a.ks[1], elem) : load_one<IO>(q + t * a.qs[1], elem);
  };
  float vn[VEC], gn = 0.0f, bn = 0.0f;
  auto fetch_v = [&](int64_t t) {
    const int64_t at = (token0 + t) * a.hv + h;
    gn = a.g ? a.g[at] : 0.0f;
    bn = a.beta[at];
#pragma unroll
    for (int c = 0; c < VEC; ++c) vn[c] = live ? load_one<IO>(v + t * a.vs[1], col + c) : 0.0f;
  };
  s_qk[0][side][elem] = fetch(0);
  fetch_v(0);
  __syncthreads();
  for (int64_t t = 0; t < a.seqlen; ++t) {
    const int par = (int)(t & 1);
    const float alpha = expf(gn), beta = bn;
    float vt[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) vt[c] = vn[c];
    float next = 0.0f;
    if (t + 1 < a.seqlen) {
      next = fetch(t + 1);
      fetch_v(t + 1);
    }
    float sk[VEC] = {}, sq[VEC] = {}, dot = 0.0f, kr[ROWS];
    const float* ql = &s_qk[par][0][row0 & (kMaxK - 1)];   // ROWS divides kMaxK: all of a thread's rows are, or none
    const float* kl = &s_qk[par][1][row0 & (kMaxK - 1)];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float qi = rows ? ql[i] : 0.0f;
      kr[i] = rows ? kl[i] : 0.0f;
      dot = fmaf(qi, kr[i], dot);
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        sk[c] = fmaf(kr[i], st[i][c], sk[c]);
        sq[c] = fmaf(qi, st[i][c], sq[c]);
      }
    }
    for (int m = groups; m < 64; m <<= 1) {
      dot += __shfl_xor(dot, m);
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        sk[c] += __shfl_xor(sk[c], m);
        sq[c] += __shfl_xor(sq[c], m);
      }
    }
    if (lane < groups) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        s_part[par][wave][0][cg * VEC + c] = sk[c];
        s_part[par][wave][1][cg * VEC + c] = sq[c];
      }
      if (lane == 0) s_dot[par][wave] = dot;
    }
    s_qk[par ^ 1][side][elem] = next;
    __syncthreads();
    float u[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      float z = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) z += s_part[par][w][0][cg * VEC + c];
      u[c] = beta * (vt[c] - alpha * z);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int c = 0; c < VEC; ++c) st[i][c] = fmaf(kr[i], u[c], alpha * st[i][c]);
    if (tid < groups && live) {
      float d = 0.0f, ov[VEC];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) d += s_dot[par][w];
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) z += s_part[par][w][1][cg * VEC + c];
        ov[c] = a.scale * fmaf(d, u[c], alpha * z);
      }
      T* o = static_cast<T*>(a.o) + ((token0 + t) * a.hv + h) * a.dv;
#pragma unroll
      for (int c = 0; c < VEC; ++c) store_one<IO>(o, col + c, ov[c]);
    }
  }
  if (a.h_final && live) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (row0 + i >= a.dk) continue;
      float* p = a.h_final + state0 + (uint32_t)((row0 + i) * a.dv + col);
      if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(st[i][0], st[i][1], st[i][2], st[i][3]);
      else *p = st[i][0];
    }
  }
}

template <typename IO>
hipError_t launch(const GdrArgs& a, hipStream_t s) {
  const bool vec = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.h0) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.h_final) % 16 == 0;
  const int per = vec ? 4 : 1;
  int lg = 0;
  while (lg < 5 && (per << lg) < a.dv) ++lg;
  const int col_blocks = (int)((a.dv + (per << lg) - 1) / (per << lg));
  const int rows = (a.dk + (kThreads >> lg) - 1) / (kThreads >> lg);
  const dim3 grid((unsigned)(a.batch * a.hv * col_blocks));
  if (vec) {
    if (rows <= 4) gdr_recur_kernel<IO, 4, 4><<<grid, kThreads, 0, s>>>(a, lg, col_blocks);
    else if (rows <= 8) gdr_recur_kernel<IO, 4, 8><<<grid, kThreads, 0, s>>>(a, lg, col_blocks);
    else gdr_recur_kernel<IO, 4, 16><<<grid, kThreads, 0, s>>>(a, lg, col_blocks);
  } else {
    if (rows <= 8) gdr_recur_kernel<IO, 1, 8><<<grid, kThreads, 0, s>>>(a, lg, col_blocks);
    else gdr_recur_kernel<IO, 1, 16><<<grid, kThreads, 0, s>>>(a, lg, col_blocks);
  }
  return hipGetLastError();
}

}  // namespace

int64_t gdr_recur_blocks(int64_t batch, int hv, int dv) { return batch * hv * ((dv + 31) / 32); }

hipError_t launch_gdr_recur(const GdrArgs& a, hipStream_t s) {
  return a.io == kIoBf16 ? launch<BF16>(a, s) : launch<F32>(a, s);
}

}  // namespace ssscan
