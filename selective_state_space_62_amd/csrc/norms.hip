// The norms before and after a block (include/ssscan.h): gated norm, residual norm, and their gradients.
//
// Bytes bound all four: a row is read once, kept in registers as it was read, its sums go over the row's lanes, and
// everything else is formed from the registers.  A row of up to 512 values (forward 1024, of two vectors to a lane) is a power of 2 of
// lanes of one wave, which hold a vector of 8 consecutive values each, and its sums need no barrier.  Wider rows are a workgroup's, of
// as many waves (up to eight) as its vectors fill, two to a lane from 4097 values on: their sums pass LDS, one barrier for each set of sums.
// The weights' gradients stay in a lane's registers over the rows of its workgroup; the workgroups' sums are then
// added in a fixed order.
// bf16 unless said: rows of 5120, 16384 of them, gated 95 us, 5.3 TB/s (178 before a row's loads went out one row ahead and a weight's
// stayed over a workgroup's rows); residual norm, rows of 2560 onto fp32, 102 us, 4.9 TB/s; backward of the heads' norm (128) 181 us,
// 4.6 TB/s; backward of the residual norm, 16379 rows of 768 in fp32, 86 us, 3.5 TB/s.
#include "device_common.h"
#include "internal.h"
#include "norms.h"

namespace ssscan {
namespace {

using namespace dev;

constexpr int kVec = 8;
constexpr int kMaxLanes = 512;

// A vector as it stands in memory, at any element alignment.
template <typename IO>
struct __attribute__((packed, aligned(sizeof(typename IO::T)))) Raw {
  uint32_t w[kVec * sizeof(typename IO::T) / 4];
};

template <typename IO>
__device__ __forceinline__ Raw<IO> load_raw(const typename IO::T* __restrict__ p, int valid) {
  Raw<IO> r;
  if (valid >= kVec) return *reinterpret_cast<const Raw<IO>*>(p);
#pragma unroll
  for (int j = 0; j < (int)(sizeof(r.w) / 4); ++j) r.w[j] = 0u;
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    if (j < valid) {
      if constexpr (IO::kPerSpan == 4) r.w[j] = __float_as_uint(p[j]);
      else r.w[j >> 1] |= (uint32_t)p[j] << ((j & 1) * 16);
    }
  return r;
}

template <typename IO>
__device__ __forceinline__ float value(const Raw<IO>& r, int j) {
  if constexpr (IO::kPerSpan == 4) return __uint_as_float(r.w[j]);
  else return (j & 1) ? __uint_as_float(r.w[j >> 1] & 0xffff0000u) : __uint_as_float(r.w[j >> 1] << 16);
}

template <typename IO>
__device__ __forceinline__ Raw<IO> pack(const float (&v)[kVec]) {
  Raw<IO> r;
#pragma unroll
  for (int j = 0; j < kVec; j += 2) {
    if constexpr (IO::kPerSpan == 4) {
      r.w[j] = __float_as_uint(v[j]);
      r.w[j + 1] = __float_as_uint(v[j + 1]);
    } else {
      r.w[j >> 1] = pack_bf16x2(v[j], v[j + 1]);
    }
  }
  return r;
}

template <typename IO>
__device__ __forceinline__ void store_raw(typename IO::T* __restrict__ p, int valid, const Raw<IO>& r) {
  if (valid >= kVec) {
    *reinterpret_cast<Raw<IO>*>(p) = r;
    return;
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    if (j < valid) {
      if constexpr (IO::kPerSpan == 4) p[j] = __uint_as_float(r.w[j]);
      else p[j] = (uint16_t)(r.w[j >> 1] >> ((j & 1) * 16));
    }
}

// 8 fp32 values of a vector of weights; `none` where there are no weights, 0 past the row's end.
__device__ __forceinline__ void load_weights(const float* __restrict__ p, int at, int valid, float none, float (&w)[kVec]) {
#pragma unroll
  for (int j = 0; j < kVec; ++j) w[j] = j < valid ? none : 0.0f;
  if (!p) return;
  const Raw<F32> r = load_raw<F32>(p + at, valid);
#pragma unroll
  for (int j = 0; j < kVec; ++j) w[j] = value<F32>(r, j);
}

// Sums of K values over the lanes of a row, in every one of them.  Rows wider than a wave are their workgroup's own:
// `slot` alternates, so that one barrier is enough.
template <int K>
__device__ __forceinline__ void row_sums(float (&v)[K], int lanes, int& slot) {
  __shared__ float s_sum[2][kMaxLanes / 64][K];
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = group_sum(v[i], lanes < 64 ? lanes : 64);
  if (lanes <= 64) return;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < K; ++i) s_sum[slot][wave][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = 0.0f;
  for (int w = 0; w < lanes >> 6; ++w)
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += s_sum[slot][w][i];
  slot ^= 1;
}

// 1 / sqrt(mean + eps), for the sum of n squares (the hardware's root is within one step).
__device__ __forceinline__ float inv_rms(float sum, float inv_n, float eps) { return __builtin_amdgcn_rsqf(fmaf(sum, inv_n, eps)); }

// A workgroup's sums over its rows of every column, from its lanes' (lane l of a row holds vectors l, l + lanes, ...),
// written as one row of n.
template <int NV>
__device__ __forceinline__ void block_columns(float (&acc)[NV][kVec], const NormPlan& pl, int n, float* __restrict__ out) {
  constexpr int kMost = 64 * NV * kVec;
  __shared__ float s_col[3][kMost];
  const int tid = threadIdx.x, l = pl.lanes > 64 ? tid : tid & (pl.lanes - 1), wave = tid >> 6;
  if (pl.lanes < 64) {
    for (int m = pl.lanes; m < 64; m <<= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[i][j] += __shfl_xor(acc[i][j], m);
  }
  const bool several = pl.lanes <= 64;                     // four waves with rows of their own
  if (several) {
    __syncthreads();
    if (wave > 0 && (tid & 63) < pl.lanes) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) s_col[wave - 1][(i * kVec + j) * 64 + l] = acc[i][j];
    }
    __syncthreads();
    if (wave > 0 || (tid & 63) >= pl.lanes) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int col = (i * pl.lanes + l) * kVec + j;
      float v = acc[i][j];
      if (several)
        for (int w = 0; w < 3; ++w) v += s_col[w][(i * kVec + j) * 64 + l];
      if (col < n) out[col] = v;
    }
}

// Where row `row` of the call starts in a tensor.
struct RowPlace {
  int64_t b, t;
  int32_t h;
};

__device__ __forceinline__ RowPlace place(const GatedNormArgs& a, int64_t row) {
  RowPlace r;
  uint32_t tok = (uint32_t)row;
  r.h = 0;
  if (a.per_head) {
    r.h = blockIdx.y;
  } else if (a.heads > 1) {
    const uint32_t t = tok / (uint32_t)a.heads;
    r.h = (int)(tok - t * (uint32_t)a.heads);
    tok = t;
  }
  r.b = 0;
  if (a.seqlen < a.tokens) {
    r.b = tok / (uint32_t)a.seqlen;
    tok -= (uint32_t)r.b * (uint32_t)a.seqlen;
  }
  r.t = tok;
  return r;
}

__device__ __forceinline__ int64_t offset(const NormRows& m, const RowPlace& r) {
  return r.b * m.stride[0] + r.t * m.stride[1] + r.h * m.stride[2];
}

// silu(z) and its derivative.
__device__ __forceinline__ float silu_slope(float z, float& slope) {
  const float sig = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
  slope = sig * fmaf(z, 1.0f - sig, 1.0f);
  return z * sig;
}

template <typename IO, int NV, bool GATE, int THREADS>
__global__ __launch_bounds__(THREADS) void gated_norm_kernel(GatedNormArgs a) {
  using T = typename IO::T;
  const NormPlan& pl = a.plan;
  const int tid = threadIdx.x, l = pl.lanes > 64 ? tid : tid & (pl.lanes - 1), per = pl.threads / pl.lanes;
  const int64_t rows = a.per_head ? a.tokens : a.tokens * a.heads;
  int slot = 0;
  float w[NV][kVec];
  int valid[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * pl.lanes + l) * kVec;
    valid[i] = a.n - at;
    load_weights(a.per_head && a.w ? a.w + (int64_t)blockIdx.y * a.n : a.w, at, valid[i], 1.0f, w[i]);
  }
  const int64_t step = (int64_t)gridDim.x * per;
  Raw<IO> nx[NV], nz[NV];
  auto fetch = [&](int64_t row) {
    const RowPlace at = place(a, row);
    const T* x = static_cast<const T*>(a.x.p) + offset(a.x, at);
#pragma unroll
    for (int i = 0; i < NV; ++i) nx[i] = load_raw<IO>(x + (i * pl.lanes + l) * kVec, valid[i]);
    if constexpr (GATE) {
      const T* z = static_cast<const T*>(a.z.p) + offset(a.z, at);
#pragma unroll
      for (int i = 0; i < NV; ++i) nz[i] = load_raw<IO>(z + (i * pl.lanes + l) * kVec, valid[i]);
    }
  };
  // every lane stays to the end, as sums pass barriers; rows behind the last are the last again, and not stored
  int64_t row = (int64_t)blockIdx.x * per + tid / pl.lanes;
  fetch(min(row, rows - 1));
  for (int64_t first = (int64_t)blockIdx.x * per; first < rows; first += step, row += step) {
    float v[NV][kVec], sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float xv = value<IO>(nx[i], j);
        const float gate = GATE ? silu(value<IO>(nz[i], j)) : 1.0f;
        const float m = GATE && a.gate_first ? xv * gate : xv;
        sum[0] = fmaf(m, m, sum[0]);
        v[i][j] = xv * gate;
      }
    if (first + step < rows) fetch(min(row + step, rows - 1));
    row_sums(sum, pl.lanes, slot);
    const float rho = inv_rms(sum[0], a.inv_n, a.eps);
    if (row >= rows) continue;
    T* y = static_cast<T*>(a.y) + (a.per_head ? row * a.heads + blockIdx.y : row) * a.n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[i][j] *= rho * w[i][j];
      store_raw<IO>(y + (i * pl.lanes + l) * kVec, valid[i], pack<IO>(v[i]));
    }
  }
}

// With m = x silu(z) (gate first) or x, rho its inverse RMS, dn the gradient of rho m w (dy, or dy silu(z)) and p = dn w:
// dm = rho (p - m rho^2 mean(p m)), dw = sum of dn m rho; both means are sums over the row at once.
template <typename IO, int NV, bool GATE, int THREADS>
__global__ __launch_bounds__(THREADS) void gated_norm_bwd_kernel(GatedNormArgs a) {
  using T = typename IO::T;
  const NormPlan& pl = a.plan;
  const int tid = threadIdx.x, l = pl.lanes > 64 ? tid : tid & (pl.lanes - 1), per = pl.threads / pl.lanes;
  const int64_t rows = a.per_head ? a.tokens : a.tokens * a.heads;
  int slot = 0;
  float w[NV][kVec], dw[NV][kVec] = {};
  int valid[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * pl.lanes + l) * kVec;
    valid[i] = a.n - at;
    load_weights(a.per_head && a.w ? a.w + (int64_t)blockIdx.y * a.n : a.w, at, valid[i], 1.0f, w[i]);
  }
  const int64_t step = (int64_t)gridDim.x * per;
  Raw<IO> nx[NV], nz[NV], nd[NV];
  auto fetch = [&](int64_t row) {
    const RowPlace at = place(a, row);
    const T* x = static_cast<const T*>(a.x.p) + offset(a.x, at);
    const T* dy = static_cast<const T*>(a.dy) + (a.per_head ? row * a.heads + blockIdx.y : row) * a.n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      nx[i] = load_raw<IO>(x + (i * pl.lanes + l) * kVec, valid[i]);
      nd[i] = load_raw<IO>(dy + (i * pl.lanes + l) * kVec, valid[i]);
    }
    if constexpr (GATE) {
      const T* z = static_cast<const T*>(a.z.p) + offset(a.z, at);
#pragma unroll
      for (int i = 0; i < NV; ++i) nz[i] = load_raw<IO>(z + (i * pl.lanes + l) * kVec, valid[i]);
    }
  };
  int64_t row = (int64_t)blockIdx.x * per + tid / pl.lanes;
  fetch(min(row, rows - 1));
  for (int64_t first = (int64_t)blockIdx.x * per; first < rows; first += step, row += step) {
    Raw<IO> rx[NV], rz[NV], rd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i] = nx[i];
      rd[i] = nd[i];
      if constexpr (GATE) rz[i] = nz[i];
    }
    if (first + step < rows) fetch(min(row + step, rows - 1));
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float gate = GATE ? silu(value<IO>(rz[i], j)) : 1.0f;
        float m = value<IO>(rx[i], j), dn = value<IO>(rd[i], j);
        if (GATE && a.gate_first) m *= gate;
        else dn *= gate;
        sum[0] = fmaf(m, m, sum[0]);
        sum[1] = fmaf(dn * w[i][j], m, sum[1]);
      }
    row_sums(sum, pl.lanes, slot);
    const float rho = inv_rms(sum[0], a.inv_n, a.eps);
    const float c = rho * rho * (sum[1] * a.inv_n);
    if (row >= rows) continue;
    const RowPlace at = place(a, row);
    T* dx = static_cast<T*>(const_cast<void*>(a.dx.p)) + offset(a.dx, at);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float gx[kVec], gz[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float xv = value<IO>(rx[i], j), d = value<IO>(rd[i], j);
        float slope = 0.0f;
        const float gate = GATE ? silu_slope(value<IO>(rz[i], j), slope) : 1.0f;
        const bool before = GATE && a.gate_first;
        const float m = before ? xv * gate : xv, dn = before ? d : d * gate;
        const float dm = rho * fmaf(-m, c, dn * w[i][j]);
        gx[j] = before ? dm * gate : dm;
        gz[j] = (before ? dm * xv : d * (m * (rho * w[i][j]))) * slope;
        dw[i][j] = fmaf(dn, m * rho, dw[i][j]);
      }
      const int e = (i * pl.lanes + l) * kVec;
      store_raw<IO>(dx + e, valid[i], pack<IO>(gx));
      if constexpr (GATE) store_raw<IO>(static_cast<T*>(const_cast<void*>(a.dz.p)) + offset(a.dz, at) + e, valid[i], pack<IO>(gz));
    }
  }
  if (a.part) block_columns<NV>(dw, pl, a.n, a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.n);
}

template <typename IO, typename RO, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void residual_norm_kernel(ResidualNormArgs a) {
  using T = typename IO::T;
  using R = typename RO::T;
  const NormPlan& pl = a.plan;
  const int tid = threadIdx.x, l = pl.lanes > 64 ? tid : tid & (pl.lanes - 1), per = pl.threads / pl.lanes;
  int slot = 0, slot_post = 0;
  float w[NV][kVec], by[NV][kVec];
  int valid[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * pl.lanes + l) * kVec;
    valid[i] = a.n - at;
    load_weights(a.w, at, valid[i], 1.0f, w[i]);
    load_weights(a.scale, at, valid[i], 1.0f, by[i]);
    float wp[kVec];
    load_weights(a.post ? a.w_post : nullptr, at, valid[i], 1.0f, wp);
#pragma unroll
    for (int j = 0; j < kVec; ++j) by[i][j] *= a.alpha * wp[j];
  }
  const int64_t step = (int64_t)gridDim.x * per;
  Raw<IO> nx[NV];
  Raw<RO> nr[NV];
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(a.x) + row * a.n;
    const R* res = static_cast<const R*>(a.res) + row * a.n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      nx[i] = load_raw<IO>(x + (i * pl.lanes + l) * kVec, valid[i]);
      nr[i] = load_raw<RO>(res + (i * pl.lanes + l) * kVec, a.res ? valid[i] : 0);
    }
  };
  int64_t row = (int64_t)blockIdx.x * per + tid / pl.lanes;
  fetch(min(row, a.rows - 1));
  for (int64_t first = (int64_t)blockIdx.x * per; first < a.rows; first += step, row += step) {
    Raw<IO> rx[NV];
    Raw<RO> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i] = nx[i];
      rr[i] = nr[i];
    }
    // in place: a row is read by the lanes that write it, and the next one is another
    if (first + step < a.rows) fetch(min(row + step, a.rows - 1));
    float rho_x = 1.0f;
    if (a.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) s[0] = fmaf(value<IO>(rx[i], j), value<IO>(rx[i], j), s[0]);
      row_sums(s, pl.lanes, slot_post);
      rho_x = inv_rms(s[0], a.inv_n, a.eps);
    }
    float sum[2] = {0.0f, 0.0f};                           // (two: the sums of x have a place of their own in LDS)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = fmaf(value<IO>(rx[i], j) * rho_x, by[i][j], value<RO>(rr[i], j));
      rr[i] = pack<RO>(v);                                 // the norm is of the sum as it is kept
#pragma unroll
      for (int j = 0; j < kVec; ++j) sum[0] = fmaf(value<RO>(rr[i], j), value<RO>(rr[i], j), sum[0]);
    }
    row_sums(sum, pl.lanes, slot);
    const float rho = inv_rms(sum[0], a.inv_n, a.eps);
    if (row >= a.rows) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * pl.lanes + l) * kVec;
      if (a.res_out) store_raw<RO>(static_cast<R*>(a.res_out) + row * a.n + e, valid[i], rr[i]);
      float v[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = value<RO>(rr[i], j) * (rho * w[i][j]);
      store_raw<IO>(static_cast<T*>(a.y) + row * a.n + e, valid[i], pack<IO>(v));
    }
  }
}

// With r the kept sum and m what was scaled onto it (x, or rho_x x w_post): dr = dres + the norm's gradient, dm = alpha
// scale dr, dscale = sum of alpha dr m, and for m as the other norm's.
template <typename IO, typename RO, int NV, int THREADS>
__global__ __launch_bounds__(THREADS) void residual_norm_bwd_kernel(ResidualNormArgs a) {
  using T = typename IO::T;
  using R = typename RO::T;
  const NormPlan& pl = a.plan;
  const int tid = threadIdx.x, l = pl.lanes > 64 ? tid : tid & (pl.lanes - 1), per = pl.threads / pl.lanes;
  int slot = 0, slot_post = 0;
  float w[NV][kVec], wp[NV][kVec], by[NV][kVec], dw[NV][kVec] = {}, dp[NV][kVec] = {}, ds[NV][kVec] = {};
  int valid[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * pl.lanes + l) * kVec;
    valid[i] = a.n - at;
    load_weights(a.w, at, valid[i], 1.0f, w[i]);
    load_weights(a.scale, at, valid[i], 1.0f, by[i]);
    load_weights(a.post ? a.w_post : nullptr, at, valid[i], 1.0f, wp[i]);
#pragma unroll
    for (int j = 0; j < kVec; ++j) by[i][j] *= a.alpha;
  }
  const int64_t step = (int64_t)gridDim.x * per;
  Raw<IO> nx[NV], nd[NV];
  Raw<RO> nr[NV], no[NV];
  auto fetch = [&](int64_t row) {
    const int64_t base = row * a.n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * pl.lanes + l) * kVec;
      nd[i] = load_raw<IO>(static_cast<const T*>(a.dy) + base + e, valid[i]);
      nr[i] = load_raw<RO>(static_cast<const R*>(a.res) + base + e, valid[i]);
      no[i] = load_raw<RO>(static_cast<const R*>(a.dres_out) + base + e, a.dres_out ? valid[i] : 0);
      nx[i] = load_raw<IO>(static_cast<const T*>(a.x) + base + e, a.x ? valid[i] : 0);
    }
  };
  int64_t row = (int64_t)blockIdx.x * per + tid / pl.lanes;
  fetch(min(row, a.rows - 1));
  for (int64_t first = (int64_t)blockIdx.x * per; first < a.rows; first += step, row += step) {
    const bool live = row < a.rows;
    const int64_t base = row * a.n;
    Raw<IO> rx[NV], rd[NV];
    Raw<RO> rr[NV], ro[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i] = nx[i];
      rd[i] = nd[i];
      rr[i] = nr[i];
      ro[i] = no[i];
    }
    if (first + step < a.rows) fetch(min(row + step, a.rows - 1));
    float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float r = value<RO>(rr[i], j), x = value<IO>(rx[i], j);
        sum[0] = fmaf(r, r, sum[0]);
        sum[1] = fmaf(value<IO>(rd[i], j) * w[i][j], r, sum[1]);
        sum[2] = fmaf(x, x, sum[2]);
      }
    row_sums(sum, pl.lanes, slot);
    const float rho = inv_rms(sum[0], a.inv_n, a.eps), c = rho * rho * (sum[1] * a.inv_n);
    const float rho_x = a.post ? inv_rms(sum[2], a.inv_n, a.eps) : 1.0f;
    float dm[NV][kVec], s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dr[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float r = value<RO>(rr[i], j), d = value<IO>(rd[i], j), x = value<IO>(rx[i], j) * rho_x;
        dr[j] = fmaf(rho, fmaf(-r, c, d * w[i][j]), value<RO>(ro[i], j));
        if (live) {
          dw[i][j] = fmaf(d, r * rho, dw[i][j]);
          ds[i][j] = fmaf(dr[j], x * wp[i][j], ds[i][j]);
        }
        dm[i][j] = dr[j] * by[i][j];
        if (a.post) {
          if (live) dp[i][j] = fmaf(dm[i][j], x, dp[i][j]);
          dm[i][j] *= wp[i][j];
          s[0] = fmaf(dm[i][j], value<IO>(rx[i], j), s[0]);
        }
      }
      if (live && a.dres) store_raw<RO>(static_cast<R*>(a.dres) + base + (i * pl.lanes + l) * kVec, valid[i], pack<RO>(dr));
    }
    float cx = 0.0f;
    if (a.post) {
      row_sums(s, pl.lanes, slot_post);
      cx = rho_x * rho_x * (s[0] * a.inv_n);
    }
    if (!live || !a.dx) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = rho_x * fmaf(-value<IO>(rx[i], j), cx, dm[i][j]);
      store_raw<IO>(static_cast<T*>(a.dx) + base + (i * pl.lanes + l) * kVec, valid[i], pack<IO>(v));
    }
  }
  if (a.part[0]) block_columns<NV>(dw, pl, a.n, a.part[0] + (int64_t)blockIdx.x * a.n);
  if (a.part[1]) block_columns<NV>(dp, pl, a.n, a.part[1] + (int64_t)blockIdx.x * a.n);
  if (a.part[2]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) ds[i][j] *= a.alpha;
    block_columns<NV>(ds, pl, a.n, a.part[2] + (int64_t)blockIdx.x * a.n);
  }
}

struct Columns {
  const float* part[3];
  float* out[3];
};

// out[y][j] of weights z: the sum of rows of partial sums in a fixed order.  64 threads to a column, four loads ahead.
__global__ __launch_bounds__(1024) void norm_columns_kernel(Columns c, int rows, int n) {
  __shared__ float s_run[64][17];
  const int lane = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + lane;
  const float* p = c.part[blockIdx.z] + (int64_t)blockIdx.y * rows * n;
  float v = 0.0f;
  if (col < n)
#pragma unroll 4
    for (int r = run; r < rows; r += 64) v += p[(int64_t)r * n + col];
  s_run[run][lane] = v;
  __syncthreads();
  if (run < 4) {
#pragma unroll
    for (int k = 4; k < 64; k += 4) v += s_run[run + k][lane];
    s_run[run][lane] = v;
  }
  __syncthreads();
  if (run == 0 && col < n)
    c.out[blockIdx.z][(int64_t)blockIdx.y * n + col] = (s_run[0][lane] + s_run[1][lane]) + (s_run[2][lane] + s_run[3][lane]);
}

hipError_t launch_columns(const Columns& c, int count, int rows, int n, int heads, hipStream_t s) {
  norm_columns_kernel<<<dim3((n + 15) / 16, heads, count), 1024, 0, s>>>(c, rows, n);
  return hipGetLastError();
}

// About as many workgroups as the card holds at once: each takes several rows, with its weights in registers and
// the next row's loads ahead.
NormPlan plan(int64_t rows, int n, int heads_apart, bool backward) {
  NormPlan p{};
  const int vec = (n + kVec - 1) / kVec;
  // two vectors to a lane where a row would not fit a workgroup of 512, and forward where it then fits a wave (the backward has up to
  // three sums for every value of a lane)
  p.vectors = vec > 512 || (!backward && vec > 64 && vec <= 128) ? 2 : 1;
  const int need_lanes = (vec + p.vectors - 1) / p.vectors;
  p.lanes = 1;
  while (p.lanes < need_lanes && p.lanes < 64) p.lanes <<= 1;
  if (need_lanes > 64) p.lanes = (need_lanes + 63) / 64 * 64;
  p.threads = p.lanes > 64 ? p.lanes : 256;
  const int64_t per = p.threads / p.lanes, need = (rows + per - 1) / per;
  int64_t most = 256 * ((backward ? 768 : 1024) / p.threads) / heads_apart;
  if (most < 1) most = 1;
  p.blocks = (int32_t)(need < most ? need : most);
  if (p.blocks < 1) p.blocks = 1;
  return p;
}

// f with the kernel's vectors to a lane and bound on threads.
template <bool BACKWARD, typename F>
hipError_t by_plan(const NormPlan& p, F f) {
  using std::integral_constant;
  if (p.vectors == 1 && p.threads <= 256) {
    f(integral_constant<int, 1>(), integral_constant<int, 256>());
  } else if (p.threads <= 256) {
    if constexpr (!BACKWARD) f(integral_constant<int, 2>(), integral_constant<int, 256>());
  } else if (p.vectors == 2) {
    f(integral_constant<int, 2>(), integral_constant<int, 512>());
  } else {
    f(integral_constant<int, 1>(), integral_constant<int, 512>());
  }
  return hipGetLastError();
}

}  // namespace

NormPlan gated_norm_plan(int64_t rows, int n, int heads_apart, bool backward) { return plan(rows, n, heads_apart, backward); }

NormPlan residual_norm_plan(int64_t rows, int n, bool backward) { return plan(rows, n, 1, backward); }

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t s) {
  const dim3 grid(a.plan.blocks, a.per_head ? a.heads : 1), block(a.plan.threads);
  return by_plan<false>(a.plan, [&](auto nv, auto nt) {
    constexpr int NV = decltype(nv)::value, NT = decltype(nt)::value;
    if (a.io == kIoBf16) {
      if (a.z.p) gated_norm_kernel<BF16, NV, true, NT><<<grid, block, 0, s>>>(a);
      else gated_norm_kernel<BF16, NV, false, NT><<<grid, block, 0, s>>>(a);
    } else {
      if (a.z.p) gated_norm_kernel<F32, NV, true, NT><<<grid, block, 0, s>>>(a);
      else gated_norm_kernel<F32, NV, false, NT><<<grid, block, 0, s>>>(a);
    }
  });
}

hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, float* dw, hipStream_t s) {
  const int heads = a.per_head ? a.heads : 1;
  const dim3 grid(a.plan.blocks, heads), block(a.plan.threads);
  const hipError_t e = by_plan<true>(a.plan, [&](auto nv, auto nt) {
    constexpr int NV = decltype(nv)::value, NT = decltype(nt)::value;
    if (a.io == kIoBf16) {
      if (a.z.p) gated_norm_bwd_kernel<BF16, NV, true, NT><<<grid, block, 0, s>>>(a);
      else gated_norm_bwd_kernel<BF16, NV, false, NT><<<grid, block, 0, s>>>(a);
    } else {
      if (a.z.p) gated_norm_bwd_kernel<F32, NV, true, NT><<<grid, block, 0, s>>>(a);
      else gated_norm_bwd_kernel<F32, NV, false, NT><<<grid, block, 0, s>>>(a);
    }
  });
  return e == hipSuccess && dw ? launch_columns({{a.part}, {dw}}, 1, a.plan.blocks, a.n, heads, s) : e;
}

template <typename F>
static hipError_t by_types(const ResidualNormArgs& a, F f) {
  if (a.io == kIoBf16) return a.rio == kIoBf16 ? f(BF16(), BF16()) : f(BF16(), F32());
  return f(F32(), F32());
}

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t s) {
  return by_types(a, [&](auto io, auto ro) {
    return by_plan<false>(a.plan, [&](auto nv, auto nt) {
      residual_norm_kernel<decltype(io), decltype(ro), decltype(nv)::value, decltype(nt)::value>
          <<<a.plan.blocks, a.plan.threads, 0, s>>>(a);
    });
  });
}

hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a, float* const (&dw)[3], hipStream_t s) {
  hipError_t e = by_types(a, [&](auto io, auto ro) {
    return by_plan<true>(a.plan, [&](auto nv, auto nt) {
      residual_norm_bwd_kernel<decltype(io), decltype(ro), decltype(nv)::value, decltype(nt)::value>
          <<<a.plan.blocks, a.plan.threads, 0, s>>>(a);
    });
  });
  Columns c{};
  int count = 0;
  for (int i = 0; i < 3; ++i) {
    if (!dw[i]) continue;
    c.part[count] = a.part[i];
    c.out[count++] = dw[i];
  }
  return e == hipSuccess && count ? launch_columns(c, count, a.plan.blocks, a.n, 1, s) : e;
}

}  // namespace ssscan
