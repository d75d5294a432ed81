// Norm and position rotation of queries and keys, token-major, for heads whose
// rotated pairs come in runs of K = 2, 4 or 8 (gfx950).
//
// G lanes take the heads of one token in turn.  A lane holds K pairs of a vector: two
// runs of K values (j .. j + K - 1 and the same at + half, or 2 K consecutive ones
// where pairs are adjacent or not rotated), each one vector load; the sum of squares
// crosses the G lanes and nothing else does.  The lane's K angles are formed once for
// all of the token's heads.
#include "qk_device.h"

namespace ssscan {
namespace {

using namespace qk;

// Sum over aligned groups of g lanes (a power of 2), in every lane of the group:
// quad permutes, mirrors of 8 and of 16 lanes, then exchanges across rows.
__device__ __forceinline__ float group_sum(float v, int g) {
  if (g > 1) v += __builtin_amdgcn_update_dpp(0.0f, v, 0xB1, 0xf, 0xf, false);
  if (g > 2) v += __builtin_amdgcn_update_dpp(0.0f, v, 0x4E, 0xf, 0xf, false);
  if (g > 4) v += __builtin_amdgcn_update_dpp(0.0f, v, 0x141, 0xf, 0xf, false);
  if (g > 8) v += __builtin_amdgcn_update_dpp(0.0f, v, 0x140, 0xf, 0xf, false);
  if (g > 16) v += __shfl_xor(v, 16);
  if (g > 32) v += __shfl_xor(v, 32);
  return v;
}

// What a lane has of every vector.
template <int K, bool INTER>
struct Lane {
  int j1, j2;      // first values of its runs
  bool act, rot;   // it has values; they are rotated
  __device__ __forceinline__ Lane(const QkArgs& a, int c) {
    act = c * 2 * K < a.n;
    rot = c * K < a.half;
    const int p = act ? c * K : 0;
    const bool apart = !INTER && rot;
    j1 = apart ? p : 2 * p;
    j2 = apart ? p + a.half : 2 * p + K;
  }
};

// Value h of pair i in a lane's 2 K values.
template <int K, bool INTER>
__device__ __forceinline__ constexpr int at(int i, int h) { return INTER ? 2 * i + h : i + h * K; }

template <typename IO, int K>
__device__ __forceinline__ void load_two(const typename IO::T* __restrict__ p, int j1, int j2, bool act, float (&x)[2 * K]) {
  float u[K] = {}, v[K] = {};
  if (act) {
    load_run<IO, K>(p + j1, u);
    load_run<IO, K>(p + j2, v);
  }
#pragma unroll
  for (int i = 0; i < K; ++i) {
    x[i] = u[i];
    x[K + i] = v[i];
  }
}

template <typename IO, int K>
__device__ __forceinline__ void store_two(typename IO::T* __restrict__ p, int j1, int j2, const float (&x)[2 * K]) {
  float u[K], v[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    u[i] = x[i];
    v[i] = x[K + i];
  }
  store_run<IO, K>(p + j1, u);
  store_run<IO, K>(p + j2, v);
}

template <int K>
__device__ __forceinline__ void load_weight(const float* __restrict__ w, int j1, int j2, float (&v)[2 * K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    v[i] = w ? w[j1 + i] : 1.0f;
    v[K + i] = w ? w[j2 + i] : 1.0f;
  }
}

template <int K>
__device__ __forceinline__ void angles(const QkArgs& a, double pos, int c, bool rot, float (&cs)[K], float (&sn)[K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    cs[i] = 1.0f;
    sn[i] = 0.0f;
    if (rot) angle(pos, a.inv_freq[c * K + i], cs[i], sn[i]);
  }
}

// Heads of a workgroup: heads [y * per, ...) of the queries followed by the keys.
template <typename IO, int K, bool INTER>
__global__ __launch_bounds__(256) void qk_rows_fwd_kernel(QkArgs a, int g, int per) {
  using T = typename IO::T;
  constexpr int U = 4;   // vectors in flight
  const int c = threadIdx.x & (g - 1);
  const Lane<K, INTER> ln(a, c);
  const int64_t tokens = a.batch * a.seqlen;
  const int64_t step = (int64_t)gridDim.x * (256 / g);
  const int first = blockIdx.y * per;
  for (int64_t tok = (int64_t)blockIdx.x * (256 / g) + threadIdx.x / g; tok < tokens; tok += step) {
    const int64_t b = tok / a.seqlen, t = tok - b * a.seqlen;
    float cs[K], sn[K];
    angles<K>(a, position(a, tok, t), c, ln.rot, cs, sn);
    int lo = first, hi = first + per;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const QkSide& sd = a.side[side];
      const int h0 = lo > 0 ? lo : 0, h1 = hi < sd.heads ? hi : sd.heads;
      lo -= sd.heads;
      hi -= sd.heads;
      if (h0 >= h1) continue;
      float w[2 * K];
      load_weight<K>(sd.w, ln.j1, ln.j2, w);
      const T* in = (const T*)sd.in + b * sd.stride[0] + t * sd.stride[1];
      T* out = (T*)sd.out + tok * sd.heads * a.n;
      for (int hb = h0; hb < h1; hb += U) {
        float x[U][2 * K];
#pragma unroll
        for (int u = 0; u < U; ++u)
          load_two<IO, K>(in + (hb + u < h1 ? hb + u : h1 - 1) * sd.stride[2], ln.j1, ln.j2, ln.act, x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (hb + u >= h1) break;
          float sq = 0.0f;
#pragma unroll
          for (int k = 0; k < 2 * K; ++k) sq = fmaf(x[u][k], x[u][k], sq);
          const float rho = inv_norm(group_sum(sq, g), a);
#pragma unroll
          for (int i = 0; i < K; ++i) {
            const int k1 = at<K, INTER>(i, 0), k2 = at<K, INTER>(i, 1);
            const float n1 = x[u][k1] * rho * w[k1], n2 = x[u][k2] * rho * w[k2];
            x[u][k1] = ln.rot ? n1 * cs[i] - n2 * sn[i] : n1;
            x[u][k2] = ln.rot ? fmaf(n2, cs[i], n1 * sn[i]) : n2;
          }
          if (ln.act) store_two<IO, K>(out + (int64_t)(hb + u) * a.n, ln.j1, ln.j2, x[u]);
        }
      }
    }
  }
}

// The backward (its formulas: qk_cols.hip).  A workgroup has heads of one side, and
// keeps the sums of dw of its tokens; blockIdx.y counts the queries' head blocks, then the keys'.
template <typename IO, int K, bool INTER>
__global__ __launch_bounds__(256) void qk_rows_bwd_kernel(QkArgs a, int g, int per, int q_blocks) {
  using T = typename IO::T;
  __shared__ float s_dw[4][256];
  const int side = (int)blockIdx.y >= q_blocks;
  const int block = (int)blockIdx.y - (side ? q_blocks : 0);
  const QkSide& sd = a.side[side];
  const int c = threadIdx.x & (g - 1);
  const Lane<K, INTER> ln(a, c);
  const int64_t tokens = a.batch * a.seqlen;
  const int64_t step = (int64_t)gridDim.x * (256 / g);
  const int h0 = block * per, h1 = h0 + per < sd.heads ? h0 + per : sd.heads;
  float w[2 * K], dw[2 * K] = {};
  load_weight<K>(sd.w, ln.j1, ln.j2, w);
  for (int64_t tok = (int64_t)blockIdx.x * (256 / g) + threadIdx.x / g; tok < tokens; tok += step) {
    const int64_t b = tok / a.seqlen, t = tok - b * a.seqlen;
    float cs[K], sn[K];
    angles<K>(a, position(a, tok, t), c, ln.rot, cs, sn);
    const T* in = (const T*)sd.in + b * sd.stride[0] + t * sd.stride[1];
    T* din = (T*)sd.din + b * sd.dstride[0] + t * sd.dstride[1];
    const T* dout = (const T*)sd.dout + tok * sd.heads * a.n;
    for (int h = h0; h < h1; ++h) {
      float x[2 * K], d[2 * K];
      load_two<IO, K>(in + h * sd.stride[2], ln.j1, ln.j2, ln.act, x);
      load_two<IO, K>(dout + (int64_t)h * a.n, ln.j1, ln.j2, ln.act, d);
      float sq = 0.0f, pv = 0.0f;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int k1 = at<K, INTER>(i, 0), k2 = at<K, INTER>(i, 1);
        const float d1 = d[k1], d2 = d[k2];
        d[k1] = ln.rot ? fmaf(d1, cs[i], d2 * sn[i]) : d1;
        d[k2] = ln.rot ? d2 * cs[i] - d1 * sn[i] : d2;
      }
#pragma unroll
      for (int k = 0; k < 2 * K; ++k) {
        sq = fmaf(x[k], x[k], sq);
        pv = fmaf(d[k] * w[k], x[k], pv);
      }
      const float rho = inv_norm(group_sum(sq, g), a);
      const float back = rho * rho * (group_sum(pv, g) / (float)a.n);
#pragma unroll
      for (int k = 0; k < 2 * K; ++k) {
        dw[k] = fmaf(d[k], rho * x[k], dw[k]);
        x[k] = rho * (d[k] * w[k] - x[k] * back);
      }
      if (ln.act) store_two<IO, K>(din + h * sd.dstride[2], ln.j1, ln.j2, x);
    }
  }
  if (!sd.dw) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < 2 * K; ++k) {
    float v = dw[k];
    for (int m = g; m < 64; m <<= 1) v += __shfl_xor(v, m);
    if (lane < g && ln.act) s_dw[wave][(k < K ? ln.j1 : ln.j2 - K) + k] = v;
  }
  __syncthreads();
  const int j = threadIdx.x;
  if (j < a.n)
    a.part[(a.part_row[side] + (int64_t)block * gridDim.x + blockIdx.x) * a.n + j] =
        (s_dw[0][j] + s_dw[1][j]) + (s_dw[2][j] + s_dw[3][j]);
}

// The longest run that the shape allows: half and the rest's pairs in whole runs, and
// 16 bytes at most.  0: none.
int run_of(const QkArgs& a) {
  for (int k = a.io == kIoBf16 ? 8 : 4; k >= 2; k >>= 1)
    if (a.half % k == 0 && (a.n - 2 * a.half) % (2 * k) == 0) return k;
  return 0;
}

int lanes_of(const QkArgs& a, int k) {
  int g = 1;
  while (g * 2 * k < a.n) g <<= 1;
  return g;
}

struct Shape {
  dim3 grid;
  int g, per, q_blocks;
};

template <typename IO, int K, bool INTER>
void launch(const QkArgs& a, bool back, const Shape& sh, hipStream_t s) {
  if (back) hipLaunchKernelGGL((qk_rows_bwd_kernel<IO, K, INTER>), sh.grid, dim3(256), 0, s, a, sh.g, sh.per, sh.q_blocks);
  else hipLaunchKernelGGL((qk_rows_fwd_kernel<IO, K, INTER>), sh.grid, dim3(256), 0, s, a, sh.g, sh.per);
}

template <typename IO, int K>
void by_pairs(const QkArgs& a, bool back, const Shape& sh, hipStream_t s) {
  if (a.interleaved) launch<IO, K, true>(a, back, sh, s);
  else launch<IO, K, false>(a, back, sh, s);
}

hipError_t go(const QkArgs& a, bool back, int k, const Shape& sh, hipStream_t s) {
  if (a.io == kIoBf16) {
    if (k == 8) by_pairs<BF16, 8>(a, back, sh, s);
    else if (k == 4) by_pairs<BF16, 4>(a, back, sh, s);
    else by_pairs<BF16, 2>(a, back, sh, s);
  } else {
    if (k == 4) by_pairs<F32, 4>(a, back, sh, s);
    else by_pairs<F32, 2>(a, back, sh, s);
  }
  return hipGetLastError();
}

}  // namespace

bool qk_rows_take(const QkArgs& a) { return run_of(a) > 0; }

hipError_t launch_qk_rows(const QkArgs& a, hipStream_t s) {
  const int k = run_of(a);
  const int64_t tokens = a.batch * a.seqlen;
  const int heads = a.side[0].heads + a.side[1].heads;
  Shape sh{};
  sh.g = lanes_of(a, k);
  // all heads of a token in one group, unless that leaves fewer than 2^18 lanes busy
  const int64_t lanes = tokens * sh.g;
  int64_t split = ((int64_t(1) << 18) + lanes - 1) / lanes;
  if (split > heads) split = heads;
  sh.per = (int)((heads + split - 1) / split);
  int64_t blocks = (tokens + 256 / sh.g - 1) / (256 / sh.g);
  if (blocks > (1 << 20)) blocks = 1 << 20;
  sh.grid = dim3((unsigned)blocks, (unsigned)((heads + sh.per - 1) / sh.per));
  if (sh.grid.y > 65535) {
    sh.per = (heads + 65534) / 65535;
    sh.grid.y = (unsigned)((heads + sh.per - 1) / sh.per);
  }
  return go(a, false, k, sh, s);
}

hipError_t launch_qk_rows_bwd(QkArgs& a, const QkBwdPlan& p, hipStream_t s) {
  const int k = run_of(a);
  Shape sh{};
  sh.g = lanes_of(a, k);
  sh.per = p.heads_per_block;
  sh.q_blocks = p.blocks[0];
  int64_t blocks = (a.batch * a.seqlen + 256 / sh.g - 1) / (256 / sh.g);
  if (blocks > p.token_blocks) blocks = p.token_blocks;
  sh.grid = dim3((unsigned)blocks, (unsigned)(p.blocks[0] + p.blocks[1]));
  for (int i = 0; i < 2; ++i) a.part_rows[i] = blocks * p.blocks[i];
  a.part_row[1] = a.part_rows[0];
  return go(a, true, k, sh, s);
}

}  // namespace ssscan
