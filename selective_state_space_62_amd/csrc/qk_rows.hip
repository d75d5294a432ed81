// Norm and position rotation of queries and keys, token-major, for heads whose
// rotated pairs come in runs of K = 2, 4 or 8 (gfx950).
//
// A workgroup takes the heads of one side (queries or keys) of some consecutive
// tokens, so that it reads and writes runs of whole rows.  Its threads first put the
// tokens' cosines and sines into LDS, each formed once; then G lanes take a vector
// (one head of one token) at a time.  A lane holds K pairs of it: two runs of K values (j .. j + K - 1
// and the same at + half, or 2 K consecutive ones where pairs are adjacent or not
// rotated), each one vector load; the sum of squares crosses the G lanes and nothing
// else does.
#include "qk_device.h"

namespace ssscan {
namespace {

using namespace qk;

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

constexpr int kThreads = 256;
constexpr int kAngles = 2048;   // pairs of a workgroup's tokens
constexpr int kTokens = 64;     // most tokens of a workgroup

// The tokens of a workgroup: cosines and sines, and where the tokens' rows start.
struct Tokens {
  float cos[kAngles], sin[kAngles];
  double pos[kTokens];
  int64_t in[kTokens], din[kTokens];

  __device__ __forceinline__ void fill(const QkArgs& a, const QkSide& sd, int64_t tok0, int count) {
    if ((int)threadIdx.x < count) {
      const int64_t tok = tok0 + threadIdx.x, b = tok / a.seqlen, t = tok - b * a.seqlen;
      pos[threadIdx.x] = position(a, tok, t);
      in[threadIdx.x] = b * sd.stride[0] + t * sd.stride[1];
      din[threadIdx.x] = b * sd.dstride[0] + t * sd.dstride[1];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < count * a.half; k += kThreads) {
      const int l = k / a.half, p = k - l * a.half;
      float c, s;
      angle(pos[l], a.inv_freq[p], c, s);
      cos[k] = c;
      sin[k] = s;
    }
  }
};

template <int K>
__device__ __forceinline__ void load_angles(const Tokens& tk, int at, float (&cs)[K], float (&sn)[K]) {
  const Run<F32, K> c = *reinterpret_cast<const Run<F32, K>*>(tk.cos + at);
  const Run<F32, K> s = *reinterpret_cast<const Run<F32, K>*>(tk.sin + at);
#pragma unroll
  for (int i = 0; i < K; ++i) {
    cs[i] = c.v[i];
    sn[i] = s.v[i];
  }
}

// blockIdx.x counts the queries' token blocks, then the keys'.
template <typename IO, int K, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_rows_fwd_kernel(QkArgs a, QkRowsShape sh) {
  using T = typename IO::T;
  __shared__ Tokens tk;
  const int side = (int)blockIdx.x >= sh.blocks[0];
  const QkSide& sd = a.side[side];
  const int g = sh.lanes, groups = kThreads / g, mine = threadIdx.x / g;
  const int c = threadIdx.x & (g - 1);
  const Lane<K, INTER> ln(a, c);
  float w[2 * K];
  load_weight<K>(sd.w, ln.j1, ln.j2, w);
  const int64_t tokens = a.batch * a.seqlen;
  const int64_t step = (int64_t)sh.blocks[side] * sh.tokens[side];
  for (int64_t tok0 = (int64_t)((int)blockIdx.x - (side ? sh.blocks[0] : 0)) * sh.tokens[side]; tok0 < tokens; tok0 += step) {
    const int count = (int)(tokens - tok0 < sh.tokens[side] ? tokens - tok0 : sh.tokens[side]);
    tk.fill(a, sd, tok0, count);
    __syncthreads();
    const int items = count * sd.heads;
    T* out = (T*)sd.out + tok0 * sd.heads * a.n;
    for (int it = mine; it < items; it += groups) {
      const int tl = it / sd.heads;
      float x[2 * K], cs[K], sn[K];
      load_two<IO, K>((const T*)sd.in + tk.in[tl] + (it - tl * sd.heads) * sd.stride[2], ln.j1, ln.j2, ln.act, x);
      if (ln.rot) load_angles<K>(tk, tl * a.half + c * K, cs, sn);
      float sq = 0.0f;
#pragma unroll
      for (int k = 0; k < 2 * K; ++k) sq = fmaf(x[k], x[k], sq);
      const float rho = inv_norm(group_sum(sq, g), a);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int k1 = at<K, INTER>(i, 0), k2 = at<K, INTER>(i, 1);
        const float n1 = x[k1] * rho * w[k1], n2 = x[k2] * rho * w[k2];
        x[k1] = ln.rot ? n1 * cs[i] - n2 * sn[i] : n1;
        x[k2] = ln.rot ? fmaf(n2, cs[i], n1 * sn[i]) : n2;
      }
      if (ln.act) store_two<IO, K>(out + (int64_t)it * a.n, ln.j1, ln.j2, x);
    }
    __syncthreads();
  }
}

// The backward (its formulas: qk_cols.hip); a workgroup keeps its sums of dw.
template <typename IO, int K, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_rows_bwd_kernel(QkArgs a, QkRowsShape sh) {
  using T = typename IO::T;
  __shared__ Tokens tk;
  __shared__ float s_dw[4][256];
  const int side = (int)blockIdx.x >= sh.blocks[0];
  const int block = (int)blockIdx.x - (side ? sh.blocks[0] : 0);
  const QkSide& sd = a.side[side];
  const int g = sh.lanes, groups = kThreads / g, mine = threadIdx.x / g;
  const int c = threadIdx.x & (g - 1);
  const Lane<K, INTER> ln(a, c);
  float w[2 * K], dw[2 * K] = {};
  load_weight<K>(sd.w, ln.j1, ln.j2, w);
  const int64_t tokens = a.batch * a.seqlen;
  const int64_t step = (int64_t)sh.blocks[side] * sh.tokens[side];
  for (int64_t tok0 = (int64_t)block * sh.tokens[side]; tok0 < tokens; tok0 += step) {
    const int count = (int)(tokens - tok0 < sh.tokens[side] ? tokens - tok0 : sh.tokens[side]);
    tk.fill(a, sd, tok0, count);
    __syncthreads();
    const int items = count * sd.heads;
    const T* dout = (const T*)sd.dout + tok0 * sd.heads * a.n;
    for (int it = mine; it < items; it += groups) {
      const int tl = it / sd.heads, h = it - tl * sd.heads;
      float x[2 * K], d[2 * K], cs[K], sn[K];
      load_two<IO, K>((const T*)sd.in + tk.in[tl] + h * sd.stride[2], ln.j1, ln.j2, ln.act, x);
      load_two<IO, K>(dout + (int64_t)it * a.n, ln.j1, ln.j2, ln.act, d);
      if (ln.rot) load_angles<K>(tk, tl * a.half + c * K, cs, sn);
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
      const float back = rho * rho * (group_sum(pv, g) * a.inv_n);
#pragma unroll
      for (int k = 0; k < 2 * K; ++k) {
        dw[k] = fmaf(d[k], rho * x[k], dw[k]);
        x[k] = rho * (d[k] * w[k] - x[k] * back);
      }
      if (ln.act) store_two<IO, K>((T*)sd.din + tk.din[tl] + h * sd.dstride[2], ln.j1, ln.j2, x);
    }
    __syncthreads();
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
    a.part[(a.part_row[side] + block) * a.n + j] = (s_dw[0][j] + s_dw[1][j]) + (s_dw[2][j] + s_dw[3][j]);
}

// The longest run that the shape allows: half and the rest's pairs in whole runs, and 16
// bytes at most (40 bf16 heads of 128 at 16384 tokens, forward: runs of 4 73, of 8 68 us); in the
// backward 4 values, whose registers leave room for more waves (6 bf16 heads of 128 at 21879 tokens: runs
// of 8 43.8, of 4 35.2 us; 40 at 16384 142.9 and 141.3 us).  0: none.
int run_of(const QkArgs& a, bool back) {
  for (int k = a.io == kIoBf16 && !back ? 8 : 4; k >= 2; k >>= 1)
    if (a.half % k == 0 && (a.n - 2 * a.half) % (2 * k) == 0) return k;
  return 0;
}

int lanes_of(const QkArgs& a, int k) {
  int g = 1;
  while (g * 2 * k < a.n) g <<= 1;
  return g;
}

// A workgroup's tokens.  Forward: two rounds of vectors for its groups of lanes, fewer
// where the tokens would not give 1024 workgroups.  (40 bf16 heads of 128 at 16384 tokens: one
// round 76, two 68, three 69 us; two or four vectors in flight to a group, which cost
// waves their registers, 71 and 80 us.)  Backward, where the workgroups are few and keep
// their sums: an equal share of the tokens, in as few turns as the angles' LDS allows.
QkRowsShape shape_of(const QkArgs& a, int k, bool back, const int64_t (&most)[2]) {
  QkRowsShape sh{};
  const int64_t tokens = a.batch * a.seqlen;
  sh.lanes = lanes_of(a, k);
  const int groups = kThreads / sh.lanes;
  const int64_t cap = a.half && kAngles / a.half < kTokens ? kAngles / a.half : kTokens;
  for (int i = 0; i < 2; ++i) {
    const int heads = a.side[i].heads;
    sh.tokens[i] = 1;
    if (!heads) continue;
    int64_t n;
    if (back) {
      const int64_t share = (tokens + most[i] - 1) / most[i], turns = (share + cap - 1) / cap;
      const int64_t least = (groups + heads - 1) / heads;
      n = (share + turns - 1) / turns;
      if (n < least) n = least;
    } else {
      n = (2 * groups + heads - 1) / heads;
      if (n > tokens / 1024) n = tokens / 1024;
    }
    if (n > cap) n = cap;
    sh.tokens[i] = n > 1 ? (int)n : 1;
    const int64_t blocks = (tokens + sh.tokens[i] - 1) / sh.tokens[i];
    sh.blocks[i] = (int)(blocks < most[i] ? blocks : most[i]);
  }
  return sh;
}

template <typename IO, int K, bool INTER>
void launch(const QkArgs& a, bool back, const QkRowsShape& sh, hipStream_t s) {
  const dim3 g((unsigned)(sh.blocks[0] + sh.blocks[1]));
  if constexpr (K <= 4) {
    if (back) {
      hipLaunchKernelGGL((qk_rows_bwd_kernel<IO, K, INTER>), g, dim3(kThreads), 0, s, a, sh);
      return;
    }
  }
  hipLaunchKernelGGL((qk_rows_fwd_kernel<IO, K, INTER>), g, dim3(kThreads), 0, s, a, sh);
}

template <typename IO, int K>
void by_pairs(const QkArgs& a, bool back, const QkRowsShape& sh, hipStream_t s) {
  if (a.interleaved) launch<IO, K, true>(a, back, sh, s);
  else launch<IO, K, false>(a, back, sh, s);
}

hipError_t go(const QkArgs& a, bool back, int k, const QkRowsShape& sh, hipStream_t s) {
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

bool qk_rows_take(const QkArgs& a) { return run_of(a, false) > 0; }

hipError_t launch_qk_rows(const QkArgs& a, hipStream_t s) {
  const int k = run_of(a, false);
  return go(a, false, k, shape_of(a, k, false, {1 << 20, 1 << 20}), s);
}

hipError_t launch_qk_rows_bwd(QkArgs& a, const QkBwdPlan& p, hipStream_t s) {
  const int k = run_of(a, true);
  const QkRowsShape sh = shape_of(a, k, true, p.blocks);
  for (int i = 0; i < 2; ++i) a.part_rows[i] = sh.blocks[i];
  a.part_row[1] = a.part_rows[0];
  return go(a, true, k, sh, s);
}

}  // namespace ssscan
