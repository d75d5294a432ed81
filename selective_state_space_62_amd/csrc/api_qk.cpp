// C ABI of the norm and rotation of queries and keys: argument checks and launches.  See include/ssscan.h.
#include <cmath>
#include <utility>

#include "api_checks.h"
#include "internal.h"
#include "qk_norm_rot.h"

namespace {

using namespace ssscan;

constexpr int kMaxHeadDim = 256;
constexpr int kMaxHeads = 1 << 20;
constexpr int64_t kMaxPosition = int64_t(1) << 53;   // exact in fp64

bool scan_dstate(int n) { return n == 1 || n == 2 || n == 4 || n == 8 || n == 16; }

ss_status check_sizes(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int head_dim) {
  if (batch < 1 || seqlen < 0)
    return record_error(SS_ERR_INVALID_ARG, "sizes must be batch >= 1, seqlen >= 0 (got %lld, %lld)",
                        (long long)batch, (long long)seqlen);
  if (heads_q < 0 || heads_k < 0 || heads_q + (int64_t)heads_k < 1 || heads_q > kMaxHeads || heads_k > kMaxHeads)
    return record_error(SS_ERR_INVALID_ARG, "head counts must be 0 to 2^20 and not both 0 (got %d, %d)", heads_q,
                        heads_k);
  if (head_dim < 1 || head_dim > kMaxHeadDim)
    return record_error(SS_ERR_UNSUPPORTED, "head_dim %d is not 1 to %d", head_dim, kMaxHeadDim);
  if (batch > kMaxDim || seqlen > kMaxDim ||
      (__int128)batch * (seqlen > 0 ? seqlen : 1) * (heads_q + (int64_t)heads_k) * head_dim * 8 > ((__int128)1 << 62))
    return record_error(SS_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte offsets");
  return SS_OK;
}

// Elements from the first to one past the last value under these strides, or -1
// where that overflows.
int64_t span_of(int64_t batch, int64_t seqlen, int heads, int n, const int64_t* st) {
  if (heads == 0 || seqlen == 0) return 0;
  __int128 last = n;
  last += (__int128)(batch - 1) * st[0] + (__int128)(seqlen - 1) * st[1] + (__int128)(heads - 1) * st[2];
  return last > ((__int128)1 << 58) ? -1 : (int64_t)last;
}

ss_status check_side(const char* name, const void* p, const int64_t* st, int64_t batch, int64_t seqlen, int heads,
                     int n, ss_dtype io, int64_t* span) {
  *span = 0;
  if (heads == 0) {
    if (p) return record_error(SS_ERR_INVALID_ARG, "%s is given with 0 heads", name);
    return SS_OK;
  }
  if (!st) return record_error(SS_ERR_INVALID_ARG, "%s has no strides", name);
  if (seqlen > 0 && !p) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, elem_bytes(io))) return record_error(SS_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  for (int k = 0; k < 3; ++k)
    if (st[k] < 0)
      return record_error(SS_ERR_INVALID_ARG, "%s has a negative stride (%lld)", name, (long long)st[k]);
  *span = span_of(batch, seqlen, heads, n, st);
  if (*span < 0) return record_error(SS_ERR_INVALID_ARG, "the strides of %s overflow 64-bit byte offsets", name);
  return SS_OK;
}

// Whether runs of n values, one for each index of D dimensions, are disjoint: by stride,
// ascending, each dimension has to step over all that the ones before it reach.
template <int D>
bool distinct(int64_t n, int64_t (&size)[D], int64_t (&stride)[D]) {
  for (int i = 0; i < D; ++i)
    for (int j = i + 1; j < D; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(size[i], size[j]);
      }
  int64_t reach = n;
  for (int i = 0; i < D; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < reach) return false;
    reach += stride[i] * (size[i] - 1);
  }
  return true;
}

// Whether two strided gradients, each without shared addresses and dk's first value `apart` after
// dq's, share none: with the same batch and token strides, either all heads of the one lie behind
// those of the other in each token's columns, or their heads alternate under one head stride.
bool columns_of_one(int64_t batch, int64_t seqlen, int n, int heads_q, const int64_t* sq, int heads_k,
                    const int64_t* sk, int64_t apart) {
  if ((batch > 1 && sq[0] != sk[0]) || (seqlen > 1 && sq[1] != sk[1])) return false;
  const int64_t eq = (heads_q - 1) * sq[2] + n, ek = (heads_k - 1) * sk[2] + n;
  if (apart >= 0 ? apart >= eq : -apart >= ek) {
    const int64_t lo = apart < 0 ? apart : 0, hi = apart + ek > eq ? apart + ek : eq;
    int64_t size[] = {batch, seqlen}, stride[] = {sq[0], sq[1]};
    if (distinct(hi - lo, size, stride)) return true;
  }
  if (heads_q > 1 && heads_k > 1 && sq[2] != sk[2]) return false;
  int64_t size[] = {batch, seqlen, heads_q > heads_k ? heads_q : heads_k, 2};
  int64_t stride[] = {sq[0], sq[1], heads_q > 1 ? sq[2] : sk[2], apart < 0 ? -apart : apart};
  return distinct(n, size, stride);
}

ss_status check_common(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int head_dim, int rot_dim, ss_dtype io,
                       uint32_t flags, float eps, const void* q, const int64_t* q_stride, const void* k,
                       const int64_t* k_stride, const float* wq, const float* wk, const double* inv_freq,
                       const int64_t* positions, int64_t pos0, int64_t* q_span, int64_t* k_span) {
  if (io != SS_F32 && io != SS_BF16)
    return record_error(SS_ERR_UNSUPPORTED, "io dtype %d is not SS_F32 or SS_BF16", (int)io);
  if (flags & ~(uint32_t)(SS_QK_INTERLEAVED | SS_QK_FEATURE_MAJOR))
    return record_error(SS_ERR_UNSUPPORTED, "unknown flags 0x%x", (unsigned)flags);
  ss_status st = check_sizes(batch, seqlen, heads_q, heads_k, head_dim);
  if (st != SS_OK) return st;
  if ((flags & SS_QK_FEATURE_MAJOR) && !scan_dstate(head_dim))
    return record_error(SS_ERR_UNSUPPORTED, "head_dim %d is not one of 1, 2, 4, 8, 16 (feature-major)", head_dim);
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2)
    return record_error(SS_ERR_INVALID_ARG, "rot_dim %d is not even and 0 to head_dim (%d)", rot_dim, head_dim);
  if (!(eps > 0.0f) || !std::isnormal(eps))
    return record_error(SS_ERR_INVALID_ARG, "eps %g is not a positive normal number", (double)eps);
  if (!positions && (pos0 < -kMaxPosition || pos0 > kMaxPosition - seqlen))
    return record_error(SS_ERR_INVALID_ARG, "positions from pos0 %lld on are past 2^53", (long long)pos0);
  if (rot_dim > 0 && !inv_freq) return record_error(SS_ERR_INVALID_ARG, "inv_freq is NULL");
  if (!aligned(inv_freq, 8) || !aligned(positions, 8))
    return record_error(SS_ERR_INVALID_ARG, "%s is not 8-byte aligned", aligned(inv_freq, 8) ? "positions" : "inv_freq");
  if (!aligned(wq, 4) || !aligned(wk, 4))
    return record_error(SS_ERR_INVALID_ARG, "%s is not 4-byte aligned", aligned(wq, 4) ? "wk" : "wq");
  if ((st = check_side("q", q, q_stride, batch, seqlen, heads_q, head_dim, io, q_span)) != SS_OK) return st;
  return check_side("k", k, k_stride, batch, seqlen, heads_k, head_dim, io, k_span);
}

QkArgs make_args(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int head_dim, int rot_dim, ss_dtype io,
                 uint32_t flags, float eps, const void* q, const int64_t* q_stride, const void* k,
                 const int64_t* k_stride, const float* wq, const float* wk, const double* inv_freq,
                 const int64_t* positions, int64_t pos0) {
  QkArgs a{};
  a.batch = batch;
  a.seqlen = seqlen;
  a.n = head_dim;
  a.half = rot_dim / 2;
  a.io = io == SS_BF16 ? kIoBf16 : kIoF32;
  a.interleaved = (flags & SS_QK_INTERLEAVED) != 0;
  a.feature_major = (flags & SS_QK_FEATURE_MAJOR) != 0;
  a.eps = eps;
  a.inv_n = 1.0f / (float)head_dim;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.pos0 = pos0;
  const void* in[2] = {q, k};
  const int64_t* st[2] = {q_stride, k_stride};
  const float* w[2] = {wq, wk};
  const int heads[2] = {heads_q, heads_k};
  for (int i = 0; i < 2; ++i) {
    a.side[i].heads = heads[i];
    a.side[i].in = in[i];
    a.side[i].w = w[i];
    for (int j = 0; j < 3; ++j) a.side[i].stride[j] = heads[i] ? st[i][j] : 0;
  }
  return a;
}

}  // namespace

extern "C" {

ss_status ss_qk_norm_rot(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int head_dim, int rot_dim,
                         ss_dtype io, uint32_t flags, float eps, const void* q, const int64_t* q_stride, const void* k,
                         const int64_t* k_stride, const float* wq, const float* wk, const double* inv_freq,
                         const int64_t* positions, int64_t pos0, void* q_out, void* k_out, void* stream) {
  int64_t q_span, k_span;
  ss_status st = check_common(batch, seqlen, heads_q, heads_k, head_dim, rot_dim, io, flags, eps, q, q_stride, k,
                              k_stride, wq, wk, inv_freq, positions, pos0, &q_span, &k_span);
  if (st != SS_OK) return st;
  const int64_t eb = elem_bytes(io), tokens = batch * seqlen;
  void* out[2] = {q_out, k_out};
  const int heads[2] = {heads_q, heads_k};
  const char* names[2] = {"q_out", "k_out"};
  for (int i = 0; i < 2; ++i) {
    if ((heads[i] == 0) != (out[i] == nullptr) && (heads[i] == 0 || tokens > 0))
      return record_error(SS_ERR_INVALID_ARG, "%s is %s", names[i], out[i] ? "given with 0 heads" : "NULL");
    if (!aligned(out[i], 16)) return record_error(SS_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
  }
  const Range ins[] = {rng("q", q, q_span * eb), rng("k", k, k_span * eb), rng("wq", wq, head_dim * 4),
                       rng("wk", wk, head_dim * 4), rng("inv_freq", inv_freq, rot_dim * 4),
                       rng("positions", positions, tokens * 8)};
  const Range outs[] = {rng("q_out", q_out, tokens * heads_q * head_dim * eb),
                        rng("k_out", k_out, tokens * heads_k * head_dim * eb)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return record_error(SS_ERR_INVALID_ARG, "%s overlaps input %s", o.name, i.name);
  if (overlap(outs[0], outs[1])) return record_error(SS_ERR_INVALID_ARG, "q_out overlaps k_out");
  if (tokens == 0) return SS_OK;
  QkArgs a = make_args(batch, seqlen, heads_q, heads_k, head_dim, rot_dim, io, flags, eps, q, q_stride, k, k_stride,
                       wq, wk, inv_freq, positions, pos0);
  for (int i = 0; i < 2; ++i) a.side[i].out = out[i];
  const hipError_t e = launch_qk_norm_rot(a, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? SS_OK : record_hip_error(e, "norm and rotation launch");
}

size_t ss_qk_norm_rot_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int head_dim) {
  if (check_sizes(batch, seqlen, heads_q, heads_k, head_dim) != SS_OK || seqlen == 0) return 0;
  const QkBwdPlan p = qk_bwd_plan(batch, seqlen, heads_q, heads_k, head_dim);
  return round256((size_t)(p.blocks[0] + p.blocks[1]) * head_dim * sizeof(float));
}

ss_status ss_qk_norm_rot_bwd(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int head_dim, int rot_dim,
                             ss_dtype io, uint32_t flags, float eps, const void* q, const int64_t* q_stride,
                             const void* k, const int64_t* k_stride, const float* wq, const float* wk,
                             const double* inv_freq, const int64_t* positions, int64_t pos0, const void* dq_out,
                             const void* dk_out, void* dq, const int64_t* dq_stride, void* dk,
                             const int64_t* dk_stride, float* dwq, float* dwk, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int64_t q_span, k_span, dq_span, dk_span;
  ss_status st = check_common(batch, seqlen, heads_q, heads_k, head_dim, rot_dim, io, flags, eps, q, q_stride, k,
                              k_stride, wq, wk, inv_freq, positions, pos0, &q_span, &k_span);
  if (st != SS_OK) return st;
  if ((st = check_side("dq", dq, dq_stride, batch, seqlen, heads_q, head_dim, io, &dq_span)) != SS_OK) return st;
  if ((st = check_side("dk", dk, dk_stride, batch, seqlen, heads_k, head_dim, io, &dk_span)) != SS_OK) return st;
  const int64_t eb = elem_bytes(io), tokens = batch * seqlen;
  const void* dout[2] = {dq_out, dk_out};
  void* din[2] = {dq, dk};
  const int64_t* dst[2] = {dq_stride, dk_stride};
  float* dw[2] = {dwq, dwk};
  const int heads[2] = {heads_q, heads_k};
  const char* names[2] = {"dq_out", "dk_out"};
  for (int i = 0; i < 2; ++i) {
    if ((heads[i] == 0) != (dout[i] == nullptr) && (heads[i] == 0 || tokens > 0))
      return record_error(SS_ERR_INVALID_ARG, "%s is %s", names[i], dout[i] ? "given with 0 heads" : "NULL");
    if (!aligned(dout[i], 16)) return record_error(SS_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
    if (heads[i] == 0 && dw[i])
      return record_error(SS_ERR_INVALID_ARG, "%s is given with 0 heads", i ? "dwk" : "dwq");
    if (!aligned(dw[i], 4)) return record_error(SS_ERR_INVALID_ARG, "%s is not 4-byte aligned", i ? "dwk" : "dwq");
    if (heads[i]) {
      int64_t size[] = {batch, seqlen, heads[i]}, stride[] = {dst[i][0], dst[i][1], dst[i][2]};
      if (!distinct(head_dim, size, stride))
        return record_error(SS_ERR_INVALID_ARG, "values of %s share addresses under its strides", i ? "dk" : "dq");
    }
  }
  const size_t need = ss_qk_norm_rot_bwd_workspace_bytes(batch, seqlen, heads_q, heads_k, head_dim);
  if (need > 0) {
    if (!workspace) return record_error(SS_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (!aligned(workspace, 256)) return record_error(SS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (workspace_bytes < need)
      return record_error(SS_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace_bytes, need);
  }
  const Range ins[] = {rng("q", q, q_span * eb), rng("k", k, k_span * eb), rng("wq", wq, head_dim * 4),
                       rng("wk", wk, head_dim * 4), rng("inv_freq", inv_freq, rot_dim * 4),
                       rng("positions", positions, tokens * 8),
                       rng("dq_out", dq_out, tokens * heads_q * head_dim * eb),
                       rng("dk_out", dk_out, tokens * heads_k * head_dim * eb)};
  const Range outs[] = {rng("dq", dq, dq_span * eb), rng("dk", dk, dk_span * eb), rng("dwq", dwq, head_dim * 4),
                        rng("dwk", dwk, head_dim * 4), rng("workspace", workspace, (int64_t)need)};
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return record_error(SS_ERR_INVALID_ARG, "%s overlaps input %s", o.name, i.name);
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j) {
      if (!overlap(outs[i], outs[j])) continue;
      const int64_t apart = (int64_t)(outs[1].lo - outs[0].lo);
      if (i == 0 && j == 1 && apart % eb == 0 &&
          columns_of_one(batch, seqlen, head_dim, heads_q, dq_stride, heads_k, dk_stride, apart / eb))
        continue;
      return record_error(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (tokens == 0) {
    for (float* p : dw) {
      const hipError_t e = launch_fill_zero(p, head_dim, s);
      if (e != hipSuccess) return record_hip_error(e, "zero-fill launch");
    }
    return SS_OK;
  }
  QkArgs a = make_args(batch, seqlen, heads_q, heads_k, head_dim, rot_dim, io, flags, eps, q, q_stride, k, k_stride,
                       wq, wk, inv_freq, positions, pos0);
  for (int i = 0; i < 2; ++i) {
    a.side[i].dout = dout[i];
    a.side[i].din = din[i];
    a.side[i].dw = dw[i];
    for (int j = 0; j < 3; ++j) a.side[i].dstride[j] = heads[i] ? dst[i][j] : 0;
  }
  a.part = static_cast<float*>(workspace);
  const hipError_t e = launch_qk_norm_rot_bwd(a, s);
  return e == hipSuccess ? SS_OK : record_hip_error(e, "norm and rotation backward launch");
}

}  // extern "C"
