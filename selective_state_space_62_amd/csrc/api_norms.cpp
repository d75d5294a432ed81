// C ABI of the norms before and after a block: argument checks and launches.  See include/ssscan.h.
#include <cmath>

#include "api_rows.h"
#include "norms.h"

namespace {

using namespace ssscan;

constexpr int kMaxN = 8192;
constexpr int kMaxHeads = 1 << 20;
constexpr int64_t kMaxRows = int64_t(1) << 32;   // counted in 32 bits

ss_status check_sizes(int64_t batch, int64_t seqlen, int heads, int n) {
  if (batch < 1 || seqlen < 0)
    return record_error(SS_ERR_INVALID_ARG, "sizes must be batch >= 1, seqlen >= 0 (got %lld, %lld)",
                        (long long)batch, (long long)seqlen);
  if (heads < 1 || heads > kMaxHeads) return record_error(SS_ERR_INVALID_ARG, "heads %d is not 1 to 2^20", heads);
  if (n < 1 || n > kMaxN) return record_error(SS_ERR_UNSUPPORTED, "row length %d is not 1 to %d", n, kMaxN);
  if (batch > kMaxDim || seqlen > kMaxDim || (__int128)batch * seqlen * heads >= kMaxRows)
    return record_error(SS_ERR_UNSUPPORTED, "2^32 rows and more are not supported");
  return SS_OK;
}

ss_status check_common(ss_dtype io, uint32_t flags, uint32_t known, float eps) {
  if (io != SS_F32 && io != SS_BF16)
    return record_error(SS_ERR_UNSUPPORTED, "io dtype %d is not SS_F32 or SS_BF16", (int)io);
  if (flags & ~known) return record_error(SS_ERR_UNSUPPORTED, "unknown flags 0x%x", (unsigned)flags);
  if (!(eps > 0.0f) || !std::isnormal(eps))
    return record_error(SS_ERR_INVALID_ARG, "eps %g is not a positive normal number", (double)eps);
  return SS_OK;
}

constexpr uint32_t kGatedFlags = SS_NORM_GATE_FIRST | SS_NORM_HEAD_WEIGHTS;

GatedNormArgs make_gated(int64_t batch, int64_t seqlen, int heads, int n, ss_dtype io, uint32_t flags, float eps,
                         const float* w) {
  GatedNormArgs a{};
  a.tokens = batch * seqlen;
  a.seqlen = seqlen;
  a.heads = heads;
  a.n = n;
  a.io = io == SS_BF16 ? kIoBf16 : kIoF32;
  a.gate_first = (flags & SS_NORM_GATE_FIRST) != 0;
  a.per_head = (flags & SS_NORM_HEAD_WEIGHTS) != 0;
  a.eps = eps;
  a.inv_n = 1.0f / (float)n;
  a.w = w;
  return a;
}

NormRows rows_of(const void* p, const int64_t* st) {
  NormRows r{p, {0, 0, 0}};
  if (p)
    for (int i = 0; i < 3; ++i) r.stride[i] = st[i];
  return r;
}

NormPlan gated_plan(int64_t tokens, int heads, int n, uint32_t flags, bool backward) {
  const bool apart = (flags & SS_NORM_HEAD_WEIGHTS) != 0;
  return gated_norm_plan(apart ? tokens : tokens * heads, n, apart ? heads : 1, backward);
}

ss_status check_residual(int64_t rows, int n, ss_dtype io, ss_dtype rio, uint32_t flags, float eps, float alpha,
                         const float* w, const float* w_post, const float* scale) {
  ss_status st = check_common(io, flags, SS_NORM_POST, eps);
  if (st != SS_OK) return st;
  if (rio != SS_F32 && rio != io)
    return record_error(SS_ERR_UNSUPPORTED, "residual dtype %d is neither SS_F32 nor the io dtype", (int)rio);
  if (rows < 0) return record_error(SS_ERR_INVALID_ARG, "rows %lld is negative", (long long)rows);
  if ((st = check_sizes(1, rows, 1, n)) != SS_OK) return st;
  if (!std::isfinite(alpha)) return record_error(SS_ERR_INVALID_ARG, "alpha %g is not finite", (double)alpha);
  if (w_post && !(flags & SS_NORM_POST)) return record_error(SS_ERR_INVALID_ARG, "w_post is given without SS_NORM_POST");
  const struct { const char* name; const float* p; } vecs[] = {{"w", w}, {"w_post", w_post}, {"scale", scale}};
  for (const auto& v : vecs)
    if (!aligned(v.p, 4)) return record_error(SS_ERR_INVALID_ARG, "%s is not 4-byte aligned", v.name);
  return SS_OK;
}

ResidualNormArgs make_residual(int64_t rows, int n, ss_dtype io, ss_dtype rio, uint32_t flags, float eps, float alpha,
                               const void* x, const void* res, const float* w, const float* w_post, const float* scale) {
  ResidualNormArgs a{};
  a.rows = rows;
  a.n = n;
  a.io = io == SS_BF16 ? kIoBf16 : kIoF32;
  a.rio = rio == SS_BF16 ? kIoBf16 : kIoF32;
  a.post = (flags & SS_NORM_POST) != 0;
  a.eps = eps;
  a.inv_n = 1.0f / (float)n;
  a.alpha = alpha;
  a.x = x;
  a.res = res;
  a.w = w;
  a.w_post = w_post;
  a.scale = scale;
  return a;
}

}  // namespace

extern "C" {

ss_status ss_gated_norm(int64_t batch, int64_t seqlen, int heads, int n, ss_dtype io, uint32_t flags, float eps,
                        const void* x, const int64_t* x_stride, const void* z, const int64_t* z_stride, const float* w,
                        void* y, void* stream) {
  ss_status st = check_common(io, flags, kGatedFlags, eps);
  if (st != SS_OK) return st;
  if ((st = check_sizes(batch, seqlen, heads, n)) != SS_OK) return st;
  int64_t sx, sz = 0;
  const int64_t eb = elem_bytes(io), tokens = batch * seqlen;
  if ((st = check_rows("x", x, x_stride, batch, seqlen, heads, n, io, &sx)) != SS_OK) return st;
  if (z && (st = check_rows("z", z, z_stride, batch, seqlen, heads, n, io, &sz)) != SS_OK) return st;
  if (tokens > 0 && !y) return record_error(SS_ERR_INVALID_ARG, "y is NULL");
  if (!aligned(y, elem_bytes(io))) return record_error(SS_ERR_INVALID_ARG, "y is not aligned to its elements");
  if (!aligned(w, 4)) return record_error(SS_ERR_INVALID_ARG, "w is not 4-byte aligned");
  const int64_t nw = (int64_t)n * (flags & SS_NORM_HEAD_WEIGHTS ? heads : 1);
  const Range ins[] = {rng("x", x, sx * eb), rng("z", z, sz * eb), rng("w", w, nw * 4)};
  const Range outs[] = {rng("y", y, tokens * heads * n * eb)};
  if ((st = check_disjoint(ins, 3, outs, 1)) != SS_OK) return st;
  if (tokens == 0) return SS_OK;
  GatedNormArgs a = make_gated(batch, seqlen, heads, n, io, flags, eps, w);
  a.x = rows_of(x, x_stride);
  a.z = rows_of(z, z_stride);
  a.y = y;
  a.plan = gated_plan(tokens, heads, n, flags, false);
  const hipError_t e = launch_gated_norm(a, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? SS_OK : record_hip_error(e, "gated norm launch");
}

size_t ss_gated_norm_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int n, uint32_t flags) {
  if (check_sizes(batch, seqlen, heads, n) != SS_OK || seqlen == 0 || (flags & ~kGatedFlags)) return 0;
  const NormPlan p = gated_plan(batch * seqlen, heads, n, flags, true);
  return round256((size_t)p.blocks * (flags & SS_NORM_HEAD_WEIGHTS ? heads : 1) * n * sizeof(float));
}

ss_status ss_gated_norm_bwd(int64_t batch, int64_t seqlen, int heads, int n, ss_dtype io, uint32_t flags, float eps,
                            const void* x, const int64_t* x_stride, const void* z, const int64_t* z_stride,
                            const float* w, const void* dy, void* dx, const int64_t* dx_stride, void* dz,
                            const int64_t* dz_stride, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
  ss_status st = check_common(io, flags, kGatedFlags, eps);
  if (st != SS_OK) return st;
  if ((st = check_sizes(batch, seqlen, heads, n)) != SS_OK) return st;
  int64_t sx, sz = 0, sdx, sdz = 0;
  const int64_t eb = elem_bytes(io), tokens = batch * seqlen;
  if ((st = check_rows("x", x, x_stride, batch, seqlen, heads, n, io, &sx)) != SS_OK) return st;
  if (z && (st = check_rows("z", z, z_stride, batch, seqlen, heads, n, io, &sz)) != SS_OK) return st;
  if (tokens > 0 && !dy) return record_error(SS_ERR_INVALID_ARG, "dy is NULL");
  if (!aligned(dy, elem_bytes(io))) return record_error(SS_ERR_INVALID_ARG, "dy is not aligned to its elements");
  if ((st = check_rows("dx", dx, dx_stride, batch, seqlen, heads, n, io, &sdx)) != SS_OK) return st;
  if ((z == nullptr) != (dz == nullptr) && tokens > 0)
    return record_error(SS_ERR_INVALID_ARG, "dz is %s", dz ? "given without z" : "NULL");
  if (dz && (st = check_rows("dz", dz, dz_stride, batch, seqlen, heads, n, io, &sdz)) != SS_OK) return st;
  const struct { const char* name; const void* p; const int64_t* st; } grads[] = {{"dx", dx, dx_stride}, {"dz", dz, dz_stride}};
  for (const auto& g : grads) {
    if (!g.p) continue;
    int64_t size[] = {batch, seqlen, heads}, stride[] = {g.st[0], g.st[1], g.st[2]};
    if (!distinct(n, size, stride))
      return record_error(SS_ERR_INVALID_ARG, "values of %s share addresses under its strides", g.name);
  }
  if (!aligned(w, 4) || !aligned(dw, 4))
    return record_error(SS_ERR_INVALID_ARG, "%s is not 4-byte aligned", aligned(w, 4) ? "dw" : "w");
  const size_t need = dw ? ss_gated_norm_bwd_workspace_bytes(batch, seqlen, heads, n, flags) : 0;
  if ((st = check_scratch(workspace, workspace_bytes, need)) != SS_OK) return st;
  const int64_t nw = (int64_t)n * (flags & SS_NORM_HEAD_WEIGHTS ? heads : 1);
  const Range ins[] = {rng("x", x, sx * eb), rng("z", z, sz * eb), rng("w", w, nw * 4),
                       rng("dy", dy, tokens * heads * n * eb)};
  const Range outs[] = {rng("dx", dx, sdx * eb), rng("dw", dw, nw * 4), rng("workspace", workspace, (int64_t)need),
                        rng("dz", dz, sdz * eb)};
  if ((st = check_disjoint(ins, 4, outs, 3)) != SS_OK) return st;
  if ((st = check_disjoint(ins, 4, outs + 3, 1)) != SS_OK) return st;
  // dx and dz may be columns of one buffer's rows
  const int64_t apart = (int64_t)(outs[3].lo - outs[0].lo);
  for (int i = 0; i < 3; ++i) {
    if (!overlap(outs[i], outs[3])) continue;
    if (i == 0 && apart % eb == 0 && columns_of_one(batch, seqlen, n, heads, dx_stride, heads, dz_stride, apart / eb)) continue;
    return record_error(SS_ERR_INVALID_ARG, "%s overlaps dz", outs[i].name);
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (tokens == 0) {
    const hipError_t e = launch_fill_zero(dw, nw, s);
    return e == hipSuccess ? SS_OK : record_hip_error(e, "zero-fill launch");
  }
  GatedNormArgs a = make_gated(batch, seqlen, heads, n, io, flags, eps, w);
  a.x = rows_of(x, x_stride);
  a.z = rows_of(z, z_stride);
  a.dy = dy;
  a.dx = rows_of(dx, dx_stride);
  a.dz = rows_of(dz, dz_stride);
  a.part = dw ? static_cast<float*>(workspace) : nullptr;
  a.plan = gated_plan(tokens, heads, n, flags, true);
  const hipError_t e = launch_gated_norm_bwd(a, dw, s);
  return e == hipSuccess ? SS_OK : record_hip_error(e, "gated norm backward launch");
}

ss_status ss_residual_norm(int64_t rows, int n, ss_dtype io, ss_dtype rio, uint32_t flags, float eps, float alpha,
                           const void* x, const void* res, const float* w, const float* w_post, const float* scale,
                           void* y, void* res_out, void* stream) {
  ss_status st = check_residual(rows, n, io, rio, flags, eps, alpha, w, w_post, scale);
  if (st != SS_OK) return st;
  if (rows > 0 && (!x || !y)) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", x ? "y" : "x");
  const struct { const char* name; const void* p; int eb; } tensors[] = {
      {"x", x, elem_bytes(io)}, {"y", y, elem_bytes(io)}, {"res", res, elem_bytes(rio)}, {"res_out", res_out, elem_bytes(rio)}};
  for (const auto& t : tensors)
    if (!aligned(t.p, t.eb)) return record_error(SS_ERR_INVALID_ARG, "%s is not aligned to its elements", t.name);
  const int64_t xb = rows * n * elem_bytes(io), rb = rows * n * elem_bytes(rio);
  const Range ins[] = {rng("x", x, xb), rng("w", w, n * 4), rng("w_post", w_post, n * 4), rng("scale", scale, n * 4),
                       rng("res", res, rb)};
  const Range outs[] = {rng("y", y, xb), rng("res_out", res_out, rb)};
  if ((st = check_disjoint(ins, res_out == res ? 4 : 5, outs, 2)) != SS_OK) return st;
  if (overlap(outs[0], ins[4])) return record_error(SS_ERR_INVALID_ARG, "y overlaps input res");
  if (rows == 0) return SS_OK;
  ResidualNormArgs a = make_residual(rows, n, io, rio, flags, eps, alpha, x, res, w, w_post, scale);
  a.y = y;
  a.res_out = res_out;
  a.plan = residual_norm_plan(rows, n, false);
  const hipError_t e = launch_residual_norm(a, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? SS_OK : record_hip_error(e, "residual norm launch");
}

size_t ss_residual_norm_bwd_workspace_bytes(int64_t rows, int n) {
  if (rows < 1 || check_sizes(1, rows, 1, n) != SS_OK) return 0;
  return 3 * round256((size_t)residual_norm_plan(rows, n, true).blocks * n * sizeof(float));
}

ss_status ss_residual_norm_bwd(int64_t rows, int n, ss_dtype io, ss_dtype rio, uint32_t flags, float eps, float alpha,
                               const void* x, const void* res, const float* w, const float* w_post, const float* scale,
                               const void* dy, const void* dres_out, void* dx, void* dres, float* dw, float* dw_post,
                               float* dscale, void* workspace, size_t workspace_bytes, void* stream) {
  ss_status st = check_residual(rows, n, io, rio, flags, eps, alpha, w, w_post, scale);
  if (st != SS_OK) return st;
  const bool post = (flags & SS_NORM_POST) != 0;
  if (dw_post && !post) return record_error(SS_ERR_INVALID_ARG, "dw_post is given without SS_NORM_POST");
  if (rows > 0 && (!res || !dy)) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", res ? "dy" : "res");
  if (rows > 0 && !x && (post || dscale))
    return record_error(SS_ERR_INVALID_ARG, "x is NULL (%s needs it)", post ? "the norm after the block" : "dscale");
  const struct { const char* name; const void* p; int eb; } tensors[] = {
      {"x", x, elem_bytes(io)}, {"dy", dy, elem_bytes(io)}, {"dx", dx, elem_bytes(io)}, {"res", res, elem_bytes(rio)},
      {"dres_out", dres_out, elem_bytes(rio)}, {"dres", dres, elem_bytes(rio)}, {"dw", dw, 4}, {"dw_post", dw_post, 4},
      {"dscale", dscale, 4}};
  for (const auto& t : tensors)
    if (!aligned(t.p, t.eb)) return record_error(SS_ERR_INVALID_ARG, "%s is not aligned to its elements", t.name);
  const size_t need = dw || dw_post || dscale ? ss_residual_norm_bwd_workspace_bytes(rows, n) : 0;
  if ((st = check_scratch(workspace, workspace_bytes, need)) != SS_OK) return st;
  const int64_t xb = rows * n * elem_bytes(io), rb = rows * n * elem_bytes(rio);
  const Range ins[] = {rng("x", x, xb), rng("res", res, rb), rng("w", w, n * 4), rng("w_post", w_post, n * 4),
                       rng("scale", scale, n * 4), rng("dy", dy, xb), rng("dres_out", dres_out, rb)};
  const Range outs[] = {rng("dx", dx, xb), rng("dw", dw, n * 4), rng("dw_post", dw_post, n * 4),
                        rng("dscale", dscale, n * 4), rng("workspace", workspace, (int64_t)need), rng("dres", dres, rb)};
  if ((st = check_disjoint(ins, 7, outs, 5)) != SS_OK) return st;
  if ((st = check_disjoint(ins, dres == dres_out ? 6 : 7, outs + 5, 1)) != SS_OK) return st;
  for (int i = 0; i < 5; ++i)
    if (overlap(outs[i], outs[5])) return record_error(SS_ERR_INVALID_ARG, "%s overlaps dres", outs[i].name);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  float* const sums[3] = {dw, dw_post, dscale};
  if (rows == 0) {
    for (float* p : sums) {
      const hipError_t e = launch_fill_zero(p, n, s);
      if (e != hipSuccess) return record_hip_error(e, "zero-fill launch");
    }
    return SS_OK;
  }
  ResidualNormArgs a = make_residual(rows, n, io, rio, flags, eps, alpha, x, res, w, w_post, scale);
  a.dy = dy;
  a.dres_out = dres_out;
  a.dx = dx;
  a.dres = dres;
  a.plan = residual_norm_plan(rows, n, true);
  for (int i = 0; i < 3; ++i)
    a.part[i] = sums[i] ? reinterpret_cast<float*>(static_cast<char*>(workspace) + i * (need / 3)) : nullptr;
  const hipError_t e = launch_residual_norm_bwd(a, sums, s);
  return e == hipSuccess ? SS_OK : record_hip_error(e, "residual norm backward launch");
}

}  // extern "C"
