// C ABI of the gated linear recurrence: argument checks and launches.  See include/ssscan.h.
#include <cmath>

#include "api_checks.h"
#include "glr.h"
#include "internal.h"

namespace {

using namespace ssscan;

ss_status check_glr(int64_t batch, int64_t dim, int64_t seqlen, ss_dtype io, ss_glr_kind kind, float decay_scale,
                    const void* i, const float* decay, const float* i_bias) {
  if (io != SS_F32 && io != SS_BF16)
    return record_error(SS_ERR_UNSUPPORTED, "io dtype %d is not SS_F32 or SS_BF16", (int)io);
  if (kind != SS_GLR_CONVEX && kind != SS_GLR_NORMALISED)
    return record_error(SS_ERR_UNSUPPORTED, "kind %d is not SS_GLR_CONVEX or SS_GLR_NORMALISED", (int)kind);
  if (batch < 1 || dim < 1 || seqlen < 0)
    return record_error(SS_ERR_INVALID_ARG,
                        "sizes must be batch >= 1, dim >= 1, seqlen >= 0 (got %lld, %lld, %lld)", (long long)batch,
                        (long long)dim, (long long)seqlen);
  if (batch > kMaxDim || dim > kMaxDim || seqlen > kMaxDim)
    return record_error(SS_ERR_INVALID_ARG, "a size exceeds 2^40");
  if ((__int128)batch * dim * (seqlen > 0 ? seqlen : 1) * 16 > ((__int128)1 << 62))
    return record_error(SS_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte offsets");
  if (kind == SS_GLR_NORMALISED) {
    if (!decay) return record_error(SS_ERR_INVALID_ARG, "decay is NULL (the normalised kind needs it)");
    if (!(decay_scale > 0.0f) || !std::isfinite(decay_scale))
      return record_error(SS_ERR_INVALID_ARG, "decay_scale %g is not positive and finite", (double)decay_scale);
  }
  if (seqlen > 0 && i_bias && !i) return record_error(SS_ERR_INVALID_ARG, "i_bias is given without i");
  return SS_OK;
}

bool valid_sizes(int64_t batch, int64_t dim, int64_t seqlen) {
  return batch >= 1 && dim >= 1 && seqlen >= 0 && batch <= kMaxDim && dim <= kMaxDim && seqlen <= kMaxDim &&
         (__int128)batch * dim * (seqlen > 0 ? seqlen : 1) * 16 <= ((__int128)1 << 62);
}

struct Named {
  const char* name;
  const void* p;
};

template <size_t N>
ss_status check_aligned(const Named (&v)[N], uintptr_t a) {
  for (const Named& n : v)
    if (n.p && !aligned(n.p, a))
      return record_error(SS_ERR_INVALID_ARG, "%s is not %d-byte aligned", n.name, (int)a);
  return SS_OK;
}

template <size_t N, size_t M>
ss_status check_overlap(const Range (&ins)[N], const Range (&outs)[M]) {
  for (const Range& o : outs)
    for (const Range& i : ins)
      if (overlap(o, i)) return record_error(SS_ERR_INVALID_ARG, "%s overlaps input %s", o.name, i.name);
  for (size_t i = 0; i < M; ++i)
    for (size_t j = i + 1; j < M; ++j)
      if (overlap(outs[i], outs[j]))
        return record_error(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
  return SS_OK;
}

ss_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return SS_OK;
  if (!workspace) return record_error(SS_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned(workspace, 256)) return record_error(SS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (bytes < need) return record_error(SS_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, need);
  return SS_OK;
}

// Forward scratch: the memory through which split rows join (their chain).  Backward
// scratch: two of them (of the sweep that recomputes the states, and of the adjoint),
// the states entering the tiles of rows of several, and the sums over each row's
// (split: each tile's) tokens behind the per-channel gradients.
struct GlrBwdLayout {
  size_t chain, ckpt, sums, total;
};

size_t chain_bytes(int64_t rows, int64_t seqlen) {
  return glr_split(rows, seqlen) ? round256(glr_chain_bytes(rows, seqlen)) : 0;
}

GlrBwdLayout bwd_layout(int64_t rows, int64_t seqlen) {
  const size_t tiles = glr_split(rows, seqlen) ? glr_tiles(seqlen) : 1;
  GlrBwdLayout w{};
  w.chain = chain_bytes(rows, seqlen);
  w.ckpt = 2 * w.chain;
  w.sums = w.ckpt + (seqlen > kGlrCkptTokens ? round256((size_t)rows * glr_tiles(seqlen) * sizeof(float)) : 0);
  w.total = w.sums + (seqlen > 0 ? round256((size_t)rows * tiles * 3 * sizeof(float)) : 0);
  return w;
}

// A chain's slots start as zeros (by a kernel, so that a captured call replays).
hipError_t clear_chains(void* ws, size_t bytes, hipStream_t s) {
  return bytes ? launch_fill_zero(static_cast<float*>(ws), (int64_t)(bytes / sizeof(float)), s) : hipSuccess;
}

GlrArgs base_args(int64_t batch, int64_t dim, int64_t seqlen, ss_dtype io, ss_glr_kind kind, float decay_scale,
                  const void* x, const void* r, const void* i, const void* z, const float* decay, const float* r_bias,
                  const float* i_bias, const float* h0) {
  GlrArgs a{};
  a.rows = batch * dim;
  a.dim = dim;
  a.seqlen = seqlen;
  a.io = io == SS_BF16 ? kIoBf16 : kIoF32;
  a.kind = kind;
  a.decay_scale = decay_scale;
  a.x = x;
  a.r = r;
  a.i = i;
  a.z = z;
  a.decay = decay;
  a.r_bias = r_bias;
  a.i_bias = i_bias;
  a.h0 = h0;
  return a;
}

}  // namespace

extern "C" {

size_t ss_glr_ckpt_bytes(int64_t batch, int64_t dim, int64_t seqlen) {
  if (!valid_sizes(batch, dim, seqlen)) return 0;
  return (size_t)batch * dim * glr_tiles(seqlen) * sizeof(float);
}

size_t ss_glr_fwd_workspace_bytes(int64_t batch, int64_t dim, int64_t seqlen) {
  if (!valid_sizes(batch, dim, seqlen)) return 0;
  return chain_bytes(batch * dim, seqlen);
}

ss_status ss_glr_fwd(int64_t batch, int64_t dim, int64_t seqlen, ss_dtype io, ss_glr_kind kind, float decay_scale,
                     const void* x, const void* r, const void* i, const void* z, const float* decay,
                     const float* r_bias, const float* i_bias, const float* h0, void* y, float* h_final, float* ckpt,
                     void* workspace, size_t workspace_bytes, void* stream) {
  ss_status st = check_glr(batch, dim, seqlen, io, kind, decay_scale, i, decay, i_bias);
  if (st != SS_OK) return st;
  if (seqlen > 0) {
    const Named req[] = {{"x", x}, {"r", r}, {"y", y}};
    for (const Named& n : req)
      if (!n.p) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", n.name);
  }
  if ((st = check_aligned({{"x", x}, {"r", r}, {"i", i}, {"z", z}, {"y", y}}, elem_bytes(io))) != SS_OK) return st;
  if ((st = check_aligned({{"decay", decay}, {"r_bias", r_bias}, {"i_bias", i_bias}, {"h0", h0}, {"h_final", h_final},
                           {"ckpt", ckpt}}, 4)) != SS_OK)
    return st;
  const size_t need = ss_glr_fwd_workspace_bytes(batch, dim, seqlen);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != SS_OK) return st;
  const int64_t rows = batch * dim, seq = rows * seqlen * elem_bytes(io);
  const Range ins[] = {rng("x", x, seq), rng("r", r, seq), rng("i", i, seq), rng("z", z, seq),
                       rng("decay", decay, dim * 4), rng("r_bias", r_bias, dim * 4), rng("i_bias", i_bias, dim * 4),
                       rng("h0", h0, rows * 4)};
  const Range outs[] = {rng("y", y, seq), rng("h_final", h_final, rows * 4),
                        rng("ckpt", ckpt, rows * glr_tiles(seqlen) * 4), rng("workspace", workspace, (int64_t)need)};
  if ((st = check_overlap(ins, outs)) != SS_OK) return st;

  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (seqlen == 0) {
    if (!h_final) return SS_OK;
    const hipError_t e = h0 ? launch_copy_state(rows, h0, h_final, s) : launch_fill_zero(h_final, rows, s);
    return e == hipSuccess ? SS_OK : record_hip_error(e, "h_final launch");
  }
  GlrArgs a = base_args(batch, dim, seqlen, io, kind, decay_scale, x, r, i, z, decay, r_bias, i_bias, h0);
  a.y = y;
  a.h_final = h_final;
  a.ckpt = ckpt;
  a.chain = need ? workspace : nullptr;
  hipError_t e = clear_chains(workspace, need, s);
  if (e == hipSuccess) e = launch_glr_fwd(a, s);
  return e == hipSuccess ? SS_OK : record_hip_error(e, "recurrence launch");
}

size_t ss_glr_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t seqlen) {
  if (!valid_sizes(batch, dim, seqlen)) return 0;
  return bwd_layout(batch * dim, seqlen).total;
}

ss_status ss_glr_bwd(int64_t batch, int64_t dim, int64_t seqlen, ss_dtype io, ss_glr_kind kind, float decay_scale,
                     const void* x, const void* r, const void* i, const void* z, const float* decay,
                     const float* r_bias, const float* i_bias, const float* h0, const void* dy, const float* dh_final,
                     const float* ckpt, void* dx, void* dr, void* di, void* dz, float* ddecay, float* dr_bias,
                     float* di_bias, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  ss_status st = check_glr(batch, dim, seqlen, io, kind, decay_scale, i, decay, i_bias);
  if (st != SS_OK) return st;
  if (seqlen > 0) {
    const Named req[] = {{"x", x}, {"r", r}, {"dy", dy}, {"dx", dx}, {"dr", dr}};
    for (const Named& n : req)
      if (!n.p) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", n.name);
  }
  if (seqlen > 0) {   // an empty tensor's address may be NULL
    if ((i == nullptr) != (di == nullptr))
      return record_error(SS_ERR_INVALID_ARG, "di must be given exactly when i is (i %s, di %s)", i ? "set" : "NULL",
                          di ? "set" : "NULL");
    if ((z == nullptr) != (dz == nullptr))
      return record_error(SS_ERR_INVALID_ARG, "dz must be given exactly when z is (z %s, dz %s)", z ? "set" : "NULL",
                          dz ? "set" : "NULL");
    if (di_bias && !i) return record_error(SS_ERR_INVALID_ARG, "di_bias is given without i");
  }
  if ((st = check_aligned({{"x", x}, {"r", r}, {"i", i}, {"z", z}, {"dy", dy}, {"dx", dx}, {"dr", dr}, {"di", di},
                           {"dz", dz}}, elem_bytes(io))) != SS_OK)
    return st;
  if ((st = check_aligned({{"decay", decay}, {"r_bias", r_bias}, {"i_bias", i_bias}, {"h0", h0},
                           {"dh_final", dh_final}, {"ckpt", ckpt}, {"ddecay", ddecay}, {"dr_bias", dr_bias},
                           {"di_bias", di_bias}, {"dh0", dh0}}, 4)) != SS_OK)
    return st;
  const int64_t rows = batch * dim, seq = rows * seqlen * elem_bytes(io);
  const GlrBwdLayout wl = bwd_layout(rows, seqlen);
  if ((st = check_workspace(workspace, workspace_bytes, wl.total)) != SS_OK) return st;
  const Range ins[] = {rng("x", x, seq), rng("r", r, seq), rng("i", i, seq), rng("z", z, seq),
                       rng("decay", decay, dim * 4), rng("r_bias", r_bias, dim * 4), rng("i_bias", i_bias, dim * 4),
                       rng("h0", h0, rows * 4), rng("dy", dy, seq), rng("dh_final", dh_final, rows * 4),
                       rng("ckpt", ckpt, rows * glr_tiles(seqlen) * 4)};
  const Range outs[] = {rng("dx", dx, seq), rng("dr", dr, seq), rng("di", di, seq), rng("dz", dz, seq),
                        rng("ddecay", ddecay, dim * 4), rng("dr_bias", dr_bias, dim * 4),
                        rng("di_bias", di_bias, dim * 4), rng("dh0", dh0, rows * 4),
                        rng("workspace", workspace, (int64_t)wl.total)};
  if ((st = check_overlap(ins, outs)) != SS_OK) return st;

  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (seqlen == 0) {
    // no tokens: the final state is h0, and nothing else enters
    if (dh0) e = dh_final ? launch_copy_state(rows, dh_final, dh0, s) : launch_fill_zero(dh0, rows, s);
    float* zero[] = {ddecay, dr_bias, di_bias};
    for (float* z0 : zero)
      if (e == hipSuccess) e = launch_fill_zero(z0, dim, s);
    return e == hipSuccess ? SS_OK : record_hip_error(e, "empty-sequence launch");
  }
  char* ws = static_cast<char*>(workspace);
  GlrArgs a = base_args(batch, dim, seqlen, io, kind, decay_scale, x, r, i, z, decay, r_bias, i_bias, h0);
  a.ckpt = const_cast<float*>(ckpt);
  const bool sweep = !ckpt && seqlen > kGlrCkptTokens;
  e = clear_chains(ws, sweep ? 2 * wl.chain : wl.chain, s);
  if (e != hipSuccess) return record_hip_error(e, "zero-fill launch");
  a.chain = wl.chain ? ws : nullptr;
  if (sweep) {
    GlrArgs f = a;   // the forward again, storing its states only
    f.z = nullptr;
    f.ckpt = a.ckpt = reinterpret_cast<float*>(ws + wl.ckpt);
    if (f.chain) f.chain = ws + wl.chain;
    e = launch_glr_fwd(f, s);
    if (e != hipSuccess) return record_hip_error(e, "state sweep launch");
  }
  a.dy = dy;
  a.dh_final = dh_final;
  a.dx = dx;
  a.dr = dr;
  a.di = di;
  a.dz = dz;
  a.dh0 = dh0;
  a.sums = ddecay || dr_bias || di_bias ? reinterpret_cast<float*>(ws + wl.sums) : nullptr;
  e = launch_glr_bwd(a, s);
  if (e != hipSuccess) return record_hip_error(e, "recurrence backward launch");
  if (a.sums) {
    e = launch_glr_reduce(batch, dim, a.chain ? glr_tiles(seqlen) : 1, a.sums, ddecay, dr_bias, di_bias, s);
    if (e != hipSuccess) return record_hip_error(e, "per-channel sums launch");
  }
  return SS_OK;
}

ss_status ss_glr_step(int64_t batch, int64_t dim, ss_dtype io, ss_glr_kind kind, float decay_scale,
                      const float* state_in, float* state_out, const void* x, const void* r, const void* i,
                      const void* z, const float* decay, const float* r_bias, const float* i_bias, void* y,
                      void* stream) {
  ss_status st = check_glr(batch, dim, 1, io, kind, decay_scale, i, decay, i_bias);
  if (st != SS_OK) return st;
  if (dim > kGlrStepDim)
    return record_error(SS_ERR_UNSUPPORTED, "dim %lld exceeds %lld", (long long)dim, (long long)kGlrStepDim);
  const Named req[] = {{"state_in", state_in}, {"state_out", state_out}, {"x", x}, {"r", r}, {"y", y}};
  for (const Named& n : req)
    if (!n.p) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", n.name);
  if ((st = check_aligned({{"x", x}, {"r", r}, {"i", i}, {"z", z}, {"y", y}}, elem_bytes(io))) != SS_OK) return st;
  if ((st = check_aligned({{"decay", decay}, {"r_bias", r_bias}, {"i_bias", i_bias}, {"state_in", state_in},
                           {"state_out", state_out}}, 4)) != SS_OK)
    return st;
  const int64_t rows = batch * dim, seq = rows * elem_bytes(io);
  const Range ins[] = {rng("x", x, seq), rng("r", r, seq), rng("i", i, seq), rng("z", z, seq),
                       rng("decay", decay, dim * 4), rng("r_bias", r_bias, dim * 4), rng("i_bias", i_bias, dim * 4),
                       rng("state_in", state_in == state_out ? nullptr : state_in, rows * 4)};
  const Range outs[] = {rng("y", y, seq), rng("state_out", state_out, rows * 4)};
  if ((st = check_overlap(ins, outs)) != SS_OK) return st;
  GlrArgs a = base_args(batch, dim, 1, io, kind, decay_scale, x, r, i, z, decay, r_bias, i_bias, state_in);
  a.y = y;
  a.h_final = state_out;
  const hipError_t e = launch_glr_step(a, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? SS_OK : record_hip_error(e, "recurrence step launch");
}

}  // extern "C"
