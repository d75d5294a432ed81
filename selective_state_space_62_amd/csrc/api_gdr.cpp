// C ABI of the gated delta rule: argument checks and launches.  See include/ssscan.h.
#include <algorithm>
#include <cmath>

#include "api_rows.h"
#include "gdr.h"

namespace {

using namespace ssscan;

constexpr int kMaxDimK = 128;
constexpr int kMaxDimV = 1 << 16;
constexpr int kMaxHeads = 1 << 20;
constexpr int64_t kMaxBlocks = int64_t(1) << 23;   // of 256 or 512 threads, fewer than 2^32 of them

ss_status check_sizes(int64_t batch, int64_t seqlen, int heads_k, int heads_v, int dim_k, int dim_v) {
  if (batch < 1 || seqlen < 0)
    return record_error(SS_ERR_INVALID_ARG, "sizes must be batch >= 1, seqlen >= 0 (got %lld, %lld)",
                        (long long)batch, (long long)seqlen);
  if (heads_k < 1 || heads_v < 1 || heads_v > kMaxHeads || heads_v % heads_k)
    return record_error(SS_ERR_INVALID_ARG, "heads_v %d is not 1 to 2^20 and a multiple of heads_k %d", heads_v, heads_k);
  if (dim_k < 1 || dim_k > kMaxDimK) return record_error(SS_ERR_UNSUPPORTED, "dim_k %d is not 1 to %d", dim_k, kMaxDimK);
  if (dim_v < 1 || dim_v > kMaxDimV) return record_error(SS_ERR_UNSUPPORTED, "dim_v %d is not 1 to %d", dim_v, kMaxDimV);
  if (batch > kMaxDim || seqlen > kMaxDim ||
      (__int128)batch * (seqlen > 0 ? seqlen : 1) * heads_v * (dim_k + (int64_t)dim_v) * 8 > ((__int128)1 << 62) ||
      (__int128)batch * heads_v * (1 + seqlen / 64) * (dim_k + 128) * (dim_v + 128) * 16 > ((__int128)1 << 62))
    return record_error(SS_ERR_INVALID_ARG, "tensor sizes overflow 64-bit byte offsets");
  return SS_OK;
}

struct Inputs {
  int64_t batch, seqlen;
  int heads_k, heads_v, dim_k, dim_v;
  ss_dtype io;
  float scale;
  const void* q;
  const int64_t* q_stride;
  const void* k;
  const int64_t* k_stride;
  const void* v;
  const int64_t* v_stride;
  const float* g;
  const float* beta;
  const float* h0;
};

int64_t gates(const Inputs& in) { return in.batch * in.seqlen * in.heads_v; }
int64_t state_numel(const Inputs& in) { return in.batch * in.heads_v * in.dim_k * in.dim_v; }

// The checks that all calls share, and the inputs' spans (ranges[0..5]: q, k, v, g, beta, h0).
ss_status check_inputs(const Inputs& in, Range (&ranges)[6]) {
  if (in.io != SS_F32 && in.io != SS_BF16)
    return record_error(SS_ERR_UNSUPPORTED, "io dtype %d is not SS_F32 or SS_BF16", (int)in.io);
  ss_status st = check_sizes(in.batch, in.seqlen, in.heads_k, in.heads_v, in.dim_k, in.dim_v);
  if (st != SS_OK) return st;
  if (!std::isfinite(in.scale)) return record_error(SS_ERR_INVALID_ARG, "scale %g is not finite", (double)in.scale);
  int64_t sq, sk, sv;
  const int64_t eb = elem_bytes(in.io);
  if ((st = check_rows("q", in.q, in.q_stride, in.batch, in.seqlen, in.heads_k, in.dim_k, in.io, &sq)) != SS_OK) return st;
  if ((st = check_rows("k", in.k, in.k_stride, in.batch, in.seqlen, in.heads_k, in.dim_k, in.io, &sk)) != SS_OK) return st;
  if ((st = check_rows("v", in.v, in.v_stride, in.batch, in.seqlen, in.heads_v, in.dim_v, in.io, &sv)) != SS_OK) return st;
  if (in.seqlen > 0 && !in.beta) return record_error(SS_ERR_INVALID_ARG, "beta is NULL");
  const struct { const char* name; const float* p; } vecs[] = {{"g", in.g}, {"beta", in.beta}, {"h0", in.h0}};
  for (const auto& n : vecs)
    if (!aligned(n.p, 4)) return record_error(SS_ERR_INVALID_ARG, "%s is not 4-byte aligned", n.name);
  ranges[0] = rng("q", in.q, sq * eb);
  ranges[1] = rng("k", in.k, sk * eb);
  ranges[2] = rng("v", in.v, sv * eb);
  ranges[3] = rng("g", in.g, gates(in) * 4);
  ranges[4] = rng("beta", in.beta, gates(in) * 4);
  ranges[5] = rng("h0", in.h0, state_numel(in) * 4);
  return SS_OK;
}

GdrArgs make_args(const Inputs& in) {
  GdrArgs a{};
  a.batch = in.batch;
  a.seqlen = in.seqlen;
  a.hk = in.heads_k;
  a.hv = in.heads_v;
  a.dk = in.dim_k;
  a.dv = in.dim_v;
  a.io = in.io == SS_BF16 ? kIoBf16 : kIoF32;
  a.scale = in.scale;
  a.q = in.q;
  a.k = in.k;
  a.v = in.v;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = in.q_stride[i];
    a.ks[i] = in.k_stride[i];
    a.vs[i] = in.v_stride[i];
  }
  if (in.seqlen == 1) a.qs[1] = a.ks[1] = a.vs[1] = 0;     // a token without a next one
  a.g = in.g;
  a.beta = in.beta;
  a.h0 = in.h0;
  return a;
}

ss_status check_blocks(int64_t blocks) {
  if (blocks >= kMaxBlocks)
    return record_error(SS_ERR_UNSUPPORTED, "2^23 workgroups (of batch rows, heads, and columns or 64 tokens) and more are not supported");
  return SS_OK;
}

// Up to this many tokens go one by one, and tokens so far apart that 64 of them pass 2^31 bytes.  Where the two meet goes by the heads and
// the type too (fewer heads and bf16 sooner); this is between: one by one and in a chunk, kernels' us (values of 128, of 64 with keys of 16):
//   bf16, keys of 128:  4 heads, 8 tokens 19, 21, 10 tokens 22, 21, 16 tokens 32, 21; 128 x 40 heads, 8 tokens 222, 274, 12 tokens 282, 280
//   bf16, keys of 64:   4 heads, 10 tokens 17, 17, 16 tokens 24, 17; 8 x 40 heads, 16 tokens 29, 26; 128 x 40 heads, 16 tokens 203, 202
//   bf16, keys of 16:   4 heads, 10 tokens 16, 15, 16 tokens 23, 15; 128 x 40 heads, 16 tokens 130, 119; 512 x 40 heads, 16 tokens 458, 489
//   fp32, keys of 128:  4 heads, 10 tokens 19, 26, 16 tokens 27, 26; 128 x 40 heads, 10 tokens 203, 520, 32 tokens 476, 542
//   fp32, keys of 64:   4 heads, 16 tokens 21, 19; 128 x 40 heads, 16 tokens 162, 241, 24 tokens 222, 249
constexpr int64_t recur_tokens(int dim_k) { return dim_k <= 64 ? 16 : 10; }
constexpr int64_t kMostStride = int64_t(1) << 22;

bool far_apart(const Inputs& in) {
  if ((int64_t)in.heads_v * in.dim_v >= kMostStride) return true;
  return in.seqlen > 1 && (in.q_stride[1] >= kMostStride || in.k_stride[1] >= kMostStride || in.v_stride[1] >= kMostStride);
}

bool aligned_rows(const void* p, const int64_t* st, ss_dtype io) {
  const int64_t eb = elem_bytes(io);
  return aligned(p, 4) && st[0] * eb % 4 == 0 && st[1] * eb % 4 == 0 && st[2] * eb % 4 == 0;
}

bool whole_runs(const Inputs& in) {
  return in.dim_k % 8 == 0 && in.dim_v % 8 == 0 && aligned_rows(in.q, in.q_stride, in.io) &&
         aligned_rows(in.k, in.k_stride, in.io) && aligned_rows(in.v, in.v_stride, in.io);
}

int64_t chunks_of(int64_t seqlen) { return (seqlen + kGdrChunk - 1) / kGdrChunk; }

struct Segments {
  int64_t count, per;
};

// Segments of at least two chunks, as many as fill the GPU, but no more than 2 sqrt(chunks): a segment's join takes as long as a
// quarter of a chunk's two passes (one head of 2^20 tokens, 256 segments 1980, 512 2549; 2 heads of 32768, 64 segments 300, 256 736;
// one head of 4096, 16 segments 112, 32 130; backward, one head of 131072, 128 segments 1399, 512 2879).  Made in segments a row costs
// about 1.7 times as much, the factors and the states first, so two of them gain little.  In one and in segments, us: 16 heads of
// 131072 tokens 16973, 2577; 12 x 8 heads (fp32, keys of 64) of 2048 337, 280; 40 heads of 4096 553, 279; 8 heads of 500 76, 59; 2
// heads of 1000 133, 68; 4 x 40 heads of 2048 361, in two 347, in three 338; 8 x 40 heads of 2048, which fill it, 535 and, in three,
// 656.  Backward: 16 heads of 32768 10405, 2192; 3 x 10 heads (fp32, 72 by 80) of 1111 467, 268; 2 heads of 1000 320, 156; 4 x 40 heads
// of 2048 1308, in two 1300, in three 1280.
Segments segments_of(int64_t batch, int64_t chunks, int heads_v, int dim_k, int dim_v, int io) {
  const int64_t groups = batch * heads_v * ((dim_v + 127) / 128);
  const int64_t n = std::min({gdr_chunk_room(io, dim_k) / groups, chunks / 2, (int64_t)(2.0 * std::sqrt((double)chunks))});
  if (n < 3) return {1, chunks};
  const int64_t per = (chunks + n - 1) / n;
  return {(chunks + per - 1) / per, per};
}

// Scratch of the segments, behind what a direction has besides.
struct SegmentsLayout {
  size_t ends, moves, moves_e, total;
};

SegmentsLayout segments_layout(size_t from, int64_t batch, int64_t seqlen, int heads_v, int dim_k, int dim_v) {
  const int64_t chunks = chunks_of(seqlen), rows = (dim_k + 31) / 32 * 32, cols = ((int64_t)dim_v + 31) / 32 * 32;
  const int64_t most = std::max(segments_of(batch, chunks, heads_v, dim_k, dim_v, kIoBf16).count,
                                segments_of(batch, chunks, heads_v, dim_k, dim_v, kIoF32).count);
  const int64_t n = most > 1 ? batch * heads_v * most : 0;
  SegmentsLayout l;
  l.ends = from;
  l.moves = l.ends + round256((size_t)(n * rows * cols) * 4);
  l.moves_e = l.moves + round256((size_t)(n * rows * rows) * 4);
  l.total = l.moves_e + round256((size_t)(n * 4) * 4);
  return l;
}

void set_segments(GdrArgs& a, const SegmentsLayout& l, char* ws) {
  const Segments seg = segments_of(a.batch, a.chunks, a.hv, a.dk, a.dv, a.io);
  a.segments = seg.count;
  a.per = seg.per;
  a.ldv = ((int64_t)a.dv + 31) / 32 * 32;
  a.ends = reinterpret_cast<float*>(ws + l.ends);
  a.moves = reinterpret_cast<float*>(ws + l.moves);
  a.moves_e = reinterpret_cast<int32_t*>(ws + l.moves_e);
}

// Scratch of the chunked forward: the inverses, P, the vectors, then the segments'.
struct FwdLayout {
  size_t p, vecs;
  SegmentsLayout segments;
};

FwdLayout fwd_layout(int64_t batch, int64_t seqlen, int heads_v, int dim_k, int dim_v) {
  const int64_t n = batch * heads_v * chunks_of(seqlen);
  FwdLayout l;
  l.p = round256(gdr_tri_bytes(n));
  l.vecs = l.p + round256(gdr_tri_bytes(n));
  l.segments = segments_layout(l.vecs + round256(gdr_vecs_bytes(n)), batch, seqlen, heads_v, dim_k, dim_v);
  return l;
}

// Scratch of the backward: the preparation's, then for every chunk of a head the state before it and the gradient of the one
// behind it, U and the gradient of R, the largest values of their tiles, and dq and dk of value heads that share keys.
struct BwdLayout {
  size_t tri_t, p, vecs, states, dstates, u, dr, maxima, part_q, part_k;
  SegmentsLayout segments;
  int64_t max_apart;
};

BwdLayout bwd_layout(int64_t batch, int64_t seqlen, int heads_k, int heads_v, int dim_k, int dim_v) {
  const int64_t n = batch * heads_v * chunks_of(seqlen), rows = (dim_k + 31) / 32 * 32, ldv = ((int64_t)dim_v + 31) / 32 * 32;
  BwdLayout l;
  l.max_apart = n * (ldv / 32);
  l.tri_t = round256(gdr_tri_bytes(n));
  l.p = l.tri_t + round256(gdr_tri_bytes(n));
  l.vecs = l.p + round256(gdr_tri_bytes(n));
  l.states = l.vecs + round256(gdr_vecs_bytes(n));
  l.dstates = l.states + round256((size_t)(n * rows * ldv) * 4);
  l.u = l.dstates + round256((size_t)(n * rows * ldv) * 4);
  l.dr = l.u + round256((size_t)(n * kGdrChunk * ldv) * 4);
  l.maxima = l.dr + round256((size_t)(n * kGdrChunk * ldv) * 4);
  l.part_q = l.maxima + round256((size_t)(kMaxKinds * l.max_apart) * 4);
  l.part_k = l.part_q + (heads_v > heads_k ? round256((size_t)(n * kGdrChunk * rows) * 4) : 0);
  l.segments = segments_layout(l.part_k + (l.part_k - l.part_q), batch, seqlen, heads_v, dim_k, dim_v);
  return l;
}

}  // namespace

extern "C" {

size_t ss_gdr_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads_k, int heads_v, int dim_k, int dim_v) {
  if (check_sizes(batch, seqlen, heads_k, heads_v, dim_k, dim_v) != SS_OK || seqlen <= recur_tokens(dim_k)) return 0;
  return fwd_layout(batch, seqlen, heads_v, dim_k, dim_v).segments.total;
}

ss_status ss_gdr_fwd(int64_t batch, int64_t seqlen, int heads_k, int heads_v, int dim_k, int dim_v, ss_dtype io,
                     float scale, const void* q, const int64_t* q_stride, const void* k, const int64_t* k_stride,
                     const void* v, const int64_t* v_stride, const float* g, const float* beta, const float* h0, void* o,
                     float* h_final, void* workspace, size_t workspace_bytes, void* stream) {
  const Inputs in{batch, seqlen, heads_k, heads_v, dim_k, dim_v, io, scale, q, q_stride, k, k_stride, v, v_stride, g, beta, h0};
  Range ins[6];
  ss_status st = check_inputs(in, ins);
  if (st != SS_OK) return st;
  if (seqlen > 0 && !o) return record_error(SS_ERR_INVALID_ARG, "o is NULL");
  if (!aligned(o, 16)) return record_error(SS_ERR_INVALID_ARG, "o is not 16-byte aligned");
  if (!aligned(h_final, 4)) return record_error(SS_ERR_INVALID_ARG, "h_final is not 4-byte aligned");
  const size_t need = ss_gdr_fwd_workspace_bytes(batch, seqlen, heads_k, heads_v, dim_k, dim_v);
  if ((st = check_scratch(workspace, workspace_bytes, need)) != SS_OK) return st;
  const Range outs[] = {rng("o", o, batch * seqlen * heads_v * dim_v * elem_bytes(io)),
                        rng("h_final", h_final, state_numel(in) * 4), rng("workspace", workspace, (int64_t)need)};
  if ((st = check_disjoint(ins, 6, outs, 3)) != SS_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (seqlen == 0) {
    if (h_final) e = h0 ? launch_copy_state(state_numel(in), h0, h_final, s) : launch_fill_zero(h_final, state_numel(in), s);
    return e == hipSuccess ? SS_OK : record_hip_error(e, "state copy launch");
  }
  const bool recur = seqlen <= recur_tokens(dim_k) || far_apart(in);
  if ((st = check_blocks(recur ? gdr_recur_blocks(batch, heads_v, dim_v) : batch * heads_v * chunks_of(seqlen))) != SS_OK)
    return st;
  GdrArgs a = make_args(in);
  a.o = o;
  a.h_final = h_final;
  if (recur) {
    e = launch_gdr_recur(a, s);
  } else {
    const FwdLayout l = fwd_layout(batch, seqlen, heads_v, dim_k, dim_v);
    char* ws = static_cast<char*>(workspace);
    a.chunks = chunks_of(seqlen);
    a.whole = whole_runs(in);
    a.tri = ws;
    a.p = ws + l.p;
    a.vecs = reinterpret_cast<float*>(ws + l.vecs);
    set_segments(a, l.segments, ws);
    e = launch_gdr_prep(a, false, s);
    if (e == hipSuccess) e = launch_gdr_chunk(a, false, s);
  }
  return e == hipSuccess ? SS_OK : record_hip_error(e, "gated delta rule launch");
}

size_t ss_gdr_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads_k, int heads_v, int dim_k, int dim_v) {
  if (check_sizes(batch, seqlen, heads_k, heads_v, dim_k, dim_v) != SS_OK || seqlen == 0) return 0;
  return bwd_layout(batch, seqlen, heads_k, heads_v, dim_k, dim_v).segments.total;
}

ss_status ss_gdr_bwd(int64_t batch, int64_t seqlen, int heads_k, int heads_v, int dim_k, int dim_v, ss_dtype io,
                     float scale, const void* q, const int64_t* q_stride, const void* k, const int64_t* k_stride,
                     const void* v, const int64_t* v_stride, const float* g, const float* beta, const float* h0,
                     const void* dout, const float* dh_final, void* dq, void* dk, void* dv, float* dg, float* dbeta,
                     float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  const Inputs in{batch, seqlen, heads_k, heads_v, dim_k, dim_v, io, scale, q, q_stride, k, k_stride, v, v_stride, g, beta, h0};
  Range own[6];
  ss_status st = check_inputs(in, own);
  if (st != SS_OK) return st;
  const int64_t eb = elem_bytes(io), tokens = batch * seqlen;
  const struct { const char* name; const void* p; } rows[] = {{"dout", dout}, {"dq", dq}, {"dk", dk}, {"dv", dv}};
  for (const auto& r : rows) {
    if (seqlen > 0 && !r.p) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", r.name);
    if (!aligned(r.p, 16)) return record_error(SS_ERR_INVALID_ARG, "%s is not 16-byte aligned", r.name);
  }
  const struct { const char* name; const float* p; } vecs[] = {{"dh_final", dh_final}, {"dg", dg}, {"dbeta", dbeta}, {"dh0", dh0}};
  for (const auto& n : vecs)
    if (!aligned(n.p, 4)) return record_error(SS_ERR_INVALID_ARG, "%s is not 4-byte aligned", n.name);
  if (far_apart(in))
    return record_error(SS_ERR_UNSUPPORTED, "tokens 2^22 values and more apart are not supported here");
  const size_t need = ss_gdr_bwd_workspace_bytes(batch, seqlen, heads_k, heads_v, dim_k, dim_v);
  if ((st = check_scratch(workspace, workspace_bytes, need)) != SS_OK) return st;
  const Range ins[] = {own[0], own[1], own[2], own[3], own[4], own[5], rng("dout", dout, tokens * heads_v * dim_v * eb),
                       rng("dh_final", dh_final, state_numel(in) * 4)};
  const Range outs[] = {rng("dq", dq, tokens * heads_k * dim_k * eb), rng("dk", dk, tokens * heads_k * dim_k * eb),
                        rng("dv", dv, tokens * heads_v * dim_v * eb), rng("dg", dg, gates(in) * 4),
                        rng("dbeta", dbeta, gates(in) * 4), rng("dh0", dh0, state_numel(in) * 4),
                        rng("workspace", workspace, (int64_t)need)};
  if ((st = check_disjoint(ins, 8, outs, 7)) != SS_OK) return st;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (seqlen == 0) {
    if (dh0) e = dh_final ? launch_copy_state(state_numel(in), dh_final, dh0, s) : launch_fill_zero(dh0, state_numel(in), s);
    return e == hipSuccess ? SS_OK : record_hip_error(e, "state copy launch");
  }
  if ((st = check_blocks(batch * heads_v * chunks_of(seqlen))) != SS_OK) return st;
  const BwdLayout l = bwd_layout(batch, seqlen, heads_k, heads_v, dim_k, dim_v);
  char* ws = static_cast<char*>(workspace);
  GdrArgs a = make_args(in);
  a.chunks = chunks_of(seqlen);
  a.whole = whole_runs(in);
  a.tri = ws;
  a.tri_t = ws + l.tri_t;
  a.p = ws + l.p;
  a.vecs = reinterpret_cast<float*>(ws + l.vecs);
  set_segments(a, l.segments, ws);
  a.states = reinterpret_cast<float*>(ws + l.states);
  a.dstates = reinterpret_cast<float*>(ws + l.dstates);
  a.u = reinterpret_cast<float*>(ws + l.u);
  a.dr = reinterpret_cast<float*>(ws + l.dr);
  a.maxima = reinterpret_cast<float*>(ws + l.maxima);
  a.max_apart = l.max_apart;
  a.part_q = reinterpret_cast<float*>(ws + l.part_q);
  a.part_k = reinterpret_cast<float*>(ws + l.part_k);
  a.dout = dout;
  a.dh_final = dh_final;
  a.dq = dq;
  a.dk_out = dk;
  a.dv_out = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dh0 = dh0;
  e = launch_gdr_prep(a, true, s);
  if (e == hipSuccess) e = launch_gdr_chunk(a, true, s);
  if (e == hipSuccess) e = launch_gdr_chunk_bwd(a, s);
  if (e == hipSuccess) e = launch_gdr_grad(a, s);
  return e == hipSuccess ? SS_OK : record_hip_error(e, "gated delta rule backward launch");
}

ss_status ss_gdr_step(int64_t batch, int heads_k, int heads_v, int dim_k, int dim_v, ss_dtype io, float scale,
                      const float* state_in, float* state_out, const void* q, const int64_t* q_stride, const void* k,
                      const int64_t* k_stride, const void* v, const int64_t* v_stride, const float* g,
                      const float* beta, void* o, void* stream) {
  const Inputs in{batch, 1, heads_k, heads_v, dim_k, dim_v, io, scale, q, q_stride, k, k_stride, v, v_stride, g, beta, state_in};
  Range ins[6];
  ss_status st = check_inputs(in, ins);
  if (st != SS_OK) return st;
  if (!state_in || !state_out || !o)
    return record_error(SS_ERR_INVALID_ARG, "%s is NULL", !state_in ? "state_in" : !state_out ? "state_out" : "o");
  if (!aligned(o, 16)) return record_error(SS_ERR_INVALID_ARG, "o is not 16-byte aligned");
  if (!aligned(state_out, 4)) return record_error(SS_ERR_INVALID_ARG, "state_out is not 4-byte aligned");
  ins[5].name = "state_in";
  const Range outs[] = {rng("o", o, batch * heads_v * dim_v * elem_bytes(io)),
                        rng("state_out", state_out, state_numel(in) * 4)};
  if ((st = check_disjoint(ins, state_out == state_in ? 5 : 6, outs, 2)) != SS_OK) return st;
  if (overlap(outs[0], ins[5])) return record_error(SS_ERR_INVALID_ARG, "o overlaps input state_in");
  if ((st = check_blocks(gdr_recur_blocks(batch, heads_v, dim_v))) != SS_OK) return st;
  GdrArgs a = make_args(in);
  a.o = o;
  a.h_final = state_out;
  const hipError_t e = launch_gdr_recur(a, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? SS_OK : record_hip_error(e, "gated delta rule step launch");
}

}  // extern "C"
