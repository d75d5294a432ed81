// Internal interface of the gated linear recurrence (include/ssscan.h, ss_glr_*).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ssscan {

// Tokens between two stored states (ckpt), and of the widest tile of a row.
constexpr int64_t kGlrCkptTokens = 2048;

// Operands of one call.  Row = (batch row, channel), rows = batch * dim; I/O
// tensors are (rows, seqlen), per-row values (rows), per-channel ones (dim).
struct GlrArgs {
  int64_t rows;
  int64_t dim;
  int64_t seqlen;
  int32_t io;          // IoType
  int32_t kind;        // ss_glr_kind
  float decay_scale;
  const void* x;
  const void* r;
  const void* i;       // nullable
  const void* z;       // nullable
  const float* decay;  // nullable (convex)
  const float* r_bias; // nullable
  const float* i_bias; // nullable
  const float* h0;     // nullable; the step's state
  void* y;             // nullable: the sweep that only stores states
  float* h_final;      // nullable; the step's new state
  float* ckpt;         // nullable: (rows, ceil(seqlen / kGlrCkptTokens))
  // backward
  const void* dy;
  const float* dh_final;  // nullable
  void* dx;
  void* dr;
  void* di;            // non-null exactly when i is
  void* dz;            // non-null exactly when z is
  float* dh0;          // nullable
  float* sums;         // nullable: (3, rows) sums over a row's tokens: of decay, r_bias, i_bias
};

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s);
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s);
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t s);
// out[d] = sum over batch rows of sums[b, d], in order; null outputs are skipped
hipError_t launch_glr_reduce(int64_t batch, int64_t dim, const float* sums, float* ddecay, float* dr_bias,
                             float* di_bias, hipStream_t s);

}  // namespace ssscan
