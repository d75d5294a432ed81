// Internal interface of the norms before and after a block (include/ssscan.h).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ssscan {

// Rows of a tensor in units of elements: batch row, token, head.
struct NormRows {
  const void* p;
  int64_t stride[3];
};

// How rows are shared out: lanes to a row, vectors of 8 values to a lane, threads and workgroups.
struct NormPlan {
  int32_t lanes;
  int32_t vectors;
  int32_t threads;
  int32_t blocks;        // along x; along y a head each where every head has weights of its own
};

struct GatedNormArgs {
  int64_t tokens;        // batch * seqlen
  int64_t seqlen;
  int32_t heads;
  int32_t n;
  int32_t io;            // IoType
  int32_t gate_first;
  int32_t per_head;      // weights (heads, n) instead of (n)
  float eps;
  float inv_n;
  NormRows x, z;         // z.p nullable
  const float* w;        // nullable
  void* y;               // forward: (tokens, heads, n)
  const void* dy;        // backward, as y
  NormRows dx, dz;
  float* part;           // backward, nullable: blocks rows of n sums of dw (for every head)
  NormPlan plan;
};

struct ResidualNormArgs {
  int64_t rows;
  int32_t n;
  int32_t io;            // of x, y and their gradients
  int32_t rio;           // of the residual and its gradient
  int32_t post;
  float eps;
  float inv_n;
  float alpha;
  const void* x;         // backward: nullable without post and dscale
  const void* res;       // forward: nullable; backward: the sum that the forward wrote
  const float* w;        // these three nullable
  const float* w_post;
  const float* scale;
  void* y;
  void* res_out;         // forward, nullable
  const void* dy;
  const void* dres_out;  // nullable
  void* dx;              // nullable
  void* dres;            // nullable
  float* part[3];        // backward, each nullable: blocks rows of n sums of dw, dw_post, dscale
  NormPlan plan;
};

NormPlan gated_norm_plan(int64_t rows, int n, int heads_apart, bool backward);
NormPlan residual_norm_plan(int64_t rows, int n, bool backward);

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t s);
hipError_t launch_gated_norm_bwd(const GatedNormArgs& a, float* dw, hipStream_t s);
hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t s);
hipError_t launch_residual_norm_bwd(const ResidualNormArgs& a, float* const (&dw)[3], hipStream_t s);

}  // namespace ssscan
