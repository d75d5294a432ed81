// Internal interface of the norm and rotation of queries and keys (include/ssscan.h).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ssscan {

// One of the two inputs with what belongs to it.  Strides in elements: batch row, token, head.
struct QkSide {
  int32_t heads;
  const void* in;
  int64_t stride[3];
  const float* w;        // nullable
  void* out;             // forward
  const void* dout;      // backward: gradient of the output, in its layout
  void* din;             // backward
  int64_t dstride[3];
  float* dw;             // backward, nullable
};

struct QkArgs {
  int64_t batch;
  int64_t seqlen;
  int32_t n;             // head_dim
  int32_t half;          // rotated pairs, rot_dim / 2
  int32_t io;            // IoType
  int32_t interleaved;
  int32_t feature_major;
  float eps;
  float inv_n;           // 1 / head_dim
  const double* inv_freq;
  const int64_t* positions;  // nullable
  int64_t pos0;
  QkSide side[2];        // queries, keys
  float* part;           // backward: rows of n partial sums of dw, those of each side together
  int64_t part_row[2];   // backward: a side's first row and rows
  int64_t part_rows[2];
};

// The most workgroups, each with a row of partial sums, that a side has in the backward.
struct QkBwdPlan {
  int64_t blocks[2];
};
QkBwdPlan qk_bwd_plan(int64_t batch, int64_t seqlen, int heads_q, int heads_k, int n);

// Launch of the kernels for pairs in runs: lanes to a vector, and of each side the
// tokens of a workgroup and the workgroups.
struct QkRowsShape {
  int32_t lanes;
  int32_t tokens[2];
  int32_t blocks[2];
};

hipError_t launch_qk_norm_rot(const QkArgs& a, hipStream_t s);
// sets part_row and part_rows itself
hipError_t launch_qk_norm_rot_bwd(QkArgs a, hipStream_t s);

// The kernels behind them: feature-major outputs, token-major ones whose pairs come in
// runs (false where they do not), and token-major ones of any shape.
hipError_t launch_qk_cols(const QkArgs& a, hipStream_t s);
hipError_t launch_qk_cols_bwd(QkArgs& a, const QkBwdPlan& p, hipStream_t s);
bool qk_rows_take(const QkArgs& a);
hipError_t launch_qk_rows(const QkArgs& a, hipStream_t s);
hipError_t launch_qk_rows_bwd(QkArgs& a, const QkBwdPlan& p, hipStream_t s);

}  // namespace ssscan
