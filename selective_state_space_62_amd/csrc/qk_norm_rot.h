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
  const double* inv_freq;
  const int64_t* positions;  // nullable
  int64_t pos0;
  QkSide side[2];        // queries, keys
  float* part;           // backward: rows of n partial sums of dw, those of each side together
  int64_t part_row[2];   // backward: a side's first row and rows
  int64_t part_rows[2];
};

// Head blocks of the backward and the most rows of partial sums that any of its kernels writes.
struct QkBwdPlan {
  int32_t heads_per_block;
  int32_t blocks[2];     // head blocks of each side
  int64_t token_blocks;  // most workgroups along the tokens
  int64_t rows() const { return token_blocks * (blocks[0] + blocks[1]); }
};
QkBwdPlan qk_bwd_plan(int64_t batch, int64_t seqlen, int heads_q, int heads_k);

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
