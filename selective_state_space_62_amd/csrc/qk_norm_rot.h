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
  float* part;           // backward: (workgroups, 2, n) partial sums of dw
};

// Workgroups of the backward, each with a row of partial sums.
int64_t qk_bwd_blocks(int64_t batch, int64_t seqlen, int heads_q, int heads_k);

hipError_t launch_qk_norm_rot(const QkArgs& a, hipStream_t s);
hipError_t launch_qk_norm_rot_bwd(const QkArgs& a, hipStream_t s);

}  // namespace ssscan
