// Internal interface of the gated linear recurrence (include/ssscan.h, ss_glr_*).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ssscan {

// Tokens between two stored states (ckpt): a piece of a row.  A tile is one, two or four pieces, or a
// shorter row as a whole.
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
  float* sums;         // nullable: (3, rows, parts) sums over pieces of a row: of decay, r_bias, i_bias
  void* chain;         // split rows: glr_chain_bytes of zeros
};

constexpr int64_t glr_tiles(int64_t seqlen) { return (seqlen + kGlrCkptTokens - 1) / kGlrCkptTokens; }
// Long rows, when there are about as many as CUs or fewer, are split over workgroups, a tile
// of one or more times kGlrCkptTokens each.  Whole calls, one after another, of the normalised kind with an
// input gate, one workgroup to a row -> split, fp32 forward / backward from stored states: 16 rows of 256K
// tokens 160 / 278 -> 25 / 44 us, 96 rows of 300001 191 / 447 -> 106 / 184; 64 rows of 5000 12 / 26 -> 18 / 31.
// Past 256 rows some CUs have two: training steps of 297 rows of 116288 tokens 373 -> 316, bf16 239 -> 208, of
// 40000 133 -> 122, bf16 89 -> 81, of 10000 37 -> 48; of 384 rows of 131072 451 -> 445, bf16 275 -> 286 us.
constexpr bool glr_split(int64_t rows, int64_t seqlen) {
  return seqlen > (rows < 256 ? 4 : 16) * kGlrCkptTokens && rows < 320;
}
// Tiles joined from one state, and the memory through which the tiles of split rows join.
constexpr int kGlrGroup = 32;
constexpr size_t glr_chain_bytes(int64_t rows, int64_t seqlen) {
  const int64_t tiles = glr_tiles(seqlen);
  return (size_t)rows * (tiles + (tiles + kGlrGroup - 1) / kGlrGroup + 1) * sizeof(uint64_t);
}

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s);
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s);
// The single token's most channels: its workgroups take 128 each, and a grid dimension holds fewer than 2^32
// threads, 256 to a workgroup.
constexpr int64_t kGlrStepDim = ((int64_t(1) << 24) - 1) * 128;
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t s);
// out[d] = sum over batch rows and parts of sums[b, d, part] in a fixed order; null outputs are skipped
hipError_t launch_glr_reduce(int64_t batch, int64_t dim, int64_t parts, const float* sums, float* ddecay,
                             float* dr_bias, float* di_bias, hipStream_t s);

}  // namespace ssscan
