// Internal interface of the gated delta rule (include/ssscan.h).
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace ssscan {

// Tokens that the chunked kernels take at once.
constexpr int kGdrChunk = 64;

// Strides in elements: batch row, token, head.
struct GdrArgs {
  int64_t batch;
  int64_t seqlen;
  int32_t hk, hv;        // key heads; value heads, a multiple of them
  int32_t dk, dv;
  int32_t io;            // IoType
  float scale;
  const void* q;
  const void* k;
  const void* v;
  int64_t qs[3], ks[3], vs[3];
  const float* g;        // (batch, seqlen, hv), nullable
  const float* beta;
  const float* h0;       // (batch, hv, dk, dv), nullable
  void* o;               // (batch, seqlen, hv, dv)
  float* h_final;        // nullable
  // chunked: what the preparation leaves for every (batch row, head, chunk)
  int64_t chunks;        // of a row
  // segments that a row's chunks go in, `per` chunks each but the last: with more than one, the state's change over each of them
  // but the last comes first, as a product with the state before it and a sum
  int64_t segments, per;
  float* ends;           // the state behind a segment, then the gradient of the one before it; dk rounded up to tiles of 32 by ldv
  float* moves;          // the factor, dk by dk rounded up to tiles of 32 (the first segment has the state before it and needs none),
  int32_t* moves_e;      // over a power of 2 for each 32 of its columns, four of them to a segment: what decays leave may be below 2^-126
  int32_t whole;         // dk and dv are multiples of 8 and the rows of q, k and v are aligned to 4 bytes
  void* tri;             // operand blocks of the inverse T
  void* tri_t;           // backward: of T transposed
  void* p;               // operand blocks of P; backward: of P transposed
  float* vecs;           // kVecs vectors
  int64_t ldv;           // dv rounded up to tiles of 32
  // backward, for every chunk of a head: rows of ldv columns as operands, and of each tile the largest |value| (of every kind in a run
  // of its own, max_apart floats behind the one before)
  float* states;         // the state before it
  float* u;              // U
  float* dstates;        // the gradient of the state behind it
  float* dr;             // the gradient of R
  float* maxima;
  int64_t max_apart;
  float* part_q;         // where value heads share keys: dq and dk of each alone, rows of dk rounded up to tiles of 32
  float* part_k;
  const void* dout;      // gradient of o
  const float* dh_final; // nullable
  void* dq;              // (batch, seqlen, hk, dk)
  void* dk_out;
  void* dv_out;          // (batch, seqlen, hv, dv)
  float* dg;             // nullable
  float* dbeta;          // nullable
  float* dh0;            // nullable
};

enum GdrMax { kMaxS, kMaxU, kMaxDs, kMaxDr, kMaxDo, kMaxKinds };

// Chunk by chunk on the matrix cores: what needs no state for all chunks at once, then the states in turn.
size_t gdr_tri_bytes(int64_t chunk_heads);                    // of tri, tri_t, p
size_t gdr_vecs_bytes(int64_t chunk_heads);
hipError_t launch_gdr_prep(const GdrArgs& a, bool backward, hipStream_t s);
hipError_t launch_gdr_chunk(const GdrArgs& a, bool states, hipStream_t s);
// Of more than one segment: from what each adds to a state, or to a state's gradient, and the factors to the states behind all but
// the last, the gradients before all but the first.
hipError_t launch_gdr_join(const GdrArgs& a, bool backward, hipStream_t s);
// Workgroups of a forward chunk kernel that the GPU holds at once.
int gdr_chunk_room(int io, int dk);
// The backward after the states: their gradients in turn, from the last chunk on, then all other gradients of all chunks.
hipError_t launch_gdr_chunk_bwd(const GdrArgs& a, hipStream_t s);
hipError_t launch_gdr_grad(const GdrArgs& a, hipStream_t s);

// Token by token, the state in registers: one token of a serving loop, and short sequences.
hipError_t launch_gdr_recur(const GdrArgs& a, hipStream_t s);
// Workgroups of its launch.
int64_t gdr_recur_blocks(int64_t batch, int hv, int dv);

}  // namespace ssscan
