// Checks of the C entry points that take rows of tokens under strides.
#pragma once

#include "api_checks.h"
#include "internal.h"

namespace ssscan {

// An operand of batch x seqlen x heads runs of n values under (batch, token, head) strides; `span` receives the elements
// it reaches over.
inline ss_status check_rows(const char* name, const void* p, const int64_t* st, int64_t batch, int64_t seqlen, int heads,
                            int n, ss_dtype io, int64_t* span) {
  if (!st) return record_error(SS_ERR_INVALID_ARG, "%s has no strides", name);
  if (seqlen > 0 && !p) return record_error(SS_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, elem_bytes(io))) return record_error(SS_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  for (int k = 0; k < 3; ++k)
    if (st[k] < 0) return record_error(SS_ERR_INVALID_ARG, "%s has a negative stride (%lld)", name, (long long)st[k]);
  *span = span_of(batch, seqlen, heads, n, st);
  if (*span < 0) return record_error(SS_ERR_INVALID_ARG, "the strides of %s overflow 64-bit byte offsets", name);
  return SS_OK;
}

inline ss_status check_disjoint(const Range* ins, int n_ins, const Range* outs, int n_outs) {
  for (int o = 0; o < n_outs; ++o) {
    for (int i = 0; i < n_ins; ++i)
      if (overlap(outs[o], ins[i]))
        return record_error(SS_ERR_INVALID_ARG, "%s overlaps input %s", outs[o].name, ins[i].name);
    for (int j = 0; j < o; ++j)
      if (overlap(outs[o], outs[j]))
        return record_error(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[j].name, outs[o].name);
  }
  return SS_OK;
}

inline ss_status check_scratch(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return SS_OK;
  if (!workspace) return record_error(SS_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned(workspace, 256)) return record_error(SS_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (bytes < need) return record_error(SS_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, need);
  return SS_OK;
}

}  // namespace ssscan
