// Host-side helpers of the entry points over the paged cache (appending rows, tree attention,
// sampling, draft verification, page operations): error text, CUDA errors, alignment.
#pragma once
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cuda_runtime.h>

#include "../../include/irm.h"

namespace irm {

void set_last_error(const char* msg);  // irm_host.cu: the calling thread's irm_last_error()
// irm_host.cu: phase steps [32] and pairing of a RoPE variant (NULL: the default), checked.
irm_status select_rope(const irm_rope* rope, uint64_t* F, int* interleaved);

inline irm_status fail(irm_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

inline irm_status cuda_fail(cudaError_t e, const char* where) {
  return fail(IRM_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Offsets of a ragged batch's tree nodes: indptr[0] = 0, non-decreasing, at most IRM_MAX_TREE
// nodes a request.  Returns the largest tree in *max_nodes.
inline irm_status check_trees(const int32_t* indptr, int B, int* max_nodes) {
  if (B <= 0) return fail(IRM_ERR_INVALID_ARG, "B must be positive (got %d)", B);
  if (indptr == nullptr) return fail(IRM_ERR_INVALID_ARG, "null tree offsets");
  if (indptr[0] != 0) return fail(IRM_ERR_INVALID_ARG, "q_indptr[0] must be 0");
  int most = 0;
  for (int b = 0; b < B; ++b) {
    const int64_t n = (int64_t)indptr[b + 1] - indptr[b];
    if (n < 0) return fail(IRM_ERR_INVALID_ARG, "q_indptr decreases at request %d", b);
    if (n > IRM_MAX_TREE)
      return fail(IRM_ERR_UNSUPPORTED, "request %d has %lld tree nodes, more than %d", b, (long long)n, IRM_MAX_TREE);
    if (n > most) most = (int)n;
  }
  *max_nodes = most;
  return IRM_OK;
}

}  // namespace irm
