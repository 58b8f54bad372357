// Paged decode: the host-side problem description and workspace layouts that
// the C ABI and the kernels share.
#pragma once

#include "da_internal.h"

namespace da {

// The kernels of a step that wait on barriers, for the test hook of their waits.
enum PagedKernel { kPagedKeys, kPagedValues, kPagedPrefixKeys, kPagedPrefixValues, kPagedKernels };

// Test hook: block stall_block[k] of kernel k keeps one thing that another role of
// it waits for (-1: none), and its waits give up after limit_ns[k] (the prefix's value
// kernel after the ordinary limit: it has no register left for another).
struct PagedDebug {
  unsigned long long limit_ns[kPagedKernels];
  int stall_block[kPagedKernels];
};

// One paged decode call.
struct PagedDecode {
  dilution_attn_paged_cache c;
  const void *q;
  void *out;
  const int32_t *prefix_table;   // null without a prefix
  int prefix_len;                // tokens of the shared prefix, a multiple of page_size
  int max_len;                   // host bound of seq_lens
  HeadScale hs;
  float eps;
  bool earlier;
  int *status;
  uint8_t *ws;
  PagedDebug dbg;
};

#if defined(__CUDACC__)
// Length of sequence s, 0 where it is not valid (then recorded once by the
// caller that passes `status`).
__device__ __forceinline__ int paged_len(const PagedDecode &p, int s, int *status) {
  const int len = __ldcg(p.c.seq_lens + s);
  if (len == 0) return 0;
  if (len < 0 || len > p.max_len || len < p.prefix_len) {
    if (status != nullptr) atomicCAS(status, DA_OK, DA_ERR_INVALID);
    return 0;
  }
  return len;
}
#endif

}  // namespace da
