// Eviction from the paged cache: what the C ABI hands to the kernels.
#pragma once

#include "da_internal.h"

namespace da {

struct EvictArgs {
  dilution_attn_paged_cache c;
  const int32_t *dst_page_table, *dst_demand_table;   // null: in place
  int dst_max_pages;
  const int32_t *keep;   // [S]
  int max_keep, max_len, sinks, recent;
  int32_t *new_lens;     // [S]
  int32_t *kept;         // [S][Hkv][max_keep], or null
  int *status;
  uint8_t *ws;
};

// Keys of a sequence in a cluster's shared memory; scores of more lie in the workspace.
constexpr int kEvictCtas = 8;
constexpr int kEvictKeys = 40 * 1024;   // a CTA's

constexpr int kEvictRows = 128;         // of 256 bytes (keys and values), a block's share
constexpr int kEvictTotals = 2048;      // totals, a block's share

struct EvictWorkspace {
  size_t info_off, list_off, flag_off, key_off, total;
  int total_chunks;     // of a query head
  int cluster, slice;   // CTAs a key head; keys of each, at most
  bool shared;          // the scores fit in shared memory
};
EvictWorkspace evict_workspace(int S, int Hkv, int max_keep, int max_len);
int launch_evict(const EvictArgs &a, cudaStream_t stream);

}  // namespace da
