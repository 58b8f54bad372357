// Rotary positions and the paged append: what the C ABI hands to the kernels.
#pragma once

#include "da_internal.h"

namespace da {

struct RopeParams {
  const float *inv_freq;
  const int32_t *positions;   // [n_axes][pos_batch][T], or null
  long long pos_stride_axis;  // elements between axes
  long long pos_stride_b;     // elements between batch entries (0: shared)
  int n_pairs, n_axes;
  float sign;                 // +1 forward, -1 backward
  uint32_t axis_bits[DA_MAX_ROPE_PAIRS / 16];   // the pairs' axes, two bits each
};

// One [B, H, T, d] operand pair of the rotation (element strides).
struct RopeTensor {
  const void *in;
  void *out;
  long long in_b, in_h, in_t, out_b, out_h, out_t;
};

struct AppendArgs {
  const void *q, *k, *v;
  const float *demand;
  long long q_t, q_h, k_t, k_h, v_t, v_h, dem_t, dem_h;   // element strides (token, head)
  void *q_out;
  const int32_t *cu_tokens;
  int N, adjacent, hpt, units, tokens;                    // tokens: a block's run
  int *status;
};

// Rows in 16-byte pieces that hold whole pairs (or their halves), in 16-byte
// pieces otherwise, or of any alignment.
enum RopePath { kRopeUnits, kRopeAny, kRopeScalar };
cudaError_t launch_rope(const RopeTensor &q, const RopeTensor &k, const RopeParams &rp, bool adjacent, RopePath path,
                        int B, int Hq, int Hk, int T, int d, int dtype, cudaStream_t stream);
cudaError_t launch_append(const AppendArgs &args, const dilution_attn_paged_cache &c, const RopeParams &rp, bool vec,
                          cudaStream_t stream);

}  // namespace da
