// Grouped product of 16-bit rows and its gradients: for every expert e with the rows
// [offsets[e], offsets[e + 1])
//   out[r, c]    = sum_i a[r, i] b[e][c, i]
//   d_a[r, i]    = sum_c d_out[r, c] b[e][c, i]
//   d_b[e][c, i] = sum_r d_out[r, c] a[r, i]
// each a product left * right summed over one axis, in fp32 on the matrix cores (gemm_16.h,
// grouped_mm_tiles.h, grouped_mm_few.h).
#include "ops_launch.h"

namespace mok {

mok_status_t launch_grouped_mm(MmKind kind, const MmArgs& a, hipStream_t st) {
  if (kind == kMmOut) return launch_mm_out(a, st);
  if (kind == kMmRows) return launch_mm_rows(a, st);
  return a.scales ? launch_mm_weights_held(a, st) : launch_mm_weights(a, st);
}

}  // namespace mok
