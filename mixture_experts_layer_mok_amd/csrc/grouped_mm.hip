// Grouped product of 16-bit rows and its gradients: for every expert e with the rows
// [offsets[e], offsets[e + 1])
//   out[r, c]    = sum_i a[r, i] b[e][c, i]
//   d_a[r, i]    = sum_c d_out[r, c] b[e][c, i]
//   d_b[e][c, i] = sum_r d_out[r, c] a[r, i]
// each a product left * right summed over one axis, in fp32 on the matrix cores (gemm_16.h,
// grouped_mm_tiles.h, grouped_mm_few.h).
#include <algorithm>

#include "ops_launch.h"

namespace mok {

// Where 128 x 128 tiles leave most of the card idle and the sums may be long enough, and where whole
// tiles may run whose last round has few (the launch that joins them takes 3 us where the routed rows
// then ask for no splitting).
bool mm_may_split(MmKind kind, int64_t max_rows, int32_t groups, int32_t n, int32_t k) {
  const int64_t cols = ((kind == kMmOut ? n : k) + 127) / 128;
  if (kind == kMmWeights) return int64_t(groups) * ((n + 127) / 128) * cols <= 256 && max_rows >= 2048;
  const int64_t m = std::min<int64_t>(max_rows, (max_rows + int64_t(groups) * 127) / 128);
  const int32_t deep = kind == kMmOut ? k : n;
  return (m * cols <= 256 && deep >= 1536) || (m * cols > 512 && deep >= 4096);
}

mok_status_t launch_grouped_mm(MmKind kind, const MmArgs& a, hipStream_t st) {
  if (kind == kMmOut) return launch_mm_out(a, st);
  if (kind == kMmRows) return launch_mm_rows(a, st);
  return a.scales ? launch_mm_weights_held(a, st) : launch_mm_weights(a, st);
}

}  // namespace mok
