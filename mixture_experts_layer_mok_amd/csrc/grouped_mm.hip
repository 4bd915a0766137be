// Grouped product of 16-bit rows and its gradients: for every expert e with the rows
// [offsets[e], offsets[e + 1])
//   out[r, c]    = sum_i a[r, i] b[e][c, i]
//   d_a[r, i]    = sum_c d_out[r, c] b[e][c, i]
//   d_b[e][c, i] = sum_r d_out[r, c] a[r, i]
// each a product left * right summed over one axis, in fp32.  One thread sums 4 x 4 results of a
// 64 x 64 tile from fp32 copies in LDS.
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "ops_launch.h"

namespace mok {

namespace {

constexpr int kTile = 64, kStep = 16;

template <int TYPE>
__device__ __forceinline__ float value(const void* p, int64_t i) {
  const uint16_t u = static_cast<const uint16_t*>(p)[i];
  return TYPE == MOK_TYPE_BF16 ? bf16_to_f32(u) : float(__builtin_bit_cast(_Float16, u));
}
template <int TYPE>
__device__ __forceinline__ float rounded(float f) {
  return TYPE == MOK_TYPE_BF16 ? bf16_to_f32(f32_to_bf16(f)) : float(_Float16(f));
}

// Rows of expert e, cut to [0, max_rows).
__device__ __forceinline__ void expert_rows(const MmArgs& p, int e, int* lo, int* hi) {
  *lo = max(p.offsets[e], 0);
  *hi = int(min(int64_t(p.offsets[e + 1]), p.max_rows));
}

template <int KIND, int TYPE>
__global__ __launch_bounds__(256) void k_grouped_mm(MmArgs p) {
  __shared__ float s_l[kStep][kTile + 1], s_r[kStep][kTile + 1];
  int e = 0, lo = 0, hi = 0, m0 = 0;
  if (KIND == kMmWeights) {
    e = blockIdx.z;
    expert_rows(p, e, &lo, &hi);
    m0 = blockIdx.y * kTile;
  } else {
    int m = blockIdx.y;
    for (; e < p.groups; ++e) {
      expert_rows(p, e, &lo, &hi);
      const int tiles = hi > lo ? (hi - lo + kTile - 1) / kTile : 0;
      if (m < tiles) break;
      m -= tiles;
    }
    if (e == p.groups) return;
    m0 = lo + m * kTile;
  }
  const int n0 = blockIdx.x * kTile;
  const int M = KIND == kMmWeights ? p.n : hi, N = KIND == kMmOut ? p.n : p.k;
  const int K = KIND == kMmOut ? p.k : KIND == kMmRows ? p.n : max(hi - lo, 0);
  const int64_t b0 = int64_t(e) * p.n * p.k;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += kStep) {
    for (int i = threadIdx.x; i < kStep * kTile; i += 256) {
      const int q = KIND == kMmWeights ? i / kTile : i % kStep, m = KIND == kMmWeights ? i % kTile : i / kStep;
      float v = 0.f;
      if (k0 + q < K && m0 + m < M)
        v = KIND == kMmWeights ? value<TYPE>(p.left, int64_t(lo + k0 + q) * p.ld_left + m0 + m)
                               : value<TYPE>(p.left, int64_t(m0 + m) * p.ld_left + k0 + q);
      s_l[q][m] = v;
    }
    for (int i = threadIdx.x; i < kStep * kTile; i += 256) {
      const int q = KIND == kMmOut ? i % kStep : i / kTile, n = KIND == kMmOut ? i / kStep : i % kTile;
      float v = 0.f;
      if (k0 + q < K && n0 + n < N) {
        const int64_t r = lo + k0 + q, c = n0 + n;
        if (KIND == kMmOut) {
          v = value<TYPE>(p.right, b0 + c * p.k + k0 + q);
        } else if (KIND == kMmRows) {
          v = value<TYPE>(p.right, b0 + int64_t(k0 + q) * p.k + c);
        } else if (!p.scales) {
          v = value<TYPE>(p.right, r * p.ld_right + c);
        } else {
          const int s = p.scales[r * p.ld_scales + c / 32];
          v = __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(p.right)[r * p.ld_right + c], 0);
          v = s == 255 ? __uint_as_float(0x7FC00000u) : rounded<TYPE>(ldexpf(v, s - 127));
        }
      }
      s_r[q][n] = v;
    }
    __syncthreads();
    for (int q = 0; q < kStep; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += s_l[q][ty + 16 * i] * s_r[q][tx + 16 * j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, c = n0 + tx + 16 * j;
      if (m >= M || c >= N) continue;
      const int64_t at = (KIND == kMmWeights ? b0 : 0) + m * p.ld_out + c;
      if (p.out32) {
        float* o = static_cast<float*>(p.out) + at;
        *o = p.add ? *o + acc[i][j] : acc[i][j];
      } else if (TYPE == MOK_TYPE_BF16) {
        static_cast<uint16_t*>(p.out)[at] = f32_to_bf16(acc[i][j]);
      } else {
        static_cast<_Float16*>(p.out)[at] = _Float16(acc[i][j]);
      }
    }
}

}  // namespace

mok_status_t launch_grouped_mm(MmKind kind, const MmArgs& a, hipStream_t st) {
  if (!a.scales)
    return kind == kMmOut    ? launch_mm_out(a, st)
           : kind == kMmRows ? launch_mm_rows(a, st)
                             : launch_mm_weights(a, st);
  const int N = kind == kMmOut ? a.n : a.k;
  // every expert may end inside a tile
  const int64_t mt = std::min<int64_t>(a.max_rows, (a.max_rows + int64_t(a.groups) * (kTile - 1)) / kTile);
  const dim3 grid((N + kTile - 1) / kTile, unsigned(kind == kMmWeights ? (a.n + kTile - 1) / kTile : mt),
                  unsigned(kind == kMmWeights ? a.groups : 1));
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    return kind == kMmOut    ? launch(k_grouped_mm<kMmOut, T>, grid, dim3(256), st, a)
           : kind == kMmRows ? launch(k_grouped_mm<kMmRows, T>, grid, dim3(256), st, a)
                             : launch(k_grouped_mm<kMmWeights, T>, grid, dim3(256), st, a);
  };
  return a.type == MOK_TYPE_BF16 ? go(std::integral_constant<int, MOK_TYPE_BF16>())
                                 : go(std::integral_constant<int, MOK_TYPE_FP16>());
}

}  // namespace mok
