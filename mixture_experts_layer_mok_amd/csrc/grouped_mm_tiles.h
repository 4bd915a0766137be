// The tile kernel of the grouped product of 16-bit rows: which tiles there are and which workgroup
// computes them.  One source file for each of the three products (grouped_mm_out.hip,
// grouped_mm_rows.hip, grouped_mm_weights.hip), so that they compile side by side.
#pragma once
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "ops_launch.h"
#include "expert_rows.h"
#include "gemm_16.h"

namespace mok {
namespace g16 {

// Tile t of mt x nt: groups of kGroupM m-tiles, inside them all m-tiles of an n-tile before the
// next, so that the tiles that run at the same time share both operands' rows.
constexpr int kGroupM = 4;
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int* m, int* n) {
  const int g = t / (kGroupM * nt), r = t - g * kGroupM * nt;
  const int gm = min(kGroupM, mt - g * kGroupM);
  *n = r / gm;
  *m = g * kGroupM + r - *n * gm;
}

// The i-th tile of this workgroup, or -1: rounds of a tile for every workgroup.  Workgroups go to
// the eight XCDs in turn, and in each round XCD x takes the x-th eighth of the tiles, whose
// operands its L2 then holds.
__device__ __forceinline__ int tile_at(int i, int total) {
  const int g = int(gridDim.x), x = int(blockIdx.x & 7), j = int(blockIdx.x >> 3);
  const int first = i * g, n = min(total - first, g), per = (n + 7) / 8;
  return j < per && x * per + j < n ? first + x * per + j : -1;
}

// Results of a tile, to `out` at its first.
template <typename T>
__device__ __forceinline__ int store_tile(const T& tile, const MmArgs& p, int64_t first, int rows, int cols) {
  if (!p.out32) {
    tile.template store<false, false>(static_cast<uint16_t*>(p.out) + first, p.ld_out, rows, cols);
    return T::kStores16;
  }
  if (p.add) tile.template store<true, true>(static_cast<float*>(p.out) + first, p.ld_out, rows, cols);
  else tile.template store<true, false>(static_cast<float*>(p.out) + first, p.ld_out, rows, cols);
  return T::kStores32;
}

// out and d_a: rows of an expert times its weights.
template <int KIND, int TYPE, int IB, int JB>
__device__ __forceinline__ void walk_rows(const MmArgs& p, RowTiles<32 * IB>& til) {
  constexpr int BK = KIND == kMmOut ? kAlong : kAcross;
  const int cols = KIND == kMmOut ? p.n : p.k, deep = KIND == kMmOut ? p.k : p.n;
  const int nt = (cols + 32 * JB - 1) / (32 * JB), total = til.total * nt;
  const int steps = (deep + kDeep - 1) / kDeep;
  typedef Operand<kAlong, IB> A;
  typedef Operand<BK, JB> B;
  int i = 0, t = tile_at(0, total);
  if (t < 0) return;
  A a;
  B b;
  int m, n, e, r0, rows;
  auto open = [&]() __attribute__((always_inline)) {
    tile_of(t, til.total, nt, &m, &n);
    til.find(p, m, &e, &r0, &rows);
    const uint16_t* w = static_cast<const uint16_t*>(p.right) + int64_t(e) * p.n * p.k;
    a.init(static_cast<const uint16_t*>(p.left) + int64_t(r0) * p.ld_left, p.ld_left, rows, deep);
    b.init(KIND == kMmOut ? w + int64_t(n) * 32 * JB * p.k : w + n * 32 * JB, p.k, cols - n * 32 * JB, deep);
    Tile<TYPE, kAlong, BK, IB, JB>::begin(a, b);
  };
  open();
  int stores = 0;
  while (t >= 0) {
    Tile<TYPE, kAlong, BK, IB, JB> tile;
    tile.run(a, b, steps, stores);
    const int64_t first = int64_t(r0) * p.ld_out + n * 32 * JB;
    const int have = rows, left = cols - n * 32 * JB;
    t = tile_at(++i, total);
    if (t >= 0) open();
    stores = store_tile(tile, p, first, have, left);
  }
}

// d_b: the experts in the order of their rows, the most first, so that the tiles of a round take
// about as long as each other.
template <int TYPE, int IB, int JB>
__device__ __forceinline__ void walk_weights(const MmArgs& p) {
  const int mt = (p.n + 32 * IB - 1) / (32 * IB), nt = (p.k + 32 * JB - 1) / (32 * JB);
  const int per = mt * nt, total = per * p.groups, lane = threadIdx.x & 63;
  int rank = 0;
  if (p.groups <= 64) {
    int lo = 0, hi = 0;
    if (lane < p.groups) expert_rows(p, lane, &lo, &hi);
    const int have = lane < p.groups ? max(hi - lo, 0) : -1;
    for (int o = 0; o < p.groups; ++o) {
      const int other = __builtin_amdgcn_readlane(have, o);
      rank += other > have || (other == have && o < lane) ? 1 : 0;
    }
  }
  typedef Operand<kAcross, IB> A;
  typedef Operand<kAcross, JB> B;
  int i = 0, t = tile_at(0, total);
  if (t < 0) return;
  A a;
  B b;
  int m, n, e, rows;
  auto open = [&]() __attribute__((always_inline)) {
    e = t / per;
    tile_of(t - e * per, mt, nt, &m, &n);
    if (p.groups <= 64) e = __ffsll((unsigned long long)__ballot(rank == e && lane < p.groups)) - 1;
    int lo, hi;
    expert_rows(p, e, &lo, &hi);
    rows = __builtin_amdgcn_readfirstlane(max(hi - lo, 0));
    lo = __builtin_amdgcn_readfirstlane(lo);
    a.init(static_cast<const uint16_t*>(p.left) + int64_t(lo) * p.ld_left + m * 32 * IB, p.ld_left, p.n - m * 32 * IB,
           rows);
    b.init(static_cast<const uint16_t*>(p.right) + int64_t(lo) * p.ld_right + n * 32 * JB, p.ld_right,
           p.k - n * 32 * JB, rows);
    Tile<TYPE, kAcross, kAcross, IB, JB>::begin(a, b);
  };
  open();
  int stores = 0;
  while (t >= 0) {
    Tile<TYPE, kAcross, kAcross, IB, JB> tile;
    tile.run(a, b, (rows + kDeep - 1) / kDeep, stores);
    const int64_t first = (int64_t(e) * p.n + m * 32 * IB) * p.k + n * 32 * JB;
    const int have = p.n - m * 32 * IB, left = p.k - n * 32 * JB;
    t = tile_at(++i, total);
    if (t >= 0) open();
    stores = store_tile(tile, p, first, have, left);
  }
}

template <int KIND, int TYPE>
__global__ __launch_bounds__(kThr) void k_mm_tiles(MmArgs p) {
  if constexpr (KIND == kMmWeights) {
    walk_weights<TYPE, 8, 8>(p);
  } else {
    RowTiles<256> til;
    til.init(p);
    walk_rows<KIND, TYPE, 8, 8>(p, til);
  }
}

template <int KIND>
mok_status_t launch_tiles(const MmArgs& a, hipStream_t st) {
  const dim3 grid(256), block(kThr);
  return a.type == MOK_TYPE_BF16 ? launch(k_mm_tiles<KIND, MOK_TYPE_BF16>, grid, block, st, a)
                                 : launch(k_mm_tiles<KIND, MOK_TYPE_FP16>, grid, block, st, a);
}

}  // namespace g16
}  // namespace mok
