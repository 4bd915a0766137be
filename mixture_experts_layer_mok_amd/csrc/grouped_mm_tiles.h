// The tile kernel of the grouped product of 16-bit rows: which tiles there are and which workgroup
// computes them.  One source file for each of the three products (grouped_mm_out.hip,
// grouped_mm_rows.hip, grouped_mm_weights.hip), so that they compile side by side.
#pragma once
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "ops_launch.h"
#include "expert_rows.h"
#include "grouped_mm_few.h"
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

template <int KIND, int IB, int JB>
using RowsLds = Lds<stage_bytes<kAlong, IB>(), stage_bytes<KIND == kMmOut ? kAlong : kAcross, JB>(), JB>;

// out and d_a: rows of an expert times its weights.  Tiles of few rows (the end of an expert's, or
// all of them) run with fewer row blocks.
template <int KIND, int TYPE, int IB, int JB>
__device__ __forceinline__ void walk_rows(const MmArgs& p, RowTiles& til) {
  constexpr int BK = KIND == kMmOut ? kAlong : kAcross;
  typedef RowsLds<KIND, IB, JB> LDS;
  const int cols = KIND == kMmOut ? p.n : p.k, deep = KIND == kMmOut ? p.k : p.n;
  const int nt = (cols + 32 * JB - 1) / (32 * JB), total = til.total * nt;
  const int steps = (deep + kDeep - 1) / kDeep;
  int i = 0, t = tile_at(0, total);
  if (t < 0) return;
  Operand<kAlong, IB> a;
  Operand<BK, JB> b;
  int m, n, e, r0, rows;
  auto with = [&](auto f) __attribute__((always_inline)) {  // f with the tile of as many rows as there are
    if (IB > 2 && rows > 64 * (IB / 4)) f(Tile<TYPE, kAlong, BK, IB, JB, LDS, IB>());
    else if (IB == 8 && rows > 64) f(Tile<TYPE, kAlong, BK, 4, JB, LDS, IB>());
    else f(Tile<TYPE, kAlong, BK, 2, JB, LDS, IB>());
  };
  auto open = [&]() __attribute__((always_inline)) {
    tile_of(t, til.total, nt, &m, &n);
    til.find(p, m, &e, &r0, &rows);
    const uint16_t* w = static_cast<const uint16_t*>(p.right) + int64_t(e) * p.n * p.k;
    a.init(static_cast<const uint16_t*>(p.left) + int64_t(r0) * p.ld_left, p.ld_left, rows, deep);
    b.init(KIND == kMmOut ? w + int64_t(n) * 32 * JB * p.k : w + n * 32 * JB, p.k, cols - n * 32 * JB, deep);
    with([&](auto tile) __attribute__((always_inline)) { tile.begin(a, b); });
  };
  open();
  int stores = 0;
  while (t >= 0) {
    with([&](auto tile) __attribute__((always_inline)) {
      tile.run(a, b, steps, stores);
      const int64_t first = int64_t(r0) * p.ld_out + n * 32 * JB;
      const int have = rows, left = cols - n * 32 * JB;
      t = tile_at(++i, total);
      if (t >= 0) open();
      stores = store_tile(tile, p, first, have, left);
    });
  }
}

// d_b: the experts in the order of their rows, the most first, so that the tiles of a round take
// about as long as each other.
template <int TYPE, int BK, int IB, int JB>
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
  typedef Lds<stage_bytes<kAcross, IB>(), stage_bytes<kAcross, JB>(), JB> LDS;
  typedef Tile<TYPE, kAcross, BK, IB, JB, LDS> T;
  int i = 0, t = tile_at(0, total);
  if (t < 0) return;
  typename T::A a;
  typename T::B b;
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
    const int left = p.k - n * 32 * JB;
    if constexpr (BK == kHeld)
      b.init(static_cast<const uint8_t*>(p.right) + int64_t(lo) * p.ld_right, p.ld_right,
             p.scales + int64_t(lo) * p.ld_scales, p.ld_scales, n * 32 * JB, left, rows);
    else
      b.init(static_cast<const uint16_t*>(p.right) + int64_t(lo) * p.ld_right + n * 32 * JB, p.ld_right, left, rows);
    T::begin(a, b);
  };
  open();
  int stores = 0;
  while (t >= 0) {
    T tile;
    tile.run(a, b, (rows + kDeep - 1) / kDeep, stores);
    const int64_t first = (int64_t(e) * p.n + m * 32 * IB) * p.k + n * 32 * JB;
    const int have = p.n - m * 32 * IB, left = p.k - n * 32 * JB;
    t = tile_at(++i, total);
    if (t >= 0) open();
    stores = store_tile(tile, p, first, have, left);
  }
}

// Which kernel has a product of rows, from estimates in microseconds: rounds of tiles times steps at
// what a step was measured to take, or the weights of the experts that have rows at 5.2 TB/s.
//   few:   every pass reads its expert's weights, and takes a third longer with more than 16 rows;
//   small: 128 x 128, two workgroups a CU: a step takes 0.72 where a CU has one at most, with two
//          0.95 forward and 1.1 for the rows' gradient (transposing reads);
//   whole: 256 x 256: 1.4 a step and 6 a tile.
// Measured on MI355X, us, whole / small / few forward:
//   N 4096, K 7168, 8 experts: 16 rows 109 / 95 / 87, 64 rows 109 / 95 / 92, 128 rows 109 / 95 / 106,
//     512 rows 119 / 102 / 229, 1024 rows 140 / 143, 2048 rows 169 / 209, 4096 rows 301 / 308; one
//     expert: 64 rows 95 / 78 / 34, 256 rows 144 / 85 / 85, 1024 rows 142 / 84
//   N 7168, K 2048, 8 experts: 512 rows 57 / 57 / 115, 2000 rows 102 / 97, 4000 rows 122 / 149
//   N 1024, K 1024, 8 experts: 256 rows 13 / 10 / 11, 4096 rows 27 / 21
// and whole / small for the rows' gradient: N 4096, K 7168, 8 experts: 64 rows 81 / 85, 1024 rows
// 104 / 143, 4096 rows 269 / 295; one expert, 256 rows 83 / 49; N 7168, K 2048: 512 rows 104 / 86,
// 2000 rows 146 / 127, 4000 rows 148 / 164.
enum Form { kFew, kSmall, kWhole };
template <int KIND>
__device__ __forceinline__ Form form_of(const MmArgs& p, RowTiles& t) {
  int n256 = 0, n128 = 0, n32 = 0, n16 = 0, live = 0;
  for (int e0 = 0; e0 < p.groups; e0 += 64) {
    t.read(p, e0);
    n256 += sum64(t.tiles_of(256));
    n128 += sum64(t.tiles_of(128));
    live += __popcll(__ballot(t.hi > t.lo));
    if (KIND == kMmOut) {
      n32 += sum64(t.tiles_of(kPassRows));
      n16 += sum64(t.tiles_of(16));
    }
  }
  const int cols = KIND == kMmOut ? p.n : p.k, deep = KIND == kMmOut ? p.k : p.n;
  const float steps = float((deep + kDeep - 1) / kDeep), weights = float(p.n) * float(p.k) * (2.f / 5.2e6f);
  const int whole = n256 * ((cols + 255) / 256), small = n128 * ((cols + 127) / 128);
  const float least = 1.05f * weights * float(live);
  const float us_small = 4.f + fmaxf(least, steps * (small <= 256 ? 0.72f : float((small + 511) / 512) *
                                                                               (KIND == kMmOut ? 0.95f : 1.1f)));
  const float us_whole = 4.f + fmaxf(least, float((whole + 255) / 256) * (1.4f * steps + 6.f));
  if (KIND == kMmOut) {
    const float items = float(n32) * float((p.n + 63) / 64);
    // (a wave's pair of chunks takes 1.5 at least, and four waves share the sum)
    const float us_few = 3.f + fmaxf((0.7f * float(n32) + 0.3f * float(n16)) * weights,
                                     ceilf(items / 512.f) * ceilf(float(p.k) / 1024.f) * 1.5f);
    if (us_few < fminf(us_small, us_whole)) return kFew;
  }
  return us_small < us_whole ? kSmall : kWhole;
}

// Whole tiles, a workgroup a CU; `both`: k_mm_small is launched too and the routed rows decide.
template <int KIND, int TYPE, int BK>
__global__ __launch_bounds__(kThr) void k_mm_tiles(MmArgs p, bool both) {
  if constexpr (KIND == kMmWeights) {
    walk_weights<TYPE, BK, 8, 8>(p);
  } else {
    RowTiles til;
    if (both && form_of<KIND>(p, til) != kWhole) return;
    til.init(p, 256, 0, both && p.groups <= 64);
    walk_rows<KIND, TYPE, 8, 8>(p, til);
  }
}
// Tiles of half the rows and columns, two workgroups a CU, and the kernel of few rows.
template <int KIND, int TYPE, int BK>
__global__ __launch_bounds__(kThr, 2) void k_mm_small(MmArgs p, bool both) {
  if constexpr (KIND == kMmWeights) {
    walk_weights<TYPE, BK, 4, 4>(p);
  } else {
    RowTiles til;
    const bool look = both || KIND == kMmOut;
    const Form form = look ? form_of<KIND>(p, til) : kSmall;
    if (both && form == kWhole) return;
    const bool have = look && p.groups <= 64;
    if constexpr (KIND == kMmOut) {
      typedef RowsLds<KIND, 4, 4> LDS;
      static_assert(kFewLds <= LDS::kBytes);
      if (form == kFew) {
        til.init(p, kPassRows, 0, have);
        walk_few<TYPE>(p, til, reinterpret_cast<f32x4_t*>(LDS::mem()));
        return;
      }
    }
    til.init(p, 128, 0, have);
    walk_rows<KIND, TYPE, 4, 4>(p, til);
  }
}

// Which kernels are launched: whole tiles alone where there may be four rounds of them (buffers hold
// about as many rows as are routed), small ones (and few rows) alone where these make a round at most,
// otherwise both, one of which returns at once (2 us).  A product of weights has its tiles whatever
// the rows.
template <int KIND, int BK>
mok_status_t launch_tiles(const MmArgs& a, hipStream_t st) {
  const int64_t cols = KIND == kMmOut ? a.n : a.k;
  auto tiles = [&](int64_t tall) {
    const int64_t m = KIND == kMmWeights
                          ? a.groups * ((a.n + tall - 1) / tall)
                          : std::min<int64_t>(a.max_rows, (a.max_rows + a.groups * (tall - 1)) / tall);
    return m * ((cols + tall - 1) / tall);
  };
  bool whole = tiles(256) >= 1024, small = tiles(128) <= 512;
  if (KIND == kMmWeights) {
    whole = tiles(256) >= 256;
    small = !whole;
  }
  const bool both = !whole && !small;
  mok_status_t s = MOK_OK;
  auto go = [&](auto kern, int grid) { return launch(kern, dim3(grid), dim3(kThr), st, a, both); };
  if (!whole)
    s = a.type == MOK_TYPE_BF16 ? go(k_mm_small<KIND, MOK_TYPE_BF16, BK>, 512) : go(k_mm_small<KIND, MOK_TYPE_FP16, BK>, 512);
  if (!small && s == MOK_OK)
    s = a.type == MOK_TYPE_BF16 ? go(k_mm_tiles<KIND, MOK_TYPE_BF16, BK>, 256) : go(k_mm_tiles<KIND, MOK_TYPE_FP16, BK>, 256);
  return s;
}

}  // namespace g16
}  // namespace mok
