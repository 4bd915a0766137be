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

// Where a tile's results go.
struct Result {
  void* out;  // its first
  int64_t ld;
  bool out32, add;
};
__device__ __forceinline__ Result result(const MmArgs& p, int64_t first) {
  return {static_cast<uint8_t*>(p.out) + first * (p.out32 ? 4 : 2), p.ld_out, p.out32, p.add};
}
__device__ __forceinline__ Result partial(const MmArgs& p, int item, int tall = 128, int wide = 128) {
  return {p.ws + int64_t(item) * (tall * wide), wide, true, false};
}
template <typename T>
__device__ __forceinline__ int store_tile(const T& tile, const Result& r, int rows, int cols) {
  if (!r.out32) {
    tile.template store<false, false>(r.out, r.ld, rows, cols);
    return T::kStores16;
  }
  if (r.add) tile.template store<true, true>(r.out, r.ld, rows, cols);
  else tile.template store<true, false>(r.out, r.ld, rows, cols);
  return T::kStores32;
}

template <int KIND, int IB, int JB>
using RowsLds = Lds<stage_bytes<kAlong, IB>(), stage_bytes<KIND == kMmOut ? kAlong : kAcross, JB>(), JB>;

// Sums split over workgroups: every tile is summed in `splits` items of `per` steps each, the partial
// results go to the workspace, 64 KB an item, and k_mm_join adds them up in order.  As many items as
// take the least by estimate, in microseconds: 0.72 a step where a CU has one item at most, 0.95 with
// two, and, where sums are split, 5 for the second launch and 0.033 an item to write it and read it
// again.  Measured on MI355X, without and with splitting: 2000 rows of one expert, n 8192, k 64, rows'
// gradient 81 -> 22 us; 256 rows, n 4096, k 7168, forward 85 -> 36; weights' gradient of 16,384 rows,
// n 1024, k 1024 170 -> 55, n 64, k 64 129 -> 25; and, always split, where that does not pay: 4096
// rows, n 1024, k 1024, forward 14 -> 29.
struct Split {
  int splits, per;
};
constexpr int kItems = int(MOK_MM_WORKSPACE_BYTES / (128 * 128 * 4));  // 512: two workgroups a CU
constexpr int kLeastSteps = 8;  // of an item
__device__ __forceinline__ float split_us(int steps, int items, bool split) {
  return float(steps) * (items <= 256 ? 0.72f : 0.95f) + (split ? 5.f + 0.033f * float(items) : 0.f);
}
__device__ __forceinline__ Split split_of(const MmArgs& p, int tiles, int steps) {
  Split best = {1, steps};
  if (!p.ws || tiles <= 0) return best;
  float us = split_us(steps, tiles, false);
  for (int s = 2; s * tiles <= kItems && s * kLeastSteps <= steps; s *= 2) {
    const int per = (steps + s - 1) / s;
    const float t = split_us(per, s * tiles, true);
    if (t < us) {
      us = t;
      best = {(steps + per - 1) / per, per};
    }
  }
  return best;
}

// The last round of whole tiles, if it has at most half of the workgroups: its tiles are summed in
// `splits` items of `per` steps each, as above; an item holds `tall` rows, as many as the round's
// tallest tile needs.  A step takes 1.4 us in a whole tile, 1.1 with at most 128 rows and 0.95 with 64
// (the loads' latency: two steps are in flight, whatever the tile).  Measured on MI355X, without and
// with, us: 16,384 rows of 8 experts with about 2048 each, N 4096, K 7168 (1024 tiles and 64 of a few
// rows) 790 / 739, rows' gradient 784 / 754; 8192 rows, N 2048, K 4096 162 / 132; 4000 rows, N 4096,
// K 7168 311 / 220; 4400 rows of one expert 275 / 222; the launch that joins costs 3 to 5 where the
// routed rows leave no such round (3777 rows, skewed, N 7168, K 4096: 216 / 222), so short sums (less
// than 4096) are left alone.
constexpr int kRound = 256;  // workgroups of whole tiles
struct Tail {
  int first, tiles, splits, per, tall;
  float us;  // what the round takes
};
__device__ __forceinline__ Tail tail_of(const MmArgs& p, RowTiles& t, int nt, int steps) {
  const int total = t.total * nt, first = total / kRound * kRound, r = total - first;
  Tail best = {total, 0, 1, steps, 256, 0.f};
  if (r == 0) return best;
  best.us = 1.4f * float(steps) + 6.f;
  if (!p.ws || !t.sorted || 2 * r > kRound) return best;
  int e, r0, rows;
  t.find(p, first / (kGroupM * nt) * kGroupM, &e, &r0, &rows);  // (none after it needs more)
  const int tall = rows > 128 ? 256 : rows > 64 ? 128 : 64;
  const float step = tall == 256 ? 1.4f : tall == 128 ? 1.1f : 0.95f;
  best.us = step * float(steps) + 6.f;
  for (int n = 2; n * r <= kRound && n * r * tall <= int(MOK_MM_WORKSPACE_BYTES / 1024) && n * kLeastSteps <= steps;
       n *= 2) {
    const int per = (steps + n - 1) / n;
    const float us = step * float(per) + 11.f + 0.033f * float(n * r * (tall / 64));
    if (us < best.us) best = {first, r, (steps + per - 1) / per, per, tall, us};
  }
  return best;
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
__device__ __forceinline__ Form form_of(const MmArgs& p, RowTiles& t, bool both) {
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
  const Split sp = split_of(p, small, int(steps));
  const int items = small * sp.splits;
  const float us_small =
      4.f + (sp.splits > 1 ? 5.f : 0.f) +
      fmaxf(least, float(sp.per) * (items <= 256 ? 0.72f : float((items + 511) / 512) *
                                                               (KIND == kMmOut ? 0.95f : 1.1f)));
  float us_whole = 1e30f;
  if (both) {
    us_whole = float((whole + 255) / 256) * (1.4f * steps + 6.f);
    if (p.ws && p.groups <= 64 && whole % kRound != 0) {
      t.init_sorted(p, 256, true);
      us_whole = float(whole / 256) * (1.4f * steps + 6.f) + tail_of(p, t, (cols + 255) / 256, int(steps)).us;
    }
    us_whole = 4.f + fmaxf(least, us_whole);
  }
  if (KIND == kMmOut) {
    const float passes = float(n32) * float((p.n + 63) / 64);
    // (a wave's pair of chunks takes 1.5 at least, and four waves share the sum)
    const float us_few = 3.f + fmaxf((0.7f * float(n32) + 0.3f * float(n16)) * weights,
                                     ceilf(passes / 512.f) * ceilf(float(p.k) / 1024.f) * 1.5f);
    if (us_few < fminf(us_small, us_whole)) return kFew;
  }
  return us_small < us_whole ? kSmall : kWhole;
}

// out and d_a: rows of an expert times its weights.  Tiles of few rows (the end of an expert's, or
// all of them) run with fewer row blocks.
template <int KIND, int TYPE, int IB, int JB>
__device__ __forceinline__ void walk_rows(const MmArgs& p, RowTiles& til) {
  constexpr int BK = KIND == kMmOut ? kAlong : kAcross;
  constexpr bool kSplit = IB == 4;
  typedef RowsLds<KIND, IB, JB> LDS;
  const int cols = KIND == kMmOut ? p.n : p.k, deep = KIND == kMmOut ? p.k : p.n;
  const int nt = (cols + 32 * JB - 1) / (32 * JB), tiles = til.total * nt;
  const int steps = (deep + kDeep - 1) / kDeep;
  const Split sp = kSplit ? split_of(p, tiles, steps) : Split{1, steps};
  const Tail tail = kSplit ? Tail{0, tiles, sp.splits, sp.per, 128, 0.f} : tail_of(p, til, nt, steps);
  const int total = tail.first + tail.tiles * tail.splits;
  int i = 0, t = tile_at(0, total);
  if (t < 0) return;
  Operand<kAlong, IB> a;
  Operand<BK, JB> b;
  int m, n, e, r0, rows, item, now;  // now: steps
  auto with = [&](auto f) __attribute__((always_inline)) {  // f with the tile of as many rows as there are
    if (IB > 2 && rows > 64 * (IB / 4)) f(Tile<TYPE, kAlong, BK, IB, JB, LDS, IB>());
    else if (IB == 8 && rows > 64) f(Tile<TYPE, kAlong, BK, 4, JB, LDS, IB>());
    else f(Tile<TYPE, kAlong, BK, 2, JB, LDS, IB>());
  };
  auto open = [&]() __attribute__((always_inline)) {
    const bool cut = t >= tail.first;
    const int s = cut ? (t - tail.first) / tail.tiles : 0, per = cut ? tail.per : steps, k0 = s * per * kDeep;
    item = t;
    now = min(per, steps - s * per);
    tile_of(t - s * tail.tiles, til.total, nt, &m, &n);
    til.find(p, m, &e, &r0, &rows);
    const int sum = min(deep - k0, per * kDeep);
    const uint16_t* w = static_cast<const uint16_t*>(p.right) + int64_t(e) * p.n * p.k;
    a.init(static_cast<const uint16_t*>(p.left) + int64_t(r0) * p.ld_left + k0, p.ld_left, rows, sum);
    b.init(KIND == kMmOut ? w + int64_t(n) * 32 * JB * p.k + k0 : w + int64_t(k0) * p.k + n * 32 * JB, p.k,
           cols - n * 32 * JB, sum);
    with([&](auto tile) __attribute__((always_inline)) { tile.begin(a, b); });
  };
  open();
  int stores = 0;
  while (t >= 0) {
    with([&](auto tile) __attribute__((always_inline)) {
      tile.run(a, b, now, stores);
      const Result res = tail.splits > 1 && item >= tail.first
                             ? partial(p, item - tail.first, tail.tall, 32 * JB)
                             : result(p, int64_t(r0) * p.ld_out + n * 32 * JB);
      const int have = rows, left = cols - n * 32 * JB;
      t = tile_at(++i, total);
      if (t >= 0) open();
      stores = store_tile(tile, res, have, left);
    });
  }
}

// Opens d_b's tile (m, n) over `rows` rows from r0 on.
template <int BK, int IB, int JB, typename A, typename B>
__device__ __forceinline__ void open_weights(const MmArgs& p, A& a, B& b, int r0, int rows, int m, int n) {
  a.init(static_cast<const uint16_t*>(p.left) + int64_t(r0) * p.ld_left + m * 32 * IB, p.ld_left, p.n - m * 32 * IB,
         rows);
  const int left = p.k - n * 32 * JB;
  if constexpr (BK == kHeld)
    b.init(static_cast<const uint8_t*>(p.right) + int64_t(r0) * p.ld_right, p.ld_right,
           p.scales + int64_t(r0) * p.ld_scales, p.ld_scales, n * 32 * JB, left, rows);
  else
    b.init(static_cast<const uint16_t*>(p.right) + int64_t(r0) * p.ld_right + n * 32 * JB, p.ld_right, left, rows);
}

// d_b in small tiles.  An expert's rows are cut into units of at most `per` steps, so that all units'
// tiles make no more items than the workspace holds; an expert without rows has one, of zeros.  An
// expert of several units has its partial results joined.
__device__ __forceinline__ int unit_steps(const MmArgs& p, RowTiles& til, int per_unit) {
  int best = 1 << 18;  // (steps of 64 rows: more than there can be)
  if (!p.ws) return best;
  til.init(p, kDeep);
  const int most = til.most;
  float us = split_us(most, min(per_unit * p.groups, kItems), false);
  for (int items = 64; items <= kItems; items *= 2) {
    const int units = items / per_unit - p.groups;  // units are at most steps / per + groups
    if (units <= 0) continue;
    const int per = max(kLeastSteps, (til.total + units - 1) / units);
    const float t = split_us(per, items, true);
    if (per < most && t < us) {
      us = t;
      best = per;
    }
  }
  return best;
}
template <int TYPE, int BK, int IB, int JB>
__device__ __forceinline__ void walk_units(const MmArgs& p) {
  const int mt = (p.n + 32 * IB - 1) / (32 * IB), nt = (p.k + 32 * JB - 1) / (32 * JB), tiles = mt * nt;
  RowTiles til;
  til.init(p, kDeep * unit_steps(p, til, tiles), 1);
  const int total = tiles * til.total;
  typedef Lds<stage_bytes<kAcross, IB>(), stage_bytes<kAcross, JB>(), JB> LDS;
  typedef Tile<TYPE, kAcross, BK, IB, JB, LDS> T;
  int i = 0, t = tile_at(0, total);
  if (t < 0) return;
  typename T::A a;
  typename T::B b;
  int m, n, e, r0, rows, part, parts, item;
  auto open = [&]() __attribute__((always_inline)) {
    item = t;
    til.find(p, t / tiles, &e, &r0, &rows, &part, &parts);
    tile_of(t % tiles, mt, nt, &m, &n);
    open_weights<BK, IB, JB>(p, a, b, r0, rows, m, n);
    T::begin(a, b);
  };
  open();
  int stores = 0;
  while (t >= 0) {
    T tile;
    tile.run(a, b, (rows + kDeep - 1) / kDeep, stores);
    const Result res = parts > 1 ? partial(p, item)
                                 : result(p, (int64_t(e) * p.n + m * 32 * IB) * p.k + n * 32 * JB);
    const int have = p.n - m * 32 * IB, left = p.k - n * 32 * JB;
    t = tile_at(++i, total);
    if (t >= 0) open();
    stores = store_tile(tile, res, have, left);
  }
}

// Which kernels of a product are launched.
enum Launched { kOnlySmall, kOnlyWhole, kBoth };

// Partial results added up, in the order of their items.  A thread has eight elements.
template <int KIND, int TYPE>
__global__ __launch_bounds__(256) void k_mm_join(MmArgs p, Launched what) {
  const int rows_of = KIND == kMmWeights ? p.n : 0, cols = KIND == kMmOut ? p.n : p.k;
  const int steps = ((KIND == kMmOut ? p.k : p.n) + kDeep - 1) / kDeep;
  RowTiles til;
  int splits = 1, units = 1, tiles, tall = 128, wide = 128, begin = 0;
  if (KIND == kMmWeights) {
    tiles = ((rows_of + 127) / 128) * ((cols + 127) / 128);
    til.init(p, kDeep * unit_steps(p, til, tiles), 1);
    units = til.total;
  } else {
    const Form form = what == kOnlyWhole                   ? kWhole
                      : what == kBoth || KIND == kMmOut ? form_of<KIND>(p, til, what == kBoth)
                                                           : kSmall;
    if (form == kFew) return;
    if (form == kWhole) {
      til.init_sorted(p, 256);
      wide = 256;
      const Tail x = tail_of(p, til, (cols + 255) / 256, steps);
      tiles = x.tiles;
      splits = x.splits;
      tall = x.tall;
      begin = x.first;
    } else {
      til.init(p, 128);
      tiles = til.total * ((cols + 127) / 128);
      splits = split_of(p, tiles, steps).splits;
    }
    if (splits == 1) return;
  }
  const int mt = (rows_of + 127) / 128, nt = (cols + wide - 1) / wide;
  const int across = wide / 8, parts_of = tall * across / 256;  // threads a row, workgroups a tile
  for (int t = blockIdx.x; t < units * tiles * parts_of; t += int(gridDim.x)) {
    const int x = t / parts_of;
    const int row = (t - x * parts_of) * (256 / across) + int(threadIdx.x) / across, col = int(threadIdx.x) % across * 8;
    int m, n, e, r0, rows, part, parts = splits;
    int64_t at;
    if (KIND == kMmWeights) {
      til.find(p, x / tiles, &e, &r0, &rows, &part, &parts);
      if (part != 0 || parts == 1) continue;
      tile_of(x % tiles, mt, nt, &m, &n);
      rows = p.n - m * 128;
      at = (int64_t(e) * p.n + m * 128 + row) * p.k;
    } else {
      tile_of(begin + x, til.total, nt, &m, &n);
      til.find(p, m, &e, &r0, &rows);
      at = int64_t(r0 + row) * p.ld_out;
    }
    if (row >= rows || n * wide + col >= cols) continue;
    at += n * wide + col;
    const f32x4_t* from = reinterpret_cast<const f32x4_t*>(p.ws) + (int64_t(x) * tall + row) * (wide / 4) + col / 4;
    const int64_t stride = int64_t(tiles) * tall * (wide / 4);
    f32x4_t lo = from[0], hi = from[1];
    for (int s = 1; s < parts; ++s) {
      from += stride;
      lo += from[0];
      hi += from[1];
    }
    if (p.out32) {
      f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at);
      if (p.add) {
        lo += o[0];
        hi += o[1];
      }
      o[0] = lo;
      o[1] = hi;
    } else {
      *reinterpret_cast<v4u*>(static_cast<uint16_t*>(p.out) + at) =
          v4u{pack2<TYPE>(lo.x, lo.y), pack2<TYPE>(lo.z, lo.w), pack2<TYPE>(hi.x, hi.y), pack2<TYPE>(hi.z, hi.w)};
    }
  }
}

// d_b in whole tiles: the experts in the order of their rows, the most first, so that the tiles of a round take
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
    open_weights<BK, IB, JB>(p, a, b, lo, rows, m, n);
    T::begin(a, b);
  };
  open();
  int stores = 0;
  while (t >= 0) {
    T tile;
    tile.run(a, b, (rows + kDeep - 1) / kDeep, stores);
    const Result res = result(p, (int64_t(e) * p.n + m * 32 * IB) * p.k + n * 32 * JB);
    const int have = p.n - m * 32 * IB, left = p.k - n * 32 * JB;
    t = tile_at(++i, total);
    if (t >= 0) open();
    stores = store_tile(tile, res, have, left);
  }
}

// Whole tiles, a workgroup a CU; `both`: k_mm_small is launched too and the routed rows decide.
template <int KIND, int TYPE, int BK>
__global__ __launch_bounds__(kThr) void k_mm_tiles(MmArgs p, bool both) {
  if constexpr (KIND == kMmWeights) {
    walk_weights<TYPE, BK, 8, 8>(p);
  } else {
    RowTiles til;
    if (both && form_of<KIND>(p, til, true) != kWhole) return;
    til.init_sorted(p, 256, both && p.groups <= 64);
    walk_rows<KIND, TYPE, 8, 8>(p, til);
  }
}
// Tiles of half the rows and columns, two workgroups a CU, and the kernel of few rows.
template <int KIND, int TYPE, int BK>
__global__ __launch_bounds__(kThr, 2) void k_mm_small(MmArgs p, bool both) {
  if constexpr (KIND == kMmWeights) {
    walk_units<TYPE, BK, 4, 4>(p);
  } else {
    RowTiles til;
    const bool look = both || KIND == kMmOut;
    const Form form = look ? form_of<KIND>(p, til, both) : kSmall;
    if (form == kWhole) return;
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

// (a.ws is set only where sums may be split.)
// Which kernels are launched: whole tiles alone where there may be four rounds of them (buffers hold
// about as many rows as are routed), small ones (and few rows) alone where these make a round at most,
// otherwise both, one of which returns at once (4 us).  A product of weights has its tiles whatever
// the rows; with two steps an expert or fewer they are small ones, two of which a CU has in flight: what
// counts is to write the results.  MI355X, us, into fp32, whole / small: 2 rows of 32 experts, N 3432,
// K 128 17.6 / 13.1, 25 of 13, N 3048, K 400 20.3 / 17.6, 1000 of 8, N 2048, K 2048 32.6 / 28.9, N 4096,
// K 7168 188 / 183; with four steps 2000 of 8, N 4096, K 2048 65.8 / 68.1, with eight 94.5 / 114.
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
    // (up to 256 small ones their sums may be split)
    whole = tiles(256) >= 256 && tiles(128) > 256 && a.max_rows > 128 * int64_t(a.groups);
    small = !whole;
  }
  const bool both = !whole && !small;
  const Launched what = whole ? kOnlyWhole : small ? kOnlySmall : kBoth;
  mok_status_t s = MOK_OK;
  auto go = [&](auto kern, int grid) { return launch(kern, dim3(grid), dim3(kThr), st, a, both); };
  if (!whole)
    s = a.type == MOK_TYPE_BF16 ? go(k_mm_small<KIND, MOK_TYPE_BF16, BK>, 512) : go(k_mm_small<KIND, MOK_TYPE_FP16, BK>, 512);
  if (!small && s == MOK_OK)
    s = a.type == MOK_TYPE_BF16 ? go(k_mm_tiles<KIND, MOK_TYPE_BF16, BK>, kRound) : go(k_mm_tiles<KIND, MOK_TYPE_FP16, BK>, kRound);
  if (a.ws && s == MOK_OK) {
    const dim3 grid(512), block(256);
    s = a.type == MOK_TYPE_BF16 ? launch(k_mm_join<KIND, MOK_TYPE_BF16>, grid, block, st, a, what)
                                : launch(k_mm_join<KIND, MOK_TYPE_FP16>, grid, block, st, a, what);
  }
  return s;
}

}  // namespace g16
}  // namespace mok
