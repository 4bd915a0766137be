// The tile kernel of the grouped product of 16-bit rows: which tiles there are and which workgroup
// computes them.  One source file for each of the three products (grouped_mm_out.hip,
// grouped_mm_rows.hip, grouped_mm_weights.hip), so that they compile side by side.
#pragma once
#include <type_traits>

#include "device.h"
#include "ops_launch.h"
#include "expert_rows.h"
#include "grouped_mm_few.h"
#include "gemm_16.h"
#include "mm_forms.h"

namespace mok {
namespace g16 {

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

__device__ __forceinline__ Split split_of(const MmArgs& p, int tiles, int steps) { return split_of(p.ws != nullptr, tiles, steps); }
__device__ __forceinline__ Tail tail_of(const MmArgs& p, RowTiles& t, int nt, int steps) {
  return tail_of(p.ws && t.sorted, t.total, nt, steps, [&](int m) __attribute__((always_inline)) {
    int e, r0, rows;
    t.find(p, m, &e, &r0, &rows);
    return rows;
  });
}
template <int KIND>
__device__ __forceinline__ Form form_of(const MmArgs& p, RowTiles& t, bool both) {
  Counts c = {0, 0, 0, 0, 0};
  for (int e0 = 0; e0 < p.groups; e0 += 64) {
    t.read(p, e0);
    c.n256 += sum64(t.tiles_of(256));
    c.n128 += sum64(t.tiles_of(128));
    c.live += __popcll(__ballot(t.hi > t.lo));
    if (KIND == kMmOut) {
      c.n32 += sum64(t.tiles_of(kPassRows));
      c.n16 += sum64(t.tiles_of(16));
    }
  }
  return form_of(MmKind(KIND), c, p.n, p.k, p.ws != nullptr, p.ws && p.groups <= 64, both,
                 [&](int nt, int steps) __attribute__((always_inline)) {
                   t.init_sorted(p, 256, true);
                   return tail_of(p, t, nt, steps);
                 });
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

// d_b in small tiles.  An expert's rows are cut into units of at most `per` steps; an expert without rows
// has one, of zeros.  An expert of several units has its partial results joined.
__device__ __forceinline__ int unit_steps(const MmArgs& p, RowTiles& til, int per_unit) {
  if (!p.ws) return kWholeExpert;
  til.init(p, kDeep);
  return unit_steps(til.total, til.most, per_unit, p.groups);
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
template <int KIND, int BK>
mok_status_t launch_tiles(const MmArgs& a, hipStream_t st) {
  const Launched what = launched(MmKind(KIND), a.max_rows, a.groups, a.n, a.k);
  const bool both = what == kBoth;
  mok_status_t s = MOK_OK;
  auto go = [&](auto kern, int grid) { return launch(kern, dim3(grid), dim3(kThr), st, a, both); };
  if (what != kOnlyWhole)
    s = a.type == MOK_TYPE_BF16 ? go(k_mm_small<KIND, MOK_TYPE_BF16, BK>, 512) : go(k_mm_small<KIND, MOK_TYPE_FP16, BK>, 512);
  if (what != kOnlySmall && s == MOK_OK)
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
