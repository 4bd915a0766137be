// Which kernels a grouped product of 16-bit rows launches, which form of it then runs and how its sums
// are split, from sizes and counts of tiles alone.
//
// k_mm_small, k_mm_tiles and k_mm_join are compiled apart and have to come to the same answers: where they
// did not, nobody would write the results, or the wrong partial results would be added up.  So every
// answer is computed here, in operations that are rounded one by one (a multiplication and an addition
// that one kernel fuses and another does not differ in the last bit, and so may the comparison after them:
// 89 steps of two full rounds and 125 tiles of at most 128 rows was such a tie).  Also compiled for the
// host, where mm_forms_check.cpp says what a call's answers are.
#pragma once
#include <cstdint>

#include "../../include/mok.h"

#if defined(__HIP__)
#define MOK_FORMS __host__ __device__ __forceinline__
#else
#define MOK_FORMS inline
#endif

namespace mok {

// C = A B summed over one axis:
//   kMmOut      out[r, c]  = sum_i a[r, i] b[e][c, i]      left a, right b
//   kMmRows     d_a[r, i]  = sum_c d_out[r, c] b[e][c, i]  left d_out, right b
//   kMmWeights  d_b[e][c, i] = sum_r d_out[r, c] a[r, i]   left d_out, right a
enum MmKind { kMmOut = 0, kMmRows = 1, kMmWeights = 2 };

namespace g16 {

constexpr int kDeep = 64;      // summed elements a step
constexpr int kPassRows = 32;  // rows a pass of the few-rows form
constexpr int kRound = 256;    // workgroups of whole tiles

// Tile t of mt x nt: groups of kGroupM m-tiles, inside them all m-tiles of an n-tile before the
// next, so that the tiles that run at the same time share both operands' rows.
constexpr int kGroupM = 4;
MOK_FORMS void tile_of(int t, int mt, int nt, int* m, int* n) {
  const int g = t / (kGroupM * nt), r = t - g * kGroupM * nt;
  const int gm = mt - g * kGroupM < kGroupM ? mt - g * kGroupM : kGroupM;
  *n = r / gm;
  *m = g * kGroupM + r - *n * gm;
}

// The rows [from, to) of an expert, cut to [0, max_rows); none where hi <= lo.  Neither end is negative,
// whatever the offsets are, so that hi - lo does not overflow.
MOK_FORMS void cut_rows(int from, int to, int64_t max_rows, int* lo, int* hi) {
  *lo = from > 0 ? from : 0;
  *hi = to <= 0 ? 0 : to < max_rows ? to : int(max_rows);
}

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
MOK_FORMS float split_us(int steps, int items, bool split) {
#pragma clang fp contract(off)
  return float(steps) * (items <= 256 ? 0.72f : 0.95f) + (split ? 5.f + 0.033f * float(items) : 0.f);
}
// may: there is a workspace.
MOK_FORMS Split split_of(bool may, int tiles, int steps) {
  Split best = {1, steps};
  if (!may || tiles <= 0) return best;
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
struct Tail {
  int first, tiles, splits, per, tall;
  float us;  // what the round takes
};
// may: there is a workspace, and the tiles of few rows come last.  tallest(m): the rows of m-tile m.
template <typename F>
MOK_FORMS Tail tail_of(bool may, int mt, int nt, int steps, F tallest) {
#pragma clang fp contract(off)
  const int total = mt * nt, first = total / kRound * kRound, r = total - first;
  Tail best = {total, 0, 1, steps, 256, 0.f};
  if (r == 0) return best;
  best.us = 1.4f * float(steps) + 6.f;
  if (!may || 2 * r > kRound) return best;
  const int rows = tallest(first / (kGroupM * nt) * kGroupM);  // (none after it needs more)
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

// Steps of a unit of the weights' gradient in small tiles: an expert's rows are cut into units of at most
// so many steps, so that all units' tiles (per_unit of each) make no more items than the workspace
// holds.  total, most: steps of all experts, of one.
constexpr int kWholeExpert = 1 << 18;  // steps of 64 rows: more than there can be
MOK_FORMS int unit_steps(int total, int most, int per_unit, int groups) {
  int best = kWholeExpert;
  float us = split_us(most, per_unit * groups < kItems ? per_unit * groups : kItems, false);
  for (int items = 64; items <= kItems; items *= 2) {
    const int units = items / per_unit - groups;  // units are at most steps / per + groups
    if (units <= 0) continue;
    const int even = (total + units - 1) / units, per = even > kLeastSteps ? even : kLeastSteps;
    const float t = split_us(per, items, true);
    if (per < most && t < us) {
      us = t;
      best = per;
    }
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
struct Counts {
  int n256, n128, n32, n16;  // tiles (passes) of so many rows, of all experts; n32, n16 forward only
  int live;                  // experts with rows
};
// both: whole tiles are launched too.  tail(nt, steps): their last round, which may be split (may_tail).
template <typename F>
MOK_FORMS Form form_of(MmKind kind, const Counts& c, int n, int k, bool may_split, bool may_tail, bool both, F tail) {
#pragma clang fp contract(off)
  const int cols = kind == kMmOut ? n : k, deep = kind == kMmOut ? k : n, depth = (deep + kDeep - 1) / kDeep;
  const float steps = float(depth), weights = float(n) * float(k) * (2.f / 5.2e6f);
  const int nt = (cols + 255) / 256, whole = c.n256 * nt, small = c.n128 * ((cols + 127) / 128);
  const float least = 1.05f * weights * float(c.live);
  const Split sp = split_of(may_split, small, depth);
  const int items = small * sp.splits;
  const float us_small =
      4.f + (sp.splits > 1 ? 5.f : 0.f) +
      __builtin_fmaxf(least, float(sp.per) * (items <= 256 ? 0.72f : float((items + 511) / 512) *
                                                                         (kind == kMmOut ? 0.95f : 1.1f)));
  float us_whole = 1e30f;
  if (both) {
    us_whole = float((whole + 255) / 256) * (1.4f * steps + 6.f);
    if (may_tail && whole % kRound != 0)
      us_whole = float(whole / 256) * (1.4f * steps + 6.f) + tail(nt, depth).us;
    us_whole = 4.f + __builtin_fmaxf(least, us_whole);
  }
  if (kind == kMmOut) {
    const float passes = float(c.n32) * float((n + 63) / 64);
    // (a wave's pair of chunks takes 1.5 at least, and four waves share the sum)
    const float us_few = 3.f + __builtin_fmaxf((0.7f * float(c.n32) + 0.3f * float(c.n16)) * weights,
                                               __builtin_ceilf(passes / 512.f) * __builtin_ceilf(float(k) / 1024.f) * 1.5f);
    if (us_few < __builtin_fminf(us_small, us_whole)) return kFew;
  }
  return us_small < us_whole ? kSmall : kWhole;
}

// Which kernels are launched, by the rows that there may be: whole tiles alone where that is four rounds of
// them (buffers hold about as many rows as are routed), small ones (and few rows) alone where these make a
// round at most, otherwise both, one of which returns at once (4 us).  In a buffer that is mostly empty
// whole tiles alone have few rows too; MI355X, forward and rows' gradient, us, of 16,384 rows / of as many
// as are routed: N 4096, K 7168, 64 rows of one expert 22, 23 / 23, 19, 256 rows 36, 37 / 30, 29, 512 rows
// of eight 95, 84 / 97, 99 (their one round is split); N 7168, K 2048 (short sums are not split) 64 rows of
// one expert 22, 25 / 17, 18, 256 rows 41, 29 / 25, 23, 512 rows of eight 37, 54 / 39, 52.
// A product of weights has its tiles whatever the rows; with two steps an expert or fewer they are small
// ones, two of which a CU has in flight: what counts is to write the results.  MI355X, us, into fp32,
// whole / small: 2 rows of 32 experts, N 3432, K 128 17.6 / 13.1, 25 of 13, N 3048, K 400 20.3 / 17.6, 1000
// of 8, N 2048, K 2048 32.6 / 28.9, N 4096, K 7168 188 / 183; with four steps 2000 of 8, N 4096, K 2048
// 65.8 / 68.1, with eight 94.5 / 114.
enum Launched { kOnlySmall, kOnlyWhole, kBoth };
// Tiles of `tall` x `tall` that a call may have: an expert's rows may start a tile of their own.
inline int64_t tiles_at_most(MmKind kind, int64_t max_rows, int64_t groups, int64_t n, int64_t k, int64_t tall) {
  const int64_t cols = kind == kMmOut ? n : k, cut = (max_rows + groups * (tall - 1)) / tall;
  const int64_t m = kind == kMmWeights ? groups * ((n + tall - 1) / tall) : max_rows < cut ? max_rows : cut;
  return m * ((cols + tall - 1) / tall);
}
inline Launched launched(MmKind kind, int64_t max_rows, int32_t groups, int32_t n, int32_t k) {
  const int64_t whole = tiles_at_most(kind, max_rows, groups, n, k, 256),
                small = tiles_at_most(kind, max_rows, groups, n, k, 128);
  // (of the weights' gradient, up to 256 small ones' sums may be split)
  if (kind == kMmWeights) return whole >= 256 && small > 256 && max_rows > 128 * int64_t(groups) ? kOnlyWhole : kOnlySmall;
  return whole >= 1024 ? kOnlyWhole : small <= 512 ? kOnlySmall : kBoth;
}
// Whether a call has use for a workspace: where 128 x 128 tiles leave most of the card idle and the sums may
// be long enough, and where whole tiles may run whose last round has few (the launch that joins them
// takes 3 us where the routed rows then ask for no splitting).
inline bool may_split(MmKind kind, int64_t max_rows, int32_t groups, int32_t n, int32_t k) {
  const int64_t tiles = tiles_at_most(kind, max_rows, groups, n, k, 128);
  if (kind == kMmWeights) return tiles <= 256 && max_rows >= 2048;
  const int32_t deep = kind == kMmOut ? k : n;
  if (tiles <= 256) return deep >= 1536;
  // (with more experts than a wave has lanes the tiles of few rows do not come last, and no round of
  // whole tiles is split)
  return tiles > 512 && deep >= 4096 && (groups <= 64 || launched(kind, max_rows, groups, n, k) == kBoth);
}

}  // namespace g16
}  // namespace mok
