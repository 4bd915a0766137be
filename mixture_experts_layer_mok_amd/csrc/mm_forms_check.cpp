// Says on the host what mm_forms.h answers, for tests.  Built with a host compiler only.
//   mm_forms_check sweep   the answers of many counts of tiles, depths and columns
//   mm_forms_check calls   for every line "kind max_rows n k ws o_0 .. o_groups" (ws 0 or 1; o: offsets):
//                          launched form parts tall, as words and numbers: parts is how many items the tiles
//                          (tall 128: all of them; else those of the last round) are summed in, 1 if
//                          they are not split.  The kernels count an expert's tiles with a wave; here they are
//                          counted one after another.
//   mm_forms_check rows    for every line "max_rows from to": the ends of an expert's rows
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "mm_forms.h"

using namespace mok;
using namespace mok::g16;

static const char* const kForms[] = {"few", "small", "whole"};
static const char* const kLaunched[] = {"only_small", "only_whole", "both"};

// A last round whose tallest tile has `rows`.
static auto rows_are(int rows) {
  return [rows](int) { return rows; };
}

// Of a float all bits: one that is rounded otherwise may turn the comparison that it goes into.
static unsigned bits(float f) {
  unsigned u;
  std::memcpy(&u, &f, sizeof u);
  return u;
}

static void sweep() {
  for (int kind = kMmOut; kind <= kMmRows; ++kind)
    for (int deep = 8; deep <= 8192; deep += 168)
      for (int cols : {256, 1800, 2048, 7168})
        for (int m = 1; m <= 160; m += 3)
          for (int rows : {40, 100, 200}) {
            const int n = kind == kMmOut ? cols : deep, k = kind == kMmOut ? deep : cols, steps = (deep + 63) / 64;
            const Counts c = {m, rows > 128 ? 2 * m : m, (rows + 31) / 32 * m, (rows + 15) / 16 * m, m < 8 ? m : 8};
            const auto tail = [&](int nt, int depth) { return tail_of(true, m, nt, depth, rows_are(rows)); };
            const Form f = form_of(MmKind(kind), c, n, k, true, true, true, tail);
            const Tail t = tail((cols + 255) / 256, steps);
            const Split s = split_of(true, c.n128 * ((cols + 127) / 128), steps);
            std::printf("%d %d %d %d %d: %s %d/%d %d/%d %x\n", kind, deep, cols, m, rows, kForms[f], t.splits, t.per,
                        s.splits, s.per, bits(t.us));
          }
  for (int steps = 1; steps <= 2048; ++steps)
    for (int items : {1, 77, 256, 300, 512})
      std::printf("%d %d: %x %x\n", steps, items, bits(split_us(steps, items, false)), bits(split_us(steps, items, true)));
  for (int groups = 1; groups <= 256; groups *= 2)
    for (int tiles = 1; tiles * groups <= 256; tiles *= 2)
      for (int total = 1; total <= 4096; total += 7)
        std::printf("%d %d %d: %d\n", groups, tiles, total, unit_steps(total, (total + 1) / 2 + 1, tiles, groups));
}

static int one(const std::string& line) {
  std::istringstream in(line);
  int kind, n, k, ws;
  int64_t max_rows;
  std::vector<int> off;
  if (!(in >> kind >> max_rows >> n >> k >> ws) || kind < 0 || kind > 2) return 1;
  for (int o; in >> o;) off.push_back(o);
  if (off.size() < 2 || off.size() > 1025) return 1;
  const int groups = int(off.size()) - 1;
  const bool may = ws && may_split(MmKind(kind), max_rows, groups, n, k);
  const Launched what = launched(MmKind(kind), max_rows, groups, n, k);
  std::vector<int> rows;
  for (int e = 0; e < groups; ++e) {
    int lo, hi;
    cut_rows(off[e], off[e + 1], max_rows, &lo, &hi);
    rows.push_back(std::max(hi - lo, 0));
  }
  auto tiles = [&](int tall) {
    int t = 0;
    for (int r : rows) t += (r + tall - 1) / tall;
    return t;
  };
  if (kind == kMmWeights) {
    int parts = 1;
    if (what == kOnlySmall && may) {
      int most = 0;
      for (int r : rows) most = std::max(most, (r + kDeep - 1) / kDeep);
      const int per = unit_steps(tiles(kDeep), most, ((n + 127) / 128) * ((k + 127) / 128), groups);
      parts = std::max(1, (most + per - 1) / per);  // of the expert with the most rows
    }
    std::printf("%s %s %d 128\n", kLaunched[what], what == kOnlyWhole ? "whole" : "small", parts);
    return 0;
  }
  std::vector<int> tall;  // rows of the tiles of 256, those of few rows last
  for (int r : rows)
    for (int i = 0; i < r; i += 256)
      if (std::min(r - i, 256) > 128) tall.push_back(std::min(r - i, 256));
  for (int half : {128, 64})
    for (int r : rows)
      if (r % 256 > half / 2 * (half > 64) && r % 256 <= half) tall.push_back(r % 256);
  const bool sorted = groups <= 64;
  const int cols = kind == kMmOut ? n : k, steps = ((kind == kMmOut ? k : n) + kDeep - 1) / kDeep;
  auto tail = [&](int nt, int depth) {
    return tail_of(may && sorted, int(tall.size()), nt, depth, [&](int m) { return tall.at(m); });
  };
  int live = 0;
  for (int r : rows) live += r > 0;
  const Counts c = {tiles(256), tiles(128), tiles(kPassRows), tiles(16), live};
  Form f = kWhole;
  if (what == kBoth || (what == kOnlySmall && kind == kMmOut))
    f = form_of(MmKind(kind), c, n, k, may, may && sorted, what == kBoth, tail);
  else if (what == kOnlySmall)
    f = kSmall;
  if (f == kWhole) {
    const Tail t = tail((cols + 255) / 256, steps);
    std::printf("%s whole %d %d\n", kLaunched[what], t.splits, t.tall);
  } else {
    const Split s = split_of(may, c.n128 * ((cols + 127) / 128), steps);
    std::printf("%s %s %d 128\n", kLaunched[what], kForms[f], f == kFew ? 1 : s.splits);
  }
  return 0;
}

int main(int argc, char** argv) {
  if (argc == 2 && !std::strcmp(argv[1], "sweep")) {
    sweep();
    return 0;
  }
  if (argc == 2 && !std::strcmp(argv[1], "rows")) {
    int64_t max_rows;
    for (int from, to, lo, hi; std::cin >> max_rows >> from >> to;) {
      cut_rows(from, to, max_rows, &lo, &hi);
      std::printf("%d %d\n", lo, hi);
    }
    return 0;
  }
  if (argc != 2 || std::strcmp(argv[1], "calls")) return 2;
  for (std::string line; std::getline(std::cin, line);)
    if (one(line)) return 1;
  return 0;
}
