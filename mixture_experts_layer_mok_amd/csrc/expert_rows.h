// Which rows each expert has, and their division into tiles, on the device.
#pragma once
#include "device.h"
#include "ops_launch.h"

namespace mok {
namespace g16 {

// Rows of expert e, cut to [0, max_rows).
__device__ __forceinline__ void expert_rows(const MmArgs& p, int e, int* lo, int* hi) {
  cut_rows(p.offsets[e], p.offsets[e + 1], p.max_rows, lo, hi);
}

// Sums of x over the lanes up to this one (gfx9 DPP: within rows of 16 lanes, then across them).
__device__ __forceinline__ int scan64(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr:1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ int sum64(int x) { return __builtin_amdgcn_readlane(scan64(x), 63); }

// The largest of the lanes' x, which are not negative.
__device__ __forceinline__ int max64(int x) {
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));
  return __builtin_amdgcn_readlane(x, 63);
}

// The m-tiles of all experts (each expert's rows cut from its first row on into tiles of `tall`),
// numbered in expert order; an expert without rows has `least` of them (0 or 1).  Every wave scans
// the experts, 64 at a time, all lanes active; with at most 64 of them they are read once.
//
// init_sorted numbers those of more than half a tile first, in expert order, then the others, which take
// less time: of more than a quarter, then of less.  So the last round of tiles is the shortest.
struct RowTiles {
  int tall, least;
  int lo, hi;   // this lane's expert of the current 64: rows
  bool mine;    // there is such an expert
  int tiles, incl;  // its m-tiles, and those up to it
  int total;    // m-tiles of all experts
  int most;     // of one expert
  bool sorted = false;
  int wholes, rank;  // sorted: how many come in expert order; this lane's place among the others, or -1

  __device__ __forceinline__ void read(const MmArgs& p, int e0) {
    const int lane = threadIdx.x & 63;
    lo = hi = 0;
    mine = e0 + lane < p.groups;
    if (mine) expert_rows(p, e0 + lane, &lo, &hi);
  }
  __device__ __forceinline__ int tiles_of(int h) const { return hi > lo ? (hi - lo + h - 1) / h : 0; }
  __device__ __forceinline__ void scan() {
    tiles = hi > lo ? tiles_of(tall) : mine ? least : 0;
    incl = scan64(tiles);
  }
  // have: the experts, at most 64, are read already.
  __device__ __forceinline__ void init(const MmArgs& p, int tall_, int least_ = 0, bool have = false) {
    sorted = false;
    tall = tall_;
    least = least_;
    total = most = 0;
    for (int e0 = 0; e0 < p.groups; e0 += 64) {
      if (!have) read(p, e0);
      scan();
      total += __builtin_amdgcn_readlane(incl, 63);
      most = max(most, max64(tiles));
    }
  }
  __device__ __forceinline__ void init_sorted(const MmArgs& p, int tall_, bool have = false) {
    if (p.groups > 64) return init(p, tall_);
    sorted = true;
    tall = tall_;
    if (!have) read(p, 0);
    const int n = max(hi - lo, 0);
    const int rest = n % tall;
    tiles = n / tall + (rest > tall / 2 ? 1 : 0);
    incl = scan64(tiles);
    wholes = __builtin_amdgcn_readlane(incl, 63);
    const bool more = rest > tall / 4 && rest <= tall / 2, less = rest > 0 && rest <= tall / 4;
    const uint64_t m = __ballot(more), l = __ballot(less), before = (1ull << (threadIdx.x & 63)) - 1;
    rank = more ? __popcll(m & before) : less ? __popcll(m) + __popcll(l & before) : -1;
    total = wholes + __popcll(m) + __popcll(l);
  }
  // m-tile m < total: its expert, first row and rows, its number among the expert's m-tiles and
  // how many those are.
  __device__ __forceinline__ void find(const MmArgs& p, int m, int* e, int* r0, int* rows, int* part, int* parts) {
    int e0 = 0;
    if (p.groups > 64) {
      for (;; e0 += 64) {
        read(p, e0);
        scan();
        const int n = __builtin_amdgcn_readlane(incl, 63);
        if (m < n) break;
        m -= n;
      }
    }
    const int s = __ffsll((unsigned long long)__ballot(incl > m)) - 1;
    *e = e0 + s;
    *parts = __builtin_amdgcn_readlane(tiles, s);
    *part = m - (__builtin_amdgcn_readlane(incl, s) - *parts);
    const int first = __builtin_amdgcn_readlane(lo, s) + *part * tall;
    *r0 = first;
    *rows = max(min(__builtin_amdgcn_readlane(hi, s) - first, tall), 0);
  }
  __device__ __forceinline__ void find(const MmArgs& p, int m, int* e, int* r0, int* rows) {
    if (sorted) {
      const bool whole = m < wholes;
      const int s = __ffsll((unsigned long long)__ballot(whole ? incl > m : rank == m - wholes)) - 1;
      const int have = __builtin_amdgcn_readlane(tiles, s), first = __builtin_amdgcn_readlane(lo, s);
      *e = s;
      *r0 = first + tall * (whole ? m - (__builtin_amdgcn_readlane(incl, s) - have) : have);
      *rows = min(__builtin_amdgcn_readlane(hi, s) - *r0, tall);
      return;
    }
    int part, parts;
    find(p, m, e, r0, rows, &part, &parts);
  }
};

}  // namespace g16
}  // namespace mok
