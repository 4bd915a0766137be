// Which rows each expert has, and their division into tiles, on the device.
#pragma once
#include "device.h"
#include "ops_launch.h"

namespace mok {
namespace g16 {

// Rows of expert e, cut to [0, max_rows).
__device__ __forceinline__ void expert_rows(const MmArgs& p, int e, int* lo, int* hi) {
  *lo = max(p.offsets[e], 0);
  *hi = int(min(int64_t(p.offsets[e + 1]), p.max_rows));
}

// The m-tiles of all experts (each expert's rows cut from its first row on into tiles of TM),
// numbered in expert order.  Every wave scans the experts, 64 at a time; with at most 64 of them
// they are read once.
template <int TM>
struct RowTiles {
  int lo, hi, incl;  // this lane's expert of the current 64: rows, m-tiles up to it
  int tiles;         // this lane's expert's
  int total;         // m-tiles of all experts

  __device__ __forceinline__ void scan(const MmArgs& p, int e0) {
    const int lane = threadIdx.x & 63;
    lo = hi = 0;
    if (e0 + lane < p.groups) expert_rows(p, e0 + lane, &lo, &hi);
    tiles = hi > lo ? (hi - lo + TM - 1) / TM : 0;
    incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(incl, d);
      if (lane >= d) incl += u;
    }
  }
  __device__ __forceinline__ void init(const MmArgs& p) {
    total = 0;
    for (int e0 = 0; e0 < p.groups; e0 += 64) {
      scan(p, e0);
      total += __builtin_amdgcn_readlane(incl, 63);
    }
  }
  // m-tile m < total: its expert, first row and rows
  __device__ __forceinline__ void find(const MmArgs& p, int m, int* e, int* r0, int* rows) {
    int e0 = 0;
    if (p.groups > 64) {
      for (;; e0 += 64) {
        scan(p, e0);
        const int n = __builtin_amdgcn_readlane(incl, 63);
        if (m < n) break;
        m -= n;
      }
    }
    const int s = __ffsll((unsigned long long)__ballot(incl > m)) - 1;
    *e = e0 + s;
    const int first = __builtin_amdgcn_readlane(lo, s) + (m - __builtin_amdgcn_readlane(incl - tiles, s)) * TM;
    *r0 = first;
    *rows = min(__builtin_amdgcn_readlane(hi, s) - first, TM);
  }
};

}  // namespace g16
}  // namespace mok
