// Grouped product on MX operands: out[r, c] = sum_i A[r, i] B[e][c, i] for the rows r of
// every expert e, A in MXFP4 or MXFP8, B in MXFP4, on the scaled MFMA with fp32
// accumulation.
//
// Operands of v_mfma_scale_f32_16x16x128_f8f6f4, as measured on gfx950: lane l holds row
// l % 16 of its operand and, with g = l / 16,
//   4-bit: the 32 elements of K block g (16 bytes);
//   8-bit: elements 16 g .. +16 (first 16 bytes) and 64 + 16 g .. +16 (last 16);
// the scale of block g of row r comes from lane r + 16 g whatever the format.  The result
// has, in lane l, column l % 16 and rows 4 (l / 16) .. +4.  Weights are the first operand, so
// a lane ends with four consecutive columns of one row of out.
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "launch.h"
#include "gemm_mx4.h"

namespace mok {

namespace {

constexpr uint32_t kOut = 0x80000000u;  // added to an offset: past every buffer's range

// Rows of expert e, cut to [0, max_rows).
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int64_t max_rows,
                                            int64_t* lo, int64_t* hi) {
  *lo = max(int64_t(offsets[e]), int64_t(0));
  *hi = min(int64_t(offsets[e + 1]), max_rows);
}

__device__ __forceinline__ uint32_t ld_u8(rsrc_t r, uint32_t off) {
  return uint32_t(uint8_t(__builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0)));
}

__device__ __forceinline__ f32x4_t mfma16(i32x8_t w, i32x8_t a, f32x4_t c, int sw, int sa, bool a8) {
  return a8 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, 0, 0, sw, 0, sa)
            : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, 4, 0, sw, 0, sa);
}

// One workgroup: 16 columns of one expert, all its rows in passes of 16 MB, the K steps of
// 128 dealt to the four waves and their sums joined through LDS in wave order.  Loads
// past K, past the rows and past N read zeros (zero codes and zero scales: no product).
template <bool A8, bool OUT32, int MB>
__global__ __launch_bounds__(256) void k_grouped_rows(GroupedArgs p) {
  __shared__ f32x4_t s_part[4][MB][64];
  const int e = blockIdx.y, n0 = blockIdx.x * 16;
  int64_t lo, hi;
  expert_rows(p.offsets, e, p.max_rows, &lo, &hi);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int kb = p.k / 2, nblk = p.k / 32, steps = (p.k + 127) / 128;
  const int ncols = min(16, p.n - n0);
  const int64_t brow = int64_t(e) * p.n + n0;
  const rsrc_t rb = row_rsrc(p.b + brow * kb, uint32_t(ncols * kb));
  const rsrc_t rbs = row_rsrc(p.bs + brow * nblk, uint32_t(ncols * nblk));
  const int abytes = A8 ? p.k : kb;
  for (int64_t r0 = lo; r0 < hi; r0 += 16 * MB) {
    const int valid = int(min(hi - r0, int64_t(16 * MB)));
    const rsrc_t ra = row_rsrc(p.a + r0 * p.ld_a, uint32_t((valid - 1) * p.ld_a + abytes));
    const rsrc_t ras = row_rsrc(p.as + r0 * p.ld_as, uint32_t((valid - 1) * p.ld_as + nblk));
    f32x4_t acc[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int ks = w; ks < steps; ks += 4) {
      const int blk = 4 * ks + g;  // this lane's scale block
      const uint32_t out_s = blk < nblk ? 0u : kOut;
      const v4u wv = buf_ld16<kCpolPlain>(rb, uint32_t(r16 * kb + blk * 16) + out_s);
      const uint32_t ws = ld_u8(rbs, uint32_t(r16 * nblk + blk) + out_s);
      const i32x8_t wf = {int(wv.x), int(wv.y), int(wv.z), int(wv.w), 0, 0, 0, 0};
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const int row = 16 * m + r16;
        const uint32_t out_r = row < valid ? 0u : kOut;
        const uint32_t as = ld_u8(ras, (uint32_t(row * p.ld_as) + blk) | out_s | out_r);
        i32x8_t af;
        if (A8) {
          const int b0 = 4 * ks + (g >> 1), k0 = 128 * ks + 16 * g;
          const v4u x = buf_ld16<kCpolPlain>(
              ra, (uint32_t(row * p.ld_a) + k0) | out_r | (b0 < nblk ? 0u : kOut));
          const v4u y = buf_ld16<kCpolPlain>(
              ra, (uint32_t(row * p.ld_a) + k0 + 64) | out_r | (b0 + 2 < nblk ? 0u : kOut));
          af = i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w),
                       int(y.x), int(y.y), int(y.z), int(y.w)};
        } else {
          const v4u x =
              buf_ld16<kCpolPlain>(ra, (uint32_t(row * p.ld_a) + blk * 16) | out_s | out_r);
          af = i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
        }
        acc[m] = mfma16(wf, af, acc[m], int(ws), int(as), A8);
      }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) s_part[w][m][lane] = acc[m];
    __syncthreads();
    for (int i = threadIdx.x; i < MB * 64; i += 256) {
      const int m = i >> 6, l = i & 63;
      f32x4_t c = s_part[0][m][l];
#pragma unroll
      for (int u = 1; u < 4; ++u) c += s_part[u][m][l];
      const int row = 16 * m + (l & 15), col = n0 + 4 * (l >> 4);
      if (row < valid && col < p.n) {
        const int64_t at = (r0 + row) * p.ld_out + col;
        if (OUT32)
          *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at) = c;
        else
          *reinterpret_cast<uint64_t*>(static_cast<uint16_t*>(p.out) + at) =
              uint64_t(pack_bf16x2(c.x, c.y)) | (uint64_t(pack_bf16x2(c.z, c.w)) << 32);
      }
    }
    __syncthreads();  // s_part is rewritten by the next pass
  }
}

// The m-tiles of all experts (each expert's rows cut from its first row on into tiles of
// TM), numbered in expert order.  Every wave scans the experts, 64 at a time; with at most 64
// of them they are read once.
template <int TM>
struct Tiling {
  int lo, hi, incl;  // this lane's expert of the current 64: rows, m-tiles up to it
  int total;         // m-tiles of all experts
  int tiles;         // this lane's expert's

  __device__ __forceinline__ void scan(const GroupedArgs& p, int e0) {
    const int lane = threadIdx.x & 63;
    int64_t l = 0, h = 0;
    if (e0 + lane < p.groups) expert_rows(p.offsets, e0 + lane, p.max_rows, &l, &h);
    lo = int(l);
    hi = int(h);
    tiles = hi > lo ? (hi - lo + TM - 1) / TM : 0;
    incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(incl, d);
      if (lane >= d) incl += u;
    }
  }
  __device__ __forceinline__ void init(const GroupedArgs& p) {
    total = 0;
    for (int e0 = 0; e0 < p.groups; e0 += 64) {
      scan(p, e0);
      total += __builtin_amdgcn_readlane(incl, 63);
    }
  }
  // m-tile m < total: its expert, first row and rows
  __device__ __forceinline__ void find(const GroupedArgs& p, int m, int* e, int64_t* r0, int* rows) {
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
    const int first = __builtin_amdgcn_readlane(lo, s) +
                      (m - __builtin_amdgcn_readlane(incl - tiles, s)) * TM;
    *r0 = first;
    *rows = min(__builtin_amdgcn_readlane(hi, s) - first, TM);
  }
};

// Tile t of mt x nt: groups of kGroupM m-tiles, inside them all m-tiles of an n-tile before the next,
// so that the tiles that run at the same time share both operands' rows.
constexpr int kGroupM = 4;
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int* m, int* n) {
  const int g = t / (kGroupM * nt), r = t - g * kGroupM * nt;
  const int gm = min(kGroupM, mt - g * kGroupM);
  *n = r / gm;
  *m = g * kGroupM + r - *n * gm;
}

// A workgroup's next tile: workgroups go to the eight XCDs in turn, and XCD x takes the x-th
// eighth of the tiles, whose operands its L2 then holds; its workgroups take them in turn.
template <bool A8, bool OUT32, int SG>
__global__ __launch_bounds__(mx4::kThr) void k_grouped_tile(GroupedArgs p, int nt) {
  constexpr int TM = mx4::tile_rows<A8>();
  Tiling<TM> til;
  til.init(p);
  const int total = til.total * nt, per = (total + 7) / 8;
  const int first = int(blockIdx.x & 7) * per, end = min(first + per, total);
  int t = first + int(blockIdx.x >> 3);
  if (t >= end) return;
  mx4::Source<A8, SG> src;
  int m, n, e, rows;
  int64_t r0;
  auto open = [&]() __attribute__((always_inline)) {
    tile_of(t, til.total, nt, &m, &n);
    til.find(p, m, &e, &r0, &rows);
    src.init(p, e, r0, rows, n * mx4::kTN);
    src.begin();
  };
  open();
  int stores = 0;  // made since the tile's first loads were issued
  auto run = [&](auto tile) __attribute__((always_inline)) {
    tile.run(src, stores);
    const int64_t r = r0;
    const int have = rows, n0 = n * mx4::kTN;
    t += int(gridDim.x >> 3);
    if (t < end) open();
    tile.template store<OUT32>(p, r, have, n0);
    stores = tile.template kStores<OUT32>;
  };
  while (t < end) {
    if (rows <= 64) run(mx4::Tile<A8, SG, 1>());
    else if (A8 || rows <= 128) run(mx4::Tile<A8, SG, 2>());
    else run(mx4::Tile<A8, SG, A8 ? 2 : 4>());
  }
}

}  // namespace

mok_status_t launch_grouped_mx4(const GroupedArgs& a, hipStream_t st) {
  if (a.max_rows / a.groups >= 64) {
    const int tm = a.a8 ? mx4::tile_rows<true>() : mx4::tile_rows<false>();
    const int nt = (a.n + mx4::kTN - 1) / mx4::kTN;
    // at most this many m-tiles: every expert may end inside one
    const int64_t mt = std::min<int64_t>(a.max_rows, (a.max_rows + int64_t(a.groups) * (tm - 1)) / tm);
    const dim3 grid(unsigned(std::min<int64_t>((mt * nt + 7) / 8 * 8, 256))), block(mx4::kThr);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, block, 0, st, a, nt); };
    auto sg = [&](auto g) {
      constexpr int SG = decltype(g)::value;
      if (a.a8) {
        if (a.out32) go(k_grouped_tile<true, true, SG>);
        else go(k_grouped_tile<true, false, SG>);
      } else {
        if (a.out32) go(k_grouped_tile<false, true, SG>);
        else go(k_grouped_tile<false, false, SG>);
      }
    };
    const int64_t align = int64_t(reinterpret_cast<uintptr_t>(a.as) | reinterpret_cast<uintptr_t>(a.bs) |
                                  uintptr_t(a.ld_as) | uintptr_t(a.k / 32));
    if (align % 16 == 0) sg(std::integral_constant<int, 16>());
    else if (align % 4 == 0) sg(std::integral_constant<int, 4>());
    else sg(std::integral_constant<int, 1>());
    return hipGetLastError() == hipSuccess ? MOK_OK : MOK_E_LAUNCH;
  }
  const dim3 grid(unsigned((a.n + 15) / 16), unsigned(a.groups)), block(256);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, block, 0, st, a); };
  if (a.a8) {
    if (a.out32) go(k_grouped_rows<true, true, 2>);
    else go(k_grouped_rows<true, false, 2>);
  } else {
    if (a.out32) go(k_grouped_rows<false, true, 2>);
    else go(k_grouped_rows<false, false, 2>);
  }
  return hipGetLastError() == hipSuccess ? MOK_OK : MOK_E_LAUNCH;
}

}  // namespace mok
