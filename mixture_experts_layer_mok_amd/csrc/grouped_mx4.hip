// Grouped product on MX operands: out[r, c] = sum_i A[r, i] B[e][c, i] for the rows r of
// every expert e, A in MXFP4 or MXFP8, B in MXFP4, on the scaled MFMA with fp32
// accumulation.
//
// Operands of v_mfma_scale_f32_16x16x128_f8f6f4, as measured on gfx950: lane l holds row
// l % 16 of its operand and, with g = l / 16,
//   4-bit: the 32 elements of K block g (16 bytes);
//   8-bit: elements 16 g .. +16 (first 16 bytes) and 64 + 16 g .. +16 (last 16);
// the scale of block g of row r comes from lane r + 16 g whatever the format.  With 8-bit
// elements the products of eight neighbours are cut toward zero to 2^(E - 13), E the largest
// sum of exponents among them, before they are added; with two 4-bit operands that cuts
// nothing.  The result
// has, in lane l, column l % 16 and rows 4 (l / 16) .. +4.  Weights are the first operand, so
// a lane ends with four consecutive columns of one row of out.
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "ops_launch.h"
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

__device__ __forceinline__ f32x4_t mfma16(i32x8_t w, i32x8_t a, f32x4_t c, int sw, int sa, bool a8) {
  return a8 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, 0, 0, sw, 0, sa)
            : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, 4, 0, sw, 0, sa);
}

// The m-tiles of all experts (each expert's rows cut from its first row on into tiles of
// TM), numbered in expert order.  Every wave scans the experts, 64 at a time; with at most 64
// of them they are read once.
template <int TM>
struct Tiling {
  int lo, hi, incl;  // this lane's expert of the current 64: rows, m-tiles up to it
  int total;         // m-tiles of all experts
  int active;        // experts with rows
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
    total = active = 0;
    for (int e0 = 0; e0 < p.groups; e0 += 64) {
      scan(p, e0);
      total += __builtin_amdgcn_readlane(incl, 63);
      active += __popcll(__ballot(tiles > 0));
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

// Whether the few-rows kernel has the call: passes of at most 32 rows times 256-column blocks, an
// expert's passes after its first counted 4/3 (the bound is explained at launch_grouped_mx4).
constexpr int kPass = 32, kFew = 128;
__host__ __device__ __forceinline__ bool is_few(int64_t passes, int64_t active, int nt) {
  return (4 * passes - active) * nt <= 3 * kFew;
}

// ------------------------------------------------------------------------------------
// Few rows an expert (decoding): bound by reading the weights once.
// ------------------------------------------------------------------------------------
// One workgroup of four waves: 16 NB columns of one expert and at most 32 of its rows (a pass).
// The K chunks of 256 (two MFMA steps) are dealt to the waves; each issues its next chunk's
// loads before it multiplies the current one, straight into registers (a weight is used by one
// wave only, so LDS would add a copy).  The copy of the chunk's registers at the end of an
// iteration waits for those loads, so they overlap one chunk's products; the rest of their
// latency is covered by the CU's other waves.  The waves' sums are joined through LDS in
// wave order.  Loads past K, past the rows and past N read zeros (zero codes, zero scales: no
// product).
constexpr int kChunk = 256, kWaves = 4;

// The eight scale bytes of a row's chunk: two dwords, or, where some row's scales do not start
// at an 8-byte address or are not whole pieces of 8 (SHIFT), the three that they lie in (64 rows
// over 8 experts, N 4096, K 7200 in MXFP8 on MI355X: 62 us by bytes, 34 so; 31 for K 7168).
template <bool SHIFT>
struct Scales8 {
  uint32_t w[SHIFT ? 3 : 2];

  __device__ __forceinline__ void load(rsrc_t r, uint32_t off, int have) {
    const uint32_t past = have > 0 ? 0u : kOut;
    if (SHIFT) {
      typedef uint32_t v3u_t __attribute__((ext_vector_type(3)));
      const v3u_t v = __builtin_amdgcn_raw_buffer_load_b96(r, (off & ~3u) | past, 0, 0);
      w[0] = v.x;
      w[1] = v.y;
      w[SHIFT ? 2 : 0] = v.z;
    } else {
      typedef uint32_t v2u_t __attribute__((ext_vector_type(2)));
      const v2u_t v = __builtin_amdgcn_raw_buffer_load_b64(r, off | past, 0, 0);
      w[0] = v.x;
      w[1] = v.y;
    }
  }
  // Byte g of dword s, 0 past the row; `low`: bytes before the first in the first dword.
  __device__ __forceinline__ int at(int s, int g, uint32_t low, int have) const {
    if (!SHIFT) return int(w[s] >> (8 * g));
    const uint32_t v = __builtin_amdgcn_alignbyte(w[SHIFT ? s + 1 : s], w[s], low) >> (8 * g);
    return 4 * s + g < have ? int(v) : 0;
  }
};

// A matrix's scales from the dword that the first byte lies in to the one that the last lies
// in; loads read the dwords past it as zeros, each by itself.
__device__ __forceinline__ rsrc_t scales_rsrc(const uint8_t* base, uint32_t bytes) {
  const uint32_t low = uint32_t(reinterpret_cast<uintptr_t>(base) & 3);
  return row_rsrc(base - low, (low + bytes + 3) & ~3u);
}

template <bool A8, bool SHIFT, int NB, int MB>
struct Chunk {
  v4u b[NB][2];         // a column block's codes, one 16-byte K block a step
  Scales8<SHIFT> bs[NB];
  v4u a[MB][2][A8 ? 2 : 1];
  Scales8<SHIFT> as[MB];

  // lb, la: bytes of the scale resources before the first scale
  __device__ __forceinline__ void load(const GroupedArgs& p, rsrc_t rb, rsrc_t rbs, uint32_t lb, rsrc_t ra,
                                       rsrc_t ras, uint32_t la, int valid, int ck) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int kb = p.k / 2, nblk = p.k / 32, have = nblk - 8 * ck;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const uint32_t row = 16 * j + r16;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        b[j][s] = buf_ld16<kCpolPlain>(
            rb, (row * kb + (8 * ck + 4 * s + g) * 16) | (4 * s + g < have ? 0u : kOut));
      bs[j].load(rbs, lb + row * nblk + 8 * ck, have);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int row = 16 * m + r16;
      const uint32_t out_r = row < valid ? 0u : kOut;
      const uint32_t at = uint32_t(row * p.ld_a);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (A8) {
          const int b0 = 4 * s + (g >> 1);
          const uint32_t k0 = kChunk * ck + 128 * s + 16 * g;
          a[m][s][0] = buf_ld16<kCpolPlain>(ra, (at + k0) | out_r | (b0 < have ? 0u : kOut));
          a[m][s][A8 ? 1 : 0] = buf_ld16<kCpolPlain>(ra, (at + k0 + 64) | out_r | (b0 + 2 < have ? 0u : kOut));
        } else {
          a[m][s][0] = buf_ld16<kCpolPlain>(
              ra, (at + (8 * ck + 4 * s + g) * 16) | out_r | (4 * s + g < have ? 0u : kOut));
        }
      }
      as[m].load(ras, (la + uint32_t(row * p.ld_as) + 8 * ck) | out_r, have);
    }
  }

  // The lane's K block of step s is 4 s + g: byte g of the step's scale dword.  shb, sha: where
  // the lane's rows start in their first dwords (16 rows on it is the same byte); `have`: the
  // chunk's K blocks.
  __device__ __forceinline__ void multiply(f32x4_t (&acc)[MB][NB], uint32_t shb, uint32_t sha, int have) const {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const v4u x = a[m][s][0], y = a[m][s][A8 ? 1 : 0];
        const i32x8_t af = {int(x.x), int(x.y), int(x.z), int(x.w), int(y.x), int(y.y), int(y.z), int(y.w)};
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const v4u w = b[j][s];
          const i32x8_t wf = {int(w.x), int(w.y), int(w.z), int(w.w), 0, 0, 0, 0};
          acc[m][j] = mfma16(wf, af, acc[m][j], bs[j].at(s, g, shb, have), as[m].at(s, g, sha, have), A8);
        }
      }
  }
};

template <bool A8, bool SHIFT, int NB, int MB>
__device__ __forceinline__ void rows_pass(const GroupedArgs& p, f32x4_t* s_part, int64_t r0, int valid,
                                          rsrc_t rb, rsrc_t rbs, uint32_t lb, int n0) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb = p.k / 2, nblk = p.k / 32, chunks = (p.k + kChunk - 1) / kChunk;
  const rsrc_t ra = row_rsrc(p.a + r0 * p.ld_a, uint32_t((valid - 1) * p.ld_a + (A8 ? p.k : kb)));
  const uint8_t* as = p.as + r0 * p.ld_as;
  const rsrc_t ras = scales_rsrc(as, uint32_t((valid - 1) * p.ld_as + nblk));
  const uint32_t la = uint32_t(reinterpret_cast<uintptr_t>(as) & 3);
  const uint32_t shb = (lb + uint32_t(lane & 15) * uint32_t(nblk)) & 3;
  const uint32_t sha = (la + uint32_t(lane & 15) * uint32_t(p.ld_as)) & 3;
  f32x4_t acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (w < chunks) {
    Chunk<A8, SHIFT, NB, MB> cur, nxt;
    cur.load(p, rb, rbs, lb, ra, ras, la, valid, w);
    for (int ck = w; ck < chunks; ck += kWaves) {
      nxt.load(p, rb, rbs, lb, ra, ras, la, valid, ck + kWaves);  // past the last: reads nothing
      cur.multiply(acc, shb, sha, nblk - 8 * ck);
      cur = nxt;
    }
  }
  // s_part[wave][block][lane]
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NB; ++j) s_part[(w * MB * NB + m * NB + j) * 64 + lane] = acc[m][j];
  __syncthreads();
  for (int i = threadIdx.x; i < MB * NB * 64; i += kWaves * 64) {
    const int blk = i >> 6, l = i & 63, m = blk / NB, j = blk % NB;
    f32x4_t c = s_part[i];
#pragma unroll
    for (int u = 1; u < kWaves; ++u) c += s_part[u * MB * NB * 64 + i];
    const int row = 16 * m + (l & 15), col = n0 + 16 * j + 4 * (l >> 4);
    if (row < valid && col < p.n) {
      const int64_t at = (r0 + row) * p.ld_out + col;
      if (p.out32)
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at) = c;
      else
        *reinterpret_cast<uint64_t*>(static_cast<uint16_t*>(p.out) + at) =
            uint64_t(pack_bf16x2(c.x, c.y)) | (uint64_t(pack_bf16x2(c.z, c.w)) << 32);
    }
  }
}

// Item t: passes of all experts times blocks of 16 NB columns, columns first, so that the passes
// that read the same weights run on the same XCD, at about the same time.
template <bool A8, bool SHIFT, int NB>
__device__ __forceinline__ void rows_item(const GroupedArgs& p, Tiling<kPass>& til, f32x4_t* s_part, int t) {
  const int ncb = (p.n + 16 * NB - 1) / (16 * NB);
  const int m = t / ncb, n0 = (t - m * ncb) * 16 * NB, ncols = min(16 * NB, p.n - n0);
  if (m >= til.total) return;
  int e, rows;
  int64_t r0;
  til.find(p, m, &e, &r0, &rows);
  const int64_t brow = int64_t(e) * p.n + n0;
  const rsrc_t rb = row_rsrc(p.b + brow * (p.k / 2), uint32_t(ncols * (p.k / 2)));
  const uint8_t* bs = p.bs + brow * (p.k / 32);
  const rsrc_t rbs = scales_rsrc(bs, uint32_t(ncols * (p.k / 32)));
  const uint32_t lb = uint32_t(reinterpret_cast<uintptr_t>(bs) & 3);
  if (rows <= 16) rows_pass<A8, SHIFT, NB, 1>(p, s_part, r0, rows, rb, rbs, lb, n0);
  else rows_pass<A8, SHIFT, NB, 2>(p, s_part, r0, rows, rb, rbs, lb, n0);
}

// Columns a workgroup: the most that leave an item a CU (every item reads its rows again).
// Measured on MI355X with a bound of 256 / 512 items, us: 128 rows of one expert, N 4096, K 7168,
// MXFP8 20 / 25 (45 with 16 columns); 256 rows of 8, N 2048, K 4096 15.6 / 19.2.  64 rows of 8
// experts, N 4096, K 7168, MXFP8: 64 columns 32, 32 39, 16 42.
template <bool A8, bool SHIFT>
__global__ __launch_bounds__(kWaves * 64) void k_grouped_rows(GroupedArgs p, int max_passes, int nt, bool both) {
  __shared__ f32x4_t s_part[kWaves * 2 * 4 * 64];
  Tiling<kPass> til;
  til.init(p);
  til.total = min(til.total, max_passes);  // more only where ranges overlap
  if (both && !is_few(til.total, til.active, nt)) return;
  if ((p.n + 63) / 64 * til.total >= 256) rows_item<A8, SHIFT, 4>(p, til, s_part, blockIdx.x);
  else if ((p.n + 31) / 32 * til.total >= 256) rows_item<A8, SHIFT, 2>(p, til, s_part, blockIdx.x);
  else rows_item<A8, SHIFT, 1>(p, til, s_part, blockIdx.x);
}

// Tile t of mt x nt: groups of kGroupM m-tiles, inside them all m-tiles of an n-tile before the next,
// so that the tiles that run at the same time share both operands' rows.
constexpr int kGroupM = 4;
__device__ __forceinline__ void tile_of(int t, int mt, int nt, int* m, int* n) {
  const int g = t / (kGroupM * nt), r = t - g * kGroupM * nt;
  const int gm = min(kGroupM, mt - g * kGroupM);
  *n = r / gm;
  *m = g * kGroupM + r - *n * gm;
}

// The tiles of 64 JB columns and the rows of til, by workgroups that take several: workgroups go to
// the eight XCDs in turn, and XCD x takes the x-th eighth of the tiles, whose operands its L2
// then holds; its workgroups take them in turn.
template <bool A8, bool OUT32, bool SHIFT, int JB>
__device__ __forceinline__ void walk_tiles(const GroupedArgs& p, Tiling<mx4::tile_rows<A8, JB>()>& til) {
  constexpr int TN = mx4::tile_cols<JB>(), kIB = A8 ? JB / 2 : JB;
  const int nt = (p.n + TN - 1) / TN;
  const int total = til.total * nt, per = (total + 7) / 8;
  const int first = int(blockIdx.x & 7) * per, end = min(first + per, total);
  int t = first + int(blockIdx.x >> 3);
  if (t >= end) return;
  mx4::Source<A8, SHIFT, JB> src;
  int m, n, e, rows;
  int64_t r0;
  auto open = [&]() __attribute__((always_inline)) {
    tile_of(t, til.total, nt, &m, &n);
    til.find(p, m, &e, &r0, &rows);
    src.init(p, e, r0, rows, n * TN);
    src.begin();
  };
  open();
  int stores = 0;  // made since the tile's first loads were issued
  auto run = [&](auto tile) __attribute__((always_inline)) {
    tile.run(src, stores);
    const int64_t r = r0;
    const int have = rows, n0 = n * TN;
    t += int(gridDim.x >> 3);
    if (t < end) open();
    tile.template store<OUT32>(p, r, have, n0);
    stores = tile.template kStores<OUT32>;
  };
  while (t < end) {
    if (kIB == 1 || rows <= 64) run(mx4::Tile<A8, SHIFT, 1, JB>());
    else if (kIB == 2 || rows <= 128) run(mx4::Tile<A8, SHIFT, kIB < 2 ? 1 : 2, JB>());
    else run(mx4::Tile<A8, SHIFT, kIB, JB>());
  }
}

// Tiles of half the rows and columns where these make one a CU at most: four times the
// workgroups, each with a fourth of the work of a K step.  Measured on MI355X, whole tiles /
// halves, us: 512 MXFP4 rows of one expert, N 4096, K 7168 43 / 27; 2000 rows of 4, N 2048, K 4096
// 30.6 / 19.8 (MXFP8, 512 tiles of half the size, 29 / 32); 1024 rows of 8, N 4096, K 7168 50 / 39.
template <bool A8, bool OUT32, bool SHIFT>
__global__ __launch_bounds__(mx4::kThr) void k_grouped_tile(GroupedArgs p, int max_mt, int nt, bool both) {
  if (both) {
    Tiling<kPass> passes;
    passes.init(p);
    if (is_few(passes.total, passes.active, nt)) return;
  }
  Tiling<mx4::tile_rows<A8, 2>()> halves;
  halves.init(p);
  if (int64_t(halves.total) * ((p.n + mx4::tile_cols<2>() - 1) / mx4::tile_cols<2>()) <= 256) {
    walk_tiles<A8, OUT32, SHIFT, 2>(p, halves);
  } else {
    Tiling<mx4::tile_rows<A8, 4>()> til;
    til.init(p);
    til.total = min(til.total, max_mt);  // more only where ranges overlap
    walk_tiles<A8, OUT32, SHIFT, 4>(p, til);
  }
}

// Whether every row's scales are whole pieces of `piece` bytes at multiples of it.
bool scales_whole(const GroupedArgs& a, uintptr_t piece) {
  return (reinterpret_cast<uintptr_t>(a.as) | reinterpret_cast<uintptr_t>(a.bs) | uintptr_t(a.ld_as) |
          uintptr_t(a.k / 32)) % piece == 0;
}

mok_status_t launch_tiles(const GroupedArgs& a, int nt, bool both, hipStream_t st) {
  const int tm = a.a8 ? mx4::tile_rows<true, 4>() : mx4::tile_rows<false, 4>();
  // at most this many m-tiles: every expert may end inside one
  const int64_t mt = std::min<int64_t>(a.max_rows, (a.max_rows + int64_t(a.groups) * (tm - 1)) / tm);
  // (a tile makes four at most of half the rows and columns)
  const dim3 grid(unsigned(std::min<int64_t>((4 * mt * nt + 7) / 8 * 8, 256))), block(mx4::kThr);
  auto go = [&](auto kern) { return launch(kern, grid, block, st, a, int(mt), nt, both); };
  auto form = [&](auto shift) {
    constexpr bool SHIFT = decltype(shift)::value;
    if (a.a8) return a.out32 ? go(k_grouped_tile<true, true, SHIFT>) : go(k_grouped_tile<true, false, SHIFT>);
    return a.out32 ? go(k_grouped_tile<false, true, SHIFT>) : go(k_grouped_tile<false, false, SHIFT>);
  };
  return scales_whole(a, 16) ? form(std::false_type()) : form(std::true_type());
}

// At most 512 items: few passes (is_few) of 64 columns, or fewer than 256 of twice the columns
// of what is taken.
mok_status_t launch_rows(const GroupedArgs& a, int64_t passes, int nt, bool both, hipStream_t st) {
  const dim3 grid(unsigned(std::min<int64_t>((a.n + 15) / 16 * passes, 4 * kFew)));
  auto go = [&](auto kern) { return launch(kern, grid, dim3(64 * kWaves), st, a, int(passes), nt, both); };
  const bool whole = scales_whole(a, 8);
  if (a.a8) return whole ? go(k_grouped_rows<true, false>) : go(k_grouped_rows<true, true>);
  return whole ? go(k_grouped_rows<false, false>) : go(k_grouped_rows<false, true>);
}

}  // namespace

// Which kernel.  The few-rows kernel reads the weights once for 32 rows, all passes at the same
// time: its time grows with passes times columns; a tile takes its K loop's time however few
// there are.  Measured on MI355X, weights from HBM, few-rows / tile kernel alone, us, by u =
// passes times 256-column blocks, MXFP8 rows and then MXFP4:
//   N 4096, K 7168, one expert: u 16 13 / 23, 9 / 22; u 32 15 / 24, 11 / 22; u 64 20 / 24, 17 / 24;
//     u 128 34 / 24, 28 / 24.  8 experts, u 128: 8 rows each 30 / 34, 28 / 33; 32 rows each 42 / 35,
//     36 / 34.  u 256 72 / 36, 61 / 34
//   N 7168, K 2048: u 56 11 / 10, 10 / 10; u 112 17 / 12, 15 / 11; u 224 32 / 19, 28 / 18
//   N 1024, K 2048: u 32 8 / 10, 7 / 9; u 128 17 / 10, 15 / 10
//   N 2048, K 4096: u 64, one expert 15 / 15, 12 / 16; u 128, 8 experts 28 / 19, 24 / 17, 16 experts
//     31 / 22, 27 / 21; 64 experts of 4 rows (u 512) 71 / 54, 66 / 54
// The bound is 128, an expert's passes after its first counted 4/3 (the tiles do not repeat those).
// It was set against tiles of one size; the half-size tiles have since moved the crossing: they
// are ahead from u of about 60 on, bar experts of few rows with long K, so that calls of u 60 to
// 128 may take the slower kernel, by at most the 10 us above.
// max_rows bounds the passes; where that leaves the choice open, both are launched, the routed
// rows decide on the device, and one returns at once (2.2-2.5 us in a captured loop; 2.3-4.8 in a
// trace of single calls).  The tiles alone above 4096 rows and where a pass an expert would
// already be too many: there are few passes then only if nearly all of max_rows or most experts
// are unused.
mok_status_t launch_grouped_mx4(const GroupedArgs& a, hipStream_t st) {
  const int nt = (a.n + mx4::tile_cols<4>() - 1) / mx4::tile_cols<4>();
  const int64_t passes = std::min<int64_t>(a.max_rows, (a.max_rows + int64_t(a.groups) * (kPass - 1)) / kPass);
  const bool rows = is_few(passes, 0, nt), tiles = !rows && (a.max_rows > 4096 || nt * std::min<int64_t>(a.groups, a.max_rows) >= 192);
  mok_status_t s = MOK_OK;
  if (!rows) s = launch_tiles(a, nt, !tiles, st);
  if (!tiles && s == MOK_OK) s = launch_rows(a, passes, nt, !rows, st);
  return s;
}

}  // namespace mok
