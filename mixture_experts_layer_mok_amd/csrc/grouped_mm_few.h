// Grouped product of few 16-bit rows an expert (decoding): bound by reading the weights once, or, where
// there is little to read, by the launch and the latency of a wave's chunks, one pair after another.
// MI355X, bf16: 64 rows of 8 experts, N 4096, K 7168 92 to 95 us (5.0 TB/s; 180 on tiles); one row of
// one expert 18 us (58.7 MB: seven pairs of chunks a wave, 2.2 us each); 4 rows of 12, N 1000, K 520,
// fp16 3.9 us, of which the launch is most.
#pragma once
#include "expert_rows.h"

namespace mok {
namespace g16 {

constexpr int kWaves = 4;
constexpr uint32_t kFewLds = kWaves * 2 * 4 * 64 * 16;  // bytes of s_part
constexpr int kUnits = 16;               // 16-byte units of a row that a chunk holds: 128 elements
constexpr uint32_t kNone = 0x80000000u;  // added to an offset: out of every resource's range

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

template <int TYPE>
__device__ __forceinline__ f32x4_t mfma16(v4u a, v4u b, f32x4_t c) {
  if (TYPE == MOK_TYPE_BF16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                0, 0, 0);
}

// One workgroup of four waves: 16 NB columns of one expert and at most 32 of its rows (a pass).  The
// chunks of 128 summed elements are dealt to the waves, whose sums are joined through LDS in wave
// order.  A wave's weights go straight into its registers (they are used once, LDS would add a copy),
// two chunks at a time: while one is multiplied the other's loads are in flight.  What lies past K,
// past the rows and past N is read as zeros.
template <int TYPE, int NB, int MB>
struct Chunk {
  v4u b[NB][4], a[MB][4];

  __device__ __forceinline__ void load(const MmArgs& p, rsrc_t rb, rsrc_t ra, int valid, int ck) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t unit = ck * kUnits + 4 * s + g, past = int(unit) < p.k / 8 ? 0u : kNone;
#pragma unroll
      for (int j = 0; j < NB; ++j)
        b[j][s] = buf_ld16<kCpolPlain>(rb, (uint32_t(16 * j + r16) * uint32_t(p.k * 2) + unit * 16) | past);
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const int row = 16 * m + r16;
        a[m][s] = buf_ld16<kCpolPlain>(ra, (uint32_t(row) * uint32_t(p.ld_left * 2) + unit * 16) | past |
                                               (row < valid ? 0u : kNone));
      }
    }
  }
  __device__ __forceinline__ void multiply(f32x4_t (&acc)[MB][NB]) const {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[m][j] = mfma16<TYPE>(b[j][s], a[m][s], acc[m][j]);
  }
};

template <int TYPE, int NB, int MB>
__device__ __forceinline__ void pass(const MmArgs& p, f32x4_t* s_part, int e, int r0, int valid, int n0) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = (p.k / 8 + kUnits - 1) / kUnits, cols = min(16 * NB, p.n - n0);
  const rsrc_t rb = row_rsrc(static_cast<const uint16_t*>(p.right) + (int64_t(e) * p.n + n0) * p.k,
                             uint32_t(cols) * uint32_t(p.k * 2));
  const rsrc_t ra = row_rsrc(static_cast<const uint16_t*>(p.left) + int64_t(r0) * p.ld_left,
                             uint32_t(valid - 1) * uint32_t(p.ld_left * 2) + uint32_t(p.k * 2));
  f32x4_t acc[MB][NB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  if (w < chunks) {
    Chunk<TYPE, NB, MB> x, y;
    x.load(p, rb, ra, valid, w);
    for (int ck = w; ck < chunks; ck += 2 * kWaves) {
      y.load(p, rb, ra, valid, ck + kWaves);  // past the last: reads nothing
      x.multiply(acc);
      x.load(p, rb, ra, valid, ck + 2 * kWaves);
      y.multiply(acc);
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
      const int64_t at = int64_t(r0 + row) * p.ld_out + col;
      if (p.out32) {
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + at) = c;
      } else if (TYPE == MOK_TYPE_BF16) {
        *reinterpret_cast<uint64_t*>(static_cast<uint16_t*>(p.out) + at) =
            uint64_t(pack_bf16x2(c.x, c.y)) | (uint64_t(pack_bf16x2(c.z, c.w)) << 32);
      } else {
        typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
        *reinterpret_cast<f16x4_t*>(static_cast<uint16_t*>(p.out) + at) =
            f16x4_t{_Float16(c.x), _Float16(c.y), _Float16(c.z), _Float16(c.w)};
      }
    }
  }
}

// Passes of all experts times blocks of 16 NB columns, columns first, so that the passes that read
// the same weights run on the same XCD, at about the same time.
template <int TYPE, int NB>
__device__ __forceinline__ void few_items(const MmArgs& p, RowTiles& til, f32x4_t* s_part) {
  const int blocks = (p.n + 16 * NB - 1) / (16 * NB), total = til.total * blocks;
  for (int t = blockIdx.x; t < total; t += int(gridDim.x)) {
    const int m = t / blocks, n0 = (t - m * blocks) * 16 * NB;
    int e, r0, rows;
    til.find(p, m, &e, &r0, &rows);
    if (rows <= 16) pass<TYPE, NB, 1>(p, s_part, e, r0, rows, n0);
    else pass<TYPE, NB, 2>(p, s_part, e, r0, rows, n0);
    __syncthreads();  // s_part is read before the next item writes it
  }
}

// Columns a workgroup: the most that leave an item a CU (every item reads its rows again).
template <int TYPE>
__device__ __forceinline__ void walk_few(const MmArgs& p, RowTiles& til, f32x4_t* s_part) {
  if ((p.n + 63) / 64 * til.total >= 256) few_items<TYPE, 4>(p, til, s_part);
  else if ((p.n + 31) / 32 * til.total >= 256) few_items<TYPE, 2>(p, til, s_part);
  else few_items<TYPE, 1>(p, til, s_part);
}

}  // namespace g16
}  // namespace mok
