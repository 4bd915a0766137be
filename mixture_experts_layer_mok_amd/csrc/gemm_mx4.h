// Tile of the grouped MX product for many rows: one workgroup of four waves computes
// kTM x 256 outputs, 256 rows with MXFP4 activations and 128 with MXFP8, each wave half of
// the rows by 128 columns (32 x 32 MFMA blocks of v_mfma_scale_f32_32x32x64_f8f6f4).
//
// A K step is 256 elements: 32 KB of A and 32 KB of B, whole 128-byte lines, moved by
// direct-to-LDS loads through a ring of two stages.  Four waves of 128 x 128 read 128 KB of
// LDS a step (eight waves of 128 x 64 would read 192 KB: with the 64 KB the loads write,
// the LDS would then be as busy as the MFMA).  One wave a SIMD leaves 512 registers: 256
// accumulators and the fragments of two slices.
//
// Operand layout of 32 x 32 x 64, as measured: lane l holds row l % 32; with h = l / 32, a
// 4-bit operand's 16 bytes are K block h (32 elements), an 8-bit operand's first 16 bytes
// are elements 16 h .. +16 of block 0 and its last 16 the same of block 1; the scale of
// block h comes from lane r + 32 h.  Which blocks of the step a slice multiplies is free as
// long as both operands agree: slice s takes blocks s and 4 + s, so that lane group h needs
// the four blocks 4 h .. 4 h + 3 over the step's four slices, whose scales are one dword of
// the row, its byte s selected by the instruction.
//
// Scales: a ring of eight steps (64 bytes a row) in LDS, refilled four steps at a time once
// every wave has read the four (32 bytes a row, so that a cache line is not fetched for a
// few bytes each step), by direct-to-LDS loads too where their alignment allows it.
//
// LDS data rows: 128 bytes hold 8 chunks of 16, chunk c of row r at c ^ (r & 7) ^ ((r >> 3)
// & 1); 256 bytes hold 16, at c ^ (r & 15): the 16 rows that one pass of a 16-byte read
// takes then cover all 64 banks.
//
// Rows past the expert's last are read as its last one (never stored); weight rows past N
// as the last one; chunks past K as zeros (an out-of-range offset reads no memory), with
// zero scales.
#pragma once
#include "gemm_bf16.h"

namespace mok {
namespace mx4 {

constexpr int kThr = 256;
constexpr int kTN = 256;
constexpr int kStep = 256;                // K elements a step
constexpr int kRing = 8;                  // steps of scales in LDS
constexpr uint32_t kStageB = 32768;       // bytes of one operand's stage
#ifndef KD1
#define KD1 8
#define KD2 8
#endif
constexpr int kD1 = KD1, kD2 = KD2;       // data loads issued under slices 1 and 2 (the rest: 3)
constexpr uint32_t kPastRange = 0x80000000u;

template <bool A8>
constexpr int tile_rows() { return A8 ? 128 : 256; }

static __shared__ __align__(1024) v4u g_a[2 * kStageB / 16];
static __shared__ __align__(1024) v4u g_b[2 * kStageB / 16];
// Scales: two dwords a row and step.  With 16-byte loads piece q (of the ring's four, two
// steps each) of row r lies at 16-byte place q * rows + r; otherwise dword d (of sixteen) of
// row r at dword place d * rows + r.
static __shared__ __align__(1024) uint32_t g_sa[2 * kRing * 256];
static __shared__ __align__(1024) uint32_t g_sb[2 * kRing * 256];

typedef __attribute__((address_space(3))) const v4u lds_v4u;
typedef __attribute__((address_space(3))) v4u lds_wv4u;
typedef __attribute__((address_space(3))) uint64_t lds_wu64;

__device__ __forceinline__ i32x4_t rsrc_2g(const void* base) {
  i32x4_t r = make_rsrc(base);
  r.z = int(kPastRange);
  return r;
}

// Four scale bytes at byte `off` of r, of which `have` exist; the others are zeros.
__device__ __forceinline__ uint32_t scale_bytes4(rsrc_t r, uint32_t off, int have) {
  uint32_t w = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    w |= uint32_t(uint8_t(__builtin_amdgcn_raw_buffer_load_b8(r, have > c ? off + c : kPastRange, 0, 0)))
         << (8 * c);
  return w;
}

// Direct-to-LDS load of one dword a lane (see dma16_at).
__device__ __forceinline__ void dma4_at(const i32x4_t& rsrc, uint32_t voff, uint32_t lds_wave_addr) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_wave_addr);
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "s"(m0)
               : "memory", "m0");
}

// SG: bytes a scale load moves: 16 where every row's scales are whole 16-byte pieces at
// 16-byte addresses, 4 where they are whole dwords, 1 otherwise (through registers).
template <bool A8, int SG>
struct Tile {
  static constexpr int kTM = tile_rows<A8>();
  static constexpr int kIB = A8 ? 2 : 4;  // 32-row blocks of A a wave
  static constexpr int kJB = 4;           // 32-row blocks of B a wave

  i32x4_t ra, rb;
  uint32_t oa[8], ob[8];     // byte offsets of this lane's chunks in step 0
  uint32_t la[4];            // LDS byte address of the A fragment of slice s, block 0, stage 0
  uint32_t lb[4];            // the same of B
  const uint8_t *psa, *psb;  // scales of A from the tile's first row, of the expert's B
  uint32_t osa, osb;         // this thread's scale rows (past the range: none)
  int nblk, steps, ca, cb;   // K blocks, steps; this lane's chunk of an A and of a B row
  f32x16_t acc[kIB][kJB];

  __device__ __forceinline__ void init(const GroupedArgs& p, int e, int64_t r0, int rows, int n0) {
    const int t = threadIdx.x, l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int kb = p.k / 2;
    nblk = p.k / 32;
    steps = (p.k + kStep - 1) / kStep;
    ra = rsrc_2g(p.a + r0 * p.ld_a);
    rb = rsrc_2g(p.b + int64_t(e) * p.n * kb);
    ca = A8 ? ((l & 15) ^ (((w & 3) * 4 + (l >> 4)) & 15)) : ((l & 7) ^ (l >> 3) ^ (w & 1));
    cb = (l & 7) ^ (l >> 3) ^ (w & 1);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int ar = A8 ? (q * 4 + w) * 4 + (l >> 4) : (q * 4 + w) * 8 + (l >> 3);
      const int br = (q * 4 + w) * 8 + (l >> 3);
      oa[q] = uint32_t(int64_t(min(ar, rows - 1)) * p.ld_a) + ca * 16;
      ob[q] = uint32_t(min(n0 + br, p.n - 1)) * uint32_t(kb) + cb * 16;
    }
    const int wm = w >> 1, wn = w & 1, r = l & 31, h = l >> 5;
    const int sw = (r & 7) ^ ((r >> 3) & 1);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      la[s] = lds_addr(g_a) + (A8 ? uint32_t(wm * 64 + r) * 256 + (((2 * s + h) ^ (r & 15)) * 16)
                                  : uint32_t(wm * 128 + r) * 128 + (((4 * h + s) ^ sw) * 16));
      lb[s] = lds_addr(g_b) + uint32_t(wn * 128 + r) * 128 + (((4 * h + s) ^ sw) * 16);
    }
    psa = p.as + r0 * p.ld_as;
    psb = p.bs + int64_t(e) * p.n * nblk;
    osa = t < kTM ? uint32_t(min(t, rows - 1) * p.ld_as) : kPastRange;
    osb = uint32_t(min(n0 + t, p.n - 1)) * uint32_t(nblk);
#pragma unroll
    for (int i = 0; i < kIB; ++i)
#pragma unroll
      for (int j = 0; j < kJB; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  }

  // Direct-to-LDS load q (0..7 A, 8..15 B) of step ks into the stage at byte `stage` of the
  // rings.  A step past the last reads nothing.
  __device__ __forceinline__ void issue(int ks, int q, uint32_t stage) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (q < 8) {
      const uint32_t past = (A8 ? 16 * ks + ca < 2 * nblk : 8 * ks + ca < nblk) ? 0u : kPastRange;
      dma16_at<false>(ra, oa[q] | past, uint32_t(ks) * (A8 ? 256 : 128),
                      lds_addr(g_a) + stage + (q * 4 + w) * 1024);
    } else {
      const uint32_t past = 8 * ks + cb < nblk ? 0u : kPastRange;
      dma16_at<false>(rb, ob[q - 8] | past, uint32_t(ks) * 128,
                      lds_addr(g_b) + stage + ((q - 8) * 4 + w) * 1024);
    }
  }

  // Scales of steps 4 quad .. 4 quad + 3 (32 bytes a row) into their half of the ring; each
  // wave moves those of 64 rows of A and of B.
  __device__ __forceinline__ void issue_scales(int quad) {
    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int at = quad * 32, half = quad & 1;
    const i32x4_t rsa = rsrc_2g(psa), rsb = rsrc_2g(psb);
    if (SG == 16) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t past = at + 16 * i < nblk ? 0u : kPastRange;
        if (w * 64 < kTM)
          dma16_at<false>(rsa, (osa + at + 16 * i) | past, 0,
                          lds_addr(g_sa) + uint32_t((half * 2 + i) * kTM + w * 64) * 16);
        dma16_at<false>(rsb, (osb + at + 16 * i) | past, 0,
                        lds_addr(g_sb) + uint32_t((half * 2 + i) * 256 + w * 64) * 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int have = nblk - at - 4 * i;
        if (SG == 4) {
          const uint32_t past = have > 0 ? 0u : kPastRange;
          if (w * 64 < kTM)
            dma4_at(rsa, (osa + at + 4 * i) | past,
                    lds_addr(g_sa) + uint32_t((half * 8 + i) * kTM + w * 64) * 4);
          dma4_at(rsb, (osb + at + 4 * i) | past,
                  lds_addr(g_sb) + uint32_t((half * 8 + i) * 256 + w * 64) * 4);
        } else {
          if (w * 64 < kTM)
            g_sa[(half * 8 + i) * kTM + t] = scale_bytes4(row_rsrc(psa, kPastRange), osa + at + 4 * i, have);
          g_sb[(half * 8 + i) * 256 + t] = scale_bytes4(row_rsrc(psb, kPastRange), osb + at + 4 * i, have);
        }
      }
    }
  }

  struct Scales {
    uint32_t a[kIB], b[kJB];
  };
  __device__ __forceinline__ void read_scales(Scales& s, int ks) const {
    const int t = threadIdx.x, l = t & 63, w = t >> 6;
    const int wm = w >> 1, wn = w & 1, r = l & 31, h = l >> 5;
    const int d = 2 * (ks & (kRing - 1)) + h;  // dword of the ring
    const int ra_ = wm * (kTM / 2) + r, rb_ = wn * 128 + r;
#pragma unroll
    for (int i = 0; i < kIB; ++i)
      s.a[i] = SG == 16 ? g_sa[((d >> 2) * kTM + ra_ + 32 * i) * 4 + (d & 3)] : g_sa[d * kTM + ra_ + 32 * i];
#pragma unroll
    for (int j = 0; j < kJB; ++j)
      s.b[j] = SG == 16 ? g_sb[((d >> 2) * 256 + rb_ + 32 * j) * 4 + (d & 3)] : g_sb[d * 256 + rb_ + 32 * j];
  }

  __device__ __forceinline__ i32x8_t read_a(int s, int i, uint32_t stage) const {
    const uint32_t o = uint32_t(i) * 32 * (A8 ? 256 : 128) + stage;
    const v4u x = *reinterpret_cast<lds_v4u*>(uintptr_t(la[s] + o));
    if (A8) {
      const v4u y = *reinterpret_cast<lds_v4u*>(uintptr_t((la[s] ^ 128u) + o));
      return i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w), int(y.x), int(y.y), int(y.z), int(y.w)};
    }
    return i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
  }
  __device__ __forceinline__ i32x8_t read_b(int s, int j, uint32_t stage) const {
    const v4u x = *reinterpret_cast<lds_v4u*>(uintptr_t(lb[s] + stage + uint32_t(j) * 32 * 128));
    return i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
  }

  struct Frag {
    i32x8_t a[kIB], b[kJB];
  };

  // One slice's MFMAs on f, and between them: the fragments of slice RS (of the stage that la,
  // lb plus rd point at) read into fr, and data loads D0 .. D0 + DN - 1 of step ks + 2 issued
  // into stage `wr`.
  template <int SL, int RS, int D0, int DN>
  __device__ __forceinline__ void slice(const Frag& f, Frag& fr, const Scales& sc, uint32_t rd, int ks,
                                        uint32_t wr) {
    constexpr int kM = kIB * kJB;  // MFMAs
    constexpr int kR = kIB + kJB;  // fragment reads, one or two after each of the first MFMAs
    constexpr int kPer = (kR + kM / 2 - 1) / (kM / 2);
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int i = m / kJB, j = m % kJB;
      __builtin_amdgcn_sched_barrier(0);
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          f.b[j], f.a[i], acc[i][j], 4, A8 ? 0 : 4, SL, int(sc.b[j]), SL, int(sc.a[i]));
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int r = m * kPer + x;
        if (r < kIB) fr.a[r] = read_a(RS, r, rd);
        else if (r < kR) fr.b[r - kIB] = read_b(RS, r - kIB, rd);
      }
#pragma unroll
      for (int q = 0; q < DN; ++q)
        if (q * kM / (DN > 0 ? DN : 1) == m) issue(ks + 2, D0 + q, wr);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ __forceinline__ void run() {
    asm volatile("" ::: "memory");
    issue_scales(0);
    issue_scales(1);
#pragma unroll
    for (int q = 0; q < 16; ++q) issue(0, q, 0);
#pragma unroll
    for (int q = 0; q < 16; ++q) issue(1, q, kStageB);
    wait_loads_and_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // f[s]: the fragments of slice s.  Those of slices 0..2 are read one step ahead, those of
    // slice 3 under slice 0 of their own step.
    Frag f[4];
    Scales sc, sn;
    read_scales(sc, 0);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
#pragma unroll
      for (int i = 0; i < kIB; ++i) f[s].a[i] = read_a(s, i, 0);
#pragma unroll
      for (int j = 0; j < kJB; ++j) f[s].b[j] = read_b(s, j, 0);
    }
    uint32_t cur = 0;  // stage of step ks
    for (int ks = 0; ks < steps; ++ks) {
      slice<0, 3, 0, 0>(f[0], f[3], sc, cur, ks, cur);
      // step ks + 1 has landed (mine by the wait, everyone's by the barrier), and every wave
      // has read the last of this step's stage and its scales
      wait_loads_and_lds();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const uint32_t nxt = cur ^ kStageB;
      if ((ks & 3) == 3) issue_scales(ks / 4 + 2);  // into the half of the ring just read
      read_scales(sn, ks + 1);
      slice<1, 0, 0, kD1>(f[1], f[0], sc, nxt, ks, cur);
      slice<2, 1, kD1, kD2>(f[2], f[1], sc, nxt, ks, cur);
      slice<3, 2, kD1 + kD2, 16 - kD1 - kD2>(f[3], f[2], sc, nxt, ks, cur);
      sc = sn;
      cur = nxt;
    }
    // every load has landed and every wave has read its last fragments: the stages are free
    wait_loads_and_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  // Block (i, j): lane l holds row l % 32 of A and, of B's 32 rows, 8 q + 4 h + u (q, u =
  // 0..3): four consecutive columns of out each.
  template <bool OUT32>
  __device__ __forceinline__ void store(const GroupedArgs& p, int64_t r0, int rows, int n0) {
    const int t = threadIdx.x, l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = w >> 1, wn = w & 1, r = l & 31, h = l >> 5;
    const int row0 = wm * (kTM / 2), col0 = n0 + wn * 128;
    if (OUT32) {
      float* o = static_cast<float*>(p.out);
#pragma unroll
      for (int i = 0; i < kIB; ++i) {
        const int row = row0 + 32 * i + r;
        float* orow = o + (r0 + row) * p.ld_out;
#pragma unroll
        for (int j = 0; j < kJB; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = col0 + 32 * j + 8 * q + 4 * h;
            if (row < rows && col < p.n)
              *reinterpret_cast<f32x4_t*>(orow + col) =
                  f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          }
      }
      return;
    }
    // bf16: the wave's rows of 128 columns (256 bytes, 16-byte chunk c of row r at c ^ (r &
    // 15)) through its own 32 KB of the stages, then whole row segments, 16 bytes a lane
    const uint32_t base = (w & 2 ? lds_addr(g_b) : lds_addr(g_a)) + uint32_t(w & 1) * kStageB;
#pragma unroll
    for (int i = 0; i < kIB; ++i) {
      const uint32_t at = base + uint32_t(32 * i + r) * 256 + 8 * h;
#pragma unroll
      for (int j = 0; j < kJB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<lds_wu64*>(uintptr_t(at + (((4 * j + q) ^ (r & 15)) * 16))) =
              uint64_t(pack_bf16x2(acc[i][j][4 * q], acc[i][j][4 * q + 1])) |
              (uint64_t(pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])) << 32);
    }
    uint16_t* o = static_cast<uint16_t*>(p.out);
#pragma unroll 4
    for (int it = 0; it < kTM / 8; ++it) {
      const int lr = it * 4 + (l >> 4), row = row0 + lr;
      const int col = col0 + (((l & 15) ^ (lr & 15)) * 8);
      const v4u v = *reinterpret_cast<lds_v4u*>(uintptr_t(base + uint32_t(lr) * 256 + (l & 15) * 16));
      if (row < rows && col < p.n) *reinterpret_cast<v4u*>(o + (r0 + row) * p.ld_out + col) = v;
    }
  }
};

}  // namespace mx4
}  // namespace mok
