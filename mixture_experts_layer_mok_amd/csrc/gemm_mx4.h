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
// Scales: eight steps' worth (64 bytes a row, so no cache line is fetched for a few
// bytes) go through registers into LDS at a time, as [dword of the window][row], which
// the lanes of a fragment read without bank conflicts.
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
constexpr int kWin = 8;                   // steps a scale window
constexpr uint32_t kStageB = 32768;       // bytes of one operand's stage
constexpr uint32_t kPastRange = 0x80000000u;

template <bool A8>
constexpr int tile_rows() { return A8 ? 128 : 256; }

static __shared__ __align__(1024) v4u g_a[2 * kStageB / 16];
static __shared__ __align__(1024) v4u g_b[2 * kStageB / 16];
static __shared__ uint32_t g_sa[2 * kWin * 256];  // [dword of the window][row]
static __shared__ uint32_t g_sb[2 * kWin * 256];

typedef __attribute__((address_space(3))) const v4u lds_v4u;
typedef __attribute__((address_space(3))) v4u lds_wv4u;
typedef __attribute__((address_space(3))) uint64_t lds_wu64;

__device__ __forceinline__ i32x4_t rsrc_2g(const void* base) {
  i32x4_t r = make_rsrc(base);
  r.z = int(kPastRange);
  return r;
}

// Sixteen scale bytes at byte `off` of r, of which `have` exist (a multiple of SG, or all);
// the others are zeros.  SG: bytes a load, 16 where every row's scales are whole 16-byte
// pieces, 4 where they are whole dwords, 1 otherwise.
template <int SG>
__device__ __forceinline__ v4u load_scales16(rsrc_t r, uint32_t off, int have) {
  if (SG == 16) return buf_ld16<kCpolPlain>(r, have >= 16 ? off : kPastRange);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (SG == 4) {
      w[i] = __builtin_amdgcn_raw_buffer_load_b32(r, have > 4 * i ? off + 4 * i : kPastRange, 0, 0);
    } else {
      w[i] = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        w[i] |= uint32_t(uint8_t(__builtin_amdgcn_raw_buffer_load_b8(
                    r, have > 4 * i + c ? off + 4 * i + c : kPastRange, 0, 0)))
                << (8 * c);
    }
  }
  return v4u{w[0], w[1], w[2], w[3]};
}

template <bool A8, int SG>
struct Tile {
  static constexpr int kTM = tile_rows<A8>();
  static constexpr int kIB = A8 ? 2 : 4;  // 32-row blocks of A a wave
  static constexpr int kJB = 4;           // 32-row blocks of B a wave

  i32x4_t ra, rb;
  uint32_t oa[8], ob[8];     // byte offsets of this lane's chunks in step 0
  uint32_t la[4];            // LDS byte address of the A fragment of slice s, block 0, stage 0
  uint32_t lb[4];            // the same of B
  rsrc_t rsa, rsb;           // scales of A from the tile's first row, of the expert's B
  uint32_t osa, osb;         // this thread's scale rows (past the range: none)
  int nblk, steps, ca, cb;   // K blocks, steps; this lane's chunk of an A and of a B row
  v4u wa[4], wb[4];          // the next window's scales of this thread's rows
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
    rsa = row_rsrc(p.as + r0 * p.ld_as, kPastRange);
    rsb = row_rsrc(p.bs + int64_t(e) * p.n * nblk, kPastRange);
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

  __device__ __forceinline__ void load_window(int win) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = win * 64 + 16 * i, have = nblk - at;
      wa[i] = load_scales16<SG>(rsa, osa + at, have);
      wb[i] = load_scales16<SG>(rsb, osb + at, have);
    }
  }
  __device__ __forceinline__ void store_window() {
    const int t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!A8 || t < kTM) g_sa[(4 * i + c) * kTM + t] = wa[i][c];
        g_sb[(4 * i + c) * 256 + t] = wb[i][c];
      }
  }

  struct Scales {
    uint32_t a[kIB], b[kJB];
  };
  __device__ __forceinline__ void read_scales(Scales& s, int ks) const {
    const int t = threadIdx.x, l = t & 63, w = t >> 6;
    const int wm = w >> 1, wn = w & 1, r = l & 31, h = l >> 5;
    const int d = 2 * (ks & (kWin - 1)) + h;
#pragma unroll
    for (int i = 0; i < kIB; ++i) s.a[i] = g_sa[d * kTM + wm * (kTM / 2) + 32 * i + r];
#pragma unroll
    for (int j = 0; j < kJB; ++j) s.b[j] = g_sb[d * 256 + wn * 128 + 32 * j + r];
  }

  __device__ __forceinline__ i32x8_t read_a(int s, int i) const {
    const uint32_t o = uint32_t(i) * 32 * (A8 ? 256 : 128);
    const v4u x = *reinterpret_cast<lds_v4u*>(uintptr_t(la[s] + o));
    if (A8) {
      const v4u y = *reinterpret_cast<lds_v4u*>(uintptr_t((la[s] ^ 128u) + o));
      return i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w), int(y.x), int(y.y), int(y.z), int(y.w)};
    }
    return i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
  }
  __device__ __forceinline__ i32x8_t read_b(int s, int j) const {
    const v4u x = *reinterpret_cast<lds_v4u*>(uintptr_t(lb[s] + uint32_t(j) * 32 * 128));
    return i32x8_t{int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
  }

  template <int SL>
  __device__ __forceinline__ void mma_row(const i32x8_t& a, const i32x8_t (&b)[kJB], uint32_t sa_,
                                          const uint32_t (&sb_)[kJB], f32x16_t (&c)[kJB]) {
#pragma unroll
    for (int j = 0; j < kJB; ++j)
      c[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[j], a, c[j], 4, A8 ? 0 : 4, SL,
                                                             int(sb_[j]), SL, int(sa_));
  }

  // One slice: its MFMAs, with the next slice's fragments (slice NSL, at la, lb) read under
  // them: B into bn, each A block in place once its row of MFMAs has issued.  With DMA, the
  // loads of step ks + 2 into the current stage are issued between the rows too.
  template <int SL, int NSL, bool DMA>
  __device__ __forceinline__ void slice(i32x8_t (&a)[kIB], i32x8_t (&b)[kJB], const Scales& sc, int ks,
                                        uint32_t stage) {
    i32x8_t bn[kJB];
#pragma unroll
    for (int i = 0; i < kIB; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      constexpr int kRB = 2;  // rows over which the B reads are spread
      if (i < kRB) {
#pragma unroll
        for (int j = 0; j < kJB / kRB; ++j) bn[i * (kJB / kRB) + j] = read_b(NSL, i * (kJB / kRB) + j);
      }
      mma_row<SL>(a[i], b, sc.a[i], sc.b, acc[i]);
      if (DMA) {
#pragma unroll
        for (int q = 0; q < 16 / kIB; ++q) issue(ks + 2, i * (16 / kIB) + q, stage);
      }
      __builtin_amdgcn_sched_barrier(0);
      a[i] = read_a(NSL, i);
    }
#pragma unroll
    for (int j = 0; j < kJB; ++j) b[j] = bn[j];
  }

  __device__ __forceinline__ void run() {
    asm volatile("" ::: "memory");
    load_window(0);
#pragma unroll
    for (int q = 0; q < 16; ++q) issue(0, q, 0);
#pragma unroll
    for (int q = 0; q < 16; ++q) issue(1, q, kStageB);
    store_window();
    wait_loads_and_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    i32x8_t a[kIB], b[kJB];
    Scales sc;
    read_scales(sc, 0);
#pragma unroll
    for (int i = 0; i < kIB; ++i) a[i] = read_a(0, i);
#pragma unroll
    for (int j = 0; j < kJB; ++j) b[j] = read_b(0, j);
    // Step ks: on entry a, b hold its slice 0 and sc its scales.
    uint32_t stage = 0;
    for (int ks = 0; ks < steps; ++ks) {
      slice<0, 1, false>(a, b, sc, ks, stage);
      slice<1, 2, false>(a, b, sc, ks, stage);
      slice<2, 3, false>(a, b, sc, ks, stage);
      __builtin_amdgcn_sched_barrier(0);
      // step ks + 1 has landed (mine by the wait, everyone's by the barrier), and every wave
      // has read the last of this stage and the scales of step ks
      wait_loads_and_lds();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const int nx = ks + 1;
      if ((nx & (kWin - 1)) == 0) {  // the next step opens a scale window
        store_window();
        wait_loads_and_lds();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      if ((nx & (kWin - 1)) == kWin / 2) load_window(nx / kWin + 1);
      const uint32_t turn = stage ? 0u - kStageB : kStageB;
      la[0] += turn;
      lb[0] += turn;
      Scales sn;
      read_scales(sn, nx);
      slice<3, 0, true>(a, b, sc, ks, stage);
      sc = sn;
#pragma unroll
      for (int s = 1; s < 4; ++s) {
        la[s] += turn;
        lb[s] += turn;
      }
      stage ^= kStageB;
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
