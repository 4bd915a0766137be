// Tile of the grouped MX product for many rows: one workgroup of four waves computes
// kTM x 256 outputs, 256 rows with MXFP4 activations and 128 with MXFP8, each wave half of
// the rows by 128 columns (32 x 32 MFMA blocks of v_mfma_scale_f32_32x32x64_f8f6f4).  Bound
// by the card's power and by moving the data: 16,384 rows, N 4096, K 7168 in MXFP4 on MI355X take
// 250 us in a captured loop over one input and 280 over changing ones (3.4-3.9 PFLOP/s, by card),
// at 1.9 of 2.4 GHz with the matrix cores half busy; the kernel without its loads and stores 188
// at the same clock, its matrix instructions alone, on random data, 162.
//
// A K step is 256 elements: 32 KB of A and 32 KB of B, whole 128-byte lines, moved by
// direct-to-LDS loads through a ring of two stages.  Four waves of 128 x 128 read 128 KB of
// LDS a step (eight waves of 128 x 64 would read 192 KB: with the 64 KB the loads write,
// the LDS would then be as busy as the MFMA).  One wave a SIMD leaves 512 registers: 256
// accumulators and the fragments of the step's four slices.
//
// Operand layout of 32 x 32 x 64, as measured: lane l holds row l % 32; with h = l / 32, a
// 4-bit operand's 16 bytes are K block h (32 elements), an 8-bit operand's first 16 bytes
// are elements 16 h .. +16 of block 0 and its last 16 the same of block 1; the scale of
// block h comes from lane r + 32 h.  Which blocks of the step a slice multiplies is free as
// long as both operands agree: slice s takes blocks s and 4 + s, so that lane group h needs
// the four blocks 4 h .. 4 h + 3 over the step's four slices, whose scales are one dword of
// the row, its byte s selected by the instruction.
//
// Scales: a ring of eight steps (64 bytes a row) in LDS, refilled four steps at a time (32
// bytes a row, so that a cache line is not fetched for a few bytes each step) once every wave
// has read the four, by direct-to-LDS loads too.  These take dword addresses; where a row's
// scales start inside a dword, the ring holds the dwords from that one on, and a reader
// shifts two of them together (16,384 rows, N 4096, K 7200 in MXFP4 on MI355X: 516 us with the
// scales brought in by bytes, 287 so; 250 for the whole pieces of K 7168).
//
// LDS data rows: 128 bytes hold 8 chunks of 16, chunk c of row r at c ^ (r & 7) ^ ((r >> 3)
// & 1); 256 bytes hold 16, at c ^ (r & 15): the 16 rows that one pass of a 16-byte read
// takes then cover all 64 banks.
//
// Rows past the expert's last are read as its last one (never stored); weight rows past N
// as the last one; chunks past K as zeros (an out-of-range offset reads no memory), with
// zero scales.
//
// Tiles of few rows (the end of an expert's rows, or all of them) run with fewer row blocks
// a wave: IB = 1 covers 64 rows, 2 covers 128, 4 covers 256.  Where whole tiles would leave
// CUs idle, tiles of half the rows and columns (JB = 2).
//
// A workgroup walks several tiles: the next one's first loads are in flight while the current
// one's results are stored, through LDS that those loads leave free.
#pragma once
#include "gemm_bf16.h"

namespace mok {
namespace mx4 {

constexpr int kThr = 256;
constexpr int kRing = 8;                  // steps of scales in LDS
constexpr uint32_t kStageB = 32768;       // bytes of one operand's stage
constexpr uint32_t kPastRange = 0x80000000u;

// JB: blocks of 32 columns a wave, 4 for whole tiles, 2 for tiles of half the rows and columns.
template <int JB>
constexpr int tile_cols() { return 64 * JB; }
template <bool A8, int JB>
constexpr int tile_rows() { return (A8 ? 32 : 64) * JB; }

static __shared__ __align__(1024) v4u g_a[2 * kStageB / 16];
static __shared__ __align__(1024) v4u g_b[2 * kStageB / 16];
// Scales: two dwords a row and step.  The two 16-byte pieces (two steps each) that a row has in
// half a ring are fetched by two lanes of one load, so that it touches 32 lines and not 64;
// piece q of row r lies at 16-byte place
//   half * 2 rows + 2 (r & ~7) + (r & 7) + 8 (q ^ ((r >> 3) & 1)),
// where reading one dword of 32 rows meets each bank twice.
static __shared__ __align__(1024) uint32_t g_sa[2 * kRing * 256];
static __shared__ __align__(1024) uint32_t g_sb[2 * kRing * 256];

typedef __attribute__((address_space(3))) const v4u lds_v4u;
typedef __attribute__((address_space(3))) v4u lds_wv4u;
typedef __attribute__((address_space(3))) uint64_t lds_wu64;

// A wave-uniform value into a scalar register, whatever the compiler holds it in: the loads
// below are inline asm, which cannot take a resource from vector registers.  (The builtin is
// dropped where its operand is known to be uniform, also when that lies in a vector register.)
// The compiler does not see into the asm, so it has the wait states that gfx950 asks for:
// one between a vector write and the lane read of its result, five between a scalar result
// of a vector instruction and a vector memory operation that reads it.
__device__ __forceinline__ int scalar(int v) {
  int s;
  asm volatile("s_nop 0\n\tv_readfirstlane_b32 %0, %1\n\ts_nop 4" : "=s"(s) : "v"(v));
  return s;
}
__device__ __forceinline__ i32x4_t rsrc_2g(const void* base) {
  const uint64_t x = reinterpret_cast<uint64_t>(base);
  return i32x4_t{scalar(int(uint32_t(x))), scalar(int(uint32_t(x >> 32) & 0xFFFFu)), int(kPastRange),
                 0x00020000};
}

// The same for `bytes` bytes, from the dword that the first lies in to the one that the last
// lies in: what a load of several dwords has past it reads as zeros (each dword by itself).
__device__ __forceinline__ i32x4_t rsrc_dwords(const uint8_t* base, uint32_t bytes) {
  const uint32_t low = uint32_t(reinterpret_cast<uintptr_t>(base) & 3);
  i32x4_t r = rsrc_2g(base - low);
  r.z = scalar(int((low + bytes + 3) & ~3u));
  return r;
}

// Direct-to-LDS load of 16 bytes a lane: lane l's land at lds_wave_addr + 16 l.  The string has
// the wait states itself: one after the write of M0, and five after whatever vector instruction
// may have written a scalar that the load reads (v_readlane reloads spilled ones).
__device__ __forceinline__ void lds_load16(const i32x4_t& rsrc, uint32_t voff, uint32_t soff,
                                           uint32_t lds_wave_addr) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_wave_addr);
  soff = __builtin_amdgcn_readfirstlane(soff);
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff),
               "s"(rsrc), "s"(soff), "s"(m0)
               : "memory", "m0");
}

// SHIFT: some row's scales do not start at a 16-byte address or are not whole 16-byte pieces.
//
// Where a tile's operands come from, and its direct-to-LDS loads.
template <bool A8, bool SHIFT, int JB>
struct Source {
  static constexpr int kTM = tile_rows<A8, JB>(), kTN = tile_cols<JB>();
  static constexpr int kSRows = kTM < 128 ? 128 : kTM;         // rows of A in the scale ring
  static constexpr int kSA = kSRows / 128, kSB = kTN / 128;    // 16-byte loads of scales a wave
  static constexpr int kQ = 2 * JB;                            // data loads of A, and of B, at most
  i32x4_t ra, rb;            // codes of A from the tile's first row, of the expert's B
  i32x4_t rsa, rsb;          // their scales
  uint32_t oa[kQ], ob[kQ];   // byte offsets of this lane's chunks in step 0
  uint32_t osa[kSA], osb[kSB];  // this lane's pieces of the scales
  uint32_t sha, shb;          // bytes of its rows' first dword before their first scale
  int nblk;                  // K blocks
  int ca, cb;                // this lane's chunk of an A and of a B row

  __device__ __forceinline__ void init(const GroupedArgs& p, int e, int64_t r0, int rows, int n0) {
    const int t = threadIdx.x, l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int kb = p.k / 2;
    nblk = p.k / 32;
    ra = rsrc_2g(p.a + r0 * p.ld_a);
    rb = rsrc_2g(p.b + int64_t(e) * p.n * kb);
    ca = A8 ? ((l & 15) ^ (((w & 3) * 4 + (l >> 4)) & 15)) : ((l & 7) ^ (l >> 3) ^ (w & 1));
    cb = (l & 7) ^ (l >> 3) ^ (w & 1);
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int ar = A8 ? (q * 4 + w) * 4 + (l >> 4) : (q * 4 + w) * 8 + (l >> 3);
      const int br = (q * 4 + w) * 8 + (l >> 3);
      oa[q] = uint32_t(int64_t(min(ar, rows - 1)) * p.ld_a) + ca * 16;
      ob[q] = uint32_t(min(n0 + br, p.n - 1)) * uint32_t(kb) + cb * 16;
    }
    const uint8_t *as = p.as + r0 * p.ld_as, *bs = p.bs + int64_t(e) * p.n * nblk;
    rsa = rsrc_dwords(as, uint32_t((rows - 1) * p.ld_as) + nblk);
    rsb = rsrc_dwords(bs, uint32_t(p.n) * nblk);
    const uint32_t la = uint32_t(reinterpret_cast<uintptr_t>(as) & 3);
    const uint32_t lb = uint32_t(reinterpret_cast<uintptr_t>(bs) & 3);
    // (32 rows on the first dword starts at the same byte)
    sha = (la + uint32_t(l & 31) * uint32_t(p.ld_as)) & 3;
    shb = (lb + uint32_t(l & 31) * uint32_t(nblk)) & 3;
    const int row = 8 * (l >> 4) + (l & 7);
    const uint32_t piece = 16u * (((l >> 3) ^ (l >> 4)) & 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i < kSA) osa[i] = ((la + uint32_t(min((w * kSA + i) * 32 + row, rows - 1) * p.ld_as)) & ~3u) + piece;
      if (i < kSB) osb[i] = ((lb + uint32_t(min(n0 + (w * kSB + i) * 32 + row, p.n - 1)) * uint32_t(nblk)) & ~3u) + piece;
    }
  }

  // Load q (0..7 A, 8..15 B) of step ks into the stage at byte `stage` of the rings.  A step
  // past the last reads nothing.
  __device__ __forceinline__ void issue(int ks, int q, uint32_t stage) const {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (q < 8) {
      const uint32_t past = (A8 ? 16 * ks + ca < 2 * nblk : 8 * ks + ca < nblk) ? 0u : kPastRange;
      lds_load16(ra, oa[q] | past, uint32_t(ks) * (A8 ? 256 : 128),
                      lds_addr(g_a) + stage + (q * 4 + w) * 1024);
    } else {
      const uint32_t past = 8 * ks + cb < nblk ? 0u : kPastRange;
      lds_load16(rb, ob[q - 8] | past, uint32_t(ks) * 128,
                      lds_addr(g_b) + stage + ((q - 8) * 4 + w) * 1024);
    }
  }

  // Part 0..3 of the scales of steps 4 quad .. 4 quad + 3 (32 bytes a row) into their half of the
  // ring; each wave moves those of a quarter of the rows.
  __device__ __forceinline__ void issue_scales(int quad, int part) const {
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int at = quad * 32, half = quad & 1, i = part & 1;
    const int last = SHIFT ? nblk + 3 : nblk;  // no scale of a row lies in a piece from here on
    const uint32_t past = at + 16 * (((l >> 3) ^ (l >> 4)) & 1) < last ? 0u : kPastRange;
    if (part >= 2 && i < kSB)
      lds_load16(rsb, (osb[i < kSB ? i : 0] + at) | past, 0,
                 lds_addr(g_sb) + uint32_t(half * 2 * kTN + (kSB * w + i) * 64) * 16);
    if (part < 2 && i < kSA)
      lds_load16(rsa, (osa[i < kSA ? i : 0] + at) | past, 0,
                 lds_addr(g_sa) + uint32_t(half * 2 * kSRows + (kSA * w + i) * 64) * 16);
  }

  // The same with what is wave-uniform in scalar registers again (values that were chosen on
  // several paths may have lost them).
  __device__ __forceinline__ Source uniform() const {
    Source s = *this;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.ra[i] = scalar(ra[i]);
      s.rb[i] = scalar(rb[i]);
      s.rsa[i] = scalar(rsa[i]);
      s.rsb[i] = scalar(rsb[i]);
    }
    s.ra.z = s.rb.z = int(kPastRange);
    s.rsa.z = scalar(rsa.z);
    s.rsb.z = scalar(rsb.z);
    s.ra.w = s.rb.w = s.rsa.w = s.rsb.w = 0x00020000;
    s.nblk = scalar(nblk);
    return s;
  }

  // The scales of the first four steps, then the data of step 0, then of step 1: kAhead loads
  // a wave may be in flight when step 0 has landed.
  static constexpr int kAhead = 2 * kQ;
  __device__ __forceinline__ void begin() const {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int part = 0; part < 4; ++part) issue_scales(0, part);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int q = 0; q < 2 * kQ; ++q) issue(ks, q < kQ ? q : q - kQ + 8, ks * kStageB);
    asm volatile("" ::: "memory");
  }
};

// The wave's LDS operations have completed (lgkmcnt 0; gfx9 encoding).
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
}

// At most n (wave-uniform, one of the counts of stores a tile makes) of the wave's memory
// operations still in flight: those it issued before its last n have completed.
__device__ __forceinline__ void wait_all_but(int n) {
  if (n >= 63) wait_vmcnt<63>();
  else if (n >= 48) wait_vmcnt<48>();
  else if (n >= 32) wait_vmcnt<32>();
  else if (n >= 24) wait_vmcnt<24>();
  else if (n >= 16) wait_vmcnt<16>();
  else if (n >= 8) wait_vmcnt<8>();
  else wait_vmcnt<0>();
}

// IB, JB: 32-row blocks of A and of B a wave.
template <bool A8, bool SHIFT, int IB, int JB>
struct Tile {
  typedef Source<A8, SHIFT, JB> Src;
  static constexpr int kJB = JB;
  static constexpr int kQA = A8 ? 4 * IB : 2 * IB;  // A loads a step

  uint32_t la[4];  // LDS byte address of the A fragment of slice s, block 0, stage 0
  uint32_t lb[4];  // the same of B
  f32x16_t acc[IB][kJB];

  __device__ __forceinline__ void init() {
    const int t = threadIdx.x, l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = w >> 1, wn = w & 1, r = l & 31, h = l >> 5;
    const int sw = (r & 7) ^ ((r >> 3) & 1);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      la[s] = lds_addr(g_a) + (A8 ? uint32_t(wm * 32 * IB + r) * 256 + (((2 * s + h) ^ (r & 15)) * 16)
                                  : uint32_t(wm * 32 * IB + r) * 128 + (((4 * h + s) ^ sw) * 16));
      lb[s] = lds_addr(g_b) + uint32_t(wn * 32 * JB + r) * 128 + (((4 * h + s) ^ sw) * 16);
    }
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j = 0; j < kJB; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  }

  struct Scales {
    uint32_t a[IB], b[kJB];
  };
  // Place, in dwords, of dword d of this lane's row in block 0 of A's (B's) ring; a block of 32
  // rows is 256 dwords on.
  __device__ __forceinline__ int scale_place(int d, bool b) const {
    const int t = threadIdx.x, l = t & 63, w = t >> 6, r = l & 31;
    const int place = 2 * (r & ~7) + (r & 7) + 8 * (((d >> 2) ^ (r >> 3)) & 1);
    const int half = (d >> 3) & 1;
    return 4 * ((b ? half * 2 * Src::kTN + (w & 1) * 64 * JB : half * 2 * Src::kSRows + (w >> 1) * 64 * IB) + place) + (d & 3);
  }
  // Dwords of the ring for this lane's scales of step ks in N row blocks of A or of B, and, where
  // they are shifted together, the next ones.
  template <int N>
  struct Dwords {
    uint32_t w[N], w1[SHIFT ? N : 1];

    __device__ __forceinline__ void read(const Tile& t, int ks, bool b) {
      const uint32_t* ring = b ? g_sb : g_sa;
      const int d = 2 * ks + int((threadIdx.x & 63) >> 5);
      const int at = t.scale_place(d, b), at1 = t.scale_place(d + 1, b);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        w[i] = ring[at + 256 * i];
        if (SHIFT) w1[SHIFT ? i : 0] = ring[at1 + 256 * i];
      }
    }
    // The four bytes that start `low` bytes into the first dword, without those past the row.
    __device__ __forceinline__ void scales(uint32_t (&s)[N], uint32_t low, int ks, int nblk) const {
      const int have = nblk - 8 * ks - 4 * int((threadIdx.x & 63) >> 5);
      const uint32_t keep = have >= 4 ? ~0u : have <= 0 ? 0u : ~(~0u << (8 * have));
#pragma unroll
      for (int i = 0; i < N; ++i)
        s[i] = SHIFT ? __builtin_amdgcn_alignbyte(w1[SHIFT ? i : 0], w[i], low) & keep : w[i];
    }
  };

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
    i32x8_t a[IB], b[kJB];
  };

  // One slice's MFMAs on f, and between them: the fragments of slice RS (of the stage at rd)
  // read into fr, and the data loads D0 .. D0 + DN - 1 of step ks + 2 issued into stage `wr`.
  template <int SL, int RS, int D0, int DN>
  __device__ __forceinline__ void slice(const Src& src, const Frag& f, Frag& fr, const Scales& sc,
                                        uint32_t rd, int ks, uint32_t wr) {
    constexpr int kM = IB * kJB;  // MFMAs
    constexpr int kR = IB + kJB;  // fragment reads, after each of the first MFMAs
    constexpr int kPer = IB == 1 ? 2 : 1;
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int i = m / kJB, j = m % kJB;
      __builtin_amdgcn_sched_barrier(0);
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          f.b[j], f.a[i], acc[i][j], 4, A8 ? 0 : 4, SL, int(sc.b[j]), SL, int(sc.a[i]));
#pragma unroll
      for (int x = 0; x < kPer; ++x) read_one(fr, RS, m * kPer + x, rd);
      if (m == kM - 1) {
#pragma unroll
        for (int r = kM * kPer; r < kR; ++r) read_one(fr, RS, r, rd);
      }
#pragma unroll
      for (int q = 0; q < DN; ++q)
        if (q * kM / (DN > 0 ? DN : 1) == m) {
          const int d = D0 + q;
          src.issue(ks + 2, d < kQA ? d : d - kQA + 8, wr);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ void read_one(Frag& fr, int s, int r, uint32_t rd) const {
    if (r < IB) fr.a[r] = read_a(s, r, rd);
    else if (r < IB + kJB) fr.b[r - IB] = read_b(s, r - IB, rd);
  }

  // The K loop; src.begin() has been issued, and after it `stores` stores of the wave.
  __device__ __forceinline__ void run(const Src& opened, int stores) {
    const Src src = opened.uniform();
    init();
    wait_all_but(Src::kAhead + stores);  // step 0 and its scales
    wait_lds();  // the last tile's results read back
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // f[s]: the fragments of slice s.  Those of slices 0..2 are read one step ahead, those of
    // slice 3 under slice 0 of their own step: a stage is free from then on, and the loads of
    // two steps ahead have the rest of the step to be issued in.
    Frag f[4];
    Scales sc, sn;
    Dwords<IB> da;
    Dwords<kJB> db;
    da.read(*this, 0, false);
    db.read(*this, 0, true);
    da.scales(sc.a, src.sha, 0, src.nblk);
    db.scales(sc.b, src.shb, 0, src.nblk);
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int r = 0; r < IB + kJB; ++r) read_one(f[s], s, r, 0);
    const int steps = (src.nblk + 7) / 8;
    uint32_t cur = 0;  // stage of step ks
    constexpr int kD = kQA + Src::kQ;  // data loads a step
    constexpr int kD1 = kD / 2, kD2 = kD - kD1;
    for (int ks = 0; ks < steps; ++ks) {
      slice<0, 3, 0, 0>(src, f[0], f[3], sc, cur, ks, cur);
      // step ks + 1 has landed (mine by the wait, everyone's by the barrier), and every wave
      // has read the last of this step's stage and its scales
      if (ks == 0) wait_all_but(stores);
      else wait_vmcnt<0>();
      wait_lds();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const uint32_t nxt = cur ^ kStageB;
      // Scales of the four steps that follow the ring's, once their half is read by all (from step
      // ks = 4 q - 5 on for the q-th four; at step 0 it is the half that the last tile's results
      // went through), and there at step 4 q - 2, where a shifted read takes their first dword.
      // With 4-bit rows, whose steps are shorter, over three steps.
      const int ph = (ks + 1) & 3, quad = (ks + 1) / 4 + 1;
      if (ks == 0 || ph == 0) {
        src.issue_scales(quad, 0);
        src.issue_scales(quad, 1);
        if (A8) src.issue_scales(quad, 2);
        if (A8) src.issue_scales(quad, 3);
      }
      if (!A8 && ph == 1) src.issue_scales(quad, 2);
      if (!A8 && ph == 2) src.issue_scales(quad, 3);
      db.read(*this, ks + 1, true);
      slice<1, 0, 0, kD1>(src, f[1], f[0], sc, nxt, ks, cur);
      db.scales(sn.b, src.shb, ks + 1, src.nblk);
      da.read(*this, ks + 1, false);
      slice<2, 1, kD1, kD2>(src, f[2], f[1], sc, nxt, ks, cur);
      da.scales(sn.a, src.sha, ks + 1, src.nblk);
      slice<3, 2, 0, 0>(src, f[3], f[2], sc, nxt, ks, cur);
      sc = sn;
      cur = nxt;
    }
    // every load has landed and every wave has read its last fragments: the stages are free
    wait_loads_and_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  // Block (i, j): lane l holds row l % 32 of A and, of B's 32 rows, 8 q + 4 h + u (q, u =
  // 0..3): four consecutive columns of out each.  Stored as they are, an instruction would write
  // 16 or 32 bytes of 32 rows, and the results cost as much as if nothing ran beside them.  So 32
  // rows of 128 bytes at a time go through 4 KB a wave of the scale ring's second half, which
  // the next tile fills later, and leave as whole 128-byte lines, non-temporally (8 chunks of 16
  // bytes, chunk c of row r at c ^ (r & 7) ^ ((r >> 3) & 1)).  16,384 rows, N 7168, K 2048 in
  // MXFP4 on MI355X: 171 us with 32-byte stores, 167 with whole lines, 157 non-temporally.
  // The stores go through a buffer resource whose range drops what lies outside the expert's
  // rows and N, so that every wave makes the same number of them: kStores.
  template <bool OUT32>
  static constexpr int kStores = IB * kJB * (OUT32 ? 4 : 2);

  template <bool OUT32>
  __device__ __forceinline__ void store(const GroupedArgs& p, int64_t r0, int rows, int n0) const {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));  // the addresses below are not kept over the K loop
    const int l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = w >> 1, wn = w & 1, r = l & 31, h = l >> 5;
    constexpr int kSize = OUT32 ? 4 : 2;
    constexpr int kJ = OUT32 ? 1 : 2;  // column blocks that make 128 bytes
    const rsrc_t ro = row_rsrc(static_cast<uint8_t*>(p.out) + r0 * p.ld_out * kSize, kPastRange);
    const uint32_t area = (w & 2 ? lds_addr(g_sb) : lds_addr(g_sa)) + 8192 + uint32_t(w & 1) * 4096;
    const uint32_t wr = area + uint32_t(r) * 128;
    const int sw = (r & 7) ^ ((r >> 3) & 1);
    // read back: instruction x takes rows 8 x + l / 8, place l % 8
    const int rr = l >> 3, rsw = rr & 7;
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j0 = 0; j0 < kJB; j0 += kJ) {
#pragma unroll
        for (int j = j0; j < j0 + kJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& c = acc[i][j];
            if (OUT32)
              *reinterpret_cast<lds_wv4u*>(uintptr_t(wr + (((2 * q + h) ^ sw) * 16))) = __builtin_bit_cast(
                  v4u, f32x4_t{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]});
            else
              *reinterpret_cast<lds_wu64*>(uintptr_t(wr + (((4 * (j - j0) + q) ^ sw) * 16) + 8 * h)) =
                  uint64_t(pack_bf16x2(c[4 * q], c[4 * q + 1])) |
                  (uint64_t(pack_bf16x2(c[4 * q + 2], c[4 * q + 3])) << 32);
          }
        asm volatile("" ::: "memory");  // the wave's LDS operations run in order
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = (wm * IB + i) * 32 + 8 * x + rr;
          const int chunk = (l & 7) ^ rsw ^ (x & 1);
          const int col = n0 + wn * 32 * JB + 32 * j0 + chunk * (16 / kSize);
          const v4u v = *reinterpret_cast<lds_v4u*>(uintptr_t(area + uint32_t(8 * x + rr) * 128 + (l & 7) * 16));
          const bool in = row < rows && col < p.n;
          buf_st16<kCpolStream>(ro, in ? uint32_t(row) * uint32_t(p.ld_out) * kSize + col * kSize : kPastRange, v);
        }
        asm volatile("" ::: "memory");
      }
    asm volatile("" ::: "memory");
  }
};

}  // namespace mx4
}  // namespace mok
