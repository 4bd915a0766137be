// Tile of the grouped product of 16-bit rows: one workgroup of four waves computes up to 256 x 256
// results, each wave half of the rows by half of the columns, in 16 x 16 blocks of
// v_mfma_f32_16x16x32_{bf16,f16}.
//
// Either operand is one of two kinds: a row of it contiguous along the axis that is summed over
// (kAlong: a, and b forward), or contiguous across it (kAcross: b for the rows' gradient, both for
// the weights').  A step sums over 64 elements: up to 32 KB of each operand, moved by direct-to-LDS
// loads through a ring of two stages.
//
// Fragments of 16 x 16 x 32: lane l holds row l % 16 of its operand, elements 8 (l / 16) .. +8 of
// the slice's 32.
//   kAlong: LDS rows of 128 bytes, 8 chunks of 16 bytes, chunk c of row r at place c ^ (r & 7).  A
//     read of 16 rows at 4 chunks each takes the LDS 4.1 clocks so, 8.0 with another term
//     (r >> 3) & 1 in the place (which suits reads of 32 rows at 2 chunks), 16 as the rows come.
//   kAcross: LDS rows of one summed element, 16 columns (32 bytes) a block; the fragment comes
//     from two transposing reads (ds_read_b64_tr_b16: lane i of 16 receives element i % 4 of the
//     8 bytes that lanes i / 4, 4 + i / 4, 8 + i / 4 and 12 + i / 4 address), summed elements
//     8 g .. +4 and 8 g + 4 .. +4 for lane group g.  A pass reads a block of eight elements, 0..3
//     and 8..11 for one; they lie in eight places of the 256 bytes that cover the banks: within a
//     load (two rows of 512 bytes, or four of 256) block c of its row x lies at c ^ x, and the loads
//     lie further apart than their 1 KB.  So a lane needs two (or four) read addresses for all
//     blocks, the rest being the reads' own offset.
//
// An operand across the sum may be held in 8 bits (kHeld): e4m3 codes and a scale for 32 columns of an
// element.  Its codes come through registers, a step ahead of their conversion (a scaled
// instruction for two codes) into the same LDS layout, which falls between the MFMAs of the step
// before their own.
//
// Rows past an operand's last are read as its last one and never stored (kAlong); chunks and
// columns past the end, and summed elements past the last, as zeros (an out-of-range offset reads
// no memory).
//
// Why this tile: of 256 x 256, a step of 64 reads 64 KB for 8.4 M operations, 2048 clocks of the matrix
// cores: 32 of the 59 bytes a clock that a CU gets from its L2 when it does nothing else.  Four waves
// of 128 x 128 leave each SIMD one wave, whose sums fill the 256 accumulation registers and whose
// fragments of two slices fit beside its loads' offsets; half the tile has the same latency a step and
// half the work.  Bound by the matrix cores and the clock that the card's power allows under them.
// MI355X, bf16, 8 experts of 2048 rows, in loops one after another on one card, us (and a library product
// of the same kind, of one expert with all the rows, into bf16):
//   N 4096, K 7168  forward 691 (613 to 629)  rows' gradient 718 (728 to 731)  weights' gradient 798 (986)
//   N 7168, K 2048  forward 375 (333)         rows' gradient 365 (363 to 365)  weights' gradient 419 (547)
// (the weights' into fp32; into bf16 752 to 759 and 392).  691 is 1393 TFLOP/s.  Counters with uneven experts:
// matrix cores busy 66% of the time forward, 63% rows' gradient, 58% weights' gradient, at 2.0 GHz of 2.4;
// waits for loads and barriers 12 to 13%, LDS bank conflicts below 1%.
//
// Known to be slow: results added to what is there (store() with ADD).  Every 16 bytes are a load, a wait for
// it and a store, 64 times a whole tile: the weights' gradients above take 1210 and 619 so, and 1000 rows of
// 8 experts, N 4096, K 7168 505 where 180 do without.
#pragma once
#include "ops_launch.h"
#include "gemm_mx4.h"

namespace mok {
namespace g16 {

constexpr int kThr = 256;
constexpr uint32_t kPast = 0x80000000u;      // added to an offset: out of every resource's range

enum Kind { kAlong = 0, kAcross = 1, kHeld = 2 };

// Bytes of one operand's stage, NB blocks of 16 rows a wave.
template <int KIND, int NB>
constexpr uint32_t stage_bytes() { return KIND == kAlong ? 4096 * NB : NB == 8 ? 35840 : 17408; }

// The LDS of a kernel: two stages of each operand, then the results on their way out, 512 JB bytes a
// wave.
template <uint32_t STAGE_A, uint32_t STAGE_B, int JB>
struct Lds {
  static constexpr uint32_t kA = STAGE_A, kB = STAGE_B;
  static constexpr uint32_t kBytes = 2 * STAGE_A + 2 * STAGE_B + 4 * 512 * JB;
  static __device__ __forceinline__ v4u* mem() {
    static __shared__ __align__(1024) v4u s_mem[kBytes / 16];
    return s_mem;
  }
  static __device__ __forceinline__ uint32_t a() { return lds_addr(mem()); }
  static __device__ __forceinline__ uint32_t b() { return a() + 2 * STAGE_A; }
  static __device__ __forceinline__ uint32_t out() { return a() + 2 * STAGE_A + 2 * STAGE_B; }
};

typedef uint32_t v2u_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v4u lds_w16;
typedef __attribute__((address_space(3))) v2u_t lds_w8;

// c += a * b.  All MFMAs of a tile are inline asm with their sums in accumulation registers: 64 blocks
// take all 256 of those, and with the builtin the compiler moved blocks between the register files
// inside the loop as soon as some of them were named by asm (lds_load16_mfma4).  What the compiler
// then does not see to: before the first MFMA come waits and reads (the sums' zeros are long
// written), a block is used again only after all others, and run() ends with wait states before the
// sums are read otherwise.
template <int TYPE>
__device__ __forceinline__ void mfma(v4u a, v4u b, f32x4_t& c) {
  if (TYPE == MOK_TYPE_BF16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// (Two bf16 conversions, not one of a pair: that instruction makes the compiler move accumulators
// between its register files inside the loop that sums them.)
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  if (TYPE == MOK_TYPE_BF16) return uint32_t(f32_to_bf16(a)) | (uint32_t(f32_to_bf16(b)) << 16);
  return __builtin_bit_cast(uint32_t, f16x2_t{_Float16(a), _Float16(b)});
}

// A wave-uniform value into a scalar register, whatever the compiler holds it in: the loads are
// inline asm, which cannot take a resource from vector registers (the wait states are the
// caller's too: one between a vector write and the lane read of its result, five between a scalar
// result of a vector instruction and a vector memory operation that reads it).
__device__ __forceinline__ int scalar(int v) {
  int s;
  asm volatile("s_nop 0\n\tv_readfirstlane_b32 %0, %1\n\ts_nop 4" : "=s"(s) : "v"(v));
  return s;
}

// One operand of a tile.  NB: blocks of 16 rows a wave (8 or 4, along also 2); the tile has 32 NB
// rows, and a wave NB loads a step.
template <int KIND, int NB>
struct Operand {
  static constexpr int kLanes = KIND == kAlong ? 8 : 4 * NB;  // lanes of a load that one LDS row takes
  static constexpr int kRows = 64 / kLanes;                   // LDS rows a load
  static_assert(KIND == kAlong || NB >= 4);
  i32x4_t r;
  uint32_t off[NB];
  int left;       // what is left of the summed axis at the next step to be loaded: chunks of 8
                  // elements (kAlong), elements (kAcross)
  uint32_t step;  // bytes from step to step

  // This lane's chunk, or its element of load q, of a step.
  static __device__ __forceinline__ int at(int q) {
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return KIND == kAlong ? (l & 7) ^ (l >> 3) : (q * 4 + w) * kRows + l / kLanes;
  }
  // base: element 0 of the operand's first row (kAlong) or of its first summed element (kAcross);
  // rows: rows, or columns, that there are; ld: elements from line to line.
  __device__ __forceinline__ void init(const void* base, int64_t ld, int rows, int summed) {
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t x = reinterpret_cast<uint64_t>(base);
    r = i32x4_t{scalar(int(uint32_t(x))), scalar(int(uint32_t(x >> 32) & 0xFFFFu)), int(kPast), 0x00020000};
    left = KIND == kAlong ? summed / 8 : summed;
    step = KIND == kAlong ? kDeep * 2 : uint32_t(kDeep * ld * 2);
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      if (KIND == kAlong) {
        off[q] = uint32_t(min((q * 4 + w) * 8 + (l >> 3), rows - 1)) * uint32_t(ld * 2) + at(q) * 16;
      } else {
        const int p = l % kLanes, chunk = 2 * ((p >> 1) ^ (l / kLanes)) + (p & 1);
        off[q] = (uint32_t(at(q)) * uint32_t(ld * 2) + chunk * 16) | (8 * chunk < rows ? 0u : kPast);
      }
    }
    cut();
  }
  // Chunks or elements that the next step no longer has: out of range from here on.
  __device__ __forceinline__ void cut() {
#pragma unroll
    for (int q = 0; q < NB; ++q) off[q] |= at(q) < left ? 0u : kPast;
  }
  __device__ __forceinline__ void next() {
    left -= KIND == kAlong ? kDeep / 8 : kDeep;
    const uint64_t base = (uint64_t(uint32_t(r.y)) << 32 | uint32_t(r.x)) + step;
    r.x = scalar(int(uint32_t(base)));
    r.y = scalar(int(uint32_t(base >> 32)));
  }
  __device__ __forceinline__ bool whole() const { return left >= (KIND == kAlong ? kDeep / 8 : kDeep); }
  // LDS byte of load j = 4 q + w in its stage.
  static constexpr uint32_t place_of(int j) {
    return KIND == kAlong ? j * 1024 : NB == 8 ? j * 1088 + (j >> 2) * 128 : j * 1024 + (j >> 1) * 128;
  }
  static __device__ __forceinline__ uint32_t place(int q, uint32_t to) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return to + place_of(4 * q) + place_of(w);
  }
  __device__ __forceinline__ void load(int q, uint32_t to) const { dma16_at<false>(r, off[q], 0u, place(q, to)); }
  __device__ __forceinline__ void uniform() {
    r.x = scalar(r.x);
    r.y = scalar(r.y);
    r.z = int(kPast);
    r.w = 0x00020000;
    left = scalar(left);
    step = uint32_t(scalar(int(step)));
  }
};

// Finite fp16 rows are held as up to 65,536 (63,488 and more: code 256 at scale byte 135), which fp16 does
// not have: it becomes 65,504, off by half a step.  So from that scale byte on (with END; without, it
// becomes infinite) half the value is converted, y, which is exact where the whole is finite, and y and
// the nearest to it of +-32,736 are added: twice y up to 61,440, 65,504 for y = 32,768, infinite above,
// where y is at least 36,864.  At smaller scale bytes the whole is converted and 0 added.  (The bounds as
// integers, whose order is that of the magnitudes of either sign: as floats an instruction more
// quiets NaNs, which y keeps.)
constexpr uint32_t kEndOfFp16 = 135;
// What a unit's conversion takes of its scale byte: a float of which the instructions read the exponent
// alone (0 stands for 2^-127, 255 for NaN), and with END below it the bits of 32,736 in fp16, or 0.
template <bool END>
__device__ __forceinline__ uint32_t held_scale(uint32_t scale) {
  const bool half = END && scale >= kEndOfFp16 && scale != 255;
  return ((scale - half) << 23) | (half ? 0x77FEu : 0u);
}
// Two e4m3 codes (the low or the high half of c) times 2^(scale byte - 127) in the product's type.
template <int TYPE, bool HIGH, bool END>
__device__ __forceinline__ uint32_t held2(uint32_t c, uint32_t scale) {
  const float f = __uint_as_float(scale);
  if (TYPE == MOK_TYPE_BF16)
    return __builtin_bit_cast(uint32_t, bf16x2_t(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, f, HIGH)));
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  typedef int16_t i16x2_t __attribute__((ext_vector_type(2)));
  typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
  const f16x2_t y = f16x2_t(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, f, HIGH));
  if (!END) return __builtin_bit_cast(uint32_t, y);
  const uint16_t top = uint16_t(scale), bottom = uint16_t(scale | 0x8000u);
  const i16x2_t at_most = __builtin_elementwise_min(__builtin_bit_cast(i16x2_t, y), i16x2_t{int16_t(top), int16_t(top)});
  const u16x2_t near = __builtin_elementwise_min(__builtin_bit_cast(u16x2_t, at_most), u16x2_t{bottom, bottom});
  return __builtin_bit_cast(uint32_t, f16x2_t(y + __builtin_bit_cast(f16x2_t, near)));
}

// An operand across the sum held in 8 bits, of 32 NB columns.  A lane takes 16 codes at a time, a
// block of 16 columns of one element.
template <int TYPE, int NB>
struct Held {
  typedef Operand<kAcross, NB> Op;
  static constexpr int kUnits = NB / 2;                // of 16 codes a lane and step
  static constexpr int kLanes = 2 * NB;                // lanes that one element takes
  static constexpr int kOps = 6 * kUnits;              // pieces that a step's conversion is cut into
  rsrc_t rc, rs;
  uint64_t codes, scales;  // of the step to be loaded
  int64_t ld, lds;
  uint32_t off[kUnits], offs[kUnits];
  int left;
  v4u q[kUnits];
  uint32_t s[kUnits];
  v4u half;  // eight converted elements

  static __device__ __forceinline__ int at(int u) {
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return (u * 4 + w) * (64 / kLanes) + l / kLanes;
  }
  // c, sc: code and scales' first byte of the operand's first element; col: its first column.
  __device__ __forceinline__ void init(const uint8_t* c, int64_t ld_, const uint8_t* sc, int64_t lds_, int col,
                                       int cols, int summed) {
    codes = reinterpret_cast<uint64_t>(c) + uint32_t(col);
    scales = reinterpret_cast<uint64_t>(sc) + uint32_t(col / 32);
    ld = ld_;
    lds = lds_;
    left = summed;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int b = int(threadIdx.x & 63) % kLanes;
      const uint32_t past = 16 * b < cols ? 0u : kPast;
      off[u] = (uint32_t(at(u)) * uint32_t(ld) + b * 16) | past;
      offs[u] = (uint32_t(at(u)) * uint32_t(lds) + b / 2) | past;
    }
  }
  __device__ __forceinline__ void next() {
    left -= kDeep;
    codes += uint64_t(kDeep * ld);
    scales += uint64_t(kDeep * lds);
  }
  // Load 0 .. 2 kUnits - 1 of a step: a unit's codes, its scale.
  __device__ __forceinline__ void load(int x) {
    const int u = x >> 1;
    const uint32_t past = at(u) < left ? 0u : kPast;
    if (x == 0) {
      rc = row_rsrc(reinterpret_cast<const void*>(codes), kPast);
      rs = row_rsrc(reinterpret_cast<const void*>(scales), kPast);
    }
    if (x & 1) s[u] = uint32_t(uint8_t(__builtin_amdgcn_raw_buffer_load_b8(rs, offs[u] | past, 0, 0)));
    else q[u] = buf_ld16<kCpolPlain>(rc, off[u] | past);
  }
  // Whether a lane of the wave holds scales at the end of fp16's range.
  __device__ __forceinline__ bool at_the_end() const {
    uint32_t m = s[0];
#pragma unroll
    for (int v = 1; v < kUnits; ++v) m = max(m, s[v]);
    return __builtin_amdgcn_ballot_w64(m >= kEndOfFp16) != 0;
  }
  // Piece o of the conversion into the stage at LDS address `to`.
  template <int O, bool END>
  __device__ __forceinline__ void convert(uint32_t to) {
    constexpr int u = O / 6, x = O % 6, w = x < 3 ? x : x - 1;
    if constexpr (O == 0) {
      // All of them are waited for here: a later wait would be for the loads to LDS too, which the
      // compiler does not count and which have been issued since.
#pragma unroll
      for (int v = 0; v < kUnits; ++v) asm volatile("" : "+v"(q[v]), "+v"(s[v]));
    }
    if constexpr (x == 2 || x == 5) {
      const int l = threadIdx.x & 63, k = at(u), b = l % kLanes, y = k % Op::kRows;
      // (element k's place: units and waves are whole loads of the 16-bit operand apart)
      const uint32_t place = to + Op::place_of(4 * (64 / kLanes) / Op::kRows) * u + lane_place() + uint32_t(b ^ y) * 32;
      *reinterpret_cast<lds_w16*>(uintptr_t(place + (x == 5 ? 16 : 0))) = half;
    } else {
      const uint32_t scale = held_scale<END>(s[u]);
      const uint32_t c = w == 0 ? q[u].x : w == 1 ? q[u].y : w == 2 ? q[u].z : q[u].w;
      half[2 * (w & 1)] = held2<TYPE, false, END>(c, scale);
      half[2 * (w & 1) + 1] = held2<TYPE, true, END>(c, scale);
    }
  }
  // LDS byte, in its stage, of the element that this lane has of unit 0.
  static __device__ __forceinline__ uint32_t lane_place() {
    const int k = at(0), j = k / Op::kRows;
    return (NB == 8 ? j * 1088 + (j >> 2) * 128 : j * 1024 + (j >> 1) * 128) + (k % Op::kRows) * (64 * NB);
  }
};

// LDS byte addresses of this lane's fragment reads.
template <int KIND, int NB>
struct FragAt {
  typedef Operand<KIND == kHeld ? kAcross : KIND, NB> Op;
  static constexpr int kAddr = KIND == kAlong ? 2 : Op::kRows;
  static_assert(Op::place_of(4 * NB - 1) + 1024 <= stage_bytes<KIND, NB>());
  uint32_t p[kAddr];

  // half: which half of the tile's rows the wave has
  __device__ __forceinline__ void init(uint32_t base, int half) {
    const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
#pragma unroll
    for (int x = 0; x < kAddr; ++x) {
      if (KIND == kAlong) {
        p[x] = base + uint32_t(half * 16 * NB + r) * 128 + (((4 * x + g) ^ (r & 7)) * 16);
      } else {
        const int k = 8 * g + (r >> 2), y = k % Op::kRows;
        p[x] = base + Op::place_of(k / Op::kRows) + y * (64 * NB) + half * (32 * NB) + (x ^ y) * 32 + (r & 3) * 8;
      }
    }
  }
  // The same in the stage at byte `stage`, opaque, so that what differs by block and slice becomes
  // the reads' own offset and no address is computed between the MFMAs.
  __device__ __forceinline__ FragAt in(uint32_t stage) const {
    FragAt f;
#pragma unroll
    for (int x = 0; x < kAddr; ++x) {
      f.p[x] = p[x] + stage;
      asm volatile("" : "+v"(f.p[x]));
    }
    return f;
  }
  // Fragment i of slice s; part: 0 or 1 of kAcross' two reads.
  __device__ __forceinline__ v4u along(int s, int i) const {
    return *reinterpret_cast<lds_cv4u*>(uintptr_t(p[KIND == kAlong ? s : 0] + uint32_t(i) * 2048));
  }
  __device__ __forceinline__ v2u_t across(int s, int i, int part) const {
    // (32 elements on, and 4 on, the places of the loads are the same distance apart for every lane)
    const uint32_t o = Op::place_of(32 / Op::kRows) * s + Op::place_of(4 / Op::kRows) * part;
    const v4s_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        reinterpret_cast<lds_v4s*>(uintptr_t(p[i % kAddr] + o + i / kAddr * (32 * kAddr))));
    return __builtin_bit_cast(v2u_t, v);
  }
};

// At most n (wave-uniform) of the wave's memory operations still in flight; n is rounded down to a
// count that the instruction can name.
__device__ __forceinline__ void wait_all_but(int n) {
  if (n >= 63) wait_vmcnt<63>();
  else if (n >= 48) wait_vmcnt<48>();
  else if (n >= 40) wait_vmcnt<40>();
  else if (n >= 32) wait_vmcnt<32>();
  else if (n >= 24) wait_vmcnt<24>();
  else if (n >= 16) wait_vmcnt<16>();
  else if (n >= 8) wait_vmcnt<8>();
  else wait_vmcnt<0>();
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14)); }

// IB, JB: blocks of 16 rows of A and of B a wave.  A may be opened for a taller tile (AB blocks), of
// which this one's rows are the first.
template <int TYPE, int AK, int BK, int IB, int JB, typename LDS, int AB = IB>
struct Tile {
  typedef Operand<AK, AB> A;
  static constexpr bool kHolds = BK == kHeld;
  typedef std::conditional_t<kHolds, Held<TYPE, JB>, Operand<kHolds ? kAcross : BK, JB>> B;
  static_assert(AB == IB || AK == kAlong);
  static constexpr int kLoads = kHolds ? IB : IB + JB;  // direct to LDS, a wave and step
  static constexpr int kReads = (AK == kAlong ? IB : 2 * IB) + (BK == kAlong ? JB : 2 * JB);

  FragAt<AK, IB> fa;
  FragAt<BK, JB> fb;
  f32x4_t acc[IB][JB];

  struct Frag {
    v4u a[IB], b[JB];
  };

  // Read r of a slice's kReads.
  static __device__ __forceinline__ void read(Frag& f, const FragAt<AK, IB>& fa, const FragAt<BK, JB>& fb, int s, int r) {
    constexpr int kB = BK == kAlong ? JB : 2 * JB;
    if (r < kB) {
      if (BK == kAlong) {
        f.b[r % JB] = fb.along(s, r);
      } else {
        const v2u_t v = fb.across(s, r >> 1, r & 1);
        f.b[(r >> 1) % JB][2 * (r & 1)] = v.x;
        f.b[(r >> 1) % JB][2 * (r & 1) + 1] = v.y;
      }
    } else {
      const int x = r - kB;
      if (AK == kAlong) {
        f.a[x % IB] = fa.along(s, x);
      } else {
        const v2u_t v = fa.across(s, x >> 1, x & 1);
        f.a[(x >> 1) % IB][2 * (x & 1)] = v.x;
        f.a[(x >> 1) % IB][2 * (x & 1) + 1] = v.y;
      }
    }
  }

  // A step's MFMAs, 2 kM of them, slice 0's on f0 and then slice 1's on f1, and what happens
  // between them, by the MFMA it follows:
  //   0 .. kRead0        slice 1's fragments are read into f1;
  //   kFree              every wave has read the last of this step's stage;
  //   from kFree on      the loads of the step after the next into it, spread over the rest of the
  //                      step: in a burst they hold up the MFMAs behind them;
  //   kM + kLanded       the next step has landed (mine by the wait, everyone's by the barrier);
  //   from there on      its slice 0 is read into f0.
  // One wave a SIMD issues everything, an MFMA every 16 clocks and three other instructions beside
  // it, so nothing stands between MFMAs that waits for the instruction before it: read addresses are
  // ready before the step (FragAt::in; computed at each read they cost 7% of the product), and the
  // loads' wait states are MFMAs (11%).
  static constexpr int kM = IB * JB;
  static constexpr int kRead0 = kM * 5 / 16, kFree = kM / 2 - 1, kLanded = kM / 4 - 1, kRead1 = kM / 2;
  // Whole tiles take a load with four MFMAs (lds_load16_mfma4), never the step's last eight.
  static constexpr bool kWith4 = kM == 64;
  // (with B in 8 bits, before its own loads, which come first in slice 1: those are waited for first)
  static constexpr int load_slot(int q) {
    return kHolds ? kFree + 1 + q * (kM - kFree - 1) / kLoads
           : kWith4 ? kFree + 1 + q * 22 / 16 * 4 : kFree + 1 + q * (2 * kM - kFree - 2) / kLoads;
  }
  static constexpr int kHeldLoads = kHolds ? JB : 0;
  static constexpr int held_before(int slot) { return slot <= kM ? 0 : 2 * (slot - kM) < kHeldLoads ? 2 * (slot - kM) : kHeldLoads; }
  // (its conversion, from a quarter of slice 0 to the end)
  static constexpr int convert_before(int m) {
    return !kHolds || m <= kM / 4 ? 0 : (m - kM / 4) * (3 * JB) / (kM - kM / 4);
  }
  static constexpr int loads_before(int slot) {
    int n = 0;
    while (n < kLoads && load_slot(n) < slot) ++n;
    return n;
  }
  static constexpr int reads_before(int x, int span) {
    return x <= 0 ? 0 : x >= span ? kReads : (x * kReads + span - 1) / span;
  }
  template <int H, int M>
  __device__ __forceinline__ void slot(const A& a, B& b, const Frag& f, Frag& fr, const FragAt<AK, IB>& ra,
                                       const FragAt<BK, JB>& rb, uint32_t wa, uint32_t wb) {
    constexpr int i = M / JB, j = M % JB;
    constexpr int q0 = loads_before(H * kM + M), q1 = loads_before(H * kM + M + 1);
    static_assert(!kWith4 || load_slot(kLoads - 1) < 2 * kM - 8);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kWith4 && q1 > q0) {
      i32x4_t r = a.r;
      uint32_t off = a.off[q0 % IB], to = A::place(q0, LDS::a() + wa);
      if constexpr (q0 >= IB) {
        r = b.r;
        off = b.off[q0 - IB];
        to = B::place(q0 - IB, LDS::b() + wb);
      }
      mx4::lds_load16_mfma4<TYPE == MOK_TYPE_FP16>(r, off, to, f.a[i], f.b[j], f.b[j + 1], f.b[j + 2], f.b[j + 3],
                                                   acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
    } else if constexpr (!kWith4 || loads_before(H * kM + M + 1) == loads_before((H * kM + M) / 4 * 4)) {
      mfma<TYPE>(f.b[j], f.a[i], acc[i][j]);
    }  // (else it was one of the four of a load)
    if constexpr (H == 0 && M == kFree) {
      wait_lds();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    if constexpr (H == 1 && M == kLanded) {
      wait_vmcnt<loads_before(kM + kLanded) + held_before(kM + kLanded)>();
      if (kHolds) wait_lds();  // what was converted is written
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }
    constexpr int kFirst = H == 0 ? 0 : kLanded + 1, kSpan = H == 0 ? kRead0 : kRead1;
    constexpr int r0 = reads_before(M - kFirst, kSpan), r1 = reads_before(M - kFirst + 1, kSpan);
#pragma unroll
    for (int r = r0; r < r1; ++r) read(fr, ra, rb, H == 0 ? 1 : 0, r);
    if constexpr (!kWith4) {
#pragma unroll
      for (int q = q0; q < q1; ++q) load(a, b, q, wa, wb);
    }
    if constexpr (kHolds) {
      if constexpr (H == 0) {  // the next step's elements, into its stage
        convert<convert_before(M), false>(b, LDS::b() + (LDS::kB - wb),
                                          std::make_integer_sequence<int, convert_before(M + 1) - convert_before(M)>());
      } else {  // the codes of the step after
#pragma unroll
        for (int x = held_before(kM + M); x < held_before(kM + M + 1); ++x) b.load(x);
      }
    }
  }
  static __device__ __forceinline__ void load(const A& a, const B& b, int q, uint32_t wa, uint32_t wb) {
    if constexpr (kHolds) {
      a.load(q, LDS::a() + wa);
    } else {
      if (q < IB) a.load(q, LDS::a() + wa);
      else b.load(q - IB, LDS::b() + wb);
    }
  }
  template <int O, bool END, int... X>
  static __device__ __forceinline__ void convert(B& b, uint32_t to, std::integer_sequence<int, X...>) {
    (b.template convert<O + X, END>(to), ...);
  }
  // The conversion of a step again, where a lane has values at the end of fp16's range.  MI355X, 16,384 rows
  // of 8 experts, N 4096, K 7168, us: 769 where no lane has them (760 without the question), 906 where
  // all have; with END in the conversion between the MFMAs 836 for every step.  (A branch that holds
  // MFMAs makes the compiler move the sums; this one leaves them where they are.)
  static __device__ __forceinline__ void convert_end(B& b, uint32_t to) {
    if constexpr (kHolds && TYPE == MOK_TYPE_FP16) {
      if (b.at_the_end()) convert<0, true>(b, to, std::make_integer_sequence<int, 3 * JB>());
    }
  }
  template <int H, int... M>
  __device__ __forceinline__ void half(const A& a, B& b, const Frag& f, Frag& fr, const FragAt<AK, IB>& ra,
                                       const FragAt<BK, JB>& rb, uint32_t wa, uint32_t wb, std::integer_sequence<int, M...>) {
    (slot<H, M>(a, b, f, fr, ra, rb, wa, wb), ...);
    __builtin_amdgcn_sched_barrier(0);
  }

  // The loads of two steps (of one, of what is held in 8 bits).
  static __device__ __forceinline__ void begin(A& a, B& b) {
    asm volatile("" ::: "memory");
    if constexpr (kHolds) {
#pragma unroll
      for (int x = 0; x < kHeldLoads; ++x) b.load(x);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int q = 0; q < IB; ++q) a.load(q, LDS::a() + ks * LDS::kA);
      a.next();
      a.cut();
      if constexpr (!kHolds) {
#pragma unroll
        for (int q = 0; q < JB; ++q) b.load(q, LDS::b() + ks * LDS::kB);
        b.next();
        b.cut();
      }
    }
    if constexpr (kHolds) b.next();
    asm volatile("" ::: "memory");
  }

  // The sum over `steps` steps; begin() has been called, and after it the wave has issued `stores`
  // memory operations.
  __device__ __forceinline__ void run(A a, B b, int steps, int stores) {
    a.uniform();
    if constexpr (!kHolds) b.uniform();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    fa.init(LDS::a(), w >> 1);
    fb.init(LDS::b(), w & 1);
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j = 0; j < JB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // (written here, well before the first MFMA, and not made again next to one)
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j = 0; j < JB; ++j) asm volatile("" : "+a"(acc[i][j]));
    wait_all_but(stores);  // steps 0 and 1
    if constexpr (kHolds) {
      convert<0, false>(b, LDS::b(), std::make_integer_sequence<int, 3 * JB>());
      convert_end(b, LDS::b());
#pragma unroll
      for (int x = 0; x < kHeldLoads; ++x) b.load(x);
      b.next();
      wait_lds();
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Frag f0, f1;
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(f0, fa, fb, 0, r);
    uint32_t ca = 0, cb = 0;  // this step's stages
    FragAt<AK, IB> na = fa.in(0);
    FragAt<BK, JB> nb = fb.in(0);
    for (int ks = 0; ks < steps; ++ks) {
      half<0>(a, b, f0, f1, na, nb, ca, cb, std::make_integer_sequence<int, kM>());
      convert_end(b, LDS::b() + (LDS::kB - cb));
      na = fa.in(LDS::kA - ca);
      nb = fb.in(LDS::kB - cb);
      half<1>(a, b, f1, f0, na, nb, ca, cb, std::make_integer_sequence<int, kM>());
      a.next();
      b.next();
      if (!a.whole()) {
        asm volatile("");  // a branch: as selects the cut would stand in every step
        a.cut();
      }
      if constexpr (!kHolds) {
        if (!b.whole()) {
          asm volatile("");
          b.cut();
        }
      }
      ca = LDS::kA - ca;
      cb = LDS::kB - cb;
    }
    // every load has landed and every wave has read its last fragments: the stages are free; and the
    // last sums are there (seven wait states after an MFMA of four passes)
    wait_loads_and_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("s_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // Memory operations that store() issues for results in 16 and in 32 bits.
  static constexpr int kStores16 = IB * JB / 2, kStores32 = IB * JB;

  // Block (i, j): lane l holds, of row l % 16, the columns 4 (l / 16) .. +4.  16 rows of 256 bytes
  // (JB = 4: 128) at a time go through the wave's own LDS and leave as whole 128-byte lines (16 or 8
  // chunks of 16 bytes a row, chunk c of row r at c ^ r).
  // The resource's range drops what lies outside `rows` and `cols`, so that every wave makes the
  // same number of stores.
  template <bool OUT32, bool ADD>
  __device__ __forceinline__ void store(void* out, int64_t ld, int rows, int cols) const {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));  // the addresses below are not kept over the sum's loop
    const int l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = w >> 1, wn = w & 1, r = l & 15, g = l >> 4;
    constexpr int kSize = OUT32 ? 4 : 2;
    constexpr int kChunks = JB == 8 ? 16 : 8;  // 16-byte chunks a row that go out together
    constexpr int kJ = kChunks / kSize;                 // column blocks that make them
    constexpr int kRows = 64 / kChunks;                 // rows that an instruction stores
    const rsrc_t ro = row_rsrc(out, kPast);
    const uint32_t area = LDS::out() + uint32_t(w) * (512 * JB);
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j0 = 0; j0 < JB; j0 += kJ) {
#pragma unroll
        for (int j = j0; j < j0 + kJ; ++j) {
          f32x4_t c = acc[i][j];
          asm volatile("" : "+a"(c));  // read out here, not for all blocks before the kinds of store part
          if (OUT32)
            *reinterpret_cast<lds_w16*>(uintptr_t(area + r * (16 * kChunks) + (((4 * (j - j0) + g) ^ (r & (kChunks - 1))) * 16))) =
                __builtin_bit_cast(v4u, c);
          else
            *reinterpret_cast<lds_w8*>(uintptr_t(area + r * (16 * kChunks) +
                                                 (((2 * (j - j0) + (g >> 1)) ^ (r & (kChunks - 1))) * 16) + 8 * (g & 1))) =
                v2u_t{pack2<TYPE>(c.x, c.y), pack2<TYPE>(c.z, c.w)};
        }
        asm volatile("" ::: "memory");  // the wave's LDS operations run in order
#pragma unroll
        for (int x = 0; x < 16 / kRows; ++x) {
          const int rr = x * kRows + l / kChunks, c = (l & (kChunks - 1)) ^ (rr & (kChunks - 1));
          const int row = (wm * IB + i) * 16 + rr;
          const int col = (wn * JB + j0) * 16 + c * (16 / kSize);
          v4u v = *reinterpret_cast<lds_cv4u*>(uintptr_t(area + rr * (16 * kChunks) + (l & (kChunks - 1)) * 16));
          const bool in = row < rows && col < cols;
          const uint32_t at = in ? uint32_t(row) * uint32_t(ld * kSize) + uint32_t(col) * kSize : kPast;
          if (ADD) {
            const f32x4_t old = __builtin_bit_cast(f32x4_t, buf_ld16<kCpolPlain>(ro, at));
            v = __builtin_bit_cast(v4u, __builtin_bit_cast(f32x4_t, v) + old);
          }
          buf_st16<kCpolStream>(ro, at, v);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);  // (else the compiler holds so many at once that it spills)
      }
  }
};

}  // namespace g16
}  // namespace mok
