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
//   kAlong: LDS rows of 128 bytes, 8 chunks of 16 bytes, chunk c of row r at place
//     c ^ (r & 7) ^ ((r >> 3) & 1): the 16 rows that one pass of a 16-byte read takes at one chunk
//     then cover all 64 banks.
//   kAcross: LDS rows of one summed element, 16 columns (32 bytes) a block; the fragment comes
//     from two transposing reads (ds_read_b64_tr_b16: lane i of 16 receives element i % 4 of the
//     8 bytes that lanes i / 4, 4 + i / 4, 8 + i / 4 and 12 + i / 4 address), summed elements
//     8 g .. +4 and 8 g + 4 .. +4 for lane group g.  Block c of element k lies at place
//     c ^ (k & 3) ^ 4 ((k >> 3) & 1): the eight elements of a pass lie in eight places of the 256
//     bytes that cover the banks.
//
// Rows past an operand's last are read as its last one and never stored (kAlong); chunks and
// columns past the end, and summed elements past the last, as zeros (an out-of-range offset reads
// no memory).
#pragma once
#include "gemm_bf16.h"
#include "ops_launch.h"

namespace mok {
namespace g16 {

constexpr int kThr = 256;
constexpr int kDeep = 64;                    // summed elements a step
constexpr uint32_t kStage = 32768;           // bytes of one operand's stage
constexpr uint32_t kPast = 0x80000000u;      // added to an offset: out of every resource's range
constexpr int64_t kFar = int64_t(kPast);

static __shared__ __align__(1024) v4u s_a[2 * kStage / 16];
static __shared__ __align__(1024) v4u s_b[2 * kStage / 16];
static __shared__ __align__(1024) v4u s_out[4 * 4096 / 16];  // results on their way out, 4 KB a wave

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t v2u_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v4u lds_w16;
typedef __attribute__((address_space(3))) v2u_t lds_w8;

template <int TYPE>
__device__ __forceinline__ f32x4_t mfma(v4u a, v4u b, f32x4_t c) {
  if (TYPE == MOK_TYPE_BF16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                0, 0, 0);
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

enum Kind { kAlong = 0, kAcross = 1 };

// One operand of a tile.  NB: blocks of 16 rows a wave; the tile has 32 NB rows, and NB loads a
// wave and step.
template <int KIND, int NB>
struct Operand {
  static constexpr int kLanes = KIND == kAlong ? 8 : 4 * NB;  // lanes of a load that one LDS row takes
  i32x4_t r;
  uint32_t off[NB];
  int left;       // what is left of the summed axis at the next step to be loaded: chunks of 8
                  // elements (kAlong), elements (kAcross)
  int at;         // this lane's chunk, or its element within load 0, of a step
  uint32_t step;  // bytes from step to step

  // base: element 0 of the operand's first row (kAlong) or of its first summed element (kAcross);
  // rows: rows, or columns, that there are; ld: elements from line to line.
  __device__ __forceinline__ void init(const void* base, int64_t ld, int rows, int summed) {
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t x = reinterpret_cast<uint64_t>(base);
    r = i32x4_t{scalar(int(uint32_t(x))), scalar(int(uint32_t(x >> 32) & 0xFFFFu)), int(kPast), 0x00020000};
    if (KIND == kAlong) {
      at = (l & 7) ^ (l >> 3) ^ (w & 1);
      left = summed / 8;
      step = 128;
#pragma unroll
      for (int q = 0; q < NB; ++q)
        off[q] = uint32_t(min((q * 4 + w) * 8 + (l >> 3), rows - 1)) * uint32_t(ld * 2) + at * 16;
    } else {
      constexpr int kRows = 64 / kLanes;  // summed elements a load
      at = w * kRows + l / kLanes;
      left = summed;
      step = uint32_t(kDeep * ld * 2);
#pragma unroll
      for (int q = 0; q < NB; ++q) {
        const int k = (q * 4 + w) * kRows + l / kLanes, p = l % kLanes;
        const int chunk = 2 * ((p >> 1) ^ (k & 3) ^ (4 * ((k >> 3) & 1))) + (p & 1);
        off[q] = (uint32_t(k) * uint32_t(ld * 2) + chunk * 16) | (8 * chunk < rows ? 0u : kPast);
      }
    }
  }
  // Load q of the next step into the stage at LDS address `to`.
  __device__ __forceinline__ void load(int q, uint32_t to) const {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mine = KIND == kAlong ? at : at + q * 4 * (64 / kLanes);
    dma16_at<false>(r, off[q] | (mine < left ? 0u : kPast), 0u, to + (q * 4 + w) * 1024);
  }
  __device__ __forceinline__ void next() {
    left -= KIND == kAlong ? kDeep / 8 : kDeep;
    const uint64_t base = (uint64_t(uint32_t(r.y)) << 32 | uint32_t(r.x)) + step;
    r.x = scalar(int(uint32_t(base)));
    r.y = scalar(int(uint32_t(base >> 32)));
  }
  __device__ __forceinline__ void uniform() {
    r.x = scalar(r.x);
    r.y = scalar(r.y);
    r.z = int(kPast);
    r.w = 0x00020000;
    left = scalar(left);
    step = uint32_t(scalar(int(step)));
  }
};

// LDS byte addresses of this lane's fragment reads in stage 0.
template <int KIND, int NB>
struct FragAt {
  static constexpr int kAddr = KIND == kAlong ? 2 : NB;
  static constexpr uint32_t kRow = 64 * NB;  // kAcross: bytes of a summed element
  uint32_t p[kAddr];

  // half: which half of the tile's rows the wave has
  __device__ __forceinline__ void init(uint32_t base, int half) {
    const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
    if (KIND == kAlong) {
      const int sw = (r & 7) ^ ((r >> 3) & 1);
#pragma unroll
      for (int s = 0; s < kAddr; ++s) p[s] = base + uint32_t(half * 16 * NB + r) * 128 + (((4 * s + g) ^ sw) * 16);
    } else {
      const int k = 8 * g + (r >> 2), f = (k & 3) ^ (4 * ((k >> 3) & 1));
#pragma unroll
      for (int i = 0; i < kAddr; ++i)
        p[i] = base + uint32_t(k) * kRow + uint32_t((half * NB + i) ^ f) * 32 + (r & 3) * 8;
    }
  }
  // Fragment i of slice s of the stage at byte `stage`; part: 0 or 1 of kAcross' two reads.
  __device__ __forceinline__ v4u along(int s, int i, uint32_t stage) const {
    return *reinterpret_cast<lds_cv4u*>(uintptr_t(p[KIND == kAlong ? s : 0] + stage + uint32_t(i) * 2048));
  }
  __device__ __forceinline__ v2u_t across(int s, int i, int part, uint32_t stage) const {
    const v4s_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4s*>(
        uintptr_t(p[KIND == kAcross ? i : 0] + stage + (32 * s + 4 * part) * kRow)));
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

template <int TYPE, int AK, int BK, int IB, int JB>
struct Tile {
  typedef Operand<AK, IB> A;
  typedef Operand<BK, JB> B;
  static constexpr int kLoads = IB + JB;  // a wave and step
  static constexpr int kReads = (AK == kAlong ? IB : 2 * IB) + (BK == kAlong ? JB : 2 * JB);

  FragAt<AK, IB> fa;
  FragAt<BK, JB> fb;
  f32x4_t acc[IB][JB];

  struct Frag {
    v4u a[IB], b[JB];
  };

  // Read r of a slice's kReads.
  __device__ __forceinline__ void read(Frag& f, int s, int r, uint32_t stage) const {
    constexpr int kB = BK == kAlong ? JB : 2 * JB;
    if (r < kB) {
      if (BK == kAlong) {
        f.b[r % JB] = fb.along(s, r, stage);
      } else {
        const v2u_t v = fb.across(s, r >> 1, r & 1, stage);
        f.b[(r >> 1) % JB][2 * (r & 1)] = v.x;
        f.b[(r >> 1) % JB][2 * (r & 1) + 1] = v.y;
      }
    } else {
      const int x = r - kB;
      if (AK == kAlong) {
        f.a[x % IB] = fa.along(s, x, stage);
      } else {
        const v2u_t v = fa.across(s, x >> 1, x & 1, stage);
        f.a[(x >> 1) % IB][2 * (x & 1)] = v.x;
        f.a[(x >> 1) % IB][2 * (x & 1) + 1] = v.y;
      }
    }
  }

  // The MFMAs of a slice on f; between them the reads of slice RS (of the stage at rd) into fr,
  // and, with LOAD, the next step's loads into the stage at wr.
  template <int RS, bool LOAD>
  __device__ __forceinline__ void slice(const A& a, const B& b, const Frag& f, Frag& fr, uint32_t rd, uint32_t wr) {
    constexpr int kM = IB * JB;
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int i = m / JB, j = m % JB;
      __builtin_amdgcn_sched_barrier(0);
      acc[i][j] = mfma<TYPE>(f.b[j], f.a[i], acc[i][j]);
#pragma unroll
      for (int r = m * kReads / kM; r < (m + 1) * kReads / kM; ++r) read(fr, RS, r, rd);
      if (LOAD) {
#pragma unroll
        for (int q = m * kLoads / kM; q < (m + 1) * kLoads / kM; ++q) {
          if (q < IB) a.load(q, lds_addr(s_a) + wr);
          else b.load(q - IB, lds_addr(s_b) + wr);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  // The loads of two steps.
  static __device__ __forceinline__ void begin(A& a, B& b) {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int q = 0; q < IB; ++q) a.load(q, lds_addr(s_a) + ks * kStage);
#pragma unroll
      for (int q = 0; q < JB; ++q) b.load(q, lds_addr(s_b) + ks * kStage);
      a.next();
      b.next();
    }
    asm volatile("" ::: "memory");
  }

  // The sum over `steps` steps; begin() has been called, and after it the wave has issued `stores`
  // memory operations.
  __device__ __forceinline__ void run(A a, B b, int steps, int stores) {
    a.uniform();
    b.uniform();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    fa.init(lds_addr(s_a), w >> 1);
    fb.init(lds_addr(s_b), w & 1);
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j = 0; j < JB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    wait_all_but(kLoads + stores);  // step 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Frag f0, f1;
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(f0, 0, r, 0);
    uint32_t cur = 0;
    for (int ks = 0; ks < steps; ++ks) {
      slice<1, false>(a, b, f0, f1, cur, cur);
      // step ks + 1 has landed (mine by the wait, everyone's by the barrier), and every wave has
      // read the last of this step's stage
      if (ks == 0) wait_all_but(stores);
      else wait_vmcnt<0>();
      wait_lds();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const uint32_t nxt = cur ^ kStage;
      slice<0, true>(a, b, f1, f0, nxt, cur);
      a.next();
      b.next();
      cur = nxt;
    }
    // every load has landed and every wave has read its last fragments: the stages are free
    wait_loads_and_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  // Memory operations that store() issues for results in 16 and in 32 bits.
  static constexpr int kStores16 = IB * JB / 2, kStores32 = IB * JB;

  // Block (i, j): lane l holds, of row l % 16, the columns 4 (l / 16) .. +4.  16 rows of 256 bytes
  // at a time go through the wave's 4 KB of LDS and leave as whole 128-byte lines (16 chunks of 16
  // bytes a row, chunk c of row r at c ^ r); with JB = 4 and 16-bit results the row has 128 bytes.
  // The resource's range drops what lies outside `rows` and `cols`, so that every wave makes the
  // same number of stores.
  template <bool OUT32, bool ADD>
  __device__ __forceinline__ void store(void* out, int64_t ld, int rows, int cols) const {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));  // the addresses below are not kept over the sum's loop
    const int l = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = w >> 1, wn = w & 1, r = l & 15, g = l >> 4;
    constexpr int kSize = OUT32 ? 4 : 2;
    constexpr int kChunks = JB == 8 || OUT32 ? 16 : 8;  // 16-byte chunks a row that go out together
    constexpr int kJ = kChunks / kSize;                 // column blocks that make them
    constexpr int kRows = 64 / kChunks;                 // rows that an instruction stores
    const rsrc_t ro = row_rsrc(out, kPast);
    const uint32_t area = lds_addr(s_out) + uint32_t(w) * 4096;
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j0 = 0; j0 < JB; j0 += kJ) {
#pragma unroll
        for (int j = j0; j < j0 + kJ; ++j) {
          const f32x4_t c = acc[i][j];
          if (OUT32)
            *reinterpret_cast<lds_w16*>(uintptr_t(area + r * 256 + (((4 * (j - j0) + g) ^ r) * 16))) =
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
      }
  }
};

}  // namespace g16
}  // namespace mok
