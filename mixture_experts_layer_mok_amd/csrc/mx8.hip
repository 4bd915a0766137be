// Activations held in 8 bits: MXFP8 quantiser and its inverse for values in bf16, fp16 and fp32,
// SwiGLU that holds its inputs so, and its backward pass from what is held.  e4m3 codes in blocks
// of 32 along a row, one e8m0 scale each; the shared exponent is the smallest n with
// amax * 2^-n <= 448 (mx_shared_exp); the codes come from gfx950's conversions, which divide by a
// power-of-two scale and round to nearest even, and nothing saturates.  All are bound by HBM: one pass,
// 16 bytes of values a lane, no LDS.  MI355X, 16,384 rows, bf16, in loops over three sets of inputs (bytes at
// the 5.27 TB/s of a large copy in brackets): quantise 7168 columns 55 us (67), back 66 (67); SwiGLU of 2048
// pairs 44 (51), its backward with the activation again 52 (64).  Alone under a profiler, with the caches as
// the other kernels of a pass leave them, 61, 60, 48 and 53 at the least.
//
// A chunk is 16 bytes of values, kN elements; the 32 / kN lanes of a group (4 of a 16-bit type,
// 8 of fp32) hold one block.  Rows are whole blocks, so a group's chunks are of one row, and
// whole groups run or idle.
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "ops_launch.h"
#include "mx.h"

namespace mok {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t v2u_t __attribute__((ext_vector_type(2)));
typedef short s16x2_t __attribute__((ext_vector_type(2)));

constexpr uint32_t kInfBits = 0x7F800000u;  // magnitude bits of infinity; NaNs lie above
constexpr uint8_t kNanScale = 255;

// 2^n as a float, n in [-127, 127]
__device__ __forceinline__ float pow2(int n) {
  return __uint_as_float(n == -127 ? 0x00400000u : uint32_t(n + 127) << 23);
}

template <int CTRL>
__device__ __forceinline__ uint32_t umax_step(uint32_t v) {
  return max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xF, 0xF, true)));
}

__device__ __forceinline__ uint32_t word(v4u v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// What differs by element type.
template <int TYPE>
struct Chunk {
  static constexpr bool k32 = TYPE == MOK_TYPE_FP32;
  static constexpr int kN = k32 ? 4 : 8;
  static constexpr int kGroup = 32 / kN;  // lanes that hold a block

  // The codes of a chunk.
  struct Codes {
    uint32_t w[k32 ? 1 : 2];
    __device__ __forceinline__ void load(const uint8_t* p) {
      if (k32) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        const v2u_t v = *reinterpret_cast<const v2u_t*>(p);
        w[0] = v.x;
        w[k32 ? 0 : 1] = v.y;
      }
    }
    __device__ __forceinline__ void store(uint8_t* p) const {
      if (k32) *reinterpret_cast<uint32_t*>(p) = w[0];
      else *reinterpret_cast<v2u_t*>(p) = v2u_t{w[0], w[k32 ? 0 : 1]};
    }
  };

  static __device__ __forceinline__ void to_float(v4u v, float (&f)[kN]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = word(v, i);
      if (k32) {
        f[i] = __uint_as_float(u);
      } else if (TYPE == MOK_TYPE_BF16) {
        f[k32 ? 0 : 2 * i] = __uint_as_float(u << 16);
        f[k32 ? 0 : 2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
      } else {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, u);
        f[k32 ? 0 : 2 * i] = float(h.x);
        f[k32 ? 0 : 2 * i + 1] = float(h.y);
      }
    }
  }
  static __device__ __forceinline__ v4u from_float(const float (&f)[kN]) {
    v4u v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k32) v[i] = __float_as_uint(f[i]);
      else if (TYPE == MOK_TYPE_BF16) v[i] = pack_bf16x2(f[k32 ? 0 : 2 * i], f[k32 ? 0 : 2 * i + 1]);
      else v[i] = __builtin_bit_cast(uint32_t, f16x2_t{_Float16(f[k32 ? 0 : 2 * i]), _Float16(f[k32 ? 0 : 2 * i + 1])});
    }
    return v;
  }

  // The bits, as a float32, of the block's largest magnitude (magnitudes order as their bits do).
  static __device__ __forceinline__ uint32_t block_amax(v4u v) {
    uint32_t m = 0;
    if (k32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max(m, word(v, i) & 0x7FFFFFFFu);
    } else {
      typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
      u16x2_t p = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        p = __builtin_elementwise_max(p, __builtin_bit_cast(u16x2_t, word(v, i) & 0x7FFF7FFFu));
      const uint16_t h = p.x > p.y ? p.x : p.y;
      m = TYPE == MOK_TYPE_BF16 ? uint32_t(h) << 16 : __float_as_uint(float(__builtin_bit_cast(_Float16, h)));
    }
    m = umax_step<0xB1>(m);             // quad_perm [1,0,3,2]
    m = umax_step<0x4E>(m);             // quad_perm [2,3,0,1]
    if (k32) m = umax_step<0x141>(m);   // row_half_mirror: the other quad of eight lanes
    return m;
  }

  // The chunk's codes, and its block's scale byte.
  static __device__ __forceinline__ uint8_t quantize(v4u v, Codes* c) {
    const uint32_t amax = block_amax(v);
    const bool finite = amax < kInfBits;
    const int n = mx_shared_exp(__uint_as_float(amax));
    const float s = pow2(n);
#pragma unroll
    for (int j = 0; j < (k32 ? 1 : 2); ++j) {
      s16x2_t q = {0, 0};
      if (k32) {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, __uint_as_float(v.x), __uint_as_float(v.y), s, false);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, __uint_as_float(v.z), __uint_as_float(v.w), s, true);
      } else if (TYPE == MOK_TYPE_BF16) {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, __builtin_bit_cast(bf16x2_t, word(v, 2 * j)), s, false);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, __builtin_bit_cast(bf16x2_t, word(v, 2 * j + 1)), s, true);
      } else {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(q, __builtin_bit_cast(f16x2_t, word(v, 2 * j)), s, false);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(q, __builtin_bit_cast(f16x2_t, word(v, 2 * j + 1)), s, true);
      }
      c->w[j] = finite ? __builtin_bit_cast(uint32_t, q) : 0u;
    }
    return finite ? uint8_t(n + 127) : kNanScale;
  }

  // The chunk's values as floats (exact: four bits times a power of two; what lies above
  // float32's range, 2^127 times 2 and more, overflows to infinity).
  static __device__ __forceinline__ void values(const Codes& c, uint8_t scale, float (&f)[kN]) {
    const float s = pow2(min(int(scale), 254) - 127);
#pragma unroll
    for (int j = 0; j < (k32 ? 1 : 2); ++j) {
      const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.w[j], s, false);
      const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.w[j], s, true);
      f[4 * j] = lo.x;
      f[4 * j + 1] = lo.y;
      f[4 * j + 2] = hi.x;
      f[4 * j + 3] = hi.y;
    }
    if (scale == kNanScale) {
#pragma unroll
      for (int j = 0; j < kN; ++j) f[j] = __uint_as_float(0x7FC00000u);
    }
  }
};

// Chunks are dealt to waves in runs of 64 kBatch; a wave finds its run's row once (a 64-bit
// division of a wave-uniform number), its lanes theirs by a 32-bit one.  Chunks a lane has in
// flight: four of the quantiser and its inverse, two of SwiGLU, whose chunks are pairs.  MI355X,
// 2777 x 1056 pairs, bf16: forward and backward together 13.9 us with two, 16.2 with four;
// 20,000 x 2048, fp32: 238, 247; the quantiser is within 2% with either.
constexpr int kBatch = 4, kPairBatch = 2;

// A 16-byte chunk of values.  A call that moves more than the memory-side cache keeps
// (kStreamBytes) reads its values around the caches, so that what it writes stays there for the
// next kernel.  MI355X, bf16, 16,384 rows: SwiGLU of 3584 pairs 85 -> 72 us, quantise and back of
// 7168 columns 126 -> 108, of 4096 69 -> 64; below the limit it costs, 8192 rows of 2048 pairs
// 23.2 -> 24.1, 5000 rows 13.9 -> 15.7.  Stores stay ordinary: around the caches they take up to
// a quarter off the kernel itself and give more back to the next one (SwiGLU of 16,384 rows of
// 2048 pairs with a kernel that reads its result 58 -> 62 us, its backward 101 -> 110).
constexpr int64_t kStreamBytes = int64_t(192) << 20;
template <bool kStream>
__device__ __forceinline__ v4u load_chunk(const uint8_t* p) {
  const v4u* q = reinterpret_cast<const v4u*>(p);
  return kStream ? __builtin_nontemporal_load(q) : *q;
}

struct Geom {
  int64_t n_chunks;
  uint32_t row_chunks;
};
struct Place {
  int64_t row;
  uint32_t c;
};
__device__ __forceinline__ Place place(const Geom& g, int64_t row0, uint32_t c0, int u) {
  const uint32_t c = c0 + 64 * u + (threadIdx.x & 63);
  const uint32_t q = c / g.row_chunks;
  return {row0 + q, c - q * g.row_chunks};
}
// Calls f(first chunk, its row, its place in it) for each of this wave's runs.
template <int kBatch, typename F>
__device__ __forceinline__ void runs(const Geom& g, F f) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t b = (int64_t(blockIdx.x) * 4 + w) * 64 * kBatch; b < g.n_chunks;
       b += int64_t(gridDim.x) * 256 * kBatch) {
    const int64_t row0 = b / g.row_chunks;
    f(b, row0, uint32_t(b - row0 * g.row_chunks));
  }
}

template <int TYPE, bool kStream>
__global__ __launch_bounds__(256) void k_quantize_mx8(Mx8Args p, Geom g) {
  typedef Chunk<TYPE> C;
  const int lane = threadIdx.x & 63;
  constexpr int kSize = C::k32 ? 4 : 2;
  runs<kBatch>(g, [&](int64_t b, int64_t row0, uint32_t c0) {
    v4u v[kBatch];
    Place at[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      at[u] = place(g, row0, c0, u);
      if (b + 64 * u + lane < g.n_chunks)
        v[u] = load_chunk<kStream>(static_cast<const uint8_t*>(p.src) + at[u].row * p.ld_val * kSize + at[u].c * 16);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (b + 64 * u + lane >= g.n_chunks) break;  // whole groups
      typename C::Codes q;
      const uint8_t s = C::quantize(v[u], &q);
      q.store(p.codes + at[u].row * p.ld_codes + at[u].c * C::kN);
      if ((lane & (C::kGroup - 1)) == 0) p.scales[at[u].row * p.ld_scales + at[u].c / C::kGroup] = s;
    }
  });
}

template <int TYPE>
__global__ __launch_bounds__(256) void k_dequantize_mx8(Mx8Args p, Geom g) {
  typedef Chunk<TYPE> C;
  const int lane = threadIdx.x & 63;
  constexpr int kSize = C::k32 ? 4 : 2;
  runs<kBatch>(g, [&](int64_t b, int64_t row0, uint32_t c0) {
    typename C::Codes q[kBatch];
    uint8_t s[kBatch];
    Place at[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      at[u] = place(g, row0, c0, u);
      if (b + 64 * u + lane < g.n_chunks) {
        q[u].load(p.codes + at[u].row * p.ld_codes + at[u].c * C::kN);
        s[u] = p.scales[at[u].row * p.ld_scales + at[u].c / C::kGroup];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (b + 64 * u + lane >= g.n_chunks) break;
      float f[C::kN];
      C::values(q[u], s[u], f);
      *reinterpret_cast<v4u*>(static_cast<uint8_t*>(p.dst) + at[u].row * p.ld_val * kSize + at[u].c * 16) =
          C::from_float(f);
    }
  });
}

// s = 1 / (1 + e^-a) and 1 - s, from e = e^-|a|, which never overflows.  For 16-bit results the
// hardware's exponential and reciprocal, a few units of 2^-24 for the |a| where s is not
// negligible, far below the rounding that follows; an e below 2^-126 (|a| above 87.3) becomes 0.
// For fp32 results the library's exponential, within an ulp or two, and a division.
template <int TYPE>
__device__ __forceinline__ void sigmoid(float a, float* s, float* rest) {
  float e, q;
  if (TYPE == MOK_TYPE_FP32) {
    e = expf(-fabsf(a));
    q = 1.0f / (1.0f + e);
  } else {
    e = __expf(-fabsf(a));
    q = __builtin_amdgcn_rcpf(1.0f + e);
  }
  const float small = e * q;
  *s = a < 0 ? small : q;
  *rest = a < 0 ? q : small;
}

// Rows that the call covers: `total` holds the routed rows on the device.
__device__ __forceinline__ int64_t rows_of(const SwigluArgs& p) {
  return p.total ? min(int64_t(max(*p.total, 0)), p.rows) : p.rows;
}

template <int TYPE, bool kStream>
__global__ __launch_bounds__(256) void k_swiglu_mx8(SwigluArgs p, Geom g) {
  typedef Chunk<TYPE> C;
  const int lane = threadIdx.x & 63;
  constexpr int kSize = C::k32 ? 4 : 2;
  g.n_chunks = rows_of(p) * g.row_chunks;
  const int64_t half = int64_t(p.inter) * kSize;
  runs<kPairBatch>(g, [&](int64_t b, int64_t row0, uint32_t c0) {
    v4u va[kPairBatch], vb[kPairBatch];
    Place at[kPairBatch];
#pragma unroll
    for (int u = 0; u < kPairBatch; ++u) {
      at[u] = place(g, row0, c0, u);
      if (b + 64 * u + lane < g.n_chunks) {
        const uint8_t* src = static_cast<const uint8_t*>(p.in) + at[u].row * p.ld_in * kSize + at[u].c * 16;
        va[u] = load_chunk<kStream>(src);
        vb[u] = load_chunk<kStream>(src + half);
      }
    }
#pragma unroll
    for (int u = 0; u < kPairBatch; ++u) {
      if (b + 64 * u + lane >= g.n_chunks) break;
      float a[C::kN], c[C::kN];
      C::to_float(va[u], a);
      C::to_float(vb[u], c);
#pragma unroll
      for (int i = 0; i < C::kN; ++i) {
        float s, rest;
        sigmoid<TYPE>(a[i], &s, &rest);
        a[i] = a[i] * s * c[i];
      }
      *reinterpret_cast<v4u*>(static_cast<uint8_t*>(p.h) + at[u].row * p.ld_h * kSize + at[u].c * 16) =
          C::from_float(a);
      typename C::Codes qa, qb;
      const uint8_t sa = C::quantize(va[u], &qa), sb = C::quantize(vb[u], &qb);
      uint8_t* codes = p.codes + at[u].row * p.ld_codes + at[u].c * C::kN;
      qa.store(codes);
      qb.store(codes + p.inter);
      if ((lane & (C::kGroup - 1)) == 0) {
        uint8_t* scales = p.scales + at[u].row * p.ld_scales + at[u].c / C::kGroup;
        scales[0] = sa;
        scales[p.inter / 32] = sb;
      }
    }
  });
}

template <int TYPE, bool kStream>
__global__ __launch_bounds__(256) void k_swiglu_mx8_bwd(SwigluArgs p, Geom g) {
  typedef Chunk<TYPE> C;
  const int lane = threadIdx.x & 63;
  constexpr int kSize = C::k32 ? 4 : 2;
  g.n_chunks = rows_of(p) * g.row_chunks;
  const int64_t half = int64_t(p.inter) * kSize;
  runs<kPairBatch>(g, [&](int64_t b, int64_t row0, uint32_t c0) {
    v4u vd[kPairBatch];
    typename C::Codes qa[kPairBatch], qb[kPairBatch];
    uint8_t sa[kPairBatch], sb[kPairBatch];
    Place at[kPairBatch];
#pragma unroll
    for (int u = 0; u < kPairBatch; ++u) {
      at[u] = place(g, row0, c0, u);
      if (b + 64 * u + lane < g.n_chunks) {
        vd[u] = load_chunk<kStream>(static_cast<const uint8_t*>(p.in) + at[u].row * p.ld_in * kSize + at[u].c * 16);
        const uint8_t* codes = p.codes + at[u].row * p.ld_codes + at[u].c * C::kN;
        qa[u].load(codes);
        qb[u].load(codes + p.inter);
        const uint8_t* scales = p.scales + at[u].row * p.ld_scales + at[u].c / C::kGroup;
        sa[u] = scales[0];
        sb[u] = scales[p.inter / 32];
      }
    }
#pragma unroll
    for (int u = 0; u < kPairBatch; ++u) {
      if (b + 64 * u + lane >= g.n_chunks) break;
      float a[C::kN], c[C::kN], d[C::kN], h[C::kN];
      C::to_float(vd[u], d);
      C::values(qa[u], sa[u], a);
      C::values(qb[u], sb[u], c);
#pragma unroll
      for (int i = 0; i < C::kN; ++i) {
        float s, rest;
        sigmoid<TYPE>(a[i], &s, &rest);
        const float silu = a[i] * s;
        h[i] = silu * c[i];
        a[i] = d[i] * c[i] * s * (1.0f + a[i] * rest);
        c[i] = d[i] * silu;
      }
      uint8_t* dst = static_cast<uint8_t*>(p.d_ab) + at[u].row * p.ld_d_ab * kSize + at[u].c * 16;
      *reinterpret_cast<v4u*>(dst) = C::from_float(a);
      *reinterpret_cast<v4u*>(dst + half) = C::from_float(c);
      if (p.h)
        *reinterpret_cast<v4u*>(static_cast<uint8_t*>(p.h) + at[u].row * p.ld_h * kSize + at[u].c * 16) =
            C::from_float(h);
    }
  });
}

Geom geom_of(int32_t type, int64_t rows, int32_t cols) {
  const int32_t per = cols / (type == MOK_TYPE_FP32 ? 4 : 8);
  return {rows * per, uint32_t(per)};
}
dim3 grid_of(const Geom& g, int batch) {
  return dim3(unsigned(std::min<int64_t>((g.n_chunks + 256 * batch - 1) / (256 * batch), 1 << 20)));
}
// Calls f with the element type as a compile-time value.
template <typename F>
mok_status_t with_type(int32_t type, F f) {
  if (type == MOK_TYPE_BF16) return f(std::integral_constant<int, MOK_TYPE_BF16>());
  if (type == MOK_TYPE_FP16) return f(std::integral_constant<int, MOK_TYPE_FP16>());
  return f(std::integral_constant<int, MOK_TYPE_FP32>());
}
// Also with whether the call, at so many values and codes moved, reads around the caches.
template <typename F>
mok_status_t with_stream(int32_t type, int64_t values, int64_t codes, F f) {
  const bool stream = values * (type == MOK_TYPE_FP32 ? 4 : 2) + codes >= kStreamBytes;
  return with_type(type, [&](auto t) { return stream ? f(t, std::true_type()) : f(t, std::false_type()); });
}

}  // namespace

mok_status_t launch_quantize_mx8(const Mx8Args& a, hipStream_t st) {
  const Geom g = geom_of(a.type, a.rows, a.cols);
  const int64_t n = a.rows * a.cols;
  return with_stream(a.type, n, n, [&](auto type, auto stream) {
    return launch(k_quantize_mx8<decltype(type)::value, decltype(stream)::value>, grid_of(g, kBatch), dim3(256), st, a,
                  g);
  });
}

mok_status_t launch_dequantize_mx8(const Mx8Args& a, hipStream_t st) {
  const Geom g = geom_of(a.type, a.rows, a.cols);
  return with_type(a.type, [&](auto type) {
    return launch(k_dequantize_mx8<decltype(type)::value>, grid_of(g, kBatch), dim3(256), st, a, g);
  });
}

mok_status_t launch_swiglu_mx8(const SwigluArgs& a, hipStream_t st) {
  const Geom g = geom_of(a.type, a.rows, a.inter);
  const int64_t n = a.rows * a.inter;
  return with_stream(a.type, 3 * n, 2 * n, [&](auto type, auto stream) {
    return launch(k_swiglu_mx8<decltype(type)::value, decltype(stream)::value>, grid_of(g, kPairBatch), dim3(256), st,
                  a, g);
  });
}

mok_status_t launch_swiglu_mx8_bwd(const SwigluArgs& a, hipStream_t st) {
  const Geom g = geom_of(a.type, a.rows, a.inter);
  const int64_t n = a.rows * a.inter;
  return with_stream(a.type, (a.h ? 4 : 3) * n, 2 * n, [&](auto type, auto stream) {
    return launch(k_swiglu_mx8_bwd<decltype(type)::value, decltype(stream)::value>, grid_of(g, kPairBatch), dim3(256),
                  st, a, g);
  });
}

}  // namespace mok
