// MXFP4 quantiser and its inverse: blocks of 32 elements along a row, e2m1 codes (two a
// byte, the even element in the low half) and one e8m0 scale.  The shared exponent is the
// smallest n with amax * 2^-n <= 6, e2m1's largest value, as the MXFP8 quantiser's is for
// 448; the codes come from gfx950's conversions, which divide by a power-of-two scale and
// round to nearest even.  Nothing saturates: the rule for n bounds every magnitude by 6.
// Both are bound by HBM.
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "ops_launch.h"
#include "mx.h"

namespace mok {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr uint32_t kInfBits = 0x7F800000u;  // magnitude bits of infinity; NaNs lie above

// Shared exponent of a block from the bits of its largest magnitude (finite).
__device__ __forceinline__ int mx4_shared_exp(uint32_t b) {
  const int E = int(b >> 23) - 127;
  if (E == -127) return -127;  // zero or float32-subnormal: below 6 * 2^-127
  const int n = E - 2 + ((b & 0x7FFFFFu) > 0x400000u ? 1 : 0);  // mantissa above 1.5
  return max(-127, n);  // at most 127 - 2 + 1
}
// 2^n as a float, n in [-127, 127]
__device__ __forceinline__ float pow2(int n) {
  return __uint_as_float(n == -127 ? 0x00400000u : uint32_t(n + 127) << 23);
}

// Largest of a quad's unsigned values (DPP quad_perm [1,0,3,2], [2,3,0,1]); the quad's
// lanes are all active.
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  v = max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, true)));
  return max(v, uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, true)));
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Eight consecutive elements: 16 bytes of a 16-bit type, 32 of fp32.
template <int TYPE>
struct Eight {
  v4u v[TYPE == MOK_TYPE_FP32 ? 2 : 1];

  template <bool NT>
  __device__ __forceinline__ void load(const uint8_t* src) {
    const v4u* s = reinterpret_cast<const v4u*>(src);
#pragma unroll
    for (int i = 0; i < (TYPE == MOK_TYPE_FP32 ? 2 : 1); ++i)
      v[i] = NT ? __builtin_nontemporal_load(s + i) : s[i];
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const v4u& q = v[i >> 2];
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
  // The bits, as a float32, of the largest magnitude (magnitudes order as their bits do).
  __device__ __forceinline__ uint32_t amax() const {
    if (TYPE == MOK_TYPE_FP32) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, word(i) & 0x7FFFFFFFu);
      return m;
    }
    u16x2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, word(i) & 0x7FFF7FFFu));
    const uint16_t h = m.x > m.y ? m.x : m.y;
    return TYPE == MOK_TYPE_BF16 ? uint32_t(h) << 16
                                 : __float_as_uint(float(__builtin_bit_cast(_Float16, h)));
  }
  // Codes of the elements over s = 2^n.
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t q = 0;
    q = pair<0>(q, s);
    q = pair<1>(q, s);
    q = pair<2>(q, s);
    return pair<3>(q, s);
  }
  template <int I>
  __device__ __forceinline__ uint32_t pair(uint32_t q, float s) const {
    if (TYPE == MOK_TYPE_BF16)
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2_t, word(I)), s, I);
    if (TYPE == MOK_TYPE_FP16)
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2_t, word(I)), s, I);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(word(TYPE == MOK_TYPE_FP32 ? 2 * I : 0)),
                                                    __uint_as_float(word(TYPE == MOK_TYPE_FP32 ? 2 * I + 1 : 0)),
                                                    s, I);
  }
};

// Chunks of a few elements (8 where quantised, so that a quad of lanes holds one block: cols
// is a multiple of 32, so a quad's chunks are of one row, and whole quads run or idle).  A
// wave takes 64 kBatch consecutive chunks and loads them all before it converts any.  DENSE:
// the matrices have no gaps between rows and are taken as one row.
constexpr int kBatch = 4;

struct Mat {
  int64_t n_chunks;
  int row_chunks;
  int64_t ld_val, ld_codes, ld_scales;  // bytes from row to row
};
// Chunk i: its row and its place in it.
template <bool DENSE>
__device__ __forceinline__ void place(const Mat& m, int64_t i, int64_t* r, int64_t* c) {
  if (DENSE) {
    *r = 0;
    *c = i;
  } else {
    *r = i / m.row_chunks;
    *c = i - *r * m.row_chunks;
  }
}

template <int TYPE, bool DENSE, bool NT>
__global__ __launch_bounds__(256) void k_quantize_mx4(const uint8_t* src, Mat m, uint8_t* codes,
                                                      uint8_t* scales) {
  constexpr int kBytes = TYPE == MOK_TYPE_FP32 ? 32 : 16;
  const int lane = threadIdx.x & 63;
  for (int64_t b = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6)) * 64 * kBatch; b < m.n_chunks;
       b += int64_t(gridDim.x) * 256 * kBatch) {
    Eight<TYPE> x[kBatch];
    int64_t r[kBatch], c[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t i = b + 64 * u + lane;
      if (i < m.n_chunks) {
        place<DENSE>(m, i, &r[u], &c[u]);
        x[u].template load<NT>(src + r[u] * m.ld_val + c[u] * kBytes);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (b + 64 * u + lane >= m.n_chunks) break;  // whole quads
      const uint32_t amax = quad_umax(x[u].amax());
      const bool finite = amax < kInfBits;
      const int n = mx4_shared_exp(amax);
      const uint32_t q = x[u].codes(pow2(min(n, 127)));
      *reinterpret_cast<uint32_t*>(codes + r[u] * m.ld_codes + c[u] * 4) = finite ? q : 0u;
      if ((lane & 3) == 0)
        scales[r[u] * m.ld_scales + (c[u] >> 2)] = finite ? uint8_t(n + 127) : uint8_t(255);
    }
  }
}

// Sixteen bytes of values: code pairs 0.. of q times s.  Exact in float32 (4 or 6 times 2^126
// and what lies above overflows to infinity, as a float of that value must).
template <int TYPE>
__device__ __forceinline__ v4u values16(uint32_t q, float s, bool nan) {
  if (TYPE == MOK_TYPE_FP32) {
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 1);
    auto bits = [&](float f) { return nan ? 0x7FC00000u : __float_as_uint(f); };
    return v4u{bits(a.x), bits(a.y), bits(b.x), bits(b.y)};
  }
  if (TYPE == MOK_TYPE_BF16) {
    auto two = [&](bf16x2_t h) { return nan ? 0x7FC07FC0u : __builtin_bit_cast(uint32_t, h); };
    return v4u{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3))};
  }
  auto two = [&](f16x2_t h) { return nan ? 0x7E007E00u : __builtin_bit_cast(uint32_t, h); };
  return v4u{two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, 0)),
             two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, 1)),
             two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, 2)),
             two(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, 3))};
}

// Chunks of 16 bytes of values: a wave's stores are whole lines (fp32 in chunks of 32 bytes, two
// stores each, was 131 us at [16384, 7168] against 100 us of traffic).
template <int TYPE, bool DENSE>
__global__ __launch_bounds__(256) void k_dequantize_mx4(const uint8_t* codes, const uint8_t* scales,
                                                        Mat m, uint8_t* dst) {
  constexpr int kElems = TYPE == MOK_TYPE_FP32 ? 4 : 8;
  const int lane = threadIdx.x & 63;
  for (int64_t b = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6)) * 64 * kBatch; b < m.n_chunks;
       b += int64_t(gridDim.x) * 256 * kBatch) {
    uint32_t q[kBatch];
    int sc[kBatch];
    int64_t r[kBatch], c[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t i = b + 64 * u + lane;
      if (i < m.n_chunks) {
        place<DENSE>(m, i, &r[u], &c[u]);
        const uint8_t* at = codes + r[u] * m.ld_codes + c[u] * (kElems / 2);
        q[u] = TYPE == MOK_TYPE_FP32 ? *reinterpret_cast<const uint16_t*>(at)
                                     : *reinterpret_cast<const uint32_t*>(at);
        sc[u] = scales[r[u] * m.ld_scales + c[u] / (32 / kElems)];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (b + 64 * u + lane >= m.n_chunks) break;
      *reinterpret_cast<v4u*>(dst + r[u] * m.ld_val + c[u] * 16) =
          values16<TYPE>(q[u], pow2(min(sc[u], 254) - 127), sc[u] == 255);
    }
  }
}

Mat mat_of(const Mx4Args& a, int elems) {
  const int es = a.type == MOK_TYPE_FP32 ? 4 : 2;
  return Mat{a.rows * (a.cols / elems), a.cols / elems, a.ld_val * es, a.ld_codes, a.ld_scales};
}
bool dense(const Mx4Args& a) {
  return a.rows == 1 || (a.ld_val == a.cols && a.ld_codes == a.cols / 2 && a.ld_scales == a.cols / 32);
}
unsigned grid_of(const Mat& m) {
  return unsigned(std::min<int64_t>((m.n_chunks + 256 * kBatch - 1) / (256 * kBatch), 1 << 20));
}
// Calls f with the element type and density as compile-time values.
template <typename F>
mok_status_t with_form(const Mx4Args& a, F f) {
  auto form = [&](auto type) {
    return dense(a) ? f(type, std::true_type()) : f(type, std::false_type());
  };
  if (a.type == MOK_TYPE_BF16) return form(std::integral_constant<int, MOK_TYPE_BF16>());
  if (a.type == MOK_TYPE_FP16) return form(std::integral_constant<int, MOK_TYPE_FP16>());
  return form(std::integral_constant<int, MOK_TYPE_FP32>());
}

}  // namespace

mok_status_t launch_quantize_mx4(const Mx4Args& a, hipStream_t st) {
  const Mat m = mat_of(a, 8);
  // What the call reads and writes, against the last-level cache: a larger source is read
  // non-temporally ([16384, 7168] bf16 53 -> 47 us; [4096, 7168] 12.9 plain, 14.0 so).
  const int64_t moved = a.rows * a.cols * (a.type == MOK_TYPE_FP32 ? 4 : 2) + a.rows * (a.cols / 2);
  const bool nt = moved > (int64_t(256) << 20);
  return with_form(a, [&](auto type, auto flat) {
    constexpr int kType = decltype(type)::value;
    constexpr bool kFlat = decltype(flat)::value;
    auto go = [&](auto kern) {
      return launch(kern, dim3(grid_of(m)), dim3(256), st, static_cast<const uint8_t*>(a.src), m, a.codes,
                    a.scales);
    };
    return nt ? go(k_quantize_mx4<kType, kFlat, true>) : go(k_quantize_mx4<kType, kFlat, false>);
  });
}

mok_status_t launch_dequantize_mx4(const Mx4Args& a, hipStream_t st) {
  const Mat m = mat_of(a, a.type == MOK_TYPE_FP32 ? 4 : 8);
  return with_form(a, [&](auto type, auto flat) {
    return launch(k_dequantize_mx4<decltype(type)::value, decltype(flat)::value>, dim3(grid_of(m)), dim3(256),
                  st, static_cast<const uint8_t*>(a.codes), static_cast<const uint8_t*>(a.scales), m,
                  static_cast<uint8_t*>(a.dst));
  });
}

}  // namespace mok
