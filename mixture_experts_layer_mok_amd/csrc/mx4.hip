// MXFP4 quantiser and its inverse: blocks of 32 elements along a row, e2m1 codes (two a
// byte, the even element in the low half) and one e8m0 scale.  The shared exponent is the
// smallest n with amax * 2^-n <= 6, e2m1's largest value, as the MXFP8 quantiser's is for
// 448; the codes come from gfx950's conversions, which divide by a power-of-two scale and
// round to nearest even.  Nothing saturates: the rule for n bounds every magnitude by 6.
// Both are bound by HBM.
#include <algorithm>

#include "device.h"
#include "launch.h"
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

// Eight consecutive elements as floats.
template <int TYPE>
__device__ __forceinline__ void load8(float (&f)[8], const void* src) {
  const v4u* s = static_cast<const v4u*>(src);
  const v4u v = s[0];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (TYPE == MOK_TYPE_FP32) {
    const v4u u = s[1];
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(w[i]);
      f[4 + i] = __uint_as_float(x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (TYPE == MOK_TYPE_BF16) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, w[i]);
        f[2 * i] = float(h.x);
        f[2 * i + 1] = float(h.y);
      }
    }
  }
}

// Chunk i of the matrix: 8 elements, row i / (cols / 8).  A quad of lanes holds one block:
// cols is a multiple of 32, so a quad's chunks are of one row, and whole quads run or idle.
template <int TYPE>
__global__ __launch_bounds__(256) void k_quantize_mx4(const uint8_t* src, int64_t ld_src,
                                                      int64_t n_chunks, int row_chunks,
                                                      uint8_t* codes, int64_t ld_codes,
                                                      uint8_t* scales, int64_t ld_scales) {
  constexpr int kSize = TYPE == MOK_TYPE_FP32 ? 4 : 2;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n_chunks;
       i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / row_chunks;
    const int c = int(i - r * row_chunks);
    float f[8];
    load8<TYPE>(f, src + r * ld_src + int64_t(c) * 8 * kSize);
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    amax = quad_umax(amax);
    const bool finite = amax < kInfBits;
    const int n = mx4_shared_exp(amax);
    const float s = pow2(min(n, 127));
    uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0], f[1], s, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[2], f[3], s, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[4], f[5], s, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[6], f[7], s, 3);
    *reinterpret_cast<uint32_t*>(codes + r * ld_codes + int64_t(c) * 4) = finite ? q : 0u;
    if ((c & 3) == 0) scales[r * ld_scales + (c >> 2)] = finite ? uint8_t(n + 127) : uint8_t(255);
  }
}

// Eight codes a thread.  The value of a code is exact in float32 (at scales below 2^-126
// as a subnormal; 4 or 6 times 2^126 overflows to infinity, as a float of that value must).
template <int TYPE>
__global__ __launch_bounds__(256) void k_dequantize_mx4(const uint8_t* codes, int64_t ld_codes,
                                                        const uint8_t* scales, int64_t ld_scales,
                                                        int64_t n_chunks, int row_chunks,
                                                        uint8_t* dst, int64_t ld_dst) {
  constexpr int kSize = TYPE == MOK_TYPE_FP32 ? 4 : 2;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n_chunks;
       i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / row_chunks;
    const int c = int(i - r * row_chunks);
    const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + r * ld_codes + int64_t(c) * 4);
    const int sc = scales[r * ld_scales + (c >> 2)];
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = (q >> (4 * e)) & 15u;
      const uint32_t m = h & 7u;
      // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
      const float mag = m < 2 ? 0.5f * float(m)
                              : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
      const float v = ldexpf(h & 8u ? -mag : mag, sc - 127);
      f[e] = sc == 255 ? __uint_as_float(0x7FC00000u) : v;
    }
    v4u* d = reinterpret_cast<v4u*>(dst + r * ld_dst + int64_t(c) * 8 * kSize);
    if (TYPE == MOK_TYPE_FP32) {
      d[0] = v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                 __float_as_uint(f[3])};
      d[1] = v4u{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                 __float_as_uint(f[7])};
    } else {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = TYPE == MOK_TYPE_BF16
                   ? pack_bf16x2(f[2 * e], f[2 * e + 1])
                   : __builtin_bit_cast(uint32_t, f16x2_t{_Float16(f[2 * e]), _Float16(f[2 * e + 1])});
      d[0] = v4u{o[0], o[1], o[2], o[3]};
    }
  }
}

unsigned grid_of(int64_t n_chunks) { return unsigned(std::min<int64_t>((n_chunks + 255) / 256, 8192)); }
mok_status_t launched() { return hipGetLastError() == hipSuccess ? MOK_OK : MOK_E_LAUNCH; }

}  // namespace

mok_status_t launch_quantize_mx4(const Mx4Args& a, hipStream_t st) {
  const int rc = a.cols / 8;
  const int64_t n = a.rows * rc;
  const int es = a.type == MOK_TYPE_FP32 ? 4 : 2;
  const auto* s = static_cast<const uint8_t*>(a.src);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(grid_of(n)), dim3(256), 0, st, s, a.ld_val * es, n, rc, a.codes,
                       a.ld_codes, a.scales, a.ld_scales);
  };
  if (a.type == MOK_TYPE_BF16) go(k_quantize_mx4<MOK_TYPE_BF16>);
  else if (a.type == MOK_TYPE_FP16) go(k_quantize_mx4<MOK_TYPE_FP16>);
  else go(k_quantize_mx4<MOK_TYPE_FP32>);
  return launched();
}

mok_status_t launch_dequantize_mx4(const Mx4Args& a, hipStream_t st) {
  const int rc = a.cols / 8;
  const int64_t n = a.rows * rc;
  const int es = a.type == MOK_TYPE_FP32 ? 4 : 2;
  auto* d = static_cast<uint8_t*>(a.dst);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(grid_of(n)), dim3(256), 0, st,
                       static_cast<const uint8_t*>(a.codes), a.ld_codes,
                       static_cast<const uint8_t*>(a.scales), a.ld_scales, n, rc, d,
                       a.ld_val * es);
  };
  if (a.type == MOK_TYPE_BF16) go(k_dequantize_mx4<MOK_TYPE_BF16>);
  else if (a.type == MOK_TYPE_FP16) go(k_dequantize_mx4<MOK_TYPE_FP16>);
  else go(k_dequantize_mx4<MOK_TYPE_FP32>);
  return launched();
}

}  // namespace mok
