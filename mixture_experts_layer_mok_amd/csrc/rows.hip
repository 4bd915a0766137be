// Row operators: tokens to expert order and back (permute, unpermute) and their
// gradients.  All four read one table, pos [T, k] (the schedule's), and are owned by the
// token: the waves of token t read or write the rows pos[t, j] of its k pairs, so every
// row has one owner, sums run in ascending j in fp32, and nothing is atomic.
//   permute        rows[pos[t,j]] = x[t]                  x read once, R rows written
//   permute bwd    dx[t] = sum_j d_rows[pos[t,j]]         R rows read, dx written once
//   unpermute      y[t] = sum_j w[t,j] rows[pos[t,j]]     R rows read, y written once
//   unpermute bwd  d_rows[pos[t,j]] = w[t,j] dy[t],       dy read once, R rows read, R rows
//                  dw[t,j] = <dy[t], rows[pos[t,j]]>      written
// Owning by token rather than by row reads x and dy once instead of once per routed row.
// All are bound by HBM.
#include <type_traits>

#include "device.h"
#include "ops_launch.h"
#include "mx.h"

namespace mok {

namespace {

// A 16-byte chunk of a row as floats: 8 of a 16-bit type, 4 of fp32.
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

template <int TYPE>
struct Elem;
template <>
struct Elem<MOK_TYPE_BF16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(float (&f)[8], v4u v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ v4u store(const float (&f)[8]) {
    return v4u{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
               pack_bf16x2(f[6], f[7])};
  }
};
template <>
struct Elem<MOK_TYPE_FP16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(float (&f)[8], v4u v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2_t h = __builtin_bit_cast(f16x2_t, w[i]);
      f[2 * i] = float(h.x);
      f[2 * i + 1] = float(h.y);
    }
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2_t{_Float16(a), _Float16(b)});
  }
  static __device__ __forceinline__ v4u store(const float (&f)[8]) {
    return v4u{pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7])};
  }
};
template <>
struct Elem<MOK_TYPE_FP32> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void load(float (&f)[4], v4u v) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ v4u store(const float (&f)[4]) {
    return v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
               __float_as_uint(f[3])};
  }
};

// W waves of a workgroup share a token; a workgroup has four waves, 4 / W tokens, or, for W of 16,
// one token.
constexpr int kMaxWaves = 16;

struct RowGeom {
  int64_t T;
  int k;
  uint32_t bytes;      // of a row
  int64_t max_rows;
  int64_t ld_tok, ld_rows, ld_out;  // bytes from row to row
};

// pos of the token's pair j in lane j, -1 where the pair has no row.
__device__ __forceinline__ int32_t my_row(const RowGeom& g, const int32_t* pos, int64_t t) {
  const int lane = threadIdx.x & 63;
  const int32_t p = lane < g.k ? pos[t * g.k + lane] : -1;
  return p >= 0 && p < g.max_rows ? p : -1;
}

// Token t, chunk b of a pass: the waves of the token interleave their chunks.
template <int W>
__device__ __forceinline__ bool my_token(const RowGeom& g, int64_t* t, uint32_t* lane_of_token) {
  constexpr int kTok = (W >= 4 ? 1 : 4 / W);  // tokens per workgroup
  const uint32_t w = threadIdx.x >> 6;
  *t = int64_t(blockIdx.x) * kTok + (W >= 4 ? 0 : w / W);
  *lane_of_token = (w % W) * 64 + (threadIdx.x & 63);
  return *t < g.T;
}
template <int W>
constexpr int threads_of() { return W >= 4 ? W * 64 : 256; }

template <int W, int U>
__global__ __launch_bounds__(threads_of<W>()) void k_permute(RowGeom g, const uint8_t* x,
                                                             const int32_t* pos, uint8_t* rows) {
  int64_t t;
  uint32_t l;
  if (!my_token<W>(g, &t, &l)) return;
  const int32_t p = my_row(g, pos, t);
  const uint64_t has = __ballot(p >= 0);
  if (!has) return;
  const rsrc_t rx = row_rsrc(x + t * g.ld_tok, g.bytes);
  for (uint32_t b0 = 0; b0 < g.bytes; b0 += W * 64 * 16 * U) {
    v4u v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = buf_ld16<kCpolPlain>(rx, b0 + (l + 64 * W * u) * 16);
    for (uint64_t m = has; m; m &= m - 1) {
      const int j = __ffsll((unsigned long long)m) - 1;
      const rsrc_t rr =
          row_rsrc(rows + int64_t(__builtin_amdgcn_readlane(p, j)) * g.ld_rows, g.bytes);
#pragma unroll
      for (int u = 0; u < U; ++u) buf_st16<kCpolStream>(rr, b0 + (l + 64 * W * u) * 16, v[u]);
    }
  }
}

// dst[t] = sum_j g_j rows[pos[t,j]], g_j = w[t,j], or 1 without weights, kSlots pairs at a time;
// missing ones get an empty range, whose loads read nothing.  As compiled, a row's load stands
// right before its addition (below the branch that leaves the slots), so a wave has one row
// in flight: with many tokens the other waves cover that (86,552 rows of 7168 at 5.4 TB/s), a few
// tokens take a round trip a row (64 tokens of eight rows of 7168: 5 us).
template <int TYPE, int W, int U, bool NT>
__global__ __launch_bounds__(threads_of<W>()) void k_sum_rows(RowGeom g, const uint8_t* rows,
                                                              const int32_t* pos, const float* w,
                                                              uint8_t* dst) {
  typedef Elem<TYPE> El;
  constexpr int kSlots = U >= 8 ? 2 : 4;
  constexpr int kPol = NT ? kCpolStream : kCpolPlain;
  int64_t t;
  uint32_t l;
  if (!my_token<W>(g, &t, &l)) return;
  const int lane = threadIdx.x & 63;
  const int32_t p = my_row(g, pos, t);
  const float gate = p >= 0 ? (w ? w[t * g.k + lane] : 1.f) : 0.f;
  const uint64_t has = __ballot(p >= 0);
  const rsrc_t rd = row_rsrc(dst + t * g.ld_out, g.bytes);
  for (uint32_t b0 = 0; b0 < g.bytes; b0 += W * 64 * 16 * U) {
    float acc[U][El::kN];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < El::kN; ++e) acc[u][e] = 0.f;
    for (uint64_t m = has; m;) {
      int js[kSlots];
      v4u v[kSlots][U];
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        js[s] = m ? __ffsll((unsigned long long)m) - 1 : -1;
        if (m) m &= m - 1;
        const int64_t row = __builtin_amdgcn_readlane(p, js[s] >= 0 ? js[s] : 0);
        const rsrc_t rr = row_rsrc(rows + (js[s] >= 0 ? row : 0) * g.ld_rows, js[s] >= 0 ? g.bytes : 0u);
#pragma unroll
        for (int u = 0; u < U; ++u) v[s][u] = buf_ld16<kPol>(rr, b0 + (l + 64 * W * u) * 16);
      }
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        if (js[s] < 0) break;  // wave-uniform
        const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gate), js[s]));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[El::kN];
          El::load(f, v[s][u]);
#pragma unroll
          for (int e = 0; e < El::kN; ++e) acc[u][e] = __fadd_rn(acc[u][e], __fmul_rn(gj, f[e]));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      buf_st16<kCpolStream>(rd, b0 + (l + 64 * W * u) * 16, El::store(acc[u]));
  }
}

// Sum over the wave, the same in every lane: the butterfly inside each row of 16 lanes by DPP
// moves, then across the four rows.
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// One pair after the other: dy's row is read for each (from the caches after the first), so
// that a pair's dot product stays in registers over the whole row and is summed over the
// lanes once.
template <int TYPE, int W, int U, bool NT>
__global__ __launch_bounds__(threads_of<W>()) void k_unpermute_bwd(RowGeom g, const uint8_t* dy,
                                                                   const uint8_t* rows,
                                                                   const int32_t* pos,
                                                                   const float* w, uint8_t* d_rows,
                                                                   float* dw) {
  typedef Elem<TYPE> El;
  constexpr int kPol = NT ? kCpolStream : kCpolPlain;
  __shared__ float s_dw[W > 1 ? kMaxWaves : 1][64];
  int64_t t;
  uint32_t l;
  if (!my_token<W>(g, &t, &l)) return;  // whole waves; whole workgroups where they share a token
  const int lane = threadIdx.x & 63;
  const int32_t p = my_row(g, pos, t);
  const float gate = p >= 0 ? w[t * g.k + lane] : 0.f;
  const rsrc_t ry = row_rsrc(dy + t * g.ld_tok, g.bytes);
  float my_dw = 0.f;  // lane j: this wave's part of dw[t, j]
  for (uint64_t m = __ballot(p >= 0); m; m &= m - 1) {
    const int j = __ffsll((unsigned long long)m) - 1;
    const int64_t row = __builtin_amdgcn_readlane(p, j);
    const rsrc_t rr = row_rsrc(rows + row * g.ld_rows, g.bytes);
    const rsrc_t rd = row_rsrc(d_rows + row * g.ld_out, g.bytes);
    const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gate), j));
    float dot = 0.f;
    for (uint32_t b0 = 0; b0 < g.bytes; b0 += W * 64 * 16 * U) {
      v4u yv[U], rv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        yv[u] = buf_ld16<kCpolPlain>(ry, b0 + (l + 64 * W * u) * 16);
        rv[u] = buf_ld16<kPol>(rr, b0 + (l + 64 * W * u) * 16);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float y[El::kN], f[El::kN], o[El::kN];
        El::load(y, yv[u]);
        El::load(f, rv[u]);
#pragma unroll
        for (int e = 0; e < El::kN; ++e) {
          dot = fmaf(y[e], f[e], dot);
          o[e] = __fmul_rn(gj, y[e]);
        }
        buf_st16<kCpolStream>(rd, b0 + (l + 64 * W * u) * 16, El::store(o));
      }
    }
    dot = wave_sum(dot);
    if (lane == j) my_dw = dot;
  }
  if (W > 1) {
    const int wv = threadIdx.x >> 6;
    s_dw[wv][lane] = my_dw;
    __syncthreads();
    if (wv) return;
    my_dw = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) my_dw += s_dw[i][lane];
  }
  if (lane < g.k) dw[t * g.k + lane] = my_dw;
}

// Launch shape.
//   W: waves a token: one where the tokens alone fill the GPU (or the row is one chunk a lane),
//     else four, or sixteen for long rows, so that a lane holds one chunk of its row.  Measured
//     on MI355X, us for W = 1 / 4 / 16 (bf16, k = 8; permute, unpermute, its gradient):
//       128 tokens of 7168:  7.0 / 5.7 / 4.7, 10.1 / 8.3 / 4.6, 18.6 / 11.5 / 7.3
//       512 tokens of 2048:  4.6 / 4.3 / 5.2,  4.7 / 4.1 / 6.1,  8.0 / 6.5 / 10.1
//       1024 tokens of 2048: 6.8 / 6.6 / 7.4,  6.8 / 6.5 / 11.7, 11.6 / 11.9 / 18.9
//       4096 tokens of 512:  6.8 / 7.6 / 20.3, 7.0 / 12.5 / 36.7, 12.8 / 19.3 / 59.8
//   U: 16-byte chunks a lane in flight, the smallest that takes the row in one pass (loads past
//     its end cost an issue), at most umax.
//   nt: rows too many for the last-level cache (256 MB) are read non-temporally; smaller ones
//     may still be there from the operator that wrote them.  Measured: 86,552 rows of 7168
//     (1.24 GB) 296 us plain, 285 nt; 512 rows of 7168 4.9 us plain, 6.9 nt.
struct Shape {
  int W, U;
  bool nt;
};
Shape shape_of(const RowGeom& g, int umax) {
  Shape s;
  s.W = g.T >= 1024 || g.bytes <= 1024 ? 1 : g.bytes > 6144 ? 16 : 4;
  const int chunks = int((g.bytes + 1023) / 1024);
  s.U = s.W > 1 ? 1 : chunks <= 2 ? 2 : chunks <= 4 ? 4 : chunks <= 8 || umax == 8 ? 8 : 16;
  s.nt = s.W == 1 && (g.max_rows + g.T) * int64_t(g.bytes) > (int64_t(256) << 20);
  return s;
}
unsigned grid_for(int64_t T, int W) { return unsigned(W >= 4 ? T : (T + 3) / 4); }

// Calls f with the shape's W, U and nt as compile-time values.
template <int N>
using Int = std::integral_constant<int, N>;
template <int UMAX, typename F>
mok_status_t with_shape(const Shape& s, F f) {
  if (s.W == 4) return f(Int<4>(), Int<1>(), std::false_type());
  if (s.W == 16) return f(Int<16>(), Int<1>(), std::false_type());
  auto nt = [&](auto u) {
    return s.nt ? f(Int<1>(), u, std::true_type()) : f(Int<1>(), u, std::false_type());
  };
  if (s.U == 2) return nt(Int<2>());
  if (s.U == 4) return nt(Int<4>());
  if (UMAX == 8 || s.U == 8) return nt(Int<8>());
  return nt(Int<UMAX>());
}
template <typename F>
mok_status_t with_type(int32_t type, F f) {
  if (type == MOK_TYPE_BF16) return f(Int<MOK_TYPE_BF16>());
  if (type == MOK_TYPE_FP16) return f(Int<MOK_TYPE_FP16>());
  return f(Int<MOK_TYPE_FP32>());
}

RowGeom geom_of(const RowArgs& a) {
  const int es = a.type == MOK_TYPE_FP32 ? 4 : 2;
  return RowGeom{a.T, a.k, uint32_t(a.cols) * es, a.max_rows, a.ld_tok * es, a.ld_rows * es,
                 a.ld_out * es};
}

}  // namespace

mok_status_t launch_permute(const RowArgs& a, hipStream_t st) {
  RowGeom g = geom_of(a);
  g.ld_rows = g.ld_out;
  Shape s = shape_of(g, 16);
  s.nt = false;
  return with_shape<16>(s, [&](auto w, auto u, auto) {
    constexpr int W = decltype(w)::value, U = decltype(u)::value;
    return launch(k_permute<W, U>, dim3(grid_for(g.T, W)), dim3(threads_of<W>()), st, g,
                  static_cast<const uint8_t*>(a.tok), a.pos, static_cast<uint8_t*>(a.out));
  });
}

mok_status_t launch_sum_rows(const RowArgs& a, hipStream_t st) {
  const RowGeom g = geom_of(a);
  return with_type(a.type, [&](auto type) {
    return with_shape<8>(shape_of(g, 8), [&](auto w, auto u, auto nt) {
      constexpr int W = decltype(w)::value, U = decltype(u)::value;
      return launch(k_sum_rows<decltype(type)::value, W, U, decltype(nt)::value>, dim3(grid_for(g.T, W)),
                    dim3(threads_of<W>()), st, g, static_cast<const uint8_t*>(a.rows), a.pos, a.w,
                    static_cast<uint8_t*>(a.out));
    });
  });
}

mok_status_t launch_unpermute_bwd(const RowArgs& a, hipStream_t st) {
  const RowGeom g = geom_of(a);
  return with_type(a.type, [&](auto type) {
    return with_shape<16>(shape_of(g, 16), [&](auto w, auto u, auto nt) {
      constexpr int W = decltype(w)::value, U = decltype(u)::value;
      return launch(k_unpermute_bwd<decltype(type)::value, W, U, decltype(nt)::value>,
                    dim3(grid_for(g.T, W)), dim3(threads_of<W>()), st, g,
                    static_cast<const uint8_t*>(a.tok), static_cast<const uint8_t*>(a.rows), a.pos, a.w,
                    static_cast<uint8_t*>(a.out), a.dw);
    });
  });
}

}  // namespace mok
