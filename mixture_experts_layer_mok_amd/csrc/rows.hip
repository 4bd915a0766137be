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
#include <algorithm>

#include "device.h"
#include "launch.h"

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

// W waves of a workgroup share a token; a workgroup holds kWg / W tokens.
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

template <int W>
__global__ __launch_bounds__(threads_of<W>()) void k_permute(RowGeom g, const uint8_t* x,
                                                             const int32_t* pos, uint8_t* rows) {
  int64_t t;
  uint32_t l;
  if (!my_token<W>(g, &t, &l)) return;
  const int32_t p = my_row(g, pos, t);
  const uint64_t has = __ballot(p >= 0);
  if (!has) return;
  const rsrc_t rx = row_rsrc(x + t * g.ld_tok, g.bytes);
  constexpr int U = W == 1 ? 8 : 4;
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

// dst[t] = sum_j g_j rows[pos[t,j]], g_j = w[t,j], or 1 without weights.
template <int TYPE, int W>
__global__ __launch_bounds__(threads_of<W>()) void k_sum_rows(RowGeom g, const uint8_t* rows,
                                                              const int32_t* pos, const float* w,
                                                              uint8_t* dst) {
  typedef Elem<TYPE> El;
  int64_t t;
  uint32_t l;
  if (!my_token<W>(g, &t, &l)) return;
  const int lane = threadIdx.x & 63;
  const int32_t p = my_row(g, pos, t);
  const float gate = p >= 0 ? (w ? w[t * g.k + lane] : 1.f) : 0.f;
  const uint64_t has = __ballot(p >= 0);
  const rsrc_t rd = row_rsrc(dst + t * g.ld_out, g.bytes);
  constexpr int U = W == 1 ? 4 : 2;
  for (uint32_t b0 = 0; b0 < g.bytes; b0 += W * 64 * 16 * U) {
    float acc[U][El::kN];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < El::kN; ++e) acc[u][e] = 0.f;
    for (uint64_t m = has; m; m &= m - 1) {
      const int j = __ffsll((unsigned long long)m) - 1;
      const rsrc_t rr =
          row_rsrc(rows + int64_t(__builtin_amdgcn_readlane(p, j)) * g.ld_rows, g.bytes);
      const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gate), j));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[El::kN];
        El::load(f, buf_ld16<kCpolPlain>(rr, b0 + (l + 64 * W * u) * 16));
#pragma unroll
        for (int e = 0; e < El::kN; ++e) acc[u][e] = __fadd_rn(acc[u][e], __fmul_rn(gj, f[e]));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      buf_st16<kCpolStream>(rd, b0 + (l + 64 * W * u) * 16, El::store(acc[u]));
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int TYPE, int W>
__global__ __launch_bounds__(threads_of<W>()) void k_unpermute_bwd(RowGeom g, const uint8_t* dy,
                                                                   const uint8_t* rows,
                                                                   const int32_t* pos,
                                                                   const float* w, uint8_t* d_rows,
                                                                   float* dw) {
  typedef Elem<TYPE> El;
  __shared__ float s_dw[W > 1 ? kMaxWaves : 1][64];
  int64_t t;
  uint32_t l;
  const bool valid = my_token<W>(g, &t, &l);
  if (!valid) return;  // whole waves, and whole workgroups where waves share a token
  const int lane = threadIdx.x & 63;
  const int32_t p = my_row(g, pos, t);
  const float gate = p >= 0 ? w[t * g.k + lane] : 0.f;
  const uint64_t has = __ballot(p >= 0);
  const rsrc_t ry = row_rsrc(dy + t * g.ld_tok, g.bytes);
  float my_dw = 0.f;  // lane j: this wave's part of dw[t, j]
  constexpr int U = W == 1 ? 4 : 2;
  if (has) {
    for (uint32_t b0 = 0; b0 < g.bytes; b0 += W * 64 * 16 * U) {
      float y[U][El::kN];
#pragma unroll
      for (int u = 0; u < U; ++u)
        El::load(y[u], buf_ld16<kCpolPlain>(ry, b0 + (l + 64 * W * u) * 16));
      for (uint64_t m = has; m; m &= m - 1) {
        const int j = __ffsll((unsigned long long)m) - 1;
        const int64_t row = __builtin_amdgcn_readlane(p, j);
        const rsrc_t rr = row_rsrc(rows + row * g.ld_rows, g.bytes);
        const rsrc_t rd = row_rsrc(d_rows + row * g.ld_out, g.bytes);
        const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gate), j));
        float dot = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t off = b0 + (l + 64 * W * u) * 16;
          float f[El::kN], o[El::kN];
          El::load(f, buf_ld16<kCpolPlain>(rr, off));
#pragma unroll
          for (int e = 0; e < El::kN; ++e) {
            dot = fmaf(y[u][e], f[e], dot);
            o[e] = __fmul_rn(gj, y[u][e]);
          }
          buf_st16<kCpolStream>(rd, off, El::store(o));
        }
        dot = wave_sum(dot);
        if (lane == j) my_dw += dot;
      }
    }
  }
  if (W > 1) {
    const int wv = (threadIdx.x >> 6);
    s_dw[wv][lane] = my_dw;
    __syncthreads();
    const int w0 = wv / W * W;
    if (wv == w0) {
      my_dw = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) my_dw += s_dw[w0 + i][lane];
    }
    if (wv != w0) return;
  }
  if (lane < g.k) dw[t * g.k + lane] = my_dw;
}

mok_status_t launched() { return hipGetLastError() == hipSuccess ? MOK_OK : MOK_E_LAUNCH; }

// Waves per token: one where the tokens alone fill the GPU, sixteen for a few tokens.
int waves_for(int64_t T) { return T >= 2048 ? 1 : (T >= 512 ? 4 : 16); }
unsigned grid_for(int64_t T, int W) { return unsigned(W >= 4 ? T : (T + 4 / W - 1) / (4 / W)); }

template <int W>
void run_permute(const RowGeom& g, const RowArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(k_permute<W>, dim3(grid_for(g.T, W)), dim3(threads_of<W>()), 0, st, g,
                     static_cast<const uint8_t*>(a.tok), a.pos, static_cast<uint8_t*>(a.out));
}
template <int TYPE, int W>
void run_sum(const RowGeom& g, const RowArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((k_sum_rows<TYPE, W>), dim3(grid_for(g.T, W)), dim3(threads_of<W>()), 0, st,
                     g, static_cast<const uint8_t*>(a.rows), a.pos, a.w,
                     static_cast<uint8_t*>(a.out));
}
template <int TYPE, int W>
void run_bwd(const RowGeom& g, const RowArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((k_unpermute_bwd<TYPE, W>), dim3(grid_for(g.T, W)), dim3(threads_of<W>()), 0,
                     st, g, static_cast<const uint8_t*>(a.tok),
                     static_cast<const uint8_t*>(a.rows), a.pos, a.w,
                     static_cast<uint8_t*>(a.out), a.dw);
}
template <int TYPE>
void run_sum_w(int W, const RowGeom& g, const RowArgs& a, hipStream_t st) {
  if (W == 1) run_sum<TYPE, 1>(g, a, st);
  else if (W == 4) run_sum<TYPE, 4>(g, a, st);
  else run_sum<TYPE, 16>(g, a, st);
}
template <int TYPE>
void run_bwd_w(int W, const RowGeom& g, const RowArgs& a, hipStream_t st) {
  if (W == 1) run_bwd<TYPE, 1>(g, a, st);
  else if (W == 4) run_bwd<TYPE, 4>(g, a, st);
  else run_bwd<TYPE, 16>(g, a, st);
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
  const int W = waves_for(a.T);
  if (W == 1) run_permute<1>(g, a, st);
  else if (W == 4) run_permute<4>(g, a, st);
  else run_permute<16>(g, a, st);
  return launched();
}

mok_status_t launch_sum_rows(const RowArgs& a, hipStream_t st) {
  const RowGeom g = geom_of(a);
  const int W = waves_for(a.T);
  if (a.type == MOK_TYPE_BF16) run_sum_w<MOK_TYPE_BF16>(W, g, a, st);
  else if (a.type == MOK_TYPE_FP16) run_sum_w<MOK_TYPE_FP16>(W, g, a, st);
  else run_sum_w<MOK_TYPE_FP32>(W, g, a, st);
  return launched();
}

mok_status_t launch_unpermute_bwd(const RowArgs& a, hipStream_t st) {
  const RowGeom g = geom_of(a);
  const int W = waves_for(a.T);
  if (a.type == MOK_TYPE_BF16) run_bwd_w<MOK_TYPE_BF16>(W, g, a, st);
  else if (a.type == MOK_TYPE_FP16) run_bwd_w<MOK_TYPE_FP16>(W, g, a, st);
  else run_bwd_w<MOK_TYPE_FP32>(W, g, a, st);
  return launched();
}

}  // namespace mok
