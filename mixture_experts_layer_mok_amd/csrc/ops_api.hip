// C ABI of the row operators and the MXFP4 operators: argument checks (all before any HIP
// runtime call) and the launches.  Declarations and contracts: include/mok.h.
#include "../../include/mok.h"
#include "ops_launch.h"

using namespace mok;

namespace {

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool type_ok(int32_t t) { return t == MOK_TYPE_BF16 || t == MOK_TYPE_FP16 || t == MOK_TYPE_FP32; }

// Row strides, in elements of up to 4 bytes, whose products with 2^31 - 2 rows stay in 64 bits.
constexpr int64_t kMaxLd = int64_t(1) << 30;
constexpr int64_t kMaxLdOut = int64_t(1) << 21;  // the product's: 256 rows stay in 31-bit offsets

// A value matrix's row stride in elements; a read operand may repeat one row (ld 0).
bool ld_ok(int64_t ld, int32_t cols, bool read) {
  return ld % 8 == 0 && ld <= kMaxLd && (ld >= cols || (read && ld == 0));
}

mok_status_t check_rows(int32_t type, int64_t tokens, int32_t top_k, int32_t cols,
                        int64_t max_rows) {
  if (!type_ok(type)) return MOK_E_UNSUPPORTED;
  if (tokens < 0 || tokens > (int64_t(1) << 24) || top_k < 1 || top_k > 64 ||
      tokens * top_k > (int64_t(1) << 24) || cols < 8 || cols % 8 != 0 || cols > 65536 ||
      max_rows < 0 || max_rows > INT32_MAX)
    return MOK_E_SHAPE;
  return MOK_OK;
}

RowArgs row_args(int32_t type, int64_t tokens, int32_t top_k, int32_t cols, int64_t max_rows,
                 const int32_t* pos) {
  RowArgs a = {};
  a.type = type;
  a.T = tokens;
  a.k = top_k;
  a.cols = cols;
  a.max_rows = max_rows;
  a.pos = pos;
  return a;
}

mok_status_t sum_rows(int32_t type, const void* rows, int64_t ld_rows, int64_t max_rows,
                      const int32_t* pos, const float* w, int64_t tokens, int32_t top_k,
                      int32_t cols, void* out, int64_t ld_out, void* stream, bool weighted) {
  const mok_status_t s = check_rows(type, tokens, top_k, cols, max_rows);
  if (s != MOK_OK) return s;
  if (!ld_ok(ld_rows, cols, true) || !ld_ok(ld_out, cols, false)) return MOK_E_SHAPE;
  if (tokens == 0) return MOK_OK;
  if ((!rows && max_rows > 0) || !pos || (weighted && !w) || !out) return MOK_E_NULL;
  if (!aligned(rows, 16) || !aligned(out, 16) || !aligned(pos, 4) || !aligned(w, 4))
    return MOK_E_SHAPE;
  RowArgs a = row_args(type, tokens, top_k, cols, max_rows, pos);
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.w = w;
  a.out = out;
  a.ld_out = ld_out;
  return launch_sum_rows(a, static_cast<hipStream_t>(stream));
}

mok_status_t check_mx4(int32_t type, int64_t ld_val, int64_t rows, int32_t cols, int64_t ld_codes,
                       int64_t ld_scales) {
  if (!type_ok(type)) return MOK_E_UNSUPPORTED;
  if (rows < 0 || rows > INT32_MAX || cols < 32 || cols % 32 != 0 || cols > 65536 ||
      ld_codes < cols / 2 || ld_codes % 16 != 0 || ld_codes > kMaxLd || ld_scales < cols / 32 ||
      ld_scales > kMaxLd || !ld_ok(ld_val, cols, false))
    return MOK_E_SHAPE;
  return MOK_OK;
}

}  // namespace

extern "C" {

mok_status_t mok_schedule_layout(const mok_desc_t* desc, size_t* offsets_bytes,
                                 size_t* pos_bytes) {
  if (!desc) return MOK_E_NULL;
  Layout L;
  const mok_status_t s = make_layout(desc, &L);
  if (s != MOK_OK) return s;
  if (offsets_bytes) *offsets_bytes = L.off_offsets;
  if (pos_bytes) *pos_bytes = L.off_pos;
  return MOK_OK;
}

mok_status_t mok_permute(int32_t type, const void* x, int64_t ld_x, const int32_t* pos,
                         int64_t tokens, int32_t top_k, int32_t cols, void* rows,
                         int64_t ld_rows, int64_t max_rows, void* stream) {
  const mok_status_t s = check_rows(type, tokens, top_k, cols, max_rows);
  if (s != MOK_OK) return s;
  if (!ld_ok(ld_x, cols, true) || !ld_ok(ld_rows, cols, false)) return MOK_E_SHAPE;
  if (tokens == 0 || max_rows == 0) return MOK_OK;
  if (!x || !pos || !rows) return MOK_E_NULL;
  if (!aligned(x, 16) || !aligned(rows, 16) || !aligned(pos, 4)) return MOK_E_SHAPE;
  RowArgs a = row_args(type, tokens, top_k, cols, max_rows, pos);
  a.tok = x;
  a.ld_tok = ld_x;
  a.out = rows;
  a.ld_out = ld_rows;
  return launch_permute(a, static_cast<hipStream_t>(stream));
}

mok_status_t mok_permute_bwd(int32_t type, const void* d_rows, int64_t ld_rows,
                             int64_t max_rows, const int32_t* pos, int64_t tokens,
                             int32_t top_k, int32_t cols, void* dx, int64_t ld_x, void* stream) {
  return sum_rows(type, d_rows, ld_rows, max_rows, pos, nullptr, tokens, top_k, cols, dx, ld_x,
                  stream, false);
}

mok_status_t mok_unpermute(int32_t type, const void* rows, int64_t ld_rows, int64_t max_rows,
                           const int32_t* pos, const float* topk_w, int64_t tokens,
                           int32_t top_k, int32_t cols, void* y, int64_t ld_y, void* stream) {
  return sum_rows(type, rows, ld_rows, max_rows, pos, topk_w, tokens, top_k, cols, y, ld_y,
                  stream, true);
}

mok_status_t mok_unpermute_bwd(int32_t type, const void* dy, int64_t ld_y, const void* rows,
                               int64_t ld_rows, int64_t max_rows, const int32_t* pos,
                               const float* topk_w, int64_t tokens, int32_t top_k,
                               int32_t cols, void* d_rows, int64_t ld_d_rows, float* d_topk_w,
                               void* stream) {
  const mok_status_t s = check_rows(type, tokens, top_k, cols, max_rows);
  if (s != MOK_OK) return s;
  if (!ld_ok(ld_y, cols, true) || !ld_ok(ld_rows, cols, true) || !ld_ok(ld_d_rows, cols, false))
    return MOK_E_SHAPE;
  if (tokens == 0) return MOK_OK;
  if (!dy || !pos || !topk_w || !d_topk_w || (max_rows > 0 && (!rows || !d_rows)))
    return MOK_E_NULL;
  if (!aligned(dy, 16) || !aligned(rows, 16) || !aligned(d_rows, 16) || !aligned(pos, 4) ||
      !aligned(topk_w, 4) || !aligned(d_topk_w, 4))
    return MOK_E_SHAPE;
  RowArgs a = row_args(type, tokens, top_k, cols, max_rows, pos);
  a.tok = dy;
  a.ld_tok = ld_y;
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.w = topk_w;
  a.out = d_rows;
  a.ld_out = ld_d_rows;
  a.dw = d_topk_w;
  return launch_unpermute_bwd(a, static_cast<hipStream_t>(stream));
}

mok_status_t mok_quantize_mx4(int32_t type, const void* src, int64_t ld_src, int64_t rows,
                              int32_t cols, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                              int64_t ld_scales, void* stream) {
  const mok_status_t s = check_mx4(type, ld_src, rows, cols, ld_codes, ld_scales);
  if (s != MOK_OK) return s;
  if (rows == 0) return MOK_OK;
  if (!src || !codes || !scales) return MOK_E_NULL;
  if (!aligned(src, 16) || !aligned(codes, 16)) return MOK_E_SHAPE;
  return launch_quantize_mx4({type, rows, cols, src, nullptr, ld_src, codes, ld_codes, scales,
                              ld_scales},
                             static_cast<hipStream_t>(stream));
}

mok_status_t mok_dequantize_mx4(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales,
                                int64_t ld_scales, int64_t rows, int32_t cols, int32_t type,
                                void* dst, int64_t ld_dst, void* stream) {
  const mok_status_t s = check_mx4(type, ld_dst, rows, cols, ld_codes, ld_scales);
  if (s != MOK_OK) return s;
  if (rows == 0) return MOK_OK;
  if (!codes || !scales || !dst) return MOK_E_NULL;
  if (!aligned(codes, 16) || !aligned(dst, 16)) return MOK_E_SHAPE;
  return launch_dequantize_mx4({type, rows, cols, nullptr, dst, ld_dst,
                                const_cast<uint8_t*>(codes), ld_codes,
                                const_cast<uint8_t*>(scales), ld_scales},
                               static_cast<hipStream_t>(stream));
}

mok_status_t mok_grouped_mx4(int32_t a_format, const uint8_t* a_codes, int64_t ld_a,
                             const uint8_t* a_scales, int64_t ld_a_scales, int64_t max_rows,
                             const int32_t* offsets, int32_t groups, const uint8_t* b_codes,
                             const uint8_t* b_scales, int32_t n, int32_t k, int32_t out_type,
                             void* out, int64_t ld_out, void* stream) {
  if (a_format != MOK_MX_E4M3 && a_format != MOK_MX_E2M1) return MOK_E_UNSUPPORTED;
  if (out_type != MOK_TYPE_BF16 && out_type != MOK_TYPE_FP32) return MOK_E_UNSUPPORTED;
  const bool a8 = a_format == MOK_MX_E4M3;
  if (max_rows < 0 || max_rows > (int64_t(1) << 24) || groups < 1 || groups > 1024 || k < 32 ||
      k % 32 != 0 || k > 65536 || n < 8 || n % 8 != 0 || n > (1 << 20) ||
      int64_t(n) * k >= (int64_t(1) << 31))
    return MOK_E_SHAPE;
  if (ld_a < (a8 ? k : k / 2) || ld_a % 16 != 0 || ld_a > MOK_MX_MAX_LD || ld_a_scales < k / 32 ||
      ld_a_scales > MOK_MX_MAX_LD || ld_out < n || ld_out % 8 != 0 || ld_out > kMaxLdOut)
    return MOK_E_SHAPE;
  if (max_rows == 0) return MOK_OK;
  if (!a_codes || !a_scales || !offsets || !b_codes || !b_scales || !out) return MOK_E_NULL;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(out, 16) || !aligned(offsets, 4))
    return MOK_E_SHAPE;
  return launch_grouped_mx4({a8, a_codes, ld_a, a_scales, ld_a_scales, max_rows, offsets, groups,
                             b_codes, b_scales, n, k, out_type == MOK_TYPE_FP32, out, ld_out},
                            static_cast<hipStream_t>(stream));
}

}  // extern "C"
