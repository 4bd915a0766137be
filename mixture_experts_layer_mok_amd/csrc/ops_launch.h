// Arguments and launchers of the row operators, the MXFP4 operators, the grouped product of
// 16-bit rows and the activations in 8 bits (rows.hip, mx4.hip, grouped_mx4.hip, grouped_mm.hip,
// mx8.hip), called by ops_api.hip after its checks.
#pragma once
#include <cstddef>
#include <tuple>
#include <utility>

#include "launch.h"
#include "mm_forms.h"

namespace mok {

// Launches a kernel and gives the launch's own result.  (hipGetLastError would also report, and
// take away, an error that an earlier call of someone else left behind.)
template <typename... P, size_t... I>
hipError_t launch_with(void (*kern)(P...), dim3 grid, dim3 block, hipStream_t st, std::tuple<P...>& args,
                       std::index_sequence<I...>) {
  void* at[] = {static_cast<void*>(&std::get<I>(args))...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kern), grid, block, at, 0, st);
}
template <typename... P, typename... A>
mok_status_t launch(void (*kern)(P...), dim3 grid, dim3 block, hipStream_t st, A... args) {
  std::tuple<P...> p(args...);
  if (launch_with(kern, grid, block, st, p, std::index_sequence_for<P...>()) == hipSuccess) return MOK_OK;
  (void)hipGetLastError();  // reported here, not by the next caller's check
  return MOK_E_LAUNCH;
}

// Row operators (rows.hip).  tok: the operand with a row per token that is read (x, dy);
// rows: the routed rows that are read; out: what is written, of ld_out elements a row.
struct RowArgs {
  int32_t type;
  int64_t T;
  int32_t k, cols;
  int64_t max_rows;
  const int32_t* pos;
  const void* tok;
  int64_t ld_tok;
  const void* rows;
  int64_t ld_rows;
  const float* w;  // null: weights of 1
  void* out;
  int64_t ld_out;
  float* dw;
};
mok_status_t launch_permute(const RowArgs& a, hipStream_t st);
mok_status_t launch_sum_rows(const RowArgs& a, hipStream_t st);
mok_status_t launch_unpermute_bwd(const RowArgs& a, hipStream_t st);

// MXFP4 (mx4.hip, grouped_mx4.hip).  ld_val: elements from row to row of src or dst.
struct Mx4Args {
  int32_t type;
  int64_t rows;
  int32_t cols;
  const void* src;
  void* dst;
  int64_t ld_val;
  uint8_t* codes;
  int64_t ld_codes;
  uint8_t* scales;
  int64_t ld_scales;
};
mok_status_t launch_quantize_mx4(const Mx4Args& a, hipStream_t st);
mok_status_t launch_dequantize_mx4(const Mx4Args& a, hipStream_t st);

struct GroupedArgs {
  bool a8;  // A holds e4m3 codes, else e2m1
  const uint8_t* a;
  int64_t ld_a;
  const uint8_t* as;
  int64_t ld_as;
  int64_t max_rows;
  const int32_t* offsets;
  int32_t groups;
  const uint8_t* b;
  const uint8_t* bs;
  int32_t n, k;
  bool out32;
  void* out;
  int64_t ld_out;
};
mok_status_t launch_grouped_mx4(const GroupedArgs& a, hipStream_t st);

// Grouped product of 16-bit rows (grouped_mm.hip); kinds: mm_forms.h.
struct MmArgs {
  int32_t type;
  const void* left;
  int64_t ld_left;
  const void* right;  // b [groups, n, k], or a (ld_right; with scales: e4m3 codes, in bytes)
  int64_t ld_right;
  const uint8_t* scales;
  int64_t ld_scales;
  int64_t max_rows;
  const int32_t* offsets;
  int32_t groups, n, k;
  bool out32, add;
  void* out;
  int64_t ld_out;
  float* ws;  // MOK_MM_WORKSPACE_BYTES for partial sums, or null
};
mok_status_t launch_grouped_mm(MmKind kind, const MmArgs& a, hipStream_t st);
mok_status_t launch_mm_out(const MmArgs& a, hipStream_t st);
mok_status_t launch_mm_rows(const MmArgs& a, hipStream_t st);
mok_status_t launch_mm_weights(const MmArgs& a, hipStream_t st);
mok_status_t launch_mm_weights_held(const MmArgs& a, hipStream_t st);

// Activations in 8 bits (mx8.hip).  ld_val: elements from row to row of src or dst.
struct Mx8Args {
  int32_t type;
  int64_t rows;
  int32_t cols;
  const void* src;
  void* dst;
  int64_t ld_val;
  uint8_t* codes;
  int64_t ld_codes;
  uint8_t* scales;
  int64_t ld_scales;
};
mok_status_t launch_quantize_mx8(const Mx8Args& a, hipStream_t st);
mok_status_t launch_dequantize_mx8(const Mx8Args& a, hipStream_t st);

struct SwigluArgs {
  int32_t type;
  int64_t rows;
  int32_t inter;
  const int32_t* total;  // rows on the device, or null: all
  const void* in;        // ab, or dh
  int64_t ld_in;
  uint8_t* codes;
  int64_t ld_codes;
  uint8_t* scales;
  int64_t ld_scales;
  void* h;
  int64_t ld_h;
  void* d_ab;
  int64_t ld_d_ab;
};
mok_status_t launch_swiglu_mx8(const SwigluArgs& a, hipStream_t st);
mok_status_t launch_swiglu_mx8_bwd(const SwigluArgs& a, hipStream_t st);

}  // namespace mok
