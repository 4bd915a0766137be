// Arguments and launchers of the row operators and the MXFP4 operators (rows.hip, mx4.hip,
// grouped_mx4.hip), called by ops_api.hip after its checks.
#pragma once
#include <cstddef>
#include <tuple>
#include <utility>

#include "launch.h"

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

}  // namespace mok
