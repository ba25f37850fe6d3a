// api_ops.hpp -- the 8-bit forms of sl_gemm with fp32 scales: api.cpp sends
// such a call here.  Host only.
#pragma once
#include "../../include/sl.h"
#include "sl_ops.hpp"

namespace sl {
namespace host {

struct BlockPlan {
  sl_plan pub;
  BlockGemmParams p;
  int32_t tile;
  bool empty;
};

// a and b E4M3 with fp32 scales: the block-scaled form
inline bool is_block_gemm(const sl_gemm_args* args) {
  return args && args->a.dtype == SL_F8_E4M3 && (args->sfa.dtype == SL_F32 || args->sfb.dtype == SL_F32);
}
sl_status plan_block(const sl_gemm_args* args, BlockPlan* out);
sl_status run_block(const sl_gemm_args* args, void* stream);

struct RowsPlan {
  sl_plan pub;
  DenseParams p;
  DensePlan tile;
  bool empty;
};

// a and b int8 with one fp32 scale per row (api_gated.cpp)
inline bool is_int8_gemm(const sl_gemm_args* args) { return args && args->a.dtype == SL_I8; }
sl_status plan_int8(const sl_gemm_args* args, RowsPlan* out);
sl_status run_int8(const sl_gemm_args* args, void* stream);

}  // namespace host
}  // namespace sl
