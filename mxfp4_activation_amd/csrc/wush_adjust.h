// Internal interface of the logits' adjustments (wush_adjust.hip) for their
// C-ABI layer (wush_serving_abi.cpp).  Not part of the public ABI.
#ifndef WUSH_ADJUST_H_
#define WUSH_ADJUST_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace wush {

struct AdjustArgs {
  const void* in;  // [R][V], row stride ld_in elements
  void* out;       // [R][V], row stride ld_out; may be in
  int type;        // 0 fp32, 1 bf16, 2 fp16
  int64_t ld_in, ld_out, R, V;
  const int32_t *prompt, *output;  // [R][n_prompt], [R][n_output] or null
  int64_t n_prompt, n_output;
  const float *repetition, *frequency, *presence;  // [R] or null
  const int32_t* bias_ids;  // [R][n_bias] or null
  const float* bias;
  int64_t n_bias;
  const int32_t* allowed;  // bits [R][(V + 31) / 32] or null
};

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t s);

}  // namespace wush

#endif  // WUSH_ADJUST_H_
