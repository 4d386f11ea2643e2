// Linear layers with 4-bit weights for a few tokens: Y = X' W^T with W in
// MXFP4, NVFP4 or INT4 as the quantizers and GPTQ-WUSH write it, and X' the
// bf16 activations or their block transform T_c x_c.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"
#include "wush_w4_core.h"
#include "wush_w4_linear.h"

namespace wush {
namespace {

using namespace w4;

// ------------------------------------------------------------ transform
//
// x' = T x once per call, as bf16 planes (split_panel), rather than by every
// workgroup that reads x': at 24576 weight rows there are 768 of them.  Each wave
// takes 32 channels of 16 tokens, so that one token still has K / 32 waves.  Bound
// by its latency: 4.1 us for 4 tokens of 4096, which read 0.3 MB.
__global__ __launch_bounds__(256) void split_kernel(SplitArgs a) {
  const int64_t panel = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (panel * 32 < a.K) split_panel(a, panel, (int64_t)blockIdx.y * 16);
}

}  // namespace

hipError_t launch_split(const SplitArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.K + 127) / 128), (unsigned)((a.M + 15) / 16));
  hipLaunchKernelGGL(split_kernel, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_linear_w4(const LinearArgs& a, hipStream_t s) {
  return a.lora.ids ? launch_linear_w4_lora(a, s) : go_format<false>(a, s);
}

}  // namespace wush
