// Host stand-ins for the decode operators' launchers (see stubs.cpp).
#include "decode_stubs.h"

wush::SplitArgs g_last_split;
wush::LinearArgs g_last_linear;
wush::MoeArgs g_last_moe;
wush::LogprobArgs g_last_logprobs;
int64_t g_moe_tokens = 0;

namespace wush {

hipError_t launch_split(const SplitArgs& a, hipStream_t) {
  ++g_launches;
  g_last_split = a;
  return hipSuccess;
}
hipError_t launch_linear_w4(const LinearArgs& a, hipStream_t) {
  ++g_launches;
  g_last_linear = a;
  return hipSuccess;
}
hipError_t launch_moe(const MoeArgs& a, hipStream_t) {
  ++g_launches;
  g_last_moe = a;
  g_moe_tokens += a.M;
  return hipSuccess;
}
hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t) {
  ++g_launches;
  g_last_logprobs = a;
  return hipSuccess;
}

}  // namespace wush
