// What the stand-ins for the decode operators' launchers recorded last.
#ifndef ABI_HOST_DECODE_STUBS_H_
#define ABI_HOST_DECODE_STUBS_H_

#include "../../mxfp4_activation_amd/csrc/wush_w4.h"
#include "stubs.h"

extern wush::SplitArgs g_last_split;
extern wush::LinearArgs g_last_linear;
extern wush::MoeArgs g_last_moe;
extern wush::LogprobArgs g_last_logprobs;
extern int64_t g_moe_tokens;  // summed over the launches

#endif  // ABI_HOST_DECODE_STUBS_H_
