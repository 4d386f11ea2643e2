// What the stand-ins for the launchers of the cache, the adapters and the logits'
// adjustments recorded last.
#ifndef ABI_HOST_SERVING_STUBS_H_
#define ABI_HOST_SERVING_STUBS_H_

#include "../../mxfp4_activation_amd/csrc/wush_adjust.h"
#include "../../mxfp4_activation_amd/csrc/wush_kv4.h"
#include "decode_stubs.h"

extern wush::KvAppendArgs g_last_append;
extern wush::KvAttnArgs g_last_attention;
extern int g_last_shape;
extern wush::LoraArgs g_last_lora, g_last_expand;
extern int64_t g_lora_tokens;  // summed over the launches
extern wush::AdjustArgs g_last_adjust;

#endif  // ABI_HOST_SERVING_STUBS_H_
