// Host stand-ins for the launchers of the cache, the adapters and the logits'
// adjustments (see stubs.cpp).
#include "serving_stubs.h"

wush::KvAppendArgs g_last_append;
wush::KvAttnArgs g_last_attention;
int g_last_shape;
wush::LoraArgs g_last_lora, g_last_expand;
int64_t g_lora_tokens = 0;
wush::AdjustArgs g_last_adjust;

namespace wush {

hipError_t launch_kv4_append(const KvAppendArgs& a, hipStream_t) {
  ++g_launches;
  g_last_append = a;
  return hipSuccess;
}
static hipError_t attention(const KvAttnArgs& a, int shape) {
  ++g_launches;
  g_last_attention = a;
  g_last_shape = shape;
  return hipSuccess;
}
hipError_t launch_kv4_attention_mx(const KvAttnArgs& a, int shape, hipStream_t) { return attention(a, shape); }
hipError_t launch_kv4_attention_nv(const KvAttnArgs& a, int shape, hipStream_t) { return attention(a, shape); }
hipError_t launch_kv4_attention_int(const KvAttnArgs& a, int shape, hipStream_t) { return attention(a, shape); }
hipError_t launch_lora(const LoraArgs& a, const SplitArgs* t, hipStream_t) {
  ++g_launches;
  g_last_lora = a;
  g_lora_tokens += a.M;
  if (t) g_last_split = *t;
  return hipSuccess;
}
hipError_t launch_lora_expand(const LoraArgs& a, int64_t, hipStream_t) {
  ++g_launches;
  g_last_expand = a;
  return hipSuccess;
}
hipError_t launch_adjust(const AdjustArgs& a, hipStream_t) {
  ++g_launches;
  g_last_adjust = a;
  return hipSuccess;
}

}  // namespace wush
