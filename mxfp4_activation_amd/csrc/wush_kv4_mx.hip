// Attention over a cache in MXFP4.
#include "wush_kv4_attention.h"

namespace wush {

hipError_t launch_kv4_attention_mx(const KvAttnArgs& a, int shape, hipStream_t s) {
  return kv4::launch<w4::kMX>(a, shape, s);
}

}  // namespace wush
