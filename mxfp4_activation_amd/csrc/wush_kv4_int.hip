// Attention over a cache in INT4.
#include "wush_kv4_attention.h"

namespace wush {

hipError_t launch_kv4_attention_int(const KvAttnArgs& a, int shape, hipStream_t s) {
  return kv4::launch<w4::kINT>(a, shape, s);
}

}  // namespace wush
