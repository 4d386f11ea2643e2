// What the C-ABI files of the decode entries share: checks of formats, rows,
// weights and workspaces, and the sizes they go by.
#ifndef WUSH_DECODE_CHECKS_H_
#define WUSH_DECODE_CHECKS_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/wush.h"
#include "wush_abi_common.h"
#include "wush_kernels.h"
#include "wush_w4.h"

namespace wush {
namespace decode {

struct Range {
  const void* p;
  uint64_t n;
};

inline bool any_overlap(const Range* outs, int n_outs, const Range* ins, int n_ins) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
    for (int j = i + 1; j < n_outs; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
  }
  return false;
}

inline int group_of(int fmt) { return fmt == kNVFP4 ? 16 : 32; }
inline int scale_bytes_of(int fmt) { return fmt == kINT4 ? 2 : 1; }
inline int out_bytes_of(int out_type) { return out_type == WUSH_OUT_F32 ? 4 : 2; }
// Planes of T x and of the experts' h (split_panel says why two do for bf16).
inline int terms_of(int out_type) { return out_type == WUSH_OUT_F32 ? 3 : 2; }

inline uint64_t round16(uint64_t n) { return (n + 15) / 16 * 16; }
inline uint64_t code_bytes(int64_t rows, int64_t K) { return (uint64_t)rows * K / 2; }
inline uint64_t scale_bytes(int fmt, int64_t rows, int64_t K) {
  return (uint64_t)rows * (K / group_of(fmt)) * scale_bytes_of(fmt);
}

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 27;

inline wush_status check_fmt(int fmt, int out_type) {
  if (fmt != kMXFP4 && fmt != kNVFP4 && fmt != kINT4)
    return fail(WUSH_EUNSUPPORTED, "unknown format %d", fmt);
  if (out_type != WUSH_OUT_F32 && out_type != WUSH_OUT_BF16) return fail(WUSH_EINVAL, "unknown out_type %d", out_type);
  return WUSH_OK;
}

inline wush_status check_width(const char* name, int64_t K, int fmt) {
  if (K <= 0 || K > kMaxK || K % group_of(fmt) != 0)
    return fail(WUSH_EINVAL, "%s must be a positive multiple of %d, at most 2^27 (got %lld)", name, group_of(fmt),
                (long long)K);
  return WUSH_OK;
}

inline wush_status check_rows(const void* X, int64_t ldx, int64_t M, int64_t K) {
  if (!X) return fail(WUSH_EINVAL, "null X");
  if (M > 1 && (ldx < K || ldx > kMaxDim)) return fail(WUSH_EINVAL, "ldx must be K or more, at most 2^30 (got %lld)", (long long)ldx);
  if (!aligned(X, 16) || (M > 1 && ldx % 8 != 0))
    return fail(WUSH_EALIGN, "every row of X must be 16-byte aligned");
  return WUSH_OK;
}

inline wush_status check_weights(const char* name, int fmt, const void* codes, const void* scales, const float* gs) {
  if (!codes || !scales) return fail(WUSH_EINVAL, "null %s codes or scales", name);
  if (fmt == kNVFP4 && !gs) return fail(WUSH_EINVAL, "NVFP4 needs %s's global_scale", name);
  if (!aligned(codes, 8)) return fail(WUSH_EALIGN, "%s codes must be 8-byte aligned", name);
  if (fmt == kINT4 && !aligned(scales, 2)) return fail(WUSH_EALIGN, "%s scales must be 2-byte aligned", name);
  if (fmt == kNVFP4 && !aligned(gs, 4)) return fail(WUSH_EALIGN, "%s global_scale must be 4-byte aligned", name);
  return WUSH_OK;
}

inline wush_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return WUSH_OK;
  if (!ws || have < need)
    return fail(WUSH_EINVAL, "workspace of %lld bytes needed (got %lld)", (long long)need, (long long)(ws ? have : 0));
  if (!aligned(ws, 16)) return fail(WUSH_EALIGN, "workspace must be 16-byte aligned");
  return WUSH_OK;
}

inline wush_status launched(hipError_t e) {
  return e == hipSuccess ? WUSH_OK : fail(WUSH_EHIP, "launch: %s", hipGetErrorString(e));
}

}  // namespace decode
}  // namespace wush

#endif  // WUSH_DECODE_CHECKS_H_
