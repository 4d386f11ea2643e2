// Reductions over a wave by data-parallel moves (no LDS, no shuffles).
// Device code only.
#ifndef WUSH_WAVE_H_
#define WUSH_WAVE_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wush {

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}

// The wave's values folded by f, in all lanes.  row_shr 1, 2, 4 and 8 leave each
// row of 16 lanes' result in its lane 15, row_bcast 15 and 31 carry them on to
// lane 63; where a move has no source lane, f sees `none`.
template <typename F>
__device__ __forceinline__ uint32_t fold(uint32_t v, uint32_t none, F f) {
  v = f(v, dpp<0x111, 0xf>(none, v));
  v = f(v, dpp<0x112, 0xf>(none, v));
  v = f(v, dpp<0x114, 0xf>(none, v));
  v = f(v, dpp<0x118, 0xf>(none, v));
  v = f(v, dpp<0x142, 0xa>(none, v));
  v = f(v, dpp<0x143, 0xc>(none, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ int wave_max_int(int v) {
  return (int)fold((uint32_t)v, 0x80000000u, [](uint32_t a, uint32_t b) { return (int)a > (int)b ? a : b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return __uint_as_float(fold(__float_as_uint(v), 0xFF800000u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(fold(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

}  // namespace wush

#endif  // WUSH_WAVE_H_
