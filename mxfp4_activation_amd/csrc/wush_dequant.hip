// Dequantization of the three 4-bit formats back to fp32.
//
// Used to evaluate the layerwise loss of joint weight-activation
// quantization ("WUSH: Near-Optimal Adaptive Transforms for LLM
// Quantization", deep dive, section 3.4.1, Eq. 5): the quantized product
// q(T_W W)^T q(T_X X) needs the values the codes stand for.
//
// Value of element k of group c in row m:
//   MXFP4  e2m1(code) * 2^(E8M0 - 127)
//   NVFP4  e2m1(code) * fp32(E4M3(scale) * g)
//   INT4   int4(code) * fp16(scale)
// Rows are whole groups, so codes and scales are taken as they lie.  Writing bounds it: a lane
// takes four neighbouring elements, so that a wave writes whole lines, 1 KB per store.  8256 x
// 8 rows of 128 (33.8 MB written, 4.5 read) take 7.7 us (5.0 TB/s); with 16 neighbouring elements
// per lane, whose stores each touch 64 lines, 14.6.
#include <hip/hip_runtime.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "wush_dequant.h"

namespace wush {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float e4m3_value(uint32_t c) {
  // OCP E4M3FN, bias 7, subnormals for exponent 0; only non-negative codes occur.
  const uint32_t e = (c >> 3) & 15u, m = c & 7u;
  return e == 0 ? ldexpf((float)m, -9) : ldexpf((float)(8u + m), (int)e - 10);
}

__device__ __forceinline__ float int4_value(uint32_t nib) { return (float)((int)(nib << 28) >> 28); }

// Stores of a lane, and elements of a workgroup.
constexpr int kStores = 4, kBlock = 256 * 4 * kStores;

template <int FMT>
__global__ __launch_bounds__(256) void dequant_kernel(const uint8_t* __restrict__ codes, const void* __restrict__ scales,
                                                     const float* __restrict__ gs, int64_t total, float* __restrict__ out) {
  constexpr int G = FMT == 1 ? 16 : 32;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t base = (int64_t)blockIdx.x * kBlock + wave * (kBlock / 4) + lane * 4;
  const float g = FMT == 1 ? gs[0] : 1.0f;
  uint32_t w[kStores], b[kStores];
#pragma unroll
  for (int u = 0; u < kStores; ++u) {
    // (Behind the end: the last four, which no one stores twice.)
    const int64_t k = base + 256 * u < total ? base + 256 * u : total - 4;
    w[u] = *reinterpret_cast<const uint16_t*>(codes + k / 2);
    b[u] = FMT == 2 ? static_cast<const uint16_t*>(scales)[k / G] : static_cast<const uint8_t*>(scales)[k / G];
  }
#pragma unroll
  for (int u = 0; u < kStores; ++u) {
    float s;
    f32x4 v;
    if (FMT == 2) {
      s = __half2float(__ushort_as_half((uint16_t)b[u]));
      v = f32x4{int4_value(w[u]), int4_value(w[u] >> 4), int4_value(w[u] >> 8), int4_value(w[u] >> 12)};
    } else {
      s = FMT == 0 ? ldexpf(1.0f, (int)b[u] - 127) : e4m3_value(b[u]) * g;
      const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0);
      const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1);
      v = f32x4{lo[0], lo[1], hi[0], hi[1]};
    }
    const int64_t k = base + 256 * u;
    if (k < total) *reinterpret_cast<f32x4*>(out + k) = f32x4{v[0] * s, v[1] * s, v[2] * s, v[3] * s};
  }
}

}  // namespace

hipError_t launch_dequant(int fmt, const uint8_t* codes, const void* scales, const float* gs, int64_t M, int64_t K,
                          float* out, hipStream_t s) {
  const int64_t total = M * K;
  const dim3 grid((unsigned)((total + kBlock - 1) / kBlock)), block(256);
  if (fmt == 0) hipLaunchKernelGGL((dequant_kernel<0>), grid, block, 0, s, codes, scales, gs, total, out);
  else if (fmt == 1) hipLaunchKernelGGL((dequant_kernel<1>), grid, block, 0, s, codes, scales, gs, total, out);
  else hipLaunchKernelGGL((dequant_kernel<2>), grid, block, 0, s, codes, scales, gs, total, out);
  return hipGetLastError();
}

}  // namespace wush
