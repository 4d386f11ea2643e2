// Conversions to and from the 4-bit formats' elements and scales, shared by the
// quantizers (wush_kernels.hip) and the cache (wush_kv4.hip).  Device code only.
#ifndef WUSH_CODEC_H_
#define WUSH_CODEC_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wush {

// E2M1 conversion of a pair: v_cvt_scalef32_pk_fp4_f32 divides both values
// by 2^(exponent field of `scale`), rounds to nearest even, saturates at +-6,
// keeps the sign of zero and writes a byte (first value in the low nibble)
// into byte BYTE of `old`.  With scale = 1.0 it is plain E2M1 rounding.
template <int BYTE>
__device__ __forceinline__ uint32_t cvt_e2m1x2(uint32_t old, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, BYTE);
}

// OCP E4M3FN code of a non-negative finite x: nearest, ties to even, with
// saturation at 448 (code 126).
__device__ __forceinline__ uint32_t e4m3_code(float x) {
  if (x >= 448.0f) return 126u;
  if (x < 0.015625f) {  // below 2^-6: subnormal grid, step 2^-9
    return (uint32_t)__builtin_rintf(x * 512.0f);  // 0..8; 8 is 2^-6 = code 8
  }
  uint32_t b = __float_as_uint(x);
  b = b + 0x7FFFFu + ((b >> 20) & 1u);  // round mantissa to 3 bits, ties to even
  uint32_t c = (b >> 20) - (120u << 3);  // rebias exponent 127 -> 7
  return c > 126u ? 126u : c;
}

__device__ __forceinline__ float e4m3_value(uint32_t c) {
  uint32_t e = c >> 3, m = c & 7u;
  if (e == 0) return (float)m * 0.001953125f;  // m * 2^-9
  return __uint_as_float(((e + 120u) << 23) | (m << 20));
}

// x is rounded to fp32 before: behind an FMA the compiler would otherwise
// round its unrounded sum to fp16 at once (v_fma_mixlo_f16), and a quotient
// half way between two fp16 numbers by way of div7's correction, whose own
// error then decides, would not go to the even one.
__device__ __forceinline__ uint32_t f16_bits(float x) {
  asm("" : "+v"(x));
  _Float16 h = (_Float16)x;  // v_cvt_f16_f32: round to nearest even
  return (uint32_t)__builtin_bit_cast(uint16_t, h);
}

__device__ __forceinline__ float f16_value(uint32_t b) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
}

// fp32(x / 7), the correctly rounded quotient, for finite x >= 0: the
// product with fp32(1/7) and one FMA correction of its residual.  Equal to
// the IEEE quotient for every non-negative finite fp32 x, subnormals
// included (checked exhaustively on the host), at three instructions
// instead of the ten of a division.
__device__ __forceinline__ float div7(float x) {
  constexpr float r = 1.0f / 7.0f;
  const float q = x * r;
  return __builtin_fmaf(__builtin_fmaf(-q, 7.0f, x), r, q);
}

// fp32(1 / s) for s the value of a positive finite fp16 number: the
// hardware reciprocal with one FMA correction.  Equal to the IEEE quotient
// for every such s (checked exhaustively on the device against its own
// division and against the host's).
__device__ __forceinline__ float recip_f16_value(float s) {
  const float r0 = __builtin_amdgcn_rcpf(s);
  return __builtin_fmaf(__builtin_fmaf(-s, r0, 1.0f), r0, r0);
}

}  // namespace wush

#endif  // WUSH_CODEC_H_
