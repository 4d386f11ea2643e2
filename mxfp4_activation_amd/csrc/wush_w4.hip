// Linear layers with 4-bit weights for a few tokens: Y = X' W^T with W in
// MXFP4, NVFP4 or INT4 as the quantizers and GPTQ-WUSH write it, and X' the
// bf16 activations or their block transform T_c x_c.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"
#include "wush_w4_core.h"

namespace wush {
namespace {

using namespace w4;

// ------------------------------------------------------------ transform
//
// X' = T x per block of G channels in fp32, kept as a sum of bf16 planes:
// y = y0 + y1 (+ y2), each the rounding of what the planes before it left.
// Two planes hold 16 bits of y, three hold all 24.  One wave owns 32 channels
// of 16 tokens.
__global__ __launch_bounds__(256) void split_kernel(SplitArgs a) {
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int64_t panel = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t k0 = panel * 32, K = a.K;
  if (k0 >= K) return;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int64_t mx = m0 + n < a.M ? m0 + n : a.M - 1;
  const uint16_t* x = a.X + mx * a.ldx + k0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x4 av = {0, 0, 0, 0}, bv = {0, 0, 0, 0};
    if (a.G == 32) {
      av = *reinterpret_cast<const u32x4*>(x + 8 * q);
      bv = *reinterpret_cast<const u32x4*>(a.T + panel * 1024 + (16 * h + n) * 32 + 8 * q);
    } else {
      // G = 16: the block fills half of the instruction's 32 columns.
      if (k0 + 16 * h >= K) break;
      if (q < 2) {
        av = *reinterpret_cast<const u32x4*>(x + 16 * h + 8 * q);
        bv = *reinterpret_cast<const u32x4*>(a.T + (2 * panel + h) * 256 + n * 16 + 8 * q);
      }
    }
    const f32x4 y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av),
                                                            __builtin_bit_cast(bf16x8, bv), f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + 4 * q + i;
      if (m >= a.M) continue;
      float v = y[i];
      uint16_t* o = a.out + m * K + k0 + 16 * h + n;
      for (int t = 0; t < a.terms; ++t) {
        const __bf16 b = (__bf16)v;
        o[t * a.M * K] = __builtin_bit_cast(uint16_t, b);
        v -= (float)b;
      }
    }
  }
}

// ------------------------------------------------------------ linear
//
// A workgroup owns 16 R weight rows and up to 16 NT tokens; its W waves split
// K (step s goes to wave s % W, so that together they read contiguous
// stretches of every row) and their sums meet in LDS.
template <int FMT, int R, int NT, int TERMS, int W>
__global__ __launch_bounds__(64 * W) void linear_kernel(LinearArgs a) {
  __shared__ float red[W][R][NT][16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * R), m0 = (int64_t)blockIdx.y * (16 * NT);
  const int64_t K = a.K;
  const int rows = (int)(a.M - m0 < 16 * NT ? a.M - m0 : 16 * NT);

  const uint8_t* cp[R];
  const uint8_t* sp[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t row = n0 + 16 * r + n < a.N ? n0 + 16 * r + n : a.N - 1;
    cp[r] = a.codes + row * row_code_bytes<FMT>(K);
    sp[r] = a.scales + row * row_scale_bytes<FMT>(K);
  }
  const uint16_t* xp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xp[t] = a.x.X + (m0 + (16 * t + n < rows ? 16 * t + n : 0)) * a.x.ldx;
  f32x4 acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};
  wave_dot<FMT, R, NT, TERMS>(acc, cp, sp, xp, a.x.plane, (int)K, wave, W);

#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * t + 4 * q + i < rows) red[wave][r][t][4 * q + i][n] = acc[r][t][i];
  __syncthreads();
  const float g = FMT == kNV ? a.gs[0] : 1.0f;
  for (int o = threadIdx.x; o < rows * 16 * R; o += 64 * W) {
    const int m = o / (16 * R), c = o % (16 * R);
    const int64_t col = n0 + c;
    if (col >= a.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[w][c / 16][m / 16][m % 16][c % 16];
    if (FMT == kNV) v *= g;
    const int64_t at = (m0 + m) * a.N + col;
    if (a.bf16_out) {
      reinterpret_cast<uint16_t*>(a.Y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
    } else {
      reinterpret_cast<float*>(a.Y)[at] = v;
    }
  }
}

template <int FMT, int R, int NT, int TERMS>
hipError_t go(const LinearArgs& a, hipStream_t s) {
  constexpr int W = 8;
  const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R)), (unsigned)((a.M + 16 * NT - 1) / (16 * NT)));
  hipLaunchKernelGGL((linear_kernel<FMT, R, NT, TERMS, W>), grid, dim3(64 * W), 0, s, a);
  return hipGetLastError();
}

template <int FMT, int TERMS>
hipError_t go_tiles(const LinearArgs& a, hipStream_t s) {
  if (a.M <= 16) return go<FMT, 1, 1, TERMS>(a, s);
  if (a.M <= 32) return go<FMT, 2, 2, TERMS>(a, s);
  return go<FMT, 2, 4, TERMS>(a, s);
}

template <int FMT>
hipError_t go_terms(const LinearArgs& a, hipStream_t s) {
  if (a.x.terms == 1) return go_tiles<FMT, 1>(a, s);
  if (a.x.terms == 2) return go_tiles<FMT, 2>(a, s);
  return go_tiles<FMT, 3>(a, s);
}

}  // namespace

hipError_t launch_split(const SplitArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.K + 127) / 128), (unsigned)((a.M + 15) / 16));
  hipLaunchKernelGGL(split_kernel, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_linear_w4(const LinearArgs& a, hipStream_t s) {
  if (a.fmt == kMX) return go_terms<kMX>(a, s);
  if (a.fmt == kNV) return go_terms<kNV>(a, s);
  return go_terms<kINT>(a, s);
}

}  // namespace wush
