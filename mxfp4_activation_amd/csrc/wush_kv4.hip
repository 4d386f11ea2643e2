// Writing keys and values to a cache in 4 bits: optional block transform,
// round-to-nearest AbsMax quantization per group, scattered to the tokens'
// slots.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_codec.h"
#include "wush_kernels.h"
#include "wush_kv4.h"

namespace wush {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf16_at(const u32x4& w, int i) {
  return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
}

// max(v[l], v[l ^ 16]) and then, for groups of 32, also of l ^ 32: the lanes that
// share a group.  Non-negative floats order like their bit patterns.
template <int G>
__device__ __forceinline__ float group_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  uint32_t m = a[0] > a[1] ? a[0] : a[1];
  if (G == 32) {
    const auto b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = b[0] > b[1] ? b[0] : b[1];
  }
  return __uint_as_float(m);
}

// Scale bits of a group (as the quantizers have them: include/wush.h).
template <int FMT>
__device__ __forceinline__ uint32_t scale_bits(float amax, float g) {
  if constexpr (FMT == kINT4) {
    return f16_bits(div7(amax));
  } else if constexpr (FMT == kMXFP4) {
    const int eb = (int)(__float_as_uint(amax) & 0x7F800000u) - (2 << 23);
    return (uint32_t)(eb > 0 ? eb : 0) >> 23;
  } else {
    return g > 0.0f ? e4m3_code((amax / 6.0f) / g) : 0u;
  }
}

// The lane's eight values y(0) .. y(7) as codes of that scale.
template <int FMT, typename Y>
__device__ __forceinline__ uint32_t encode(Y y, uint32_t scale, float g) {
  uint32_t w = 0;
  if constexpr (FMT == kINT4) {
    const bool usable = (scale & 0x7FFFu) != 0u && (scale & 0x7C00u) != 0x7C00u;
    const float r = usable ? recip_f16_value(f16_value(scale)) : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // After adding 1.5 * 2^23 the low bits of the sum are the rounded integer.
      const float v = fminf(fmaxf(y(k) * r, -7.0f), 7.0f) + 12582912.0f;
      w |= (__float_as_uint(v) & 15u) << (4 * k);
    }
  } else {
    float v[8], div = 1.0f;
    if constexpr (FMT == kMXFP4) {
      div = __uint_as_float(scale << 23);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = y(k);
    } else {
      const float eff = e4m3_value(scale) * g;
      const float r = g > 0.0f && eff > 0.0f ? 1.0f / eff : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = y(k) * r;
    }
    w = cvt_e2m1x2<0>(w, v[0], v[1], div);
    w = cvt_e2m1x2<1>(w, v[2], v[3], div);
    w = cvt_e2m1x2<2>(w, v[4], v[5], div);
    w = cvt_e2m1x2<3>(w, v[6], v[7], div);
  }
  return w;
}

// A wave takes a panel of 32 channels of one head and, of its tokens, 16 at a time: lane
// (n = lane % 16, q = lane / 16) holds channels 8 q .. 8 q + 7 of token n.  (A wave per whole
// head, with wider stores, needs 148 registers and took 24.4 us where this takes 22.)
//
// A transformed value is fp32(sum_j T x), and what 4 bits it becomes has to be that value's.
// The sums are formed with v_mfma_f32_16x16x32_bf16, whose rounding is off by at most d: 32
// roundings or truncations, each within 2^-23 of sum |T x|, which a second pair of
// instructions gives; 2^-17 of it covers them and its own error, 2^-21 |y| the rounding to
// fp32, 2^-120 products below the fp32 range.  Scale and codes are formed at both ends of
// [y - d, y + d]; they grow with y, so where they agree they are y's.  Where any of the wave's
// do not (one tile in nine, INT4's fine scales one in two), the tile is summed again in float64.
// 8200 tokens of 8 heads of 128 (MXFP4, both sides transformed) take 22 us, with every sum in
// float64 31 us: half of the waves' time is waiting, a third of it behind float64 sums.
//
// Operands.  v_mfma_f32: row 4 q + r of half hf stands for output 8 q + 4 hf + r.
// v_mfma_f64_16x16x4 (A[i][k] in lane (i, k), B[k][j] in lane (j, k), D[4 r + q][j] in register
// r of lane (j, q)): instruction s takes channels 8 k + s, which lane (n, k) of B holds, and
// row i of half hf stands for output 8 (i % 4) + 4 hf + i / 4.  Either way lane (n, q) gets
// outputs 8 q .. 8 q + 7.  Two blocks of 16 stand block-diagonally.
template <int FMT>
__device__ __forceinline__ u32x4 bank_row(const uint16_t* T, int64_t panel, int o, int q) {
  if (FMT != kNVFP4) return *reinterpret_cast<const u32x4*>(T + (panel * 32 + o) * 32 + 8 * q);
  u32x4 w = {0, 0, 0, 0};
  if (o / 16 == q / 2) w = *reinterpret_cast<const u32x4*>(T + (panel * 32 + o) * 16 + 8 * (q & 1));
  return w;
}

template <int FMT>
__device__ __forceinline__ float amax8(const float (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(y[k]));
  return group_max<FMT == kNVFP4 ? 16 : 32>(m);
}

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                 f32x4{0, 0, 0, 0}, 0, 0, 0);
}

// Waves per SIMD that the registers leave room for.
template <bool TRANSFORM>
constexpr int kAppendWaves = TRANSFORM ? 6 : 8;

template <int FMT, bool TRANSFORM>
__global__ __launch_bounds__(256, kAppendWaves<TRANSFORM>) void kv4_append_kernel(KvAppendArgs a) {
  constexpr int G = FMT == kNVFP4 ? 16 : 32;
  constexpr int kScaleBytes = FMT == kINT4 ? 2 : 1;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int panels = a.D / 32;
  const int job = (int)blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (job >= a.heads * panels) return;
  const int h = job / panels, panel = job % panels;
  const KvAppendSide& e = a.side[blockIdx.z];
  const int64_t tiles = (a.n + 15) / 16;
  const float g = FMT == kNVFP4 ? e.gs[0] : 1.0f;
  const bool transform = TRANSFORM && e.T != nullptr;
  u32x4 t[2];
  if (transform) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) t[hf] = bank_row<FMT>(e.T, job, 8 * (n >> 2) + 4 * hf + (n & 3), q);
  }
  const u32x4 magnitude = {0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};
  const int64_t limit = a.pages << a.page_log2;
  const uint16_t* src = e.X + (int64_t)h * a.D + panel * 32 + 8 * q;
  u32x4 next;
  int64_t next_slot;
  const auto ask = [&](int64_t tile) {
    const int64_t tok = tile * 16 + n;
    next = u32x4{0, 0, 0, 0};
    next_slot = -1;
    if (tok < a.n) {
      next = *reinterpret_cast<const u32x4*>(src + tok * e.ld);
      next_slot = a.slots[tok];
    }
  };
  ask(blockIdx.x);
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const u32x4 x = next;
    const int64_t slot = next_slot;
    ask(tile + gridDim.x);
    float y[8];
    uint32_t scale, w;
    if (transform) {
      float d[8];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const f32x4 v = mfma(t[hf], x), s = mfma(t[hf] & magnitude, x & magnitude);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          y[4 * hf + r] = v[r];
          d[4 * hf + r] = __builtin_fmaf(s[r], 0x1p-17f, __builtin_fmaf(fabsf(v[r]), 0x1p-21f, 0x1p-120f));
        }
      }
      float dmax = d[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) dmax = fmaxf(dmax, d[k]);
      dmax = group_max<G>(dmax);
      const float amax = amax8<FMT>(y);
      scale = scale_bits<FMT>(amax + dmax, g);
      w = encode<FMT>([&](int k) { return y[k] + d[k]; }, scale, g);
      const bool unsure = scale_bits<FMT>(fmaxf(amax - dmax, 0.0f), g) != scale ||
                          encode<FMT>([&](int k) { return y[k] - d[k]; }, scale, g) != w;
      if (__any(unsure)) {
        f64x4 v[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const u32x4 row = bank_row<FMT>(e.T, job, 8 * (n & 3) + 4 * hf + (n >> 2), q);
#pragma unroll
          for (int s = 0; s < 8; ++s)
            v[hf] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)bf16_at(row, s), (double)bf16_at(x, s), v[hf], 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = (float)v[k >> 2][k & 3];
        scale = scale_bits<FMT>(amax8<FMT>(y), g);
        w = encode<FMT>([&](int k) { return y[k]; }, scale, g);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 8; ++s) y[s] = bf16_at(x, s);
      scale = scale_bits<FMT>(amax8<FMT>(y), g);
      w = encode<FMT>([&](int k) { return y[k]; }, scale, g);
    }
    if (slot >= 0 && slot < limit) {
      const int64_t row = (((slot >> a.page_log2) * a.heads + h) << a.page_log2) + (slot & (((int64_t)1 << a.page_log2) - 1));
      *reinterpret_cast<uint32_t*>(e.codes + row * (a.D / 2) + panel * 16 + 4 * q) = w;
      const int group = G == 32 ? panel : 2 * panel + (q >> 1);
      if (G == 32 ? q == 0 : (q & 1) == 0) {
        uint8_t* to = e.scales + (row * (a.D / G) + group) * kScaleBytes;
        if (kScaleBytes == 2) {
          *reinterpret_cast<uint16_t*>(to) = (uint16_t)scale;
        } else {
          *to = (uint8_t)scale;
        }
      }
    }
  }
}

template <int FMT>
hipError_t go(const KvAppendArgs& a, hipStream_t s) {
  const int64_t tiles = (a.n + 15) / 16, jobs = (int64_t)a.heads * (a.D / 32);
  // Waves take as many tiles as lets all of them be there at once: a wave reads its transform
  // once, and a second round of a few waves would cost as much as the first.
  const bool transform = a.side[0].T || a.side[1].T;
  const int64_t columns = (jobs + 3) / 4 * 2;  // workgroups side by side
  const int64_t room = 256 * (transform ? kAppendWaves<true> : kAppendWaves<false>) / columns;
  const int64_t each = room > 0 ? (tiles + room - 1) / room : tiles;
  const dim3 grid((unsigned)((tiles + each - 1) / each), (unsigned)(columns / 2), 2);
  if (transform) {
    hipLaunchKernelGGL((kv4_append_kernel<FMT, true>), grid, dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL((kv4_append_kernel<FMT, false>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(const KvAppendArgs& a, hipStream_t s) {
  if (a.fmt == kMXFP4) return go<kMXFP4>(a, s);
  if (a.fmt == kNVFP4) return go<kNVFP4>(a, s);
  return go<kINT4>(a, s);
}

}  // namespace wush
