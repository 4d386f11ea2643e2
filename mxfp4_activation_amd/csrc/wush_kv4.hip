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

// The lane's eight values as codes, and its group's scale bits (as the quantizers
// have them: include/wush.h).
template <int FMT>
__device__ __forceinline__ uint32_t encode(const float (&y)[8], float amax, float g, uint32_t& scale) {
  uint32_t w = 0;
  if constexpr (FMT == kINT4) {
    scale = f16_bits(div7(amax));
    const bool usable = (scale & 0x7FFFu) != 0u && (scale & 0x7C00u) != 0x7C00u;
    const float r = usable ? recip_f16_value(f16_value(scale)) : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // After adding 1.5 * 2^23 the low bits of the sum are the rounded integer.
      const float v = fminf(fmaxf(y[k] * r, -7.0f), 7.0f) + 12582912.0f;
      w |= (__float_as_uint(v) & 15u) << (4 * k);
    }
  } else {
    float v[8], div;
    if constexpr (FMT == kMXFP4) {
      const int eb = (int)(__float_as_uint(amax) & 0x7F800000u) - (2 << 23);
      const uint32_t sc = (uint32_t)(eb > 0 ? eb : 0);
      scale = sc >> 23;
      div = __uint_as_float(sc);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = y[k];
    } else {
      scale = g > 0.0f ? e4m3_code((amax / 6.0f) / g) : 0u;
      const float eff = e4m3_value(scale) * g;
      const float r = g > 0.0f && eff > 0.0f ? 1.0f / eff : 0.0f;
      div = 1.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = y[k] * r;
    }
    w = cvt_e2m1x2<0>(w, v[0], v[1], div);
    w = cvt_e2m1x2<1>(w, v[2], v[3], div);
    w = cvt_e2m1x2<2>(w, v[4], v[5], div);
    w = cvt_e2m1x2<3>(w, v[6], v[7], div);
  }
  return w;
}

// A wave takes a panel of 32 channels of one head and, of its tokens, 16 at a time:
// lane (n = lane % 16, q = lane / 16) holds channels 8 q .. 8 q + 7 of token n.
//
// With a transform the values are rounded to 4 bits next, so sums have to be close
// enough to the exact ones for the rounding to be theirs: they are formed in float64 on
// the matrix cores, y = fp32(sum).  (The quantizers instead bound the error of fp32
// sums and recompute what lies near a border, which pays at their sizes.)
// v_mfma_f64_16x16x4: A[i][k] in lane (i, k), B[k][j] in lane (j, k), D[4 r + q][j] in
// register r of lane (j, q).  Instruction s takes channels 8 k + s, which lane (n, k) of B
// holds, and row i of half hf stands for output 8 (i % 4) + 4 hf + i / 4, so that
// lane (n, q) gets outputs 8 q .. 8 q + 7.  Two blocks of 16 stand block-diagonally.
template <int FMT, bool TRANSFORM>
__global__ __launch_bounds__(256) void kv4_append_kernel(KvAppendArgs a) {
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
  double t[2][8];
  const bool transform = TRANSFORM && e.T != nullptr;
  if (transform) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int o = 8 * (n & 3) + 4 * hf + (n >> 2);
      u32x4 w = {0, 0, 0, 0};
      if (G == 32) {
        w = *reinterpret_cast<const u32x4*>(e.T + (((int64_t)h * panels + panel) * 32 + o) * 32 + 8 * q);
      } else if (o / 16 == q / 2) {
        w = *reinterpret_cast<const u32x4*>(e.T + (((int64_t)h * panels + panel) * 32 + o) * 16 + 8 * (q & 1));
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) t[hf][s] = (double)bf16_at(w, s);
    }
  }
  const int64_t limit = a.pages << a.page_log2;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t tok = tile * 16 + n;
    u32x4 x = {0, 0, 0, 0};
    int64_t slot = -1;
    if (tok < a.n) {
      x = *reinterpret_cast<const u32x4*>(e.X + tok * e.ld + (int64_t)h * a.D + panel * 32 + 8 * q);
      slot = a.slots[tok];
    }
    float y[8];
    if (transform) {
      f64x4 d0 = {0, 0, 0, 0}, d1 = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const double b = (double)bf16_at(x, s);
        d0 = __builtin_amdgcn_mfma_f64_16x16x4f64(t[0][s], b, d0, 0, 0, 0);
        d1 = __builtin_amdgcn_mfma_f64_16x16x4f64(t[1][s], b, d1, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        y[r] = (float)d0[r];
        y[4 + r] = (float)d1[r];
      }
    } else {
#pragma unroll
      for (int s = 0; s < 8; ++s) y[s] = bf16_at(x, s);
    }
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < 8; ++s) amax = fmaxf(amax, fabsf(y[s]));
    amax = group_max<G>(amax);
    uint32_t scale;
    const uint32_t w = encode<FMT>(y, amax, g, scale);
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
  // About 8192 waves; a wave that takes several tiles reads its transform once.
  const int64_t want = (8192 + 2 * jobs - 1) / (2 * jobs);
  const dim3 grid((unsigned)(tiles < want ? tiles : want), (unsigned)((jobs + 3) / 4), 2);
  if (a.side[0].T || a.side[1].T) {
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
