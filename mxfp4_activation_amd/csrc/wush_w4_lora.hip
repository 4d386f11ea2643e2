// Low-rank adapters beside the linear layers with 4-bit weights: what they add, and the
// product that takes it up.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"
#include "wush_w4_core.h"
#include "wush_w4_linear.h"
#include "wush_wave.h"

namespace wush {
namespace {

// h[m] = scale A x[m] of the token's adapter.  A workgroup takes kLoraRows rows of A for
// one token; its waves share the row.  Tokens of one adapter read the same rows, from the
// cache after the first.
constexpr int kLoraRows = 4;

__device__ __forceinline__ void lora_rows(const LoraArgs& a, int64_t m, int r0, float (*sums)[4]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t id = a.ids[m];
  if (id < 0 || id >= a.E) return;
  const uint16_t* x = a.X + m * a.ldx;
  const uint16_t* A = a.A + (id * a.rank + r0) * a.K;
  float s[kLoraRows] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t k = wave * 512 + lane * 8; k < a.K; k += 2048) {
    const u32x4 xv = *reinterpret_cast<const u32x4*>(x + k);
    u32x4 w[kLoraRows];
#pragma unroll
    for (int r = 0; r < kLoraRows; ++r) w[r] = *reinterpret_cast<const u32x4*>(A + r * a.K + k);
#pragma unroll
    for (int r = 0; r < kLoraRows; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r] = __builtin_fmaf(bf16_lo(w[r][i]), bf16_lo(xv[i]), s[r]);
        s[r] = __builtin_fmaf(bf16_hi(w[r][i]), bf16_hi(xv[i]), s[r]);
      }
  }
#pragma unroll
  for (int r = 0; r < kLoraRows; ++r) {
    s[r] = wave_sum(s[r]);
    if (lane == 0) sums[r][wave] = s[r];
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < kLoraRows) {
    const float v = (sums[t][0] + sums[t][1]) + (sums[t][2] + sums[t][3]);
    a.h[m * a.rank + r0 + t] = v * (a.scale ? a.scale[id] : 1.0f);
  }
}

// The transform's workgroups, if any, then the adapters': one launch.  3.0 us for one token of
// 4096 channels and rank 16, 5.1 for 64 and rank 32: a round trip to memory and a reduction.
__global__ __launch_bounds__(256) void lora_kernel(LoraArgs a, SplitArgs t, int panels, int split) {
  __shared__ float sums[kLoraRows][4];
  const int b = blockIdx.x;
  if (b < split) {
    const int64_t panel = (int64_t)(b % panels) * 4 + (threadIdx.x >> 6);
    if (panel * 32 < t.K) split_panel(t, panel, (int64_t)(b / panels) * 16);
    return;
  }
  const int per = a.rank / kLoraRows;
  lora_rows(a, (b - split) / per, (b - split) % per * kLoraRows, sums);
}

// v plus the values of the other lanes of its aligned group of 1 << LOG2 lanes.  (Once
// pairs and quads agree, mirroring a half row or row serves as well as an exchange.)
template <int LOG2>
__device__ __forceinline__ float sum_group(float v) {
  const auto plus = [&](uint32_t o) { v += __uint_as_float(o); };
  if (LOG2 > 0) plus(dpp<0xB1, 0xf>(0, __float_as_uint(v)));   // quad_perm 1 0 3 2
  if (LOG2 > 1) plus(dpp<0x4E, 0xf>(0, __float_as_uint(v)));   // quad_perm 2 3 0 1
  if (LOG2 > 2) plus(dpp<0x141, 0xf>(0, __float_as_uint(v)));  // row_half_mirror
  if (LOG2 > 3) plus(dpp<0x140, 0xf>(0, __float_as_uint(v)));  // row_mirror
  if (LOG2 > 4) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if (LOG2 > 5) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// delta[m][n] = B[ids[m]] h[m]; -0 without an adapter, NaN for one that is not there.  A row of B is read by 1 << LOG2
// neighbouring lanes, 16 bytes each, so that a wave reads whole lines, kLoraBlocks times 1 KB at
// a time; the lanes of a row add up.  Many small waves: B is most of what a batch over many
// adapters reads, and the product's own workgroups are too few to wait for it.  64 tokens,
// 40 adapters of rank 32, N = 24576: 13.5 us, 49 MB of B at 3.6 TB/s.
constexpr int kLoraBlocks = 4;
template <int LOG2>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a, int64_t N) {
  constexpr int kPer = 64 >> LOG2;  // rows of a wave's load
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m = blockIdx.y, id = a.ids[m];
  const bool with = id >= 0 && id < a.E;
  const int piece = lane & ((1 << LOG2) - 1), pieces = a.rank / 8;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave) * (kPer * kLoraBlocks) + (lane >> LOG2);
  if (!with) {
    const float none = id < 0 ? -0.0f : __builtin_nanf("");
#pragma unroll
    for (int u = 0; u < kLoraBlocks; ++u)
      if (piece == 0 && n0 + u * kPer < N) a.delta[m * N + n0 + u * kPer] = none;
    return;
  }
  f32x4 h0 = {0, 0, 0, 0}, h1 = {0, 0, 0, 0};
  if (piece < pieces) {
    h0 = *reinterpret_cast<const f32x4*>(a.h + m * a.rank + 8 * piece);
    h1 = *reinterpret_cast<const f32x4*>(a.h + m * a.rank + 8 * piece + 4);
  }
  u32x4 w[kLoraBlocks];
#pragma unroll
  for (int u = 0; u < kLoraBlocks; ++u) {
    const int64_t n = n0 + u * kPer < N ? n0 + u * kPer : N - 1;
    w[u] = *reinterpret_cast<const u32x4*>(a.B + (id * N + n) * a.rank + 8 * (piece < pieces ? piece : 0));
  }
#pragma unroll
  for (int u = 0; u < kLoraBlocks; ++u) {
    const float v = sum_group<LOG2>(piece < pieces ? dot8(w[u], h0, h1) : 0.0f);
    if (piece == 0 && n0 + u * kPer < N) a.delta[m * N + n0 + u * kPer] = v;
  }
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, const SplitArgs* t, hipStream_t s) {
  const int64_t panels = t ? (t->K + 127) / 128 : 1, split = t ? panels * ((t->M + 15) / 16) : 0;
  const int64_t groups = split + a.M * (a.rank / kLoraRows);
  if (groups > INT32_MAX) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(lora_kernel, dim3((unsigned)groups), dim3(256), 0, s, a, t ? *t : SplitArgs{}, (int)panels, (int)split);
  return hipGetLastError();
}

namespace {
template <int LOG2>
hipError_t expand(const LoraArgs& a, int64_t N, hipStream_t s) {
  constexpr int kRows = 4 * kLoraBlocks * (64 >> LOG2);
  hipLaunchKernelGGL(lora_expand_kernel<LOG2>, dim3((unsigned)((N + kRows - 1) / kRows), (unsigned)a.M), dim3(256), 0, s, a, N);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_lora_expand(const LoraArgs& a, int64_t N, hipStream_t s) {
  const int pieces = a.rank / 8;
  if (pieces == 1) return expand<0>(a, N, s);
  if (pieces == 2) return expand<1>(a, N, s);
  if (pieces <= 4) return expand<2>(a, N, s);
  if (pieces <= 8) return expand<3>(a, N, s);
  if (pieces <= 16) return expand<4>(a, N, s);
  if (pieces <= 32) return expand<5>(a, N, s);
  return expand<6>(a, N, s);
}

hipError_t launch_linear_w4_lora(const LinearArgs& a, hipStream_t s) { return go_format<true>(a, s); }

}  // namespace wush
