// Linear layers with 4-bit weights for a few tokens: Y = X' W^T with W in
// MXFP4, NVFP4 or INT4 as the quantizers and GPTQ-WUSH write it, and X' the
// bf16 activations or their block transform T_c x_c.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"
#include "wush_w4_core.h"
#include "wush_wave.h"

namespace wush {
namespace {

using namespace w4;

// ------------------------------------------------------------ transform
//
// x' = T x once per call, as bf16 planes (split_panel), rather than by every
// workgroup that reads x': at 24576 weight rows there are 768 of them.  Each wave
// takes 32 channels of 16 tokens, so that one token still has K / 32 waves.  Bound
// by its latency: 4.1 us for 4 tokens of 4096, which read 0.3 MB.
__global__ __launch_bounds__(256) void split_kernel(SplitArgs a) {
  const int64_t panel = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (panel * 32 < a.K) split_panel(a, panel, (int64_t)blockIdx.y * 16);
}

// ------------------------------------------------------------ adapters
//
// h[m] = scale A x[m] of the token's adapter.  A workgroup takes kLoraRows rows of A for
// one token; its waves share the row.  Tokens of one adapter read the same rows, from the
// cache after the first.
constexpr int kLoraRows = 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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

__device__ __forceinline__ float dot8(const u32x4& w, const f32x4& h0, const f32x4& h1) {
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v = __builtin_fmaf(bf16_lo(w[k]), k < 2 ? h0[2 * k] : h1[2 * k - 4], v);
    v = __builtin_fmaf(bf16_hi(w[k]), k < 2 ? h0[2 * k + 1] : h1[2 * k - 3], v);
  }
  return v;
}

// delta[m][n] = B[ids[m]] h[m]; 0 without an adapter, NaN for one that is not there.  A row of B is read by 1 << LOG2
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
    const float none = id < 0 ? 0.0f : __builtin_nanf("");
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

// What token m's adapter adds to result n: nothing without one, NaN for one that is not there.
__device__ __forceinline__ float lora_term(const LoraArgs& a, int64_t N, int64_t m, int64_t n) {
  const int64_t id = a.ids[m];
  if (id < 0) return 0.0f;
  if (id >= a.E) return __builtin_nanf("");
  const uint16_t* b = a.B + (id * N + n) * a.rank;
  const float* h = a.h + m * a.rank;
  float v = 0.0f;
  for (int r = 0; r < a.rank; r += 8)
    v += dot8(*reinterpret_cast<const u32x4*>(b + r), *reinterpret_cast<const f32x4*>(h + r), *reinterpret_cast<const f32x4*>(h + r + 4));
  return v;
}

// ------------------------------------------------------------ linear
//
// A workgroup owns 16 R WN weight rows and up to 16 NT tokens; group_dot
// (wush_w4_core.h) says how it multiplies.  Bound by the weights' way in where tokens are
// few, and behind that by unpacking them, which every workgroup does once per 16 NT
// tokens: NT grows with the tokens.  Measured without T:
//   1 token:   4096 x 4096 MXFP4 4.2 us (2.1 TB/s: a launch and two round trips to
//              memory), 24576 x 4096 11.5 us (4.7 TB/s), 8192 x 28672 26.2 us (4.8 TB/s),
//              INT4 39 us with T (3.4 TB/s; waves wait for 53% of their cycles,
//              vector instructions take 31% of the time, the matrix cores 27%)
//   13 tokens: 5003 x 5136 NVFP4 11.1 us (1.3 TB/s: 157 workgroups for 256 compute units)
//   64 tokens: 57344 x 8192 MXFP4 99 us (605 TFLOP/s, 2.5 TB/s: two waves per SIMD wait
//              for each other's chunks and for weights not asked for ahead; matrix cores
//              23% busy; 87 us of it remain at 17 tokens), NVFP4 115, INT4 140
template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, int WN, int WK>
__global__ __launch_bounds__(64 * WN * WK, (min_waves<FMT, R, NT, TERMS>())) void linear_kernel(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  constexpr int kRows = 16 * R * WN;
  const int wn = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WN;
  constexpr int kTokens = SPREAD ? 4 : 16 * NT;
  const int64_t n0 = (int64_t)blockIdx.x * kRows, m0 = (int64_t)blockIdx.y * kTokens;
  const int rows = (int)(a.M - m0 < kTokens ? a.M - m0 : kTokens);
  const auto p = make_rows<FMT, R, D>(
      a.codes, a.scales, a.K, [&](int r) { return n0 + 16 * (wn * R + r) < a.N ? n0 + 16 * (wn * R + r) : a.N - 1; },
      [&](int) { return a.N - 1; });
  const uint16_t* X = a.x.X + m0 * a.x.ldx;
  const int64_t ldx = a.x.ldx;
  group_dot<FMT, R, D, NT, TERMS, SPREAD, WN, WK>(
      lds, p, [] {}, [&](int row) { return X + row * ldx; }, a.x.plane, rows, a.K);
  const float g = FMT == kNV ? a.gs[0] : 1.0f;
  constexpr int kThreads = 64 * WN * WK;
  const auto result = [&](int o, auto more) {
    const int m = o / kRows, c = o % kRows;
    if (n0 + c >= a.N) return;
    float v = group_sum<R, WN, WK>(lds, c, m, rows);
    if (FMT == kNV) v *= g;
    v = more(v, m0 + m, n0 + c);
    const int64_t at = (m0 + m) * a.N + n0 + c;
    if (a.bf16_out) {
      reinterpret_cast<uint16_t*>(a.Y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
    } else {
      reinterpret_cast<float*>(a.Y)[at] = v;
    }
  };
  if (!a.lora.ids) {
    for (int o = threadIdx.x; o < rows * kRows; o += kThreads) result(o, [](float v, int64_t, int64_t) { return v; });
  } else if (!a.lora.delta) {
    for (int o = threadIdx.x; o < rows * kRows; o += kThreads)
      result(o, [&](float v, int64_t m, int64_t n) { return v + lora_term(a.lora, a.N, m, n); });
  } else {
    // Four results' parts asked for at a time: one by one they cost 12 of 54 us (64 tokens,
    // 24576 x 4096 NVFP4).
    for (int o0 = threadIdx.x; o0 < rows * kRows; o0 += 4 * kThreads) {
      float d[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int o = o0 + u * kThreads, m = o / kRows, c = o % kRows;
        d[u] = o < rows * kRows && n0 + c < a.N ? a.lora.delta[(m0 + m) * a.N + n0 + c] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (o0 + u * kThreads < rows * kRows)
          result(o0 + u * kThreads, [&](float v, int64_t, int64_t) { return v + d[u]; });
    }
  }
}

template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, int WN, int WK>
hipError_t go(const LinearArgs& a, hipStream_t s) {
  constexpr int kTokens = SPREAD ? 4 : 16 * NT;
  const dim3 grid((unsigned)((a.N + 16 * R * WN - 1) / (16 * R * WN)), (unsigned)((a.M + kTokens - 1) / kTokens));
  const int rows = (int)(a.M < kTokens ? a.M : kTokens);
  return launch_lds(linear_kernel<FMT, R, D, NT, TERMS, SPREAD, WN, WK>, grid, 64 * WN * WK,
                    lds_bytes<R, D, NT, TERMS, WN, WK>(rows, a.K), s, a);
}

constexpr int64_t kLds = 163840;

// Which shape of workgroup.  What counts is how many there are (256 compute
// units want a few waves each), how many row tiles share the activations' way
// through LDS, and that way's share of LDS.  Measured on both sides of each bound (us;
// MXFP4, K = 4096, without and with T; a call of a few us is the host's), R x D units
// and WN x WK waves:
//   up to 4 tokens, N 12288: 12288 x 1 token 1x2, 1x8 9.6, 2x2, 1x4 9.6; 4 tokens 9.0, 9.9
//     (NVFP4 10.2, 12.6; INT4 11.2, 12.0); 16384 x 4 10.8, 10.5 (14.1, 13.2; 13.3, 12.5);
//     24576 x 4 15.1, 14.3, with T 24.1, 19.9.
//   13 tokens, all 4608: 4096 rows 1x2, 1x8 9.0, 2x1, 1x8 9.1; 6144 9.6, 9.3 (NVFP4 11.0, 9.9;
//     INT4 11.3, 9.9).  8192: 8192 rows 2x1, 1x8 9.2, 2x2, 2x4 10.4; 12288 15.4, 12.2.
//     16384: 16384 rows 2x2, 2x4 12.7, 2x2, 2x2 13.6; 24576 19.8, 19.1, with T 31.2, 27.6.
//   17 tokens and more, all 32768 (rows x token tiles), 2x2 units and waves against the best of
//     the wider tiles: 16384 x 32 17.8 against 24.0, with T 35.6 against 55.6; 8192 x 64
//     15.7 against 23.4, 32.8 against 48.0 (NVFP4 20.3, 28.3; INT4 20.2, 31.9); 12288 x 64
//     24.5 against 26.3, 47.0 against 54.3; 16384 x 64 30.4 against 26.8, 60.6 against 55.2;
//     4096 x 128 15.7 against 23.3, 32.7 against 48.7.
//   6 and 16 tokens with T, 24576 rows, 4x1, 2x4 against 2x2, 2x2: 26.0 and 28.5 against 23.1
//     and 36.1; 40960 rows 40.2 and 49.9 against 31.4 and 50.6.
//   33 to 64 tokens, N 16384: 16384 x 48 four token tiles 21.8, two 25.7; 20480 x 48 39.4, 27.1.
//     N 32768: 32768 x 64 two token tiles 37.3, four 50.8; 40960 x 64 52.7, 51.7 (INT4
//     66.1, 71.0); 57344 x 8192 x 64 four 97.6, two 134.
template <int FMT, int TERMS>
hipError_t go_tiles(const LinearArgs& a, hipStream_t s) {
  const int64_t K = a.K, N = a.N;
  const int rows = (int)(a.M < 16 ? a.M : 16);
  if (a.M <= 4) {
    if (N > 12288) return go<FMT, 2, 2, 1, TERMS, true, 1, 4>(a, s);
    if (lds_bytes<1, 2, 1, TERMS, 1, 8>(rows, K) <= kLds / 2) return go<FMT, 1, 2, 1, TERMS, true, 1, 8>(a, s);
    return go<FMT, 1, 1, 1, TERMS, true, 1, 8>(a, s);
  }
  const int64_t all = N * ((a.M + 15) / 16);  // weight rows, once per token tile
  if (all <= 4608 && lds_bytes<1, 2, 1, TERMS, 1, 8>(rows, K) <= kLds / 2)
    return go<FMT, 1, 2, 1, TERMS, false, 1, 8>(a, s);
  if (all <= 8192 && lds_bytes<2, 1, 1, TERMS, 1, 8>(rows, K) <= kLds)
    return go<FMT, 2, 1, 1, TERMS, false, 1, 8>(a, s);
  if (all <= 16384 && lds_bytes<2, 2, 1, TERMS, 2, 4>(rows, K) <= kLds)
    return go<FMT, 2, 2, 1, TERMS, false, 2, 4>(a, s);
  if (all <= (a.M <= 16 ? 16384 : 32768) || (a.M <= 16 && TERMS == 1)) return go<FMT, 2, 2, 1, TERMS, false, 2, 2>(a, s);
  if (a.M <= 16) return go<FMT, 4, 1, 1, TERMS, false, 2, 4>(a, s);
  if constexpr (TERMS > 1) {
    return go<FMT, 4, 1, 2, TERMS, false, 4, 2>(a, s);
  } else {
    if (a.M <= 32) return go<FMT, 4, 1, 2, 1, false, 2, 4>(a, s);
    if (N <= 16384 && lds_bytes<2, 1, 4, 1, 2, 4>((int)(a.M < 64 ? a.M : 64), K) <= kLds)
      return go<FMT, 2, 1, 4, 1, false, 2, 4>(a, s);
    if (N <= 32768) return go<FMT, 2, 2, 2, 1, false, 4, 1>(a, s);
    return go<FMT, 2, 2, 4, 1, false, 8, 1>(a, s);
  }
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

hipError_t launch_linear_w4(const LinearArgs& a, hipStream_t s) {
  if (a.fmt == kMX) return go_terms<kMX>(a, s);
  if (a.fmt == kNV) return go_terms<kNV>(a, s);
  return go_terms<kINT>(a, s);
}

}  // namespace wush
