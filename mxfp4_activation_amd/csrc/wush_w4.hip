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
// x' = T x once per call, as bf16 planes (split_panel), rather than by every
// workgroup that reads x': at 24576 weight rows there are 768 of them.  Each wave
// takes 32 channels of 16 tokens, so that one token still has K / 32 waves.  Bound
// by its latency: 4.1 us for 4 tokens of 4096, which read 0.3 MB.
__global__ __launch_bounds__(256) void split_kernel(SplitArgs a) {
  const int64_t panel = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (panel * 32 < a.K) split_panel(a, panel, (int64_t)blockIdx.y * 16);
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
  for (int o = threadIdx.x; o < rows * kRows; o += 64 * WN * WK) {
    const int m = o / kRows, c = o % kRows;
    if (n0 + c >= a.N) continue;
    float v = group_sum<R, WN, WK>(lds, c, m, rows);
    if (FMT == kNV) v *= g;
    const int64_t at = (m0 + m) * a.N + n0 + c;
    if (a.bf16_out) {
      reinterpret_cast<uint16_t*>(a.Y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
    } else {
      reinterpret_cast<float*>(a.Y)[at] = v;
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

hipError_t launch_linear_w4(const LinearArgs& a, hipStream_t s) {
  if (a.fmt == kMX) return go_terms<kMX>(a, s);
  if (a.fmt == kNV) return go_terms<kNV>(a, s);
  return go_terms<kINT>(a, s);
}

}  // namespace wush
