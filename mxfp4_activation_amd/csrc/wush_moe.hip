// A mixture-of-experts layer on 4-bit weights for a few tokens:
//   l = Wr x,  the topk largest l_e (ties: lowest e),  softmax weights w_e,
//   y = sum_e w_e Wd_e T_mid,e (silu(Wg_e x') * (Wu_e x')),  x' = x or T_in x.
// Four launches on one stream: the router's logits; the choice of experts and the
// grouping of tokens by expert; gate, up and their product; down and the
// weighted sum.  Every sum has a fixed order, so results repeat bit for bit.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"
#include "wush_w4_core.h"

namespace wush {
namespace {

using namespace w4;

// ------------------------------------------------------------ router
//
// Logits of 16 experts for 16 tokens per workgroup, K split over the waves.
constexpr int kRouterWaves = 16;

__global__ __launch_bounds__(64 * kRouterWaves) void router_kernel(MoeArgs a) {
  __shared__ float red[kRouterWaves][16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int e0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const int rows = a.M - m0 < 16 ? a.M - m0 : 16;
  const int e = e0 + n < a.E ? e0 + n : a.E - 1;
  const uint8_t* cp[1] = {reinterpret_cast<const uint8_t*>(a.router + e * a.H)};
  const uint8_t* sp[1] = {nullptr};
  const uint16_t* xp[1] = {a.X + (int64_t)(m0 + (n < rows ? n : 0)) * a.ldx};
  f32x4 acc[1][1] = {{f32x4{0, 0, 0, 0}}};
  wave_dot<kBF, 1, 1, 1>(acc, cp, sp, xp, 0, (int)a.H, wave, kRouterWaves);
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][4 * q + i][n] = acc[0][0][i];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
    float v = 0.0f;
    for (int w = 0; w < kRouterWaves; ++w) v += red[w][m][c];
    if (m < rows && e0 + c < a.E) a.logits[(int64_t)(m0 + m) * a.E + e0 + c] = v;
  }
}

// ------------------------------------------------------------ choice
//
// One workgroup.  A wave chooses a token's experts: every lane holds the
// logits of experts lane, lane + 64, ... as keys (ordered logit, then lower
// index first), and the largest key of the wave is taken topk times.  Then
// one thread per expert collects its tokens in order.
constexpr int kRouteThreads = 1024;

// Order-preserving: larger float, larger key; NaN below everything.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v);
  if (v != v) return 0u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

template <int J>  // experts per lane
__global__ __launch_bounds__(kRouteThreads) void route_kernel(MoeArgs a, int tile_tokens) {
  __shared__ int ids[kMoeTokens * kMoeMaxTopK];
  __shared__ int scan_slots[kRouteThreads], scan_tiles[kRouteThreads];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_slots = a.M * a.topk;
  for (int m = wave; m < a.M; m += kRouteThreads / 64) {
    float l[J];
    uint64_t key[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane + 64 * j;
      l[j] = e < a.E ? a.logits[(int64_t)m * a.E + e] : 0.0f;
      key[j] = e < a.E ? ((uint64_t)order_bits(l[j]) << 32) | (0xFFFFFFFFu - (uint32_t)e) : 0u;
    }
    int my_id = 0;
    for (int p = 0; p < a.topk; ++p) {
      uint64_t best = key[0];
#pragma unroll
      for (int j = 1; j < J; ++j) best = key[j] > best ? key[j] : best;
      best = wave_max_u64(best);
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (key[j] == best) key[j] = 0;
      if (lane == p) my_id = (int)(0xFFFFFFFFu - (uint32_t)best);
    }
    const bool mine = lane < a.topk;
    const float lp = mine ? a.logits[(int64_t)m * a.E + my_id] : 0.0f;
    const float top = __shfl(lp, 0);
    const float w = mine ? expf(lp - top) : 0.0f;
    float part = w;
    if (!a.renorm) {
      part = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (lane + 64 * j < a.E) part += expf(l[j] - top);
    }
    const float total = wave_sum(part);
    if (mine) {
      a.ids[m * a.topk + lane] = my_id;
      a.weights[m * a.topk + lane] = w / total;
      ids[m * a.topk + lane] = my_id;
    }
  }
  __syncthreads();
  // Thread e: expert e's slots, in order of the tokens.
  const int e = threadIdx.x;
  int count = 0;
  if (e < a.E)
    for (int s = 0; s < n_slots; ++s) count += ids[s] == e;
  const int tiles = (count + tile_tokens - 1) / tile_tokens;
  scan_slots[e] = count;
  scan_tiles[e] = tiles;
  __syncthreads();
  for (int d = 1; d < kRouteThreads; d <<= 1) {
    const int s = e >= d ? scan_slots[e - d] : 0, t = e >= d ? scan_tiles[e - d] : 0;
    __syncthreads();
    scan_slots[e] += s;
    scan_tiles[e] += t;
    __syncthreads();
  }
  int at = scan_slots[e] - count;
  for (int t = 0; t < tiles; ++t) {
    const int left = count - t * tile_tokens;
    a.tiles[scan_tiles[e] - tiles + t] =
        MoeTile{e, at + t * tile_tokens, left < tile_tokens ? left : tile_tokens, 0};
  }
  if (count > 0)
    for (int s = 0; s < n_slots; ++s)
      if (ids[s] == e) a.slots[at++] = s;
  if (e == kRouteThreads - 1) *a.n_tiles = scan_tiles[e];
}

// ------------------------------------------------------------ gate and up
//
// A workgroup owns 32 channels of h for one tile of tokens of one expert: 32
// gate rows and 32 up rows, K split over the waves.  The 32 channels hold
// whole transform blocks, so T_mid is applied to h right here.
constexpr int kWaves = 8;

template <int FMT, int NT, int TERMS>
__global__ __launch_bounds__(64 * kWaves) void gate_up_kernel(MoeArgs a) {
  __shared__ float red[kWaves][4][NT][16][16];
  if ((int)blockIdx.y >= *a.n_tiles) return;
  const MoeTile tile = a.tiles[blockIdx.y];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int64_t H = a.H, I = a.I, i0 = (int64_t)blockIdx.x * 32;

  const uint8_t* cp[4];
  const uint8_t* sp[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t i = i0 + 16 * (r & 1) + n;
    const int64_t row = (int64_t)tile.expert * (2 * I) + (r < 2 ? 0 : I) + (i < I ? i : I - 1);
    cp[r] = a.gu_codes + row * row_code_bytes<FMT>(H);
    sp[r] = a.gu_scales + row * row_scale_bytes<FMT>(H);
  }
  const uint16_t* xp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int s = a.slots[tile.start + (16 * t + n < tile.count ? 16 * t + n : 0)];
    xp[t] = a.x.X + (int64_t)(s / a.topk) * a.x.ldx;
  }
  f32x4 acc[4][NT];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};
  wave_dot<FMT, 4, NT, TERMS>(acc, cp, sp, xp, a.x.plane, (int)H, wave, kWaves);

#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][r][t][4 * q + i][n] = acc[r][t][i];
  __syncthreads();
  const float gs = FMT == kNV ? a.gu_gs[tile.expert] : 1.0f;
  const int c = threadIdx.x & 31;
  float h[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = threadIdx.x >> 5;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      g += red[w][c >> 4][t][m][c & 15];
      u += red[w][2 + (c >> 4)][t][m][c & 15];
    }
    if (FMT == kNV) {
      g *= gs;
      u *= gs;
    }
    h[t] = g / (1.0f + expf(-g)) * u;
  }
  if (a.T_mid) {
    constexpr int G = FMT == kNV ? 16 : 32;
    __syncthreads();  // everyone has read red
    float(*hs)[16][32] = reinterpret_cast<float(*)[16][32]>(&red[0][0][0][0][0]);
#pragma unroll
    for (int t = 0; t < NT; ++t) hs[t][threadIdx.x >> 5][c] = h[t];
    __syncthreads();
    const int64_t i = i0 + c < I ? i0 + c : I - 1;
    const uint16_t* T = a.T_mid + ((int64_t)tile.expert * I + i) * G;  // row i % G of block i / G
    const int b = c / G * G;
#pragma unroll
    for (int t = 0; t < NT; ++t) h[t] = 0.0f;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float tj = __uint_as_float((uint32_t)T[j] << 16);
#pragma unroll
      for (int t = 0; t < NT; ++t) h[t] = __builtin_fmaf(tj, hs[t][threadIdx.x >> 5][b + j], h[t]);
    }
  }
  if (i0 + c >= I) return;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = 16 * t + (threadIdx.x >> 5);
    if (m >= tile.count) continue;
    const int64_t s = a.slots[tile.start + m];
    uint16_t* o = a.h + s * I + i0 + c;
    float v = h[t];
    for (int p = 0; p < a.h_terms; ++p) {
      const __bf16 bv = (__bf16)v;
      o[p * (int64_t)a.M * a.topk * I] = __builtin_bit_cast(uint16_t, bv);
      v -= (float)bv;
    }
  }
}

// ------------------------------------------------------------ down
//
// A workgroup owns 16 channels of y for all tokens and goes through all
// tiles: the steps of all tiles form one sequence, of which every wave takes
// a stretch.  Where a wave leaves a tile, it adds the tile's sums, times the
// tokens' weights, to its own y in LDS; the waves' sums meet at the end.
template <int FMT, int NT, int TERMS>
__global__ __launch_bounds__(64 * kWaves) void down_kernel(MoeArgs a) {
  __shared__ float ys[kWaves][kMoeTokens][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int64_t H = a.H, I = a.I;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t row = n0 + n < H ? n0 + n : H - 1;
  for (int m = q; m < a.M; m += 4) ys[wave][m][n] = 0.0f;
  // ys[wave] is this wave's alone; its lanes meet there in program order.
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int n_tiles = *a.n_tiles;
  const int whole = (int)(I / kStep), steps = (int)((I + kStep - 1) / kStep);
  const int64_t units = (int64_t)n_tiles * steps;
  const int64_t u0 = units * wave / kWaves, u1 = units * (wave + 1) / kWaves;
  const int64_t plane = (int64_t)a.M * a.topk * I;

  Raw<FMT> w[1], nw[1];
  auto load = [&](Raw<FMT>& to, int tile, int st) {
    const int64_t r = (int64_t)a.tiles[tile].expert * H + row;
    const uint8_t* cp = a.dn_codes + r * row_code_bytes<FMT>(I);
    const uint8_t* sp = a.dn_scales + r * row_scale_bytes<FMT>(I);
    if (st < whole) {
      load_raw<FMT>(to, cp, sp, st, q);
    } else {
      load_raw_tail<FMT>(to, cp, sp, st, q, (int)I);
    }
  };
  if (u0 < u1) {
    int tile = (int)(u0 / steps), st = (int)(u0 % steps);
    load(w[0], tile, st);
    int64_t u = u0;
    while (u < u1) {
      const MoeTile info = a.tiles[tile];
      const uint16_t* xp[NT];
      f32x4 acc[1][NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc[0][t] = f32x4{0, 0, 0, 0};
        xp[t] = a.h + (int64_t)a.slots[info.start + (16 * t + n < info.count ? 16 * t + n : 0)] * I;
      }
      // This tile's share of the stretch.
      while (true) {
        const bool last = st + 1 == steps;
        const int tile2 = last ? tile + 1 : tile, st2 = last ? 0 : st + 1;
        if (u + 1 < u1) load(nw[0], tile2, st2);
        if (st < whole) {
          step<FMT, 1, NT, TERMS, false>(acc, w, xp, plane, st, q, (int)I);
        } else {
          step<FMT, 1, NT, TERMS, true>(acc, w, xp, plane, st, q, (int)I);
        }
        w[0] = nw[0];
        ++u;
        tile = tile2;
        st = st2;
        if (last || u == u1) break;
      }
      const float gs = FMT == kNV ? a.dn_gs[info.expert] : 1.0f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = 16 * t + 4 * q + i;
          if (m >= info.count) continue;
          const int s = a.slots[info.start + m];
          ys[wave][s / a.topk][n] += a.weights[s] * (FMT == kNV ? acc[0][t][i] * gs : acc[0][t][i]);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.M * 16; o += 64 * kWaves) {
    const int m = o >> 4, c = o & 15;
    if (n0 + c >= H) continue;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += ys[k][m][c];
    const int64_t at = m * H + n0 + c;
    if (a.bf16_out) {
      reinterpret_cast<uint16_t*>(a.Y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
    } else {
      reinterpret_cast<float*>(a.Y)[at] = v;
    }
  }
}

template <int FMT, int NT, int TERMS>
hipError_t go_gate_up(const MoeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.I + 31) / 32), (unsigned)moe_max_tiles(a.M, a.topk, a.E));
  hipLaunchKernelGGL((gate_up_kernel<FMT, NT, TERMS>), grid, dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}

template <int FMT, int NT, int TERMS>
hipError_t go_down(const MoeArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((down_kernel<FMT, NT, TERMS>), dim3((unsigned)((a.H + 15) / 16)), dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}

template <int FMT, int NT>
hipError_t go_experts(const MoeArgs& a, hipStream_t s) {
  hipError_t e;
  if (a.x.terms == 1) e = go_gate_up<FMT, NT, 1>(a, s);
  else if (a.x.terms == 2) e = go_gate_up<FMT, NT, 2>(a, s);
  else e = go_gate_up<FMT, NT, 3>(a, s);
  if (e != hipSuccess) return e;
  return a.h_terms == 2 ? go_down<FMT, NT, 2>(a, s) : go_down<FMT, NT, 3>(a, s);
}

template <int FMT>
hipError_t go_fmt(const MoeArgs& a, hipStream_t s) {
  const int nt = moe_tile_nt(a.M, a.topk, a.E);
  if (nt == 1) return go_experts<FMT, 1>(a, s);
  if (nt == 2) return go_experts<FMT, 2>(a, s);
  return go_experts<FMT, 4>(a, s);
}

}  // namespace

hipError_t launch_moe(const MoeArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(router_kernel, dim3((unsigned)((a.E + 15) / 16), (unsigned)((a.M + 15) / 16)),
                     dim3(64 * kRouterWaves), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int tokens = 16 * moe_tile_nt(a.M, a.topk, a.E);
  if (a.E <= 128) hipLaunchKernelGGL((route_kernel<2>), dim3(1), dim3(kRouteThreads), 0, s, a, tokens);
  else if (a.E <= 256) hipLaunchKernelGGL((route_kernel<4>), dim3(1), dim3(kRouteThreads), 0, s, a, tokens);
  else hipLaunchKernelGGL((route_kernel<16>), dim3(1), dim3(kRouteThreads), 0, s, a, tokens);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.fmt == kMX) return go_fmt<kMX>(a, s);
  if (a.fmt == kNV) return go_fmt<kNV>(a, s);
  return go_fmt<kINT>(a, s);
}

}  // namespace wush
