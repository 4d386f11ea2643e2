// A mixture-of-experts layer on 4-bit weights for a few tokens:
//   l = Wr x,  the topk largest l_e (ties: lowest e),  softmax weights w_e,
//   y = sum_e w_e Wd_e T_mid,e (silu(Wg_e x') * (Wu_e x')),  x' = x or T_in x.
// Launches on one stream: the router's logits (and T_in x); the choice of
// experts and the grouping of tokens by expert; gate, up and their product; down; the
// weighted sum.  Every sum has a fixed order, so results repeat bit for bit.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"
#include "wush_w4_core.h"
#include "wush_wave.h"

namespace wush {
namespace {

using namespace w4;

// ------------------------------------------------------------ router
//
// Logits of 16 experts for 16 tokens: K is split over the waves of kRouterParts
// workgroups, whose sums the choice adds up in order.  The workgroups behind those
// transform: each wave 32 channels of 16 tokens (one launch for two things that
// need x alone).  Bound by the latency of reading the router, one round trip to memory
// where a compute unit has few lines to fetch: 8 tokens, 128 experts of 4096 5.0 us
// with four workgroups of eight waves per 16 experts, the same with eight of four, 8.5
// with one of sixteen (8 workgroups for 1 MB); the whole call 107 us against 110.
constexpr int kRouterWaves = 8, kRouterSlices = kRouterWaves * kRouterParts;

__global__ __launch_bounds__(64 * kRouterWaves) void router_kernel(MoeArgs a, int router_groups) {
  __shared__ float red[kRouterWaves][16][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * 16;
  if ((int)blockIdx.x >= router_groups) {
    const int64_t panel = (int64_t)(blockIdx.x - router_groups) * kRouterWaves + wave;
    if (panel * 32 < a.H)
      split_panel(SplitArgs{a.X, a.ldx, a.T_in, a.xt, a.M, a.H, a.fmt == kNV ? 16 : 32, a.terms}, panel, m0);
    return;
  }
  const int e0 = blockIdx.x / kRouterParts * 16, part = blockIdx.x % kRouterParts;
  const int slice = part * kRouterWaves + wave;
  const int rows = a.M - m0 < 16 ? a.M - m0 : 16;
  const int e = e0 + n < a.E ? e0 + n : a.E - 1;
  const uint16_t* w = a.router + (int64_t)e * a.H + 8 * q;
  const uint16_t* x = a.X + (int64_t)(m0 + (n < rows ? n : 0)) * a.ldx + 8 * q;
  f32x4 acc = {0, 0, 0, 0};
  const int vecs = (int)(a.H / 32);  // instructions of 32 elements; H may end in half of one
  constexpr int kBatch = 4;          // their loads are on their way together
  for (int i0 = slice; i0 < vecs; i0 += kBatch * kRouterSlices) {
    bf16x8 xv[kBatch], wv[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kRouterSlices, at = 32 * (i < vecs ? i : slice);
      xv[b] = *reinterpret_cast<const bf16x8*>(x + at);
      wv[b] = *reinterpret_cast<const bf16x8*>(w + at);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (i0 + b * kRouterSlices < vecs) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[b], wv[b], acc, 0, 0, 0);
  }
  if (a.H % 32 != 0 && slice == vecs % kRouterSlices) {
    u32x4 xv = {0, 0, 0, 0}, wv = {0, 0, 0, 0};
    if (q < 2) {
      xv = *reinterpret_cast<const u32x4*>(x + 32 * vecs);
      wv = *reinterpret_cast<const u32x4*>(w + 32 * vecs);
    }
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv), __builtin_bit_cast(bf16x8, wv), acc,
                                                  0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[wave][4 * q + i][n] = acc[i];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int m = threadIdx.x >> 4, c = threadIdx.x & 15;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kRouterWaves; ++k) v += red[k][m][c];
    if (m < rows && e0 + c < a.E) a.logits[((int64_t)part * a.M + m0 + m) * a.E + e0 + c] = v;
  }
}

// ------------------------------------------------------------ choice

// A logit as an integer of the same order, for comparisons in one instruction:
// NaN below every number, -0 like +0.
constexpr int kTaken = INT32_MIN;  // below all of them
__device__ __forceinline__ int order_key(float l) {
  const int b = (int)__float_as_uint(l + 0.0f);
  return l != l ? kTaken + 1 : b ^ (b >> 31 & 0x7FFFFFFF);
}

// One wave chooses B tokens' experts: every lane holds the logits of experts lane,
// lane + 64, ...; topk times the largest is found, and among its equals the
// lowest expert.  Lane p < topk ends with choice p and its weight.
template <int J, int B>
__device__ __forceinline__ void choose(const MoeArgs& a, int m0, int (&id)[B], float (&weight)[B]) {
  const int lane = threadIdx.x & 63;
  float l[B][J], chosen[B];
  int key[B][J];
#pragma unroll
  for (int b = 0; b < B; ++b)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane + 64 * j, m = m0 + b < a.M ? m0 + b : m0;
      const float* at = a.logits + (int64_t)m * a.E + (e < a.E ? e : 0);
      l[b][j] = at[0];
#pragma unroll
      for (int k = 1; k < kRouterParts; ++k) l[b][j] += at[(int64_t)k * a.M * a.E];
    }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    id[b] = 0;
    chosen[b] = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) key[b][j] = lane + 64 * j < a.E ? order_key(l[b][j]) : kTaken;
  }
  for (int p = 0; p < a.topk; ++p) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      int best = key[b][0];
#pragma unroll
      for (int j = 1; j < J; ++j) best = key[b][j] > best ? key[b][j] : best;
      best = wave_max_int(best);
      int found = 0;
#pragma unroll
      for (int j = J - 1; j >= 0; --j) {
        const uint64_t at = __ballot(key[b][j] == best);
        if (at != 0) found = 64 * j + __ffsll((unsigned long long)at) - 1;
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (found == lane + 64 * j) key[b][j] = kTaken;
      if (lane == p) {
        id[b] = found;
        // The key's logit; a chosen NaN gives NaN below.
        chosen[b] = best == kTaken + 1 ? __builtin_nanf("") : __uint_as_float((uint32_t)(best ^ (best >> 31 & 0x7FFFFFFF)));
      }
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const float t = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(chosen[b]), 0));
    const float w = lane < a.topk ? expf(chosen[b] - t) : 0.0f;
    float part = w;
    if (!a.renorm) {
      part = 0.0f;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (lane + 64 * j < a.E) part += expf(l[b][j] - t);
    }
    weight[b] = w / wave_sum(part);
  }
}

// One workgroup: the tokens' choices, and the experts' tiles.  An expert's
// tokens are the set bits of a 64-bit mask, in order, so results repeat without any
// sorting.  A wave chooses for B tokens at a time: the top_k rounds of one depend on
// each other, those of B do not.  Bound by that chain: 3.6 us for one token
// and the top 4 of 64 experts, 5.3 us for 8 tokens and 8 of 128, 10 us for 64 tokens
// and 6 of 96.
constexpr int kRouteThreads = 1024;

template <int J, int B>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(MoeArgs a, int tile_tokens) {
  constexpr int kWaves = kRouteThreads / 64;
  __shared__ unsigned long long tokens[kMoeMaxExperts];  // of each expert
  __shared__ int first[kMoeMaxExperts];                  // its first tile
  __shared__ short chosen[kMoeTokens * kMoeMaxTopK];
  __shared__ int wave_tiles[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = threadIdx.x;
  tokens[e] = 0;
  __syncthreads();
  for (int m0 = wave * B; m0 < a.M; m0 += kWaves * B) {
    int id[B];
    float weight[B];
    choose<J, B>(a, m0, id, weight);
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int m = m0 + b;
      if (lane < a.topk && m < a.M) {
        a.ids[m * a.topk + lane] = id[b];
        a.weights[m * a.topk + lane] = weight[b];
        chosen[m * a.topk + lane] = (short)id[b];
        atomicOr(&tokens[id[b]], 1ull << m);
      }
    }
  }
  __syncthreads();
  // Thread e: expert e's tiles (at most 16); their place by a prefix sum over the
  // experts, bit by bit of the counts.
  const int count = __popcll(tokens[e]), tiles = (count + tile_tokens - 1) / tile_tokens;
  const uint64_t below = (1ull << lane) - 1;
  int at = 0, all = 0;
#pragma unroll
  for (int b = 0; b < 5; ++b) {
    const uint64_t set = __ballot(tiles >> b & 1);
    at += __popcll(set & below) << b;
    all += __popcll(set) << b;
  }
  if (lane == 0) wave_tiles[wave] = all;
  __syncthreads();
  for (int k = 0; k < wave; ++k) at += wave_tiles[k];
  first[e] = at;
  for (int t = 0; t < tiles; ++t) {
    const int left = count - t * tile_tokens;
    a.tiles[at + t].expert = e;
    a.tiles[at + t].count = left < tile_tokens ? left : tile_tokens;
  }
  if (e == kRouteThreads - 1) *a.n_tiles = at + tiles;
  __syncthreads();
  for (int s = threadIdx.x; s < a.M * a.topk; s += kRouteThreads) {
    const int id = chosen[s], rank = __popcll(tokens[id] & ((1ull << (s / a.topk)) - 1));
    MoeTile& tile = a.tiles[first[id] + rank / tile_tokens];
    tile.token[rank % tile_tokens] = (int16_t)(s / a.topk);
    tile.slot[rank % tile_tokens] = (int16_t)s;
  }
}

template <int J>
hipError_t go_route(const MoeArgs& a, int tile_tokens, hipStream_t s) {
  if constexpr (J <= 4) {
    if (a.M > 32) {
      hipLaunchKernelGGL((route_kernel<J, 4>), dim3(1), dim3(kRouteThreads), 0, s, a, tile_tokens);
      return hipGetLastError();
    }
    if (a.M > 16) {
      hipLaunchKernelGGL((route_kernel<J, 2>), dim3(1), dim3(kRouteThreads), 0, s, a, tile_tokens);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((route_kernel<J, 1>), dim3(1), dim3(kRouteThreads), 0, s, a, tile_tokens);
  return hipGetLastError();
}

// ------------------------------------------------------------ gate and up
//
// A workgroup owns 8 R WN (32 or more) channels of h for one tile of tokens of
// one expert: wave wn has 8 R gate rows and the 8 R up rows of the same channels.  32
// channels hold whole transform blocks, so T_mid is applied to h right here, and
// neither gate nor up is ever written.  Bound by the experts' weights: 128 experts of
// 4096 x 1280 MXFP4, 8 tokens, T: 67 us (51 experts of 5.6 MB: 4.2 TB/s); 8 INT4
// experts of 4096 x 4096, 33 tokens: 45 us (3.3 TB/s); 96 NVFP4 experts of 2560 x
// 1440, 64 tokens: 98 us (4.0 TB/s).  Waves wait for 47 to 49% of their cycles; vector
// instructions take 25, 34 and 51% of the time.
template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, int WN, int WK>
__global__ __launch_bounds__(64 * WN * WK, (min_waves<FMT, R, NT, TERMS>())) void gate_up_kernel(MoeArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  __shared__ int slot[16 * NT], token[16 * NT];
  constexpr int kThreads = 64 * WN * WK, kWaveChannels = 8 * R, kChannels = kWaveChannels * WN, kRows = SPREAD ? 4 : 16 * NT;
  static_assert(kChannels % 32 == 0, "whole transform blocks");
  const MoeTile& tile = a.tiles[blockIdx.y];
  const int expert = tile.expert, count = tile.count, my_slot = tile.slot[threadIdx.x & 31];
  const int my_token = tile.token[threadIdx.x & 31];
  if ((int)blockIdx.y >= *a.n_tiles) return;
  const int wn = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WN;
  const int64_t H = a.H, I = a.I, i0 = (int64_t)blockIdx.x * kChannels;
  const int64_t gate = (int64_t)expert * (2 * I);
  const auto p = make_rows<FMT, R, D>(
      a.gu_codes, a.gu_scales, H,
      [&](int r) {
        const int64_t i = i0 + kWaveChannels * wn + 16 * (r % (R / 2));
        return gate + (r < R / 2 ? 0 : I) + (i < I ? i : I - 1);
      },
      [&](int r) { return gate + (r < R / 2 ? I : 2 * I) - 1; });
  const auto ready = [&] {
    if ((int)threadIdx.x < count) {
      slot[threadIdx.x] = my_slot;
      token[threadIdx.x] = my_token;
    }
    meet();
  };
  const uint16_t* X = a.T_in ? a.xt : a.X;
  const int64_t ldx = a.T_in ? H : a.ldx;
  group_dot<FMT, R, D, NT, TERMS, SPREAD, WN, WK>(
      lds, p, ready, [&](int row) { return X + token[row] * ldx; }, a.M * H, count, H);
  const float gs = FMT == kNV ? a.gu_gs[expert] : 1.0f;
  // Value v: token v / kChannels, channel v % kChannels.
  constexpr int kEach = (kRows * kChannels + kThreads - 1) / kThreads;
  const int values = count * kChannels;
  float h[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int v = threadIdx.x + k * kThreads, m = v / kChannels, c = v % kChannels;
    h[k] = 0.0f;
    if (v < values) {
      const int row = 2 * kWaveChannels * (c / kWaveChannels) + c % kWaveChannels;
      float g = group_sum<R, WN, WK>(lds, row, m, count);
      float u = group_sum<R, WN, WK>(lds, row + kWaveChannels, m, count);
      if (FMT == kNV) {
        g *= gs;
        u *= gs;
      }
      h[k] = g / (1.0f + expf(-g)) * u;
    }
  }
  if (a.T_mid) {
    constexpr int G = FMT == kNV ? 16 : 32;
    __syncthreads();  // everyone has read the sums
    float* hs = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int v = threadIdx.x + k * kThreads;
      if (v < values) hs[v] = h[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int v = threadIdx.x + k * kThreads, c = v % kChannels;
      if (v >= values || i0 + c >= I) continue;
      const uint16_t* T = a.T_mid + ((int64_t)expert * I + i0 + c) * G;  // row c % G of its block
      const float* block = hs + v / G * G;
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < G; j += 8) {
        const u32x4 t = *reinterpret_cast<const u32x4*>(T + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = __builtin_fmaf(__uint_as_float(t[i] << 16), block[j + 2 * i], s);
          s = __builtin_fmaf(__uint_as_float(t[i] & 0xFFFF0000u), block[j + 2 * i + 1], s);
        }
      }
      h[k] = s;
    }
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int v = threadIdx.x + k * kThreads, m = v / kChannels, c = v % kChannels;
    if (v >= values || i0 + c >= I) continue;
    uint16_t* o = a.h + slot[m] * I + i0 + c;
    float r = h[k];
    for (int t = 0; t < a.terms; ++t) {
      const __bf16 b = (__bf16)r;
      o[t * ((int64_t)a.M * a.topk * I)] = __builtin_bit_cast(uint16_t, b);
      r -= (float)b;
    }
  }
}

// ------------------------------------------------------------ down
//
// A workgroup owns 16 R WN channels of y for one tile; its results, one row per
// slot, wait in memory for the slots' other experts (added there by atomics, their
// order would change results).  Bound as gate and up: 35, 32 and 64 us on the same
// three (4.0, 2.4 and 3.1 TB/s: rows are short, or few workgroups).
template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, int WN, int WK>
__global__ __launch_bounds__(64 * WN * WK, (min_waves<FMT, R, NT, TERMS>())) void down_kernel(MoeArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  __shared__ int slot[16 * NT];
  constexpr int kThreads = 64 * WN * WK, kChannels = 16 * R * WN;
  const MoeTile& tile = a.tiles[blockIdx.y];
  const int expert = tile.expert, count = tile.count, my_slot = tile.slot[threadIdx.x & 31];
  if ((int)blockIdx.y >= *a.n_tiles) return;
  const int wn = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WN;
  const int64_t H = a.H, I = a.I, n0 = (int64_t)blockIdx.x * kChannels;
  const auto p = make_rows<FMT, R, D>(
      a.dn_codes, a.dn_scales, I,
      [&](int r) {
        const int64_t i = n0 + 16 * (wn * R + r);
        return expert * H + (i < H ? i : H - 1);
      },
      [&](int) { return expert * H + H - 1; });
  const auto ready = [&] {
    if ((int)threadIdx.x < count) slot[threadIdx.x] = my_slot;
    meet();
  };
  group_dot<FMT, R, D, NT, TERMS, SPREAD, WN, WK>(
      lds, p, ready, [&](int row) { return a.h + slot[row] * I; }, (int64_t)a.M * a.topk * I, count, I);
  const float gs = FMT == kNV ? a.dn_gs[expert] : 1.0f;
  for (int v = threadIdx.x; v < count * kChannels; v += kThreads) {
    const int m = v / kChannels, c = v % kChannels;
    if (n0 + c >= H) continue;
    float s = group_sum<R, WN, WK>(lds, c, m, count);
    if (FMT == kNV) s *= gs;
    a.part[slot[m] * H + n0 + c] = s;
  }
}

// ------------------------------------------------------------ weighted sum
//
// In the order of the choice, whatever workgroup was first.  1.9 us for one token,
// which is what a launch takes.
__global__ __launch_bounds__(256) void combine_kernel(MoeArgs a) {
  const int m = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.H) return;
  const float* part = a.part + (int64_t)m * a.topk * a.H + c;
  float v = 0.0f;
#pragma unroll 8
  for (int j = 0; j < a.topk; ++j) v = __builtin_fmaf(a.weights[m * a.topk + j], part[j * a.H], v);
  if (a.bf16_out) {
    reinterpret_cast<uint16_t*>(a.Y)[m * a.H + c] = __builtin_bit_cast(uint16_t, (__bf16)v);
  } else {
    reinterpret_cast<float*>(a.Y)[m * a.H + c] = v;
  }
}

template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, int WN, int WK>
hipError_t go_gate_up(const MoeArgs& a, int max_tiles, hipStream_t s) {
  constexpr int kChannels = 8 * R * WN, kRows = SPREAD ? 4 : 16 * NT;
  const dim3 grid((unsigned)((a.I + kChannels - 1) / kChannels), (unsigned)max_tiles);
  const int rows = a.M < kRows ? a.M : kRows;
  int64_t lds = lds_bytes<R, D, NT, TERMS, WN, WK>(rows, a.H);
  const int64_t hs = (int64_t)4 * rows * kChannels;
  if (hs > lds) lds = hs;
  return launch_lds(gate_up_kernel<FMT, R, D, NT, TERMS, SPREAD, WN, WK>, grid, 64 * WN * WK, lds, s, a);
}

template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, int WN, int WK>
hipError_t go_down(const MoeArgs& a, int max_tiles, hipStream_t s) {
  const dim3 grid((unsigned)((a.H + 16 * R * WN - 1) / (16 * R * WN)), (unsigned)max_tiles);
  constexpr int kRows = SPREAD ? 4 : 16 * NT;
  const int rows = a.M < kRows ? a.M : kRows;
  return launch_lds(down_kernel<FMT, R, D, NT, TERMS, SPREAD, WN, WK>, grid, 64 * WN * WK,
                    lds_bytes<R, D, NT, TERMS, WN, WK>(rows, a.I), s, a);
}

// Tokens per tile, by how many tokens an expert can expect: 4, 16 or 32.
int tile_tokens(const MoeArgs& a) {
  const float expect = (float)(a.M * a.topk) / a.E;
  return a.M <= 4 || expect <= 2.0f ? 4 : a.M <= 16 || expect <= 12.0f ? 16 : 32;
}

// Four waves of two row tiles and two steps each.  Measured on 128 experts of
// 4096 x 1280 MXFP4 with transforms, 8 tokens (the whole call): 122 us, against 133
// with eight waves of four row tiles that split K, and 144 with four of those;
// down 124 against 132 with K split over four waves.  (Both sides were timed in turn
// in one state of the rest; the call now takes 104 to 109 us.)
template <int FMT, int TERMS>
hipError_t go_gate_up_tiles(const MoeArgs& a, int max_tiles, hipStream_t s) {
  const int t = tile_tokens(a);
  if (t == 4) return go_gate_up<FMT, 2, 2, 1, TERMS, true, 2, 2>(a, max_tiles, s);
  if (t == 16) return go_gate_up<FMT, 2, 2, 1, TERMS, false, 2, 2>(a, max_tiles, s);
  return go_gate_up<FMT, 4, 1, 2, TERMS, false, 4, 2>(a, max_tiles, s);
}

template <int FMT, int TERMS>
hipError_t go_down_tiles(const MoeArgs& a, int max_tiles, hipStream_t s) {
  const int t = tile_tokens(a);
  if (t == 4) return go_down<FMT, 2, 2, 1, TERMS, true, 2, 2>(a, max_tiles, s);
  if (t == 16) {
    // Up to one workgroup per compute unit: eight waves each that split K four ways.
    // Whole calls, those against the other shape, MXFP4, NVFP4 and INT4: 128 workgroups
    // (24 tokens, 2 of 8 experts of 2048 x 1024) 27.1 : 28.8, 30.1 : 30.7, 30.7 : 31.9;
    // 256 (16 tokens, 2 of 8 of 4096 x 4096) 71.6 : 74.6, 78.3 : 80.8, 80.3 : 84.0; 320
    // (64 tokens, 2 of 16 of 2560 x 1440) 51.0 : 48.3, 60.3 : 55.2, 60.8 : 56.0; 1024
    // (40 tokens, 8 of 32 of 4096 x 1568) 124 : 116, 143 : 130, 144 : 130.
    const int slots = a.M * a.topk, experts = slots < a.E ? slots : a.E;
    if ((a.H + 127) / 128 * experts <= 256) return go_down<FMT, 4, 1, 1, TERMS, false, 2, 4>(a, max_tiles, s);
    return go_down<FMT, 2, 2, 1, TERMS, false, 4, 1>(a, max_tiles, s);
  }
  return go_down<FMT, 4, 1, 2, TERMS, false, 4, 2>(a, max_tiles, s);
}

template <int FMT>
hipError_t go_experts(const MoeArgs& a, hipStream_t s) {
  // No more tiles than slots, nor than experts and the tiles cut off full ones.
  const int slots = a.M * a.topk, cut = (slots < a.E ? slots : a.E) + slots / tile_tokens(a);
  const int max_tiles = slots < cut ? slots : cut;
  hipError_t e = !a.T_in          ? go_gate_up_tiles<FMT, 1>(a, max_tiles, s)
                 : a.terms == 2 ? go_gate_up_tiles<FMT, 2>(a, max_tiles, s)
                                : go_gate_up_tiles<FMT, 3>(a, max_tiles, s);
  if (e != hipSuccess) return e;
  return a.terms == 2 ? go_down_tiles<FMT, 2>(a, max_tiles, s) : go_down_tiles<FMT, 3>(a, max_tiles, s);
}

}  // namespace

hipError_t launch_moe(const MoeArgs& a, hipStream_t s) {
  const int router_groups = (a.E + 15) / 16 * kRouterParts;
  const int64_t split = a.T_in ? (a.H + 32 * kRouterWaves - 1) / (32 * kRouterWaves) : 0;
  hipLaunchKernelGGL(router_kernel, dim3((unsigned)(router_groups + split), (unsigned)((a.M + 15) / 16)),
                     dim3(64 * kRouterWaves), 0, s, a, router_groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int tokens = tile_tokens(a);
  e = a.E <= 128 ? go_route<2>(a, tokens, s) : a.E <= 256 ? go_route<4>(a, tokens, s) : go_route<16>(a, tokens, s);
  if (e != hipSuccess) return e;
  e = a.fmt == kMX ? go_experts<kMX>(a, s) : a.fmt == kNV ? go_experts<kNV>(a, s) : go_experts<kINT>(a, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((a.H + 255) / 256), (unsigned)a.M), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace wush
