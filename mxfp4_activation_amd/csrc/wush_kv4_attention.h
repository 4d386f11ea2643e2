// Attention of a few or many queries over a paged cache of keys and values in
// 4 bits.  Device code, included once per format (wush_kv4_*.hip).
//
//   out_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(scale q_i . k_t)
//
// over the tokens t that query i sees, with the running maximum of the scores
// taken out of the exponent.
//
// Work.  An item is one key head's queries of one sequence: up to 16, 32 or 128
// columns (query, head of the group).  Its tokens come in units of 128.  Items
// and units are counted on the device, from the lengths as they are when the kernel
// runs; every workgroup takes an equal run of units, so that one long sequence
// among short ones is spread over the whole chip.  An item that a run's border
// cuts leaves its pieces (maximum, sum, unscaled result) in the workspace, and a
// second kernel joins them.
//
// A wave's step is 32 tokens, all of it in registers: no LDS, no barrier.
//   S = K Q^T with v_mfma_f32_16x16x32_bf16, A = 16 tokens, B = 16 columns: lane
//     (n = lane % 16, q = lane / 16) of D holds column n, tokens 4 q + r.
//   O^T += V^T P^T, A = 16 channels, B = the columns: lane (n, q) of B holds 8
//     tokens of column n, which are tokens 4 q + r of the step's two halves: its own
//     eight values of D, rounded to bf16.  A's lane takes the same tokens.
// A lane's share of V is D / 16 neighbouring channels of eight tokens; channel j of
// them goes into matrix instruction j, whose D then holds, per lane, channels
// (D / 16) (4 q + r) + j.  Column n stays in lanes n, n + 16, n + 32, n + 48
// throughout, so the softmax needs one exchange between lanes where a maximum grows
// by more than 2^8, and one at the end.
//
// Exactness.  E2M1 times E8M0 or E4M3 has at most 6 significant bits and is exact in
// bf16, as are INT4's integers.  INT4's fp16 scale multiplies K's fp32 sums over
// one group; V as integer times scale is rounded to bf16 (off by up to 2^-8, as P is: P is a
// probability up to the running maximum's slack, and both errors are below the
// result's own rounding, since a result averages over its tokens).  Sums are fp32; a
// transformed query enters as two bf16 planes (16 bits).
#ifndef WUSH_KV4_ATTENTION_H_
#define WUSH_KV4_ATTENTION_H_

#include <float.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_kv4.h"
#include "wush_w4_core.h"
#include "wush_wave.h"

namespace wush {
namespace kv4 {

using namespace w4;

constexpr int kThreads = 256;
constexpr int kTile = 32;   // tokens of a wave's step
constexpr float kSlack = 8.0f;  // log2 by which scores may pass the running maximum

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ------------------------------------------------------------ plan

struct Seq {
  int start, count, len;  // first query's row, queries, tokens
  bool bad;               // more tokens than the table has room for
};

__device__ __forceinline__ Seq seq_of(const KvAttnArgs& a, int b) {
  Seq s;
  s.start = b;
  s.count = 1;
  if (a.q_start) {
    const int lo = a.q_start[b], hi = a.q_start[b + 1];
    s.start = lo < 0 ? 0 : lo < a.n ? lo : a.n;
    const int end = hi < s.start ? s.start : hi < a.n ? hi : a.n;
    s.count = end - s.start;
  }
  const int64_t room = (int64_t)a.width << a.page_log2;
  s.len = a.lengths[b];
  s.bad = s.len > room;
  s.len = s.len < 0 ? 0 : s.bad ? (int)room : s.len;
  return s;
}

// Tokens that queries i0 .. i1 of a sequence see, as a range.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span span_of(const KvAttnArgs& a, const Seq& s, int i0, int i1) {
  const int hi = s.len - s.count + i1 + 1;
  const int lo = a.window ? s.len - s.count + i0 - a.window + 1 : 0;
  return Span{lo > 0 ? lo : 0, hi > 0 ? hi : 0};
}

template <int NC>
__device__ __forceinline__ int items_of(const KvAttnArgs& a, const Seq& s) {
  return (s.count * a.group + NC - 1) / NC;
}

// Units of item t of a sequence and key head; an item without tokens has one.
template <int NC>
__device__ __forceinline__ int units_of(const KvAttnArgs& a, const Seq& s, int t) {
  const int i0 = t * NC / a.group, last = (t * NC + NC - 1) / a.group;
  const Span p = span_of(a, s, i0, last < s.count ? last : s.count - 1);
  return p.hi > p.lo ? (p.hi + kKvUnit - 1) / kKvUnit - p.lo / kKvUnit : 1;
}

// Inclusive sums over the wave.
__device__ __forceinline__ int wave_scan(int v) {
  uint32_t u = (uint32_t)v;
  u += dpp<0x111, 0xf>(0, u);
  u += dpp<0x112, 0xf>(0, u);
  u += dpp<0x114, 0xf>(0, u);
  u += dpp<0x118, 0xf>(0, u);
  u += dpp<0x142, 0xa>(0, u);
  u += dpp<0x143, 0xc>(0, u);
  return (int)u;
}

// A sequence's share of the work, per key head: units, items, the most units of an item.
struct Load {
  int units, items, most;
};
template <int NC>
__device__ __forceinline__ Load load_of(const KvAttnArgs& a, const Seq& s) {
  Load l = {0, items_of<NC>(a, s), 0};
  for (int t = 0; t < l.items; ++t) {
    const int u = units_of<NC>(a, s, t);
    l.units += u;
    l.most = l.most > u ? l.most : u;
  }
  return l;
}

struct PlanLds {
  int units[4], items[4], most[4];
  int b, base, per_head;
  Seq s;
};

// The sequences c .. c + 255, one per thread: its own, its load, the units and items
// before it, and their sums over all.
struct Chunk {
  Seq s;
  Load own;
  int units, items;                // of the chunk, before the thread's
  int all_units, all_items, most;  // of the chunk
};
template <int NC>
__device__ __forceinline__ Chunk chunk_of(const KvAttnArgs& a, PlanLds& l, int c) {
  const int b = c + (int)threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Chunk k;
  k.s = Seq{0, 0, 0, false};
  k.own = Load{0, 0, 0};
  if (b < a.B) {
    k.s = seq_of(a, b);
    k.own = load_of<NC>(a, k.s);
    k.own.units *= a.kv;
    k.own.items *= a.kv;
  }
  const int units = wave_scan(k.own.units), items = wave_scan(k.own.items), most = wave_max_int(k.own.most);
  __syncthreads();  // the chunk before is done with
  if (lane == 63) {
    l.units[wave] = units;
    l.items[wave] = items;
    l.most[wave] = most;
  }
  __syncthreads();
  k.units = units - k.own.units;
  k.items = items - k.own.items;
  k.all_units = k.all_items = k.most = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) {
      k.units += l.units[w];
      k.items += l.items[w];
    }
    k.all_units += l.units[w];
    k.all_items += l.items[w];
    k.most = k.most > l.most[w] ? k.most : l.most[w];
  }
  return k;
}

// How the call's work is shared out: by whole items, or by units.
struct Shares {
  bool whole;
  int total, share;  // items or units, in all and per workgroup
};

// Items are taken whole where nothing may be cut, and where there are enough of about the
// same length: the longest times the rounds of them is at most 1.3 times the mean share.
// (Two prompts of 1000 queries behind 16384 tokens, 456 items for 512 places: 105 us of
// joining and 60 MB of pieces less, for 12% longer runs.)
template <int NC>
__device__ __forceinline__ Shares shares_of(const KvAttnArgs& a, PlanLds& l, Chunk& first) {
  first = chunk_of<NC>(a, l, 0);
  int units = first.all_units, items = first.all_items, most = first.most;
  for (int c = kThreads; c < a.B; c += kThreads) {
    const Chunk k = chunk_of<NC>(a, l, c);
    units += k.all_units;
    items += k.all_items;
    most = most > k.most ? most : k.most;
  }
  units = uniform(units);
  items = uniform(items);
  most = uniform(most);
  Shares s;
  s.whole = a.runs == 0 ||
            (items <= a.workgroups && (float)most * (float)((items + a.runs - 1) / a.runs) * (float)a.runs <= 1.3f * (float)units);
  s.total = s.whole ? items : units;
  s.share = s.whole ? 1 : (units + a.runs - 1) / a.runs;
  return s;
}

// Where a unit (or whole item) is: sequence, key head, item, and the unit's place in it.
struct Place {
  int b, h, t, off;
  Seq s;
};

// The place of number u < total, for the whole workgroup.
template <int NC>
__device__ __forceinline__ Place find(const KvAttnArgs& a, PlanLds& l, const Chunk& first, bool whole, int u) {
  int base = 0;
  for (int c = 0; c < a.B; c += kThreads) {
    const Chunk k = c == 0 ? first : chunk_of<NC>(a, l, c);
    const int own = whole ? k.own.items : k.own.units, before = base + (whole ? k.items : k.units);
    if (u >= before && u - before < own) {
      l.b = c + (int)threadIdx.x;
      l.base = before;
      l.per_head = own / a.kv;
      l.s = k.s;
    }
    base += whole ? k.all_items : k.all_units;
    if (base > u) break;
  }
  __syncthreads();
  Place p;
  p.b = uniform(l.b);
  p.s.start = uniform(l.s.start);
  p.s.count = uniform(l.s.count);
  p.s.len = uniform(l.s.len);
  p.s.bad = uniform(l.s.bad);
  const int per_head = uniform(l.per_head), at = u - uniform(l.base);
  p.h = at / per_head;
  p.off = at - p.h * per_head;
  p.t = 0;
  if (whole) {
    p.t = p.off;
    p.off = 0;
    return p;
  }
  for (;;) {
    const int nu = units_of<NC>(a, p.s, p.t);
    if (p.off < nu) break;
    p.off -= nu;
    ++p.t;
  }
  return p;
}

// ------------------------------------------------------------ one step's data

template <int FMT, int D>
struct Raw {
  static constexpr int kK = D / 32;                       // dwords of K per lane and half
  static constexpr int kV = D / 16 > 8 ? D / 128 : 1;     // dwords of V per lane and token
  static constexpr int kKS = FMT == kINT ? D / 16 : 1;    // dwords of K's scales per lane and half
  uint32_t kc[2][kK];
  uint32_t ks[2][kKS];
  uint32_t vc[8][kV];
  uint32_t vs[8];
};

template <int D>
constexpr int kCh = D / 16;  // channels of V per lane

// Channel of element 0 of K's matrix instruction j in lane quarter q.
template <int FMT, int D>
__device__ __forceinline__ int channel(int j, int q) {
  return FMT == kINT ? 32 * j + 8 * q : q * (D / 4) + 8 * j;
}

template <int FMT, int D>
struct Offsets {
  uint32_t k, ks, v, vs;  // bytes from the first token of a half
};

template <int FMT, int D>
__device__ __forceinline__ Offsets<FMT, D> offsets() {
  constexpr int kRow = D / 2;
  constexpr int kScaleRow = FMT == kMX ? D / 32 : D / 16;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  Offsets<FMT, D> o;
  if (FMT == kINT) {
    o.k = n * kRow + (D == 64 ? 4 : 16) * q;
    o.ks = 4 * q * kScaleRow;
  } else {
    o.k = n * kRow + q * (D / 8);
    o.ks = n * kScaleRow + (FMT == kMX ? q * D / 128 : q * (D / 64));
  }
  o.v = 4 * q * kRow + n * (kCh<D> / 2);
  const int group = n * kCh<D> / (FMT == kNV ? 16 : 32);
  o.vs = 4 * q * kScaleRow + group * (FMT == kINT ? 2 : 1);
  return o;
}

// Half u of a step: 16 tokens, in one page, whose first one's rows these are.
template <int FMT, int D>
__device__ __forceinline__ void load_half(Raw<FMT, D>& w, int u, const uint8_t* kc, const uint8_t* ks, const uint8_t* vc,
                                          const uint8_t* vs, const Offsets<FMT, D>& o) {
  constexpr int kRow = D / 2;
  constexpr int kScaleRow = FMT == kMX ? D / 32 : D / 16;
  if constexpr (D == 64) {
    if constexpr (FMT == kINT) {
      w.kc[u][0] = load_unaligned<uint32_t>(kc + o.k);
      w.kc[u][1] = load_unaligned<uint32_t>(kc + o.k + 16);
    } else {
      const u32x2 v = load_unaligned<u32x2>(kc + o.k);
      w.kc[u][0] = v[0];
      w.kc[u][1] = v[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const u32x4 v = load_unaligned<u32x4>(kc + o.k + (FMT == kINT ? 64 : 16) * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) w.kc[u][4 * i + k] = v[k];
    }
  }
  if constexpr (FMT == kINT) {
#pragma unroll
    for (int i = 0; i < Raw<FMT, D>::kKS / 4; ++i) {
      const u32x4 v = load_unaligned<u32x4>(ks + o.ks + 16 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) w.ks[u][4 * i + k] = v[k];
    }
  } else if constexpr (FMT == kMX) {
    w.ks[u][0] = D == 256 ? load_unaligned<uint16_t>(ks + o.ks) : ks[o.ks];
  } else {
    w.ks[u][0] = D == 256   ? load_unaligned<uint32_t>(ks + o.ks)
                 : D == 128 ? load_unaligned<uint16_t>(ks + o.ks)
                            : ks[o.ks];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* p = vc + o.v + i * kRow;
    if constexpr (D == 64) {
      w.vc[4 * u + i][0] = load_unaligned<uint16_t>(p);
    } else if constexpr (D == 128) {
      w.vc[4 * u + i][0] = load_unaligned<uint32_t>(p);
    } else {
      const u32x2 v = load_unaligned<u32x2>(p);
      w.vc[4 * u + i][0] = v[0];
      w.vc[4 * u + i][1] = v[1];
    }
    const uint8_t* s = vs + o.vs + i * kScaleRow;
    w.vs[4 * u + i] = FMT == kINT ? load_unaligned<uint16_t>(s) : *s;
  }
}

__device__ __forceinline__ float half_value(uint32_t b) { return __half2float(__ushort_as_half((uint16_t)b)); }

// Scale of K's dword j of half u, applied to the elements (not INT4).
template <int FMT, int D>
__device__ __forceinline__ float k_scale(const Raw<FMT, D>& w, int u, int j) {
  if constexpr (FMT == kMX) {
    return __uint_as_float(((w.ks[u][0] >> (8 * (j / 4))) & 0xFFu) << 23);
  } else {
    const uint32_t v = w.ks[u][0];
    const int i = j / 2;  // two dwords share a group of 16
    return i == 0   ? __builtin_amdgcn_cvt_f32_fp8(v, 0)
           : i == 1 ? __builtin_amdgcn_cvt_f32_fp8(v, 1)
           : i == 2 ? __builtin_amdgcn_cvt_f32_fp8(v, 2)
                    : __builtin_amdgcn_cvt_f32_fp8(v, 3);
  }
}

// Byte b (two channels) of V's dword i for all eight tokens, as the A operands of two
// matrix instructions.
template <int FMT, int D>
__device__ __forceinline__ void expand_v(const Raw<FMT, D>& w, const float (&s)[8], int i, int b, u32x4& even, u32x4& odd) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t d0 = w.vc[2 * p][i], d1 = w.vc[2 * p + 1][i];
    if constexpr (FMT == kMX) {
      uint32_t c0, c1;
      switch (b) {
        case 0:
          c0 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d0, s[2 * p], 0));
          c1 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d1, s[2 * p + 1], 0));
          break;
        case 1:
          c0 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d0, s[2 * p], 1));
          c1 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d1, s[2 * p + 1], 1));
          break;
        case 2:
          c0 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d0, s[2 * p], 2));
          c1 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d1, s[2 * p + 1], 2));
          break;
        default:
          c0 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d0, s[2 * p], 3));
          c1 = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d1, s[2 * p + 1], 3));
      }
      even[p] = __builtin_amdgcn_perm(c1, c0, 0x05040100u);
      odd[p] = __builtin_amdgcn_perm(c1, c0, 0x07060302u);
    } else if constexpr (FMT == kNV) {
      f32x2 c0, c1;
      switch (b) {
        case 0:
          c0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d0, 1.0f, 0);
          c1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d1, 1.0f, 0);
          break;
        case 1:
          c0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d0, 1.0f, 1);
          c1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d1, 1.0f, 1);
          break;
        case 2:
          c0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d0, 1.0f, 2);
          c1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d1, 1.0f, 2);
          break;
        default:
          c0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d0, 1.0f, 3);
          c1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d1, 1.0f, 3);
      }
      even[p] = pack(cvt_bf16(c0[0] * s[2 * p], c1[0] * s[2 * p + 1]));
      odd[p] = pack(cvt_bf16(c0[1] * s[2 * p], c1[1] * s[2 * p + 1]));
    } else {
      // The integer, exact in fp32, times the scale: exact too (15 bits), then rounded.
      const int e0 = (int)(d0 << (28 - 8 * b)) >> 28, e1 = (int)(d1 << (28 - 8 * b)) >> 28;
      const int o0 = (int)(d0 << (24 - 8 * b)) >> 28, o1 = (int)(d1 << (24 - 8 * b)) >> 28;
      even[p] = pack(cvt_bf16((float)e0 * s[2 * p], (float)e1 * s[2 * p + 1]));
      odd[p] = pack(cvt_bf16((float)o0 * s[2 * p], (float)o1 * s[2 * p + 1]));
    }
  }
}

// ------------------------------------------------------------ a piece of an item

// Over the four lanes of a column.
__device__ __forceinline__ float column_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Orders this wave's LDS accesses.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int D>
constexpr int kQLine = D + 8;  // of a query in LDS, elements

// Whether the columns' operands stay in LDS (transformed ones in two planes, or long
// ones) rather than in registers, and the elements that a tile of them takes there.
template <int D, int PLANES>
constexpr bool kStaged = PLANES == 2 || D == 256;
template <int D, int PLANES>
constexpr int kQTile = PLANES * 16 * kQLine<D>;

// 16 channels (part c) of the lane's column n, transformed: to LDS as two bf16 planes.
template <int FMT, int D>
__device__ __forceinline__ void transform_q(const uint16_t* q, const uint16_t* T, uint16_t* lds, int c) {
  constexpr int G = FMT == kNV ? 16 : 32;
  const int lane = threadIdx.x & 63, n = lane & 15, k = lane >> 4;
  u32x4 av = {0, 0, 0, 0}, bv = {0, 0, 0, 0};
  if (G == 32) {
    av = *reinterpret_cast<const u32x4*>(T + (16 * c + n) * 32 + 8 * k);
    bv = *reinterpret_cast<const u32x4*>(q + c / 2 * 32 + 8 * k);
  } else if (k < 2) {  // the block fills half of the instruction's 32 columns
    av = *reinterpret_cast<const u32x4*>(T + (16 * c + n) * 16 + 8 * k);
    bv = *reinterpret_cast<const u32x4*>(q + 16 * c + 8 * k);
  }
  const f32x4 y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av),
                                                          __builtin_bit_cast(bf16x8, bv), f32x4{0, 0, 0, 0}, 0, 0, 0);
  u32x2 hi, lo;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const bf16x2 h = cvt_bf16(y[2 * p], y[2 * p + 1]);
    hi[p] = pack(h);
    lo[p] = pack(cvt_bf16(y[2 * p] - (float)h[0], y[2 * p + 1] - (float)h[1]));
  }
  *reinterpret_cast<u32x2*>(lds + n * kQLine<D> + 16 * c + 4 * k) = hi;
  *reinterpret_cast<u32x2*>(lds + (16 + n) * kQLine<D> + 16 * c + 4 * k) = lo;
}

// LDS of a workgroup in floats: the waves' results of one tile of columns (in two halves for
// D = 256), and in front of them the staged columns.
template <int D>
constexpr int kParts = D == 256 ? 2 : 1;
template <int D, int SHAPE, int PLANES>
constexpr int q_floats() {
  constexpr int tiles = kv_tiles(SHAPE, D) * (SHAPE == kKvPrompt ? 4 : 1);
  return kStaged<D, PLANES> ? tiles * kQTile<D, PLANES> / 2 : 0;
}
template <int D, int SHAPE, int PLANES>
constexpr int lds_floats() {
  return q_floats<D, SHAPE, PLANES>() + (SHAPE == kKvPrompt ? 0 : 4 * kCh<D> / kParts<D> * 4 * 64);
}

struct Piece {
  int b, h, t;      // sequence, key head, item
  int lo, hi;       // tokens, within the item's
  bool whole;       // of the item
  float* part;      // where it goes if not
  Seq s;
};

template <int FMT, int D, int SHAPE, int PLANES>
__device__ __forceinline__ void attend(const KvAttnArgs& a, const Piece& p, float* lds, float (&stat)[2][4][32]) {
  constexpr int NQ = kv_tiles(SHAPE, D), KJ = D / 32, CH = kCh<D>, NC = kv_columns(SHAPE, D);
  constexpr bool kInLds = kStaged<D, PLANES>;
  constexpr bool kAlone = SHAPE == kKvPrompt;  // waves have columns of their own
  using RawT = Raw<FMT, D>;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int all = p.s.count * a.group;  // columns of the sequence
  const int c0 = p.t * NC + (kAlone ? wave * 16 * NQ : 0);
  const int past = p.s.len - p.s.count;  // place of query 0

  // The wave's tokens and tiles of them.
  int lo = p.lo, hi = p.hi;
  const int i0 = c0 / a.group, end = (c0 + 16 * NQ - 1) / a.group, i1 = end < p.s.count ? end : p.s.count - 1;
  if (kAlone) {
    const Span w = c0 < all ? span_of(a, p.s, i0, i1) : Span{0, 0};
    lo = lo > w.lo ? lo : w.lo;
    hi = hi < w.hi ? hi : w.hi;
  }
  const int first = lo / kTile + (kAlone ? 0 : wave), step = kAlone ? 1 : 4;
  const int last = (hi + kTile - 1) / kTile;
  const int steps = hi > lo && last > first ? (last - first + step - 1) / step : 0;

  // Columns: query rows, their places, operands.
  int pos[NQ];
  bf16x8 held[kInLds ? 1 : NQ][kInLds ? 1 : KJ];
  uint16_t* staged = reinterpret_cast<uint16_t*>(lds) + (kAlone ? wave * NQ * kQTile<D, PLANES> : 0);
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    const int col = c0 + 16 * ct + n;
    const int used = col < all ? col : all - 1;
    const int i = used / a.group;
    pos[ct] = col < all ? past + i : -1;
    const uint16_t* row = a.q + (int64_t)(p.s.start + i) * a.ldq + (int64_t)(p.h * a.group + used - i * a.group) * D;
    if constexpr (!kInLds) {
#pragma unroll
      for (int j = 0; j < KJ; ++j) held[ct][j] = *reinterpret_cast<const bf16x8*>(row + channel<FMT, D>(j, q));
    } else {
      // Columns that the waves share are staged by all of them.
      uint16_t* to = staged + ct * kQTile<D, PLANES>;
      if constexpr (PLANES == 2) {
        for (int c = kAlone ? 0 : wave; c < D / 16; c += kAlone ? 1 : 4)
          transform_q<FMT, D>(row, a.T + (int64_t)p.h * D * (FMT == kNV ? 16 : 32), to, c);
      } else {
        for (int c = kAlone ? 0 : wave; c < D / 32; c += kAlone ? 1 : 4)
          *reinterpret_cast<u32x4*>(to + n * kQLine<D> + 32 * c + 8 * q) = *reinterpret_cast<const u32x4*>(row + 32 * c + 8 * q);
      }
    }
  }
  if constexpr (kInLds) {
    if (kAlone) {
      wave_fence();
    } else {
      __syncthreads();
    }
  }
  auto column = [&](int ct, int t, int j) {
    if constexpr (kInLds) {
      return *reinterpret_cast<const bf16x8*>(staged + ct * kQTile<D, PLANES> + (16 * t + n) * kQLine<D> + channel<FMT, D>(j, q));
    } else {
      return held[ct][j];
    }
  };
  float qs[FMT == kINT ? NQ : 1][FMT == kINT ? KJ : 1];
  if constexpr (FMT == kINT) {
    // K enters as code + 8: a group's sum starts at -8 sum q, which a matrix
    // instruction with a constant -8 gives in every row.
    const uint32_t m8 = 0xC100C100u;  // bf16 -8, twice
    const bf16x8 minus8 = __builtin_bit_cast(bf16x8, (u32x4{m8, m8, m8, m8}));
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct)
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        f32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < PLANES; ++t) v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus8, column(ct, t, j), v, 0, 0, 0);
        qs[ct][j] = v[0];
      }
  }
  // Tiles that every column of the wave sees whole need no mask.
  const int clear_to = past + i0 + 1, clear_from = a.window ? past + i1 - a.window + 1 : 0;
  // (a tensor scale of 0 must not meet a masked score)
  const float scale = FMT == kNV ? fmaxf(a.scale * a.k_gs[0], 1e-30f) : fmaxf(a.scale, 1e-30f);

  f32x4 acc[CH][NQ];
  float m[NQ], l[NQ];
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    m[ct] = -FLT_MAX;
    l[ct] = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) acc[j][ct] = f32x4{0, 0, 0, 0};
  }

  const auto o = offsets<FMT, D>();
  const int mask = (1 << a.page_log2) - 1;
  const int top = (hi - 1) & ~15, bottom = lo & ~15;  // halves that hold tokens
  // First token of half u of step k, or of the nearest half that holds tokens.
  auto half_at = [&](int k, int u) {
    const int t = (first + k * step) * kTile + 16 * u;
    return t > top ? top : t < bottom ? bottom : t;
  };
  int pages = 0;  // lane l: page of half l % 2 of step 32 i + l / 2
  bool bad = p.s.bad;
  auto read_pages = [&](int k) {
    const int at = half_at(k + (lane >> 1), lane & 1);
    int v = a.table[p.b * a.ldt + (at >> a.page_log2)];
    if (v < 0 || v >= a.pages) {
      bad = true;
      v = 0;
    }
    pages = v;
  };
  auto load = [&](RawT& w, int k) {
    if ((k & 31) == 0) read_pages(k);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int page = __builtin_amdgcn_readlane(pages, 2 * (k & 31) + u);
      const int64_t row = (((int64_t)page * a.kv + p.h) << a.page_log2) + (half_at(k, u) & mask);
      constexpr int kScaleRow = FMT == kMX ? D / 32 : D / 16;
      load_half<FMT, D>(w, u, a.k_codes + row * (D / 2), a.k_scales + row * kScaleRow, a.v_codes + row * (D / 2),
                        a.v_scales + row * kScaleRow, o);
    }
  };

  auto compute = [&](RawT& w, int k) {
    const int t0 = (first + k * step) * kTile;
    const bool clear = t0 >= clear_from && t0 + kTile <= clear_to;
    f32x4 s[2][NQ];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct) s[u][ct] = f32x4{0, 0, 0, 0};
      if constexpr (FMT == kINT && D > 64) {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
          u32x4 c = {w.kc[u][4 * i], w.kc[u][4 * i + 1], w.kc[u][4 * i + 2], w.kc[u][4 * i + 3]};
          transpose4(c);
#pragma unroll
          for (int j = 0; j < 4; ++j) w.kc[u][4 * i + j] = c[j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      bf16x8 qf[NQ][PLANES];
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct)
#pragma unroll
        for (int t = 0; t < PLANES; ++t) qf[ct][t] = column(ct, t, j);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (FMT == kINT) {
          const bf16x8 kf = expand<FMT>(w.kc[u][j], 0.0f);
          float sc[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int e = r * KJ + j;  // of the lane's four tokens' scales
            sc[r] = half_value(w.ks[u][e / 2] >> (16 * (e % 2)));
          }
#pragma unroll
          for (int ct = 0; ct < NQ; ++ct) {
            f32x4 g = {qs[ct][j], qs[ct][j], qs[ct][j], qs[ct][j]};
#pragma unroll
            for (int t = 0; t < PLANES; ++t) g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[ct][t], g, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) s[u][ct][r] = __builtin_fmaf(sc[r], g[r], s[u][ct][r]);
          }
        } else {
          const bf16x8 kf = expand<FMT>(w.kc[u][j], k_scale(w, u, j));
#pragma unroll
          for (int ct = 0; ct < NQ; ++ct)
#pragma unroll
            for (int t = 0; t < PLANES; ++t)
              s[u][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[ct][t], s[u][ct], 0, 0, 0);
        }
      }
      // Expanding more than one dword ahead costs registers, and with them waves.
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!clear) {
      asm volatile("");  // a branch, not selects on every step
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = t0 + 16 * u + 4 * q + r;
          // Places without a token may hold anything, also what 0 does not cancel.
          if (t < lo || t >= hi) {
#pragma unroll
            for (int i = 0; i < RawT::kV; ++i) w.vc[4 * u + r][i] = 0;
            w.vs[4 * u + r] = 0;
          }
#pragma unroll
          for (int ct = 0; ct < NQ; ++ct) {
            const bool seen = t >= lo && t <= pos[ct] && (!a.window || t > pos[ct] - a.window);
            s[u][ct][r] = seen ? s[u][ct][r] : -__builtin_inff();
          }
        }
    }
    // The running maximum moves where a score passes it by more than the slack.
    float high[NQ];
    bool grown = false;
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct) {
      float v = s[0][ct][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) v = fmaxf(v, s[i >> 2][ct][i & 3]);
      high[ct] = v * scale;
      grown |= high[ct] > m[ct] + kSlack;
    }
    if (__any(grown)) {
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct) {
        const float next = fmaxf(m[ct], column_max(high[ct]));
        const float f = __builtin_amdgcn_exp2f(m[ct] - next);
        m[ct] = next;
        l[ct] *= f;
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[j][ct][r] *= f;
      }
    }
    bf16x8 pf[NQ];
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][ct][i & 3], scale, -m[ct]));
        l[ct] += e[i];
      }
      pf[ct] = __builtin_bit_cast(bf16x8, (u32x4{pack(cvt_bf16(e[0], e[1])), pack(cvt_bf16(e[2], e[3])),
                                                pack(cvt_bf16(e[4], e[5])), pack(cvt_bf16(e[6], e[7]))}));
    }
    float vs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      vs[i] = FMT == kMX   ? __uint_as_float(w.vs[i] << 23)
              : FMT == kNV ? __builtin_amdgcn_cvt_f32_fp8(w.vs[i], 0)
                           : half_value(w.vs[i]);
#pragma unroll
    for (int i = 0; i < RawT::kV; ++i)
#pragma unroll
      for (int b = 0; b < (CH < 8 ? CH / 2 : 4); ++b) {
        u32x4 even, odd;
        expand_v<FMT, D>(w, vs, i, b, even, odd);
#pragma unroll
        for (int ct = 0; ct < NQ; ++ct) {
          acc[8 * i + 2 * b][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), pf[ct],
                                                                           acc[8 * i + 2 * b][ct], 0, 0, 0);
          acc[8 * i + 2 * b + 1][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), pf[ct],
                                                                               acc[8 * i + 2 * b + 1][ct], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  };

  if (steps > 0) {
    // Two register sets in turn; a load past the last step repeats a place in range.
    RawT w0, w1;
    load(w0, 0);
    for (int k = 0; k < steps; k += 2) {
      load(w1, k + 1);
      compute(w0, k);
      load(w0, k + 2);
      if (k + 1 < steps) compute(w1, k + 1);
    }
  }
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    l[ct] = column_sum(l[ct]);
    if (__any(bad)) l[ct] = __builtin_nanf("");
  }

  const float vg = FMT == kNV ? a.v_gs[0] : 1.0f;
  auto out_row = [&](int col) {
    const int i = col / a.group;
    return a.out + ((int64_t)(p.s.start + i) * a.kv * a.group + p.h * a.group + col - i * a.group) * D;
  };
  if constexpr (kAlone) {
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct) {
      const int col = c0 + 16 * ct + n, mine = col - p.t * NC;
      if (col >= all) continue;
      const float f = p.whole ? (l[ct] != 0.0f ? vg / l[ct] : 0.0f) : 1.0f;
      if (!p.whole && q == 0) {
        p.part[mine] = m[ct];
        p.part[NC + mine] = l[ct];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int ch = CH * (4 * q + r);
#pragma unroll
        for (int j = 0; j < CH; j += 4) {
          const f32x4 v = {acc[j][ct][r] * f, acc[j + 1][ct][r] * f, acc[j + 2][ct][r] * f, acc[j + 3][ct][r] * f};
          if (p.whole) {
            *reinterpret_cast<u32x2*>(out_row(col) + ch + j) = u32x2{pack(cvt_bf16(v[0], v[1])), pack(cvt_bf16(v[2], v[3]))};
          } else {
            *reinterpret_cast<f32x4*>(p.part + 2 * NC + mine * D + ch + j) = v;
          }
        }
      }
    }
  } else {
    // The four waves' results of a column meet in LDS: factors first, then quads of
    // channels, one per lane, without conflicts between banks.
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct)
      if (q == 0) {
        stat[0][wave][16 * ct + n] = m[ct];
        stat[1][wave][16 * ct + n] = l[ct];
      }
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct) {
      const int at = 16 * ct + n, col = c0 + at;
      float M = stat[0][0][at], L = 0.0f;
#pragma unroll
      for (int w = 1; w < 4; ++w) M = fmaxf(M, stat[0][w][at]);
#pragma unroll
      for (int w = 0; w < 4; ++w) L += stat[1][w][at] * __builtin_amdgcn_exp2f(stat[0][w][at] - M);
      const float f = __builtin_amdgcn_exp2f(m[ct] - M);
      const float g = p.whole ? (L != 0.0f ? vg / L : 0.0f) : 1.0f;
      if (!p.whole && wave == 0 && q == 0 && col < all) {
        p.part[at] = M;
        p.part[NC + at] = L;
      }
      constexpr int kQuads = CH / kParts<D>;  // quads of channels per lane: CH in all
#pragma unroll
      for (int part = 0; part < kParts<D>; ++part) {
        f32x4* red = reinterpret_cast<f32x4*>(lds + q_floats<D, SHAPE, PLANES>());
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          const int e = part * kQuads + i, r = e / (CH / 4), j = e % (CH / 4) * 4;
          red[(wave * kQuads + i) * 64 + lane] = f32x4{acc[j][ct][r], acc[j + 1][ct][r], acc[j + 2][ct][r], acc[j + 3][ct][r]} * f;
        }
        __syncthreads();
#pragma unroll
        for (int i0q = 0; i0q < kQuads; i0q += 4) {
          const int i = i0q + wave;
          if (i < kQuads) {
            f32x4 v = red[i * 64 + lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) v += red[(w * kQuads + i) * 64 + lane];
            const int e = part * kQuads + i, ch = CH * (4 * q + e / (CH / 4)) + e % (CH / 4) * 4;
            if (col < all) {
              if (p.whole) {
                *reinterpret_cast<u32x2*>(out_row(col) + ch) =
                    u32x2{pack(cvt_bf16(v[0] * g, v[1] * g)), pack(cvt_bf16(v[2] * g, v[3] * g))};
              } else {
                *reinterpret_cast<f32x4*>(p.part + 2 * NC + at * D + ch) = v;
              }
            }
          }
        }
        __syncthreads();
      }
    }
  }
}

template <int FMT, int D, int SHAPE, int PLANES>
__global__ __launch_bounds__(kThreads, 2) void kv4_attention_kernel(KvAttnArgs a) {
  constexpr int NC = kv_columns(SHAPE, D);
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ float stat[2][4][32];
  __shared__ PlanLds plan;
  const int w = blockIdx.x;
  Chunk chunk;
  const Shares s = shares_of<NC>(a, plan, chunk);
  const int64_t begin = (int64_t)w * s.share;
  KvJoin join = {};
  if (begin < s.total) {
    const int end = (int)(begin + s.share < s.total ? begin + s.share : s.total);
    Place at = find<NC>(a, plan, chunk, s.whole, (int)begin);
    for (int u = (int)begin; u < end;) {
      const int nu = units_of<NC>(a, at.s, at.t);
      const int take = s.whole || nu - at.off < end - u ? nu - at.off : end - u;
      Piece p;
      p.b = at.b;
      p.h = at.h;
      p.t = at.t;
      p.s = at.s;
      p.whole = take == nu;
      p.part = a.part + ((int64_t)w * 2 + (u == (int)begin ? 0 : 1)) * (NC * (D + 2));
      const int i0 = at.t * NC / a.group, il = (at.t * NC + NC - 1) / a.group;
      const Span all = span_of(a, at.s, i0, il < at.s.count ? il : at.s.count - 1);
      const int64_t from = (int64_t)(all.lo / kKvUnit + at.off) * kKvUnit, to = from + (int64_t)take * kKvUnit;
      p.lo = all.lo > from ? all.lo : (int)from;
      p.hi = all.hi < to ? all.hi : (int)to;
      attend<FMT, D, SHAPE, PLANES>(a, p, lds, stat);
      if (at.off == 0 && take < nu) {
        const int cols = at.s.count * a.group - at.t * NC;
        join = KvJoin{(u + nu - 1) / s.share - w + 1, u == (int)begin ? 0 : 1, cols < NC ? cols : NC, at.t * NC, at.s.start, at.h, {0, 0}};
      }
      u += s.whole ? 1 : take;
      if (u >= end) break;
      at.off = 0;
      if (++at.t == items_of<NC>(a, at.s)) {
        at.t = 0;
        if (++at.h == a.kv) {
          at.h = 0;
          do {
            at.s = seq_of(a, ++at.b);
          } while (at.s.count == 0);
        }
      }
      __syncthreads();  // LDS changes its use
    }
  }
  if (w < a.runs && threadIdx.x == 0) a.join[w] = join;
}

// The pieces of the item that begins in run blockIdx.x and goes on behind its end, if there is
// one.  A workgroup takes a column at a time; lanes take four channels each, so that it
// reads 1024 / D pieces at once.
template <int D, int SHAPE>
__global__ __launch_bounds__(kThreads) void kv4_join_kernel(KvAttnArgs a, int nv) {
  constexpr int NC = kv_columns(SHAPE, D), kLanes = D / 4, kAtOnce = kThreads / kLanes;
  __shared__ float wave_m[4], wave_l[kAtOnce];
  __shared__ __attribute__((aligned(16))) float sums[kAtOnce][D];
  const KvJoin j = a.join[blockIdx.x];
  if (j.pieces == 0) return;
  const int tid = threadIdx.x, mine = tid / kLanes, ch = tid % kLanes * 4;
  constexpr int64_t kPiece = NC * (D + 2);
  const float vg = nv ? a.v_gs[0] : 1.0f;
  // Piece i: the run's second place perhaps, then every run's first.
  const float* base = a.part + (int64_t)blockIdx.x * 2 * kPiece;
  auto piece = [&](int i) { return base + ((int64_t)i * 2 + (i == 0 ? j.second : 0)) * kPiece; };
  for (int c = blockIdx.y; c < j.cols; c += gridDim.y) {
    float M = -FLT_MAX;
    for (int i = tid; i < j.pieces; i += kThreads) M = fmaxf(M, piece(i)[c]);
    M = wave_max(M);
    if ((tid & 63) == 0) wave_m[tid >> 6] = M;
    __syncthreads();
    M = fmaxf(fmaxf(wave_m[0], wave_m[1]), fmaxf(wave_m[2], wave_m[3]));
    float L = 0.0f;
    f32x4 v = {0, 0, 0, 0};
#pragma unroll 4
    for (int i = mine; i < j.pieces; i += kAtOnce) {
      const float* p = piece(i);
      const float f = __builtin_amdgcn_exp2f(p[c] - M);
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + 2 * NC + c * D + ch);
      L = __builtin_fmaf(p[NC + c], f, L);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(x[e], f, v[e]);
    }
    *reinterpret_cast<f32x4*>(&sums[mine][ch]) = v;
    if (ch == 0) wave_l[mine] = L;
    __syncthreads();
    if (tid < D) {
      float sum = 0.0f, all = 0.0f;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        sum += sums[i][tid];
        all += wave_l[i];
      }
      const int col = j.col0 + c, i = col / a.group;
      uint16_t* o = a.out + ((int64_t)(j.start + i) * a.kv * a.group + j.head * a.group + col - i * a.group) * D;
      o[tid] = __builtin_bit_cast(uint16_t, (__bf16)(all != 0.0f ? sum * (vg / all) : 0.0f));
    }
    __syncthreads();
  }
}

template <int FMT, int D, int SHAPE, int PLANES>
hipError_t go(const KvAttnArgs& a, hipStream_t s) {
  hipError_t e = launch_lds(kv4_attention_kernel<FMT, D, SHAPE, PLANES>, dim3(a.workgroups), kThreads,
                            4 * lds_floats<D, SHAPE, PLANES>(), s, a);
  if (e != hipSuccess || a.runs == 0) return e;
  hipLaunchKernelGGL((kv4_join_kernel<D, SHAPE>), dim3(a.runs, kv_columns(SHAPE, D) / 4), dim3(kThreads), 0, s, a,
                     FMT == kNV ? 1 : 0);
  return hipGetLastError();
}

template <int FMT, int D, int PLANES>
hipError_t go_shape(const KvAttnArgs& a, int shape, hipStream_t s) {
  if (shape == kKvNarrow) return go<FMT, D, kKvNarrow, PLANES>(a, s);
  if constexpr (D <= 128) {
    if (shape == kKvWide) return go<FMT, D, kKvWide, PLANES>(a, s);
  }
  return go<FMT, D, kKvPrompt, PLANES>(a, s);
}

template <int FMT, int D>
hipError_t go_planes(const KvAttnArgs& a, int shape, hipStream_t s) {
  return a.T ? go_shape<FMT, D, 2>(a, shape, s) : go_shape<FMT, D, 1>(a, shape, s);
}

template <int FMT>
hipError_t launch(const KvAttnArgs& a, int shape, hipStream_t s) {
  if (a.D == 64) return go_planes<FMT, 64>(a, shape, s);
  if (a.D == 128) return go_planes<FMT, 128>(a, shape, s);
  return go_planes<FMT, 256>(a, shape, s);
}

}  // namespace kv4
}  // namespace wush

#endif  // WUSH_KV4_ATTENTION_H_
