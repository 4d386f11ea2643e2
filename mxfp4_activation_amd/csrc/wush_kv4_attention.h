// Attention of a few or many queries over a paged cache of keys and values in
// 4 bits.  Device code, included once per format (wush_kv4_*.hip).
//
//   out_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(scale q_i . k_t)
//
// over the tokens t that query i sees, with the running maximum of the scores
// taken out of the exponent.
//
// Work.  An item is one key head's queries of one sequence: up to 16, 32 or 128 (64 for heads of 256)
// columns (query, head of the group).  Its tokens come in units of 128.  Items
// and units are counted on the device, from the lengths as they are when the kernel
// runs, and items of more than a share of them are cut into pieces of about that many, one
// per workgroup, so that one long sequence among short ones is spread over the whole chip.
// Pieces (maximum, sum, unscaled result) meet in a second kernel by way of the workspace.
//
// A wave's step is 32 tokens.  K, V and the scores stay in registers, without a barrier; so do the
// queries of up to 16 columns (transformed ones, heads of 256 and more columns are read from LDS).
// Prompts have K and V in LDS, expanded once per workgroup (attend_prompt).
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
// Exactness.  K: E2M1 times E8M0 or E4M3 has at most 6 significant bits and is exact in
// bf16, as are INT4's integers, whose fp16 scale multiplies the fp32 sums over one group.
// P and V: MXFP4's values need bf16's range; P is then rounded to 8 bits, as the result is.
// NVFP4's and INT4's enter as fp16, and P with 11 bits: E2M1 times E4M3 is exact, an
// integer times INT4's scale is rounded to 11 bits.  P is at most 2^8 there and taken
// times 2^7; what fp16's range cuts off is at most 2^-32 of the largest probability.
// INT4's values are taken times 1/8, so that the largest scale's are finite: what that
// cuts off is at most 2^-22, no more than rounding so small a scale to fp16 has lost.
// Sums are fp32; a transformed query enters as two bf16 planes (16 bits).
#ifndef WUSH_KV4_ATTENTION_H_
#define WUSH_KV4_ATTENTION_H_

#include <float.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "wush_kv4.h"
#include "wush_w4_core.h"
#include "wush_wave.h"

namespace wush {
namespace kv4 {

using namespace w4;

constexpr int kThreads = 256;
constexpr int kTile = 32;   // tokens of a wave's step
constexpr float kSlack = 8.0f;  // log2 by which scores may pass the running maximum

// Whether P and V are fp16 (else bf16), log2 of the factor at P and V's factor.
template <int FMT>
constexpr bool kHalf = FMT != kMX;
template <int FMT>
constexpr float kPShift = kHalf<FMT> ? 7.0f : 0.0f;
template <int FMT>
constexpr float kVFactor = FMT == kINT ? 0.125f : 1.0f;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f16x2 half2_of(uint32_t v) { return __builtin_bit_cast(f16x2, v); }
__device__ __forceinline__ uint32_t bits_of(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ f16x2 cvt_f16(float a, float b) { return __builtin_convertvector((f32x2{a, b}), f16x2); }

// O^T += V^T P^T.
template <int FMT>
__device__ __forceinline__ f32x4 add_pv(const u32x4& v, const u32x4& p, const f32x4& c) {
  if constexpr (kHalf<FMT>) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), __builtin_bit_cast(f16x8, p), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, p), c, 0, 0, 0);
  }
}

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

// What a sequence and key head's items come to in units, all together and at most, and
// cut for a share of units: in pieces, in items that have several, and in pieces of those.
struct Load {
  int units, items, most, pieces, several, cut;
};
template <int NC>
__device__ __forceinline__ Load load_of(const KvAttnArgs& a, const Seq& s, int share) {
  Load l = {0, items_of<NC>(a, s), 0, 0, 0, 0};
  for (int t = 0; t < l.items; ++t) {
    const int u = units_of<NC>(a, s, t);
    const int p = (u - 1) / share + 1;
    l.units += u;
    l.most = l.most > u ? l.most : u;
    l.pieces += p;
    l.several += p > 1;
    l.cut += p > 1 ? p : 0;
  }
  return l;
}

// A piece: sequence, key head, item, units of the item, of it from `off` on `take`; its place
// in the workspace; how many there are of the item, and which one it is; the item's place
// among those with several.
struct Place {
  int b, h, t, units, off, take, slot, pieces, index, rank;
  Seq s;
};

struct PlanLds {
  int sums[3][4];
  int b, pieces, several, cut, per_head, several_per_head, cut_per_head;
  Seq s;
  Place at;  // of a run's piece, while the waves are at it
  int left;
};

// A sequence per lane where there are no more (every wave for itself), otherwise one per
// thread, 256 at a time.
__device__ __forceinline__ bool few(const KvAttnArgs& a) { return a.B <= 64; }
__device__ __forceinline__ int place_of(const KvAttnArgs& a) { return few(a) ? threadIdx.x & 63 : threadIdx.x; }
__device__ __forceinline__ Seq seq_or_none(const KvAttnArgs& a, int b) { return b < a.B ? seq_of(a, b) : Seq{0, 0, 0, false}; }

// How the units are shared out: pieces of items, of at most `share` units, or (by_runs) an
// equal run of units for every workgroup, which may end one item's and begin another's.
struct Shares {
  int share;
  bool by_runs;
  int total;  // units, by runs
};

// Items are taken whole where nothing may be cut, and where that takes no longer: the longest
// times the rounds of them is at most 1.1 times the mean load, and for few columns the pieces'
// meeting, as long as 6 units, more.  (33 sequences, 16 heads, windows of 1000 tokens, 8 or 9
// units: 15.9 us whole, 18.3 in two pieces each.  Two prompts of 1000 queries behind 16384
// tokens, 456 items for 512 places, 1.17 times the mean: 533 us whole, 497 by runs.)
// A share is what lets all pieces be there at once, but 4 units before it is a second
// workgroup on a CU (8 sequences of 1000 tokens, 16 heads: 10.6 us in shares of 4, 13.4 of 1).
// Short shares keep to one item, since a second one costs a second start: 48 sequences of 1 to
// 8192 tokens, 7 units each, 30.8 us by runs and 22.1 by pieces.  Long ones are better equal: 48
// of 3584 to 9557, 14 units, 45.6 and 48.7, 16 of up to 131072, 105 units, 302 and 383.  Between them it
// depends: 8 to 10 units in 48 sequences of about the same length, INT4, 31.8 and 34.5, MXFP4 37.2 and 37.4.
constexpr int kRunUnits = 12;
constexpr float kJoinUnits = 6.0f;
constexpr int kAloneUnits = 4;
template <int NC, int SHAPE>
__device__ __forceinline__ Shares shares_of(const KvAttnArgs& a, PlanLds& l, const Seq& first) {
  Shares r = {INT32_MAX, false, 0};
  if (a.runs == 0) return r;
  int units = 0, items = 0, most = 0;
  for (int c = 0; c < a.B; c += kThreads) {
    const Load o = load_of<NC>(a, c == 0 ? first : seq_or_none(a, c + (int)threadIdx.x), INT32_MAX);
    units += a.kv * o.units;
    items += a.kv * o.items;
    most = most > o.most ? most : o.most;
  }
  units = __builtin_amdgcn_readlane(wave_scan(units), 63);
  items = __builtin_amdgcn_readlane(wave_scan(items), 63);
  most = wave_max_int(most);
  if (!few(a)) {
    if ((threadIdx.x & 63) == 0) {
      const int wave = threadIdx.x >> 6;
      l.sums[0][wave] = units;
      l.sums[1][wave] = items;
      l.sums[2][wave] = most;
    }
    __syncthreads();
    units = items = most = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      units += l.sums[0][w];
      items += l.sums[1][w];
      most = most > l.sums[2][w] ? most : l.sums[2][w];
    }
    units = uniform(units);
    items = uniform(items);
    most = uniform(most);
    __syncthreads();
  }
  // (More only where q_start does not ascend: the workspace has no room for them.)
  if (items > a.items) return r;
  const float meeting = SHAPE == kKvPrompt ? 0.0f : kJoinUnits * (float)a.runs;
  if ((float)most * (float)((items + a.runs - 1) / a.runs) * (float)a.runs <= 1.1f * (float)units + meeting) return r;
  r.share = (units - 1) / a.runs + 1;
  if (SHAPE != kKvPrompt) {
    const int alone = (units - 1) / 256 + 1, least = alone < kAloneUnits ? alone : kAloneUnits;
    r.share = r.share < least ? least : r.share;
  }
  r.by_runs = r.share >= kRunUnits;
  r.total = units;
  return r;
}

// Piece number w of all, with `share` units at most, for the whole workgroup; false if there
// are not so many.  `total`: items that have several (for w = 0, or few sequences).
template <int NC>
__device__ __forceinline__ bool find(const KvAttnArgs& a, PlanLds& l, const Seq& first, int share, int w, Place& p, int& total) {
  int pieces, several, cut, per_head, several_per_head, cut_per_head;
  total = 0;
  if (few(a)) {
    const Load o = load_of<NC>(a, first, share);
    const int own = a.kv * o.pieces, items = a.kv * o.several, many = a.kv * o.cut;
    const int upto = wave_scan(own), items_upto = wave_scan(items), many_upto = wave_scan(many);
    total = __builtin_amdgcn_readlane(items_upto, 63);
    if (w >= __builtin_amdgcn_readlane(upto, 63)) return false;
    const int b = __builtin_ctzll(__ballot(w < upto));
    p.b = b;
    p.s.start = __builtin_amdgcn_readlane(first.start, b);
    p.s.count = __builtin_amdgcn_readlane(first.count, b);
    p.s.len = __builtin_amdgcn_readlane(first.len, b);
    p.s.bad = __builtin_amdgcn_readlane(first.bad, b);
    pieces = __builtin_amdgcn_readlane(upto - own, b);
    several = __builtin_amdgcn_readlane(items_upto - items, b);
    cut = __builtin_amdgcn_readlane(many_upto - many, b);
    per_head = __builtin_amdgcn_readlane(o.pieces, b);
    several_per_head = __builtin_amdgcn_readlane(o.several, b);
    cut_per_head = __builtin_amdgcn_readlane(o.cut, b);
  } else {
    int base = 0, cut_base = 0;
    bool found = false;
    for (int c = 0; c < a.B; c += kThreads) {
      const int b = c + (int)threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
      const Seq s = c == 0 ? first : seq_or_none(a, b);
      const Load o = load_of<NC>(a, s, share);
      const int own = a.kv * o.pieces, items = a.kv * o.several, many = a.kv * o.cut;
      const int upto = wave_scan(own), items_upto = wave_scan(items), many_upto = wave_scan(many);
      __syncthreads();
      if (lane == 63) {
        l.sums[0][wave] = upto;
        l.sums[1][wave] = many_upto;
        l.sums[2][wave] = items_upto;
      }
      __syncthreads();
      int before = base + upto - own, many_before = cut_base + many_upto - many, items_before = total + items_upto - items;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < wave) {
          before += l.sums[0][i];
          many_before += l.sums[1][i];
          items_before += l.sums[2][i];
        }
        base += l.sums[0][i];
        cut_base += l.sums[1][i];
        total += l.sums[2][i];
      }
      if (w >= before && w - before < own) {
        l.b = b;
        l.pieces = before;
        l.several = items_before;
        l.cut = many_before;
        l.per_head = o.pieces;
        l.several_per_head = o.several;
        l.cut_per_head = o.cut;
        l.s = s;
      }
      found = w < base;
      // The first workgroup counts them all.
      if (found && w != 0) break;
    }
    total = uniform(total);
    if (!uniform(found)) return false;
    __syncthreads();
    p.b = uniform(l.b);
    p.s.start = uniform(l.s.start);
    p.s.count = uniform(l.s.count);
    p.s.len = uniform(l.s.len);
    p.s.bad = uniform(l.s.bad);
    pieces = uniform(l.pieces);
    several = uniform(l.several);
    cut = uniform(l.cut);
    per_head = uniform(l.per_head);
    several_per_head = uniform(l.several_per_head);
    cut_per_head = uniform(l.cut_per_head);
  }
  const int at = w - pieces;
  p.h = at / per_head;
  p.index = at - p.h * per_head;
  p.rank = several + p.h * several_per_head;
  p.slot = cut + p.h * cut_per_head;
  for (p.t = 0;; ++p.t) {
    p.units = units_of<NC>(a, p.s, p.t);
    p.pieces = (p.units - 1) / share + 1;
    if (p.index < p.pieces) break;
    p.index -= p.pieces;
    p.rank += p.pieces > 1;
    p.slot += p.pieces > 1 ? p.pieces : 0;
  }
  p.slot += p.index;
  // Pieces of about the same size.
  const int each = p.pieces > 1 ? (p.units - 1) / p.pieces + 1 : p.units;
  p.off = p.index * each;
  p.take = p.units - p.off < each ? p.units - p.off : each;
  return true;
}

// The item behind p's.
template <int NC>
__device__ __forceinline__ void next_item(const KvAttnArgs& a, Place& p) {
  p.rank += p.units > 1;
  if (++p.t == items_of<NC>(a, p.s)) {
    p.t = 0;
    if (++p.h == a.kv) {
      p.h = 0;
      do {
        p.s = seq_of(a, ++p.b);
      } while (p.s.count == 0);
    }
  }
  p.units = units_of<NC>(a, p.s, p.t);
  p.off = 0;
}

// ------------------------------------------------------------ one step's data

template <int FMT, int D>
struct Raw {
  static constexpr int kK = D / 32;                       // dwords of K per lane and half
  static constexpr int kV = D / 16 > 8 ? D / 128 : 1;     // dwords of V per lane and token
  static constexpr int kKS = FMT == kINT ? D / 16 : 1;    // dwords of K's scales that a lane goes by
  uint32_t kc[2][kK];
  uint32_t ks[2];  // INT4: lane n has dword n % kKS, and hands it to its 16 lanes when it is wanted
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
__device__ __forceinline__ Offsets<FMT, D> offsets(int lane) {
  constexpr int kRow = D / 2;
  constexpr int kScaleRow = FMT == kMX ? D / 32 : D / 16;
  const int n = lane & 15, q = lane >> 4;
  Offsets<FMT, D> o;
  if (FMT == kINT) {
    o.k = n * kRow + (D == 64 ? 4 : 16) * q;
    o.ks = 4 * q * kScaleRow + 4 * (n % Raw<FMT, D>::kKS);
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
__device__ __forceinline__ void load_k(Raw<FMT, D>& w, int u, const uint8_t* kc, const uint8_t* ks, const Offsets<FMT, D>& o) {
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
    w.ks[u] = load_unaligned<uint32_t>(ks + o.ks);
  } else if constexpr (FMT == kMX) {
    w.ks[u] = D == 256 ? load_unaligned<uint16_t>(ks + o.ks) : ks[o.ks];
  } else {
    w.ks[u] = D == 256   ? load_unaligned<uint32_t>(ks + o.ks)
              : D == 128 ? load_unaligned<uint16_t>(ks + o.ks)
                         : ks[o.ks];
  }
}

template <int FMT, int D>
__device__ __forceinline__ void load_v(Raw<FMT, D>& w, int u, const uint8_t* vc, const uint8_t* vs, const Offsets<FMT, D>& o) {
  constexpr int kRow = D / 2;
  constexpr int kScaleRow = FMT == kMX ? D / 32 : D / 16;
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

// f(0) .. f(N - 1) with the numbers as constants.
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// INT4: scales of group J of the lane quarter's four tokens, out of its lanes' dwords.
template <int KJ, int J>
__device__ __forceinline__ void k_scales(uint32_t ks, float (&sc)[4]) {
  each<4>([&](auto r) {
    constexpr int e = r * KJ + J;
    sc[r] = half_value(dpp<0x150 + e / 2, 0xf>(0, ks) >> (16 * (e % 2)));  // row_newbcast
  });
}

// Scale of K's dword j of half u, applied to the elements (not INT4).
template <int FMT, int D>
__device__ __forceinline__ float k_scale(const Raw<FMT, D>& w, int u, int j) {
  if constexpr (FMT == kMX) {
    return __uint_as_float(((w.ks[u] >> (8 * (j / 4))) & 0xFFu) << 23);
  } else {
    const uint32_t v = w.ks[u];
    const int i = j / 2;  // two dwords share a group of 16
    return i == 0   ? __builtin_amdgcn_cvt_f32_fp8(v, 0)
           : i == 1 ? __builtin_amdgcn_cvt_f32_fp8(v, 1)
           : i == 2 ? __builtin_amdgcn_cvt_f32_fp8(v, 2)
                    : __builtin_amdgcn_cvt_f32_fp8(v, 3);
  }
}

// Byte B (two channels) of a dword of codes, with their scale or E2M1's own values.
template <int B>
__device__ __forceinline__ uint32_t mx_pair(uint32_t codes, float scale) {
  return pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, B));
}
template <int B>
__device__ __forceinline__ f16x2 e2m1_pair(uint32_t codes) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, B);
}

// Scales of V's eight tokens as expand_v wants them: fp32 (MXFP4), twice the same fp16
// (NVFP4), pairs of fp16 (INT4).
template <int FMT>
struct VScales {
  uint32_t s[FMT == kINT ? 4 : 8];
};
template <int FMT, int D>
__device__ __forceinline__ VScales<FMT> v_scales(const Raw<FMT, D>& w) {
  VScales<FMT> o;
#pragma unroll
  for (int i = 0; i < (FMT == kINT ? 4 : 8); ++i) {
    if constexpr (FMT == kMX) {
      o.s[i] = w.vs[i] << 23;
    } else if constexpr (FMT == kNV) {
      const float v = __builtin_amdgcn_cvt_f32_fp8(w.vs[i], 0);
      o.s[i] = bits_of(cvt_f16(v, v));
    } else {
      o.s[i] = w.vs[2 * i] | w.vs[2 * i + 1] << 16;
    }
  }
  return o;
}

// Byte B (two channels) of V's dword i for all eight tokens, as the A operands of two
// matrix instructions.
template <int FMT, int D, int B>
__device__ __forceinline__ void expand_v(const Raw<FMT, D>& w, const VScales<FMT>& v, int i, u32x4& even, u32x4& odd) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t d0 = w.vc[2 * p][i], d1 = w.vc[2 * p + 1][i];
    if constexpr (FMT == kINT) {
      // Both tokens' byte.  Codes with their sign bits turned over are codes + 8; as mantissa
      // bits of fp16 numbers they stand for eighths: 128 + (code + 8) / 8, 8 + (code + 8) / 8.
      const uint32_t t = __builtin_amdgcn_perm(d1, d0, 0x0C000C00u | (uint32_t)((4 + B) << 16 | B));
      const f16x2 s = half2_of(v.s[p]);
      even[p] = bits_of((half2_of((t & 0x000F000Fu) ^ 0x58085808u) - f16x2{129, 129}) * s);
      odd[p] = bits_of((half2_of((t & 0x00F000F0u) ^ 0x48804880u) - f16x2{9, 9}) * s);
    } else {
      uint32_t c0, c1;
      if constexpr (FMT == kMX) {
        c0 = mx_pair<B>(d0, __uint_as_float(v.s[2 * p]));
        c1 = mx_pair<B>(d1, __uint_as_float(v.s[2 * p + 1]));
      } else {
        c0 = bits_of(e2m1_pair<B>(d0) * half2_of(v.s[2 * p]));
        c1 = bits_of(e2m1_pair<B>(d1) * half2_of(v.s[2 * p + 1]));
      }
      even[p] = __builtin_amdgcn_perm(c1, c0, 0x05040100u);
      odd[p] = __builtin_amdgcn_perm(c1, c0, 0x07060302u);
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

// INT4: the lane's codes of half u, regrouped so that dword j is group j's.
template <int FMT, int D>
__device__ __forceinline__ void arrange_k(Raw<FMT, D>& w, int u) {
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

// Scales whose values may not be finite: fp16's infinities and NaN, E4M3's NaN, and the E8M0 scales
// with which a code passes bf16's range.
template <int FMT>
constexpr uint32_t kOpenBits = FMT == kMX ? 0xFF : FMT == kNV ? 0x7F : 0x7C00;
template <int FMT>
constexpr uint32_t kOpenFrom = FMT == kMX ? 253 : kOpenBits<FMT>;
template <int FMT>
__device__ __forceinline__ bool open_scale(uint32_t s) {
  return (s & kOpenBits<FMT>) >= kOpenFrom<FMT>;
}

// Zeros for the tokens outside [lo, hi) of a step that some column does not see whole, which may hold
// anything, and a scale of 0 for values that may not be finite, which a probability of 0 would
// not cancel (spoiled has what they are to the columns that see them); whether there were any of those.
template <int FMT, int D>
__device__ __forceinline__ bool clear_v(Raw<FMT, D>& w, int t0, int lo, int hi) {
  const int q = (threadIdx.x & 63) >> 4;
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int t = t0 + 16 * (e / 4) + 4 * q + e % 4;
    if (t < lo || t >= hi) {
#pragma unroll
      for (int i = 0; i < Raw<FMT, D>::kV; ++i) w.vc[e][i] = 0;
      w.vs[e] = 0;
    }
    most = max(most, w.vs[e] & kOpenBits<FMT>);
    w.vs[e] = open_scale<FMT>(w.vs[e]) ? 0 : w.vs[e];
  }
  return __any(most >= kOpenFrom<FMT>);
}

// Whether a column sees token t.
__device__ __forceinline__ bool sees(int t, int pos, int window) { return t <= pos && (!window || t > pos - window); }

// Scores of tokens that a column does not see become -inf.
template <int NQ>
__device__ __forceinline__ void mask_scores(f32x4 (&s)[2][NQ], int t0, int lo, const int (&pos)[NQ], int window) {
  const int q = (threadIdx.x & 63) >> 4;
  // (The scores pass through an empty statement, so that this stays behind its branch: as
  // selects it would be a third of every step's instructions.)
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct) asm volatile("" : "+v"(s[u][ct]));
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = t0 + 16 * u + 4 * q + r;
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct) {
        s[u][ct][r] = t >= lo && sees(t, pos[ct], window) ? s[u][ct][r] : -__builtin_inff();
      }
    }
}

// Of the scores, with K's tensor scale.  One of 0 must not meet a masked score; one that is not
// a number makes the results so, as does a negative one, with which the running maximum
// would be a minimum.
template <int FMT>
__device__ __forceinline__ float score_scale(const KvAttnArgs& a) {
  if (FMT != kNV) return fmaxf(a.scale, 0x1p-149f);  // (in a vector register: INT4 prompts 641 us, 681 from a scalar one)
  const float f = a.scale * a.k_gs[0];
  return f > 0.0f ? f : f == 0.0f ? FLT_MIN : __builtin_nanf("");
}

// Scores of 32 tokens to probabilities, up to the running maximum m, as B operands.  l sums
// what they were rounded to, so that where one token outweighs the others nothing of the
// rounding is left.
template <int FMT, int NQ, int CH>
__device__ __forceinline__ void softmax_step(const f32x4 (&s)[2][NQ], float scale, float (&m)[NQ], float (&l)[NQ],
                                             f32x4 (&acc)[CH][NQ], u32x4 (&pf)[NQ]) {
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
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    float e[8];
    const float shift = kPShift<FMT> - m[ct];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][ct][i & 3], scale, shift));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kHalf<FMT>) {
        const f16x2 c = cvt_f16(e[2 * i], e[2 * i + 1]);
        pf[ct][i] = bits_of(c);
        l[ct] = __builtin_amdgcn_fdot2(c, f16x2{1, 1}, l[ct], false);
      } else {
        const bf16x2 c = cvt_bf16(e[2 * i], e[2 * i + 1]);
        pf[ct][i] = pack(c);
        l[ct] = __builtin_amdgcn_fdot2_f32_bf16(c, bf16x2{(__bf16)1.0f, (__bf16)1.0f}, l[ct], false);
      }
    }
  }
}

// Orders this wave's LDS accesses.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int D>
constexpr int kQLine = D + 8;  // of a query in LDS, elements

// Whether the columns' operands stay in LDS (transformed ones in two planes, long ones, or two
// tiles of them, which spilled) rather than in registers, and the elements that a tile of
// them takes there.
template <int FMT, int D, int SHAPE, int PLANES>
constexpr bool kStaged = PLANES == 2 || D == 256 || SHAPE != kKvNarrow;
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
template <int FMT, int D, int SHAPE, int PLANES>
constexpr int q_floats() {
  return kStaged<FMT, D, SHAPE, PLANES> ? kv_tiles(SHAPE, D) * kQTile<D, PLANES> / 2 : 0;
}

struct Piece {
  int b, h, t;      // sequence, key head, item
  int lo, hi;       // tokens, within the item's
  bool whole;       // of the item
  float* part;      // where it goes if not
  Seq s;
};

// Tokens of the units that a place takes.
template <int NC>
__device__ __forceinline__ Span tokens_of(const KvAttnArgs& a, const Place& at) {
  const int i0 = at.t * NC / a.group, il = (at.t * NC + NC - 1) / a.group;
  const Span all = span_of(a, at.s, i0, il < at.s.count ? il : at.s.count - 1);
  const int64_t from = (int64_t)(all.lo / kKvUnit + at.off) * kKvUnit, to = from + (int64_t)at.take * kKvUnit;
  return Span{all.lo > from ? all.lo : (int)from, all.hi < to ? all.hi : (int)to};
}

// Tokens that all columns of item t see.
template <int NC>
__device__ __forceinline__ Span clear_of(const KvAttnArgs& a, const Seq& s, int t) {
  const int past = s.len - s.count, il = (t * NC + NC - 1) / a.group;
  return Span{a.window ? past + (il < s.count ? il : s.count - 1) - a.window + 1 : 0, past + t * NC / a.group + 1};
}

// Row of the result for a column of the piece's sequence.
__device__ __forceinline__ uint16_t* out_row(const KvAttnArgs& a, const Piece& p, int col, int D) {
  const int i = col / a.group;
  return a.out + ((int64_t)(p.s.start + i) * a.kv * a.group + p.h * a.group + col - i * a.group) * D;
}

// Of a piece's tokens, without a window, those of steps that do not lie before clear_to.
__device__ __forceinline__ Span behind(const Span& tokens, int clear_to, int window) {
  const int from = clear_to & -kTile;
  return Span{!window && from > tokens.lo ? from : tokens.lo, tokens.hi};
}

// What clear_v took out, for the columns that see it: their results are NaN in the channels of its
// group.  Sets bit r for row r of the lane's results, whose channels are those of lane 4 q + r of
// V.  Goes once more over the scales of these of the piece's tokens.
template <int FMT, int D, int NQ>
__device__ __forceinline__ void spoiled(const KvAttnArgs& a, int b, int h, const Span& tokens, const int (&pos)[NQ],
                                        uint32_t (&bad)[NQ]) {
  constexpr int kScaleRow = FMT == kMX ? D / 32 : D / 16;
  // (The lane is counted here, so that no register is kept for it over the steps.)
  uint32_t none = 0;
  asm volatile("" : "+s"(none));
  const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, none)), q = lane >> 4;
  const uint32_t at = offsets<FMT, D>(lane).vs;
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) bad[ct] = 0;
#pragma unroll 1
  for (int half = tokens.lo & ~15; half < tokens.hi; half += 16) {
    const int page = a.table[b * a.ldt + (half >> a.page_log2)];
    if (page < 0 || page >= a.pages) continue;
    const int64_t row = (((int64_t)page * a.kv + h) << a.page_log2) + (half & ((1 << a.page_log2) - 1));
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
      const uint8_t* s = a.v_scales + row * kScaleRow + at + e * kScaleRow;
      const int mine = half + 4 * q + e;
      const bool open =
          mine >= tokens.lo && mine < tokens.hi && open_scale<FMT>(FMT == kINT ? load_unaligned<uint16_t>(s) : *s);
      const uint64_t lanes = __ballot(open);
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const uint32_t rows = (uint32_t)(lanes >> (16 * k)) >> (4 * q) & 15u;
#pragma unroll
        for (int ct = 0; ct < NQ; ++ct) bad[ct] |= sees(half + 4 * k + e, pos[ct], a.window) ? rows : 0u;
      }
    }
  }
}

// The same for a wave's columns of a prompt's piece, c0 of the item's on, with operands from where
// they are kept anyway: registers that held them through the steps cost NVFP4 and INT4 prompts up
// to 17% of their time.
template <int FMT, int D, int NC, int NQ>
__device__ __forceinline__ void spoiled(const PlanLds& plan, int c0, uint32_t (&bad)[NQ]) {
  typedef const KvAttnArgs __attribute__((address_space(4))) Kernarg;
  Kernarg* k = (Kernarg*)__builtin_amdgcn_kernarg_segment_ptr();
  uint32_t none = 0;
  asm volatile("" : "+s"(k), "+s"(none));  // (not what was read or counted before)
  KvAttnArgs a{};
  a.table = k->table;
  a.ldt = k->ldt;
  a.v_scales = k->v_scales;
  a.kv = k->kv;
  a.group = k->group;
  a.page_log2 = k->page_log2;
  a.pages = k->pages;
  a.window = k->window;
  Place at;
  at.b = uniform(plan.at.b);
  at.h = uniform(plan.at.h);
  at.t = uniform(plan.at.t);
  at.off = uniform(plan.at.off);
  at.take = uniform(plan.at.take);
  at.s.count = uniform(plan.at.s.count);
  at.s.len = uniform(plan.at.s.len);
  const int n = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, none)) & 15, columns = at.s.count * a.group;
  int pos[NQ];
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    const int col = at.t * NC + c0 + 16 * ct + n;
    pos[ct] = col < columns ? at.s.len - at.s.count + col / a.group : -1;
  }
  spoiled<FMT, D>(a, at.b, at.h, behind(tokens_of<NC>(a, at), clear_of<NC>(a, at.s, at.t).hi, a.window), pos, bad);
}

// A piece for few columns, its 32-token steps dealt to the four waves.  Measured, with the
// joining: 16 sequences of up to 131072 tokens, 8 heads of 128, INT4, 297 to 305 us: 4.9 TB/s, nearly a
// device copy's 5.04, vector instructions two thirds of the time.  One of 131072, MXFP4, 34.7 us: 4.1 TB/s.
// 48 of up to 8192, 4 heads, NVFP4 with T_q, 21.5 us: 1.4 TB/s, a start of 5 us and 7 units of
// 0.9 (waves wait for 42% of their cycles).  One of 500, 8.2 us: a launch, the lengths, the table
// and the codes one after the other, then 4 steps.
template <int FMT, int D, int SHAPE, int PLANES>
__device__ __forceinline__ void attend(const KvAttnArgs& a, const Piece& p, float* lds, float (&stat)[2][4][32]) {
  constexpr int NQ = kv_tiles(SHAPE, D), KJ = D / 32, CH = kCh<D>, NC = kv_columns(SHAPE, D);
  constexpr bool kInLds = kStaged<FMT, D, SHAPE, PLANES>;
  using RawT = Raw<FMT, D>;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int all = p.s.count * a.group;  // columns of the sequence
  const int c0 = p.t * NC;
  const int past = p.s.len - p.s.count;  // place of query 0

  // The wave's tokens and tiles of them.
  const int lo = p.lo, hi = p.hi;
  const int i0 = c0 / a.group, end = (c0 + 16 * NQ - 1) / a.group, i1 = end < p.s.count ? end : p.s.count - 1;
  const int first = lo / kTile + wave, step = 4;
  const int last = (hi + kTile - 1) / kTile;
  const int steps = hi > lo && last > first ? (last - first + step - 1) / step : 0;

  const auto o = offsets<FMT, D>(lane);
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
      load_k<FMT, D>(w, u, a.k_codes + row * (D / 2), a.k_scales + row * kScaleRow, o);
      load_v<FMT, D>(w, u, a.v_codes + row * (D / 2), a.v_scales + row * kScaleRow, o);
    }
  };

  // The first step is asked for before the queries are looked at.
  RawT w0, w1;
  if (steps > 0) load(w0, 0);

  // Columns: query rows, their places, operands.
  int pos[NQ];
  bf16x8 held[kInLds ? 1 : NQ][kInLds ? 1 : KJ];
  uint16_t* staged = reinterpret_cast<uint16_t*>(lds);
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
        for (int c = wave; c < D / 16; c += 4)
          transform_q<FMT, D>(row, a.T + (int64_t)p.h * D * (FMT == kNV ? 16 : 32), to, c);
      } else {
        for (int c = wave; c < D / 32; c += 4)
          *reinterpret_cast<u32x4*>(to + n * kQLine<D> + 32 * c + 8 * q) = *reinterpret_cast<const u32x4*>(row + 32 * c + 8 * q);
      }
    }
  }
  if constexpr (kInLds) __syncthreads();
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
  const float scale = score_scale<FMT>(a);

  f32x4 acc[CH][NQ];
  float m[NQ], l[NQ];
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    m[ct] = -FLT_MAX;
    l[ct] = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) acc[j][ct] = f32x4{0, 0, 0, 0};
  }

  int open = 0;
  auto compute = [&](RawT& w, int k) {
    const int t0 = (first + k * step) * kTile;
    const bool clear = t0 >= clear_from && t0 + kTile <= clear_to;
    f32x4 s[2][NQ];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct) s[u][ct] = f32x4{0, 0, 0, 0};
      arrange_k(w, u);
    }
    each<KJ>([&](auto jc) {
      constexpr int j = jc;
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
          k_scales<KJ, j>(w.ks[u], sc);
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
    });
    if (!clear) {
      mask_scores<NQ>(s, t0, lo, pos, a.window);
      if (clear_v(w, t0, lo, hi)) open = 1;
    }
    u32x4 pf[NQ];
    softmax_step<FMT, NQ, CH>(s, scale, m, l, acc, pf);
    const VScales<FMT> vs = v_scales(w);
#pragma unroll
    for (int i = 0; i < RawT::kV; ++i)
      each<(CH < 8 ? CH / 2 : 4)>([&](auto bc) {
        constexpr int b = bc;
        u32x4 even, odd;
        expand_v<FMT, D, b>(w, vs, i, even, odd);
#pragma unroll
        for (int ct = 0; ct < NQ; ++ct) {
          acc[8 * i + 2 * b][ct] = add_pv<FMT>(even, pf[ct], acc[8 * i + 2 * b][ct]);
          acc[8 * i + 2 * b + 1][ct] = add_pv<FMT>(odd, pf[ct], acc[8 * i + 2 * b + 1][ct]);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
  };

  if (steps > 0) {
    // Two register sets in turn; a load past the last step repeats a place in range.
    for (int k = 0; k < steps; k += 2) {
      load(w1, k + 1);
      compute(w0, k);
      load(w0, k + 2);
      if (k + 1 < steps) compute(w1, k + 1);
    }
  }
  if (open) {
    uint32_t bad[NQ], nan = 0x7FC00000u;
    spoiled<FMT, D>(a, p.b, p.h, behind(Span{lo, hi}, clear_to, a.window), pos, bad);
    asm volatile("" : "+s"(nan));  // (no register is kept for it either)
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][ct][r] = bad[ct] >> r & 1u ? __uint_as_float(nan) : acc[j][ct][r];
  }
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    l[ct] = column_sum(l[ct]);
    if (__any(bad)) l[ct] = __builtin_nanf("");
  }

  const float vg = FMT == kNV ? a.v_gs[0] : 1.0f / kVFactor<FMT>;
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
      f32x4* red = reinterpret_cast<f32x4*>(lds + q_floats<FMT, D, SHAPE, PLANES>());
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
              *reinterpret_cast<u32x2*>(out_row(a, p, col, D) + ch) =
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

// The same for many columns: each of the four waves has 32 (16 for D = 256) of its own, and
// they share what K and V become.  Per stage every wave expands 32 tokens (for D = 256 pairs
// of waves K or V of them) into LDS, as the operands that all four then read; the next
// stage's codes are on their way meanwhile.  Two chunks of 1000 queries of 32 heads behind 15000 to
// 16384 tokens take 480 us with the joining: 957 TFLOP/s; matrix cores 38%, vector instructions
// 42% of the time, a quarter of the waves' cycles waiting.  (Prefills are bound by the plan instead:
// one sequence of 2000 queries 134 us, 243 TFLOP/s, for one lane walks all of its 63 items, in load_of
// twice and then in find, and the last items, which see most tokens, begin last.)  (Each wave expanding for itself, in
// registers, spends 136 of 263 instructions of a step on it: 640 us.  The next tile's scores
// among this one's exponentials: 607, for registers.)
template <int FMT, int D>
constexpr int kStageTiles = D == 256 ? 2 : 4;
template <int FMT, int D>
constexpr int kTileLds = (2 * (D / 32) + kCh<D>) * 512 + (FMT == kINT ? 256 : 0);  // elements of 32 tokens

template <int FMT, int D, int SHAPE, int PLANES>
constexpr int lds_floats() {
  if (SHAPE != kKvPrompt) return q_floats<FMT, D, SHAPE, PLANES>() + 4 * kCh<D> / kParts<D> * 4 * 64;
  constexpr int tiles = kStageTiles<FMT, D> * kTileLds<FMT, D> / 2, queries = PLANES == 2 ? 4 * kQTile<D, 2> / 2 : 0;
  return (tiles > queries ? tiles : queries) + 4;  // (and two flags)
}

// f, or NaN for the rows that are.
__device__ __forceinline__ f32x4 row_factors(float f, uint32_t bad) {
  uint32_t nan = 0x7FC00000u;
  asm("" : "+s"(nan));  // (not a vector register's constant over the steps)
  f32x4 v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = bad >> r & 1u ? __uint_as_float(nan) : f;
  return v;
}

template <int FMT, int D, int PLANES>
__device__ __forceinline__ void attend_prompt(const KvAttnArgs& a, const Piece& p, const PlanLds& plan, float* lds) {
  constexpr int NQ = kv_tiles(kKvPrompt, D), KJ = D / 32, CH = kCh<D>, NC = kv_columns(kKvPrompt, D);
  constexpr int NS = kStageTiles<FMT, D>, kLds = kTileLds<FMT, D>;
  using RawT = Raw<FMT, D>;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  const int all = p.s.count * a.group;  // columns of the sequence
  const int c0 = p.t * NC + wave * 16 * NQ;
  const int past = p.s.len - p.s.count;  // place of query 0
  uint16_t* tiles = reinterpret_cast<uint16_t*>(lds);
  int* any_bad = reinterpret_cast<int*>(lds + lds_floats<FMT, D, kKvPrompt, PLANES>() - 4);
  int* any_open = any_bad + 1;

  // Tokens of the wave's columns, and of the stages.
  const int i0 = c0 / a.group, end = (c0 + 16 * NQ - 1) / a.group, i1 = end < p.s.count ? end : p.s.count - 1;
  const Span mine = c0 < all ? span_of(a, p.s, i0, i1) : Span{0, 0};
  const int lo = p.lo > mine.lo ? p.lo : mine.lo, hi = p.hi < mine.hi ? p.hi : mine.hi;
  const int first = p.lo / kTile, last = p.hi > p.lo ? (p.hi + kTile - 1) / kTile : first;
  const int stages = (last - first + NS - 1) / NS;

  // What this wave expands: tile `sub` of each stage.
  const int sub = D == 256 ? wave >> 1 : wave;
  const bool does_k = D < 256 || !(wave & 1), does_v = D < 256 || (wave & 1);
  const auto o = offsets<FMT, D>(lane);
  const int mask = (1 << a.page_log2) - 1;
  const int top = (p.hi - 1) & ~15, bottom = p.lo & ~15;  // halves that hold tokens
  auto half_at = [&](int k, int u) {
    const int t = (first + k * NS + sub) * kTile + 16 * u;
    return t > top ? top : t < bottom ? bottom : t;
  };
  int pages = 0;  // lane l: page of half l % 2 of stage 32 i + l / 2
  bool bad = p.s.bad;
  RawT w;
  auto load = [&](int k) {
    if ((k & 31) == 0) {
      int v = a.table[p.b * a.ldt + (half_at(k + (lane >> 1), lane & 1) >> a.page_log2)];
      if (v < 0 || v >= a.pages) {
        bad = true;
        v = 0;
      }
      pages = v;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int page = __builtin_amdgcn_readlane(pages, 2 * (k & 31) + u);
      const int64_t row = (((int64_t)page * a.kv + p.h) << a.page_log2) + (half_at(k, u) & mask);
      constexpr int kScaleRow = FMT == kMX ? D / 32 : D / 16;
      if (does_k) load_k<FMT, D>(w, u, a.k_codes + row * (D / 2), a.k_scales + row * kScaleRow, o);
      if (does_v) load_v<FMT, D>(w, u, a.v_codes + row * (D / 2), a.v_scales + row * kScaleRow, o);
    }
  };
  if (stages > 0) load(0);

  // Columns: query rows, their places, operands.
  int pos[NQ];
  bf16x8 qf[NQ][PLANES][KJ];
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    const int col = c0 + 16 * ct + n;
    const int used = col < all ? col : all - 1;
    const int i = used / a.group;
    pos[ct] = col < all ? past + i : -1;
    const uint16_t* row = a.q + (int64_t)(p.s.start + i) * a.ldq + (int64_t)(p.h * a.group + used - i * a.group) * D;
    if constexpr (PLANES == 1) {
#pragma unroll
      for (int j = 0; j < KJ; ++j) qf[ct][0][j] = *reinterpret_cast<const bf16x8*>(row + channel<FMT, D>(j, q));
    } else {
      uint16_t* to = tiles + wave * kQTile<D, 2>;
      wave_fence();
      for (int c = 0; c < D / 16; ++c) transform_q<FMT, D>(row, a.T + (int64_t)p.h * D * (FMT == kNV ? 16 : 32), to, c);
      wave_fence();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          qf[ct][t][j] = *reinterpret_cast<const bf16x8*>(to + (16 * t + n) * kQLine<D> + channel<FMT, D>(j, q));
    }
  }
  float qs[FMT == kINT ? NQ : 1][FMT == kINT ? KJ : 1];
  if constexpr (FMT == kINT) {
    // K enters as code + 8 (see attend).
    const uint32_t m8 = 0xC100C100u;  // bf16 -8, twice
    const bf16x8 minus8 = __builtin_bit_cast(bf16x8, (u32x4{m8, m8, m8, m8}));
#pragma unroll
    for (int ct = 0; ct < NQ; ++ct)
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        f32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < PLANES; ++t) v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus8, qf[ct][t][j], v, 0, 0, 0);
        qs[ct][j] = v[0];
      }
  }
  // Tiles that every column of the four waves sees whole need no mask.
  const Span clear = clear_of<NC>(a, p.s, p.t);
  int open = 0;
  const float scale = score_scale<FMT>(a);
  f32x4 acc[CH][NQ];
  float m[NQ], l[NQ];
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    m[ct] = -FLT_MAX;
    l[ct] = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) acc[j][ct] = f32x4{0, 0, 0, 0};
  }
  if (threadIdx.x == 0) *any_bad = *any_open = 0;
  __syncthreads();  // the queries' LDS is free

  // INT4: whether a group's sums and the next operands fit the registers (two prompts as above, heads of
  // 256: 826 us with and 870 without, but with T 1158 and 1110).
  constexpr bool kGroups = FMT == kINT && (PLANES == 1 || D == 64);
  // A tile's operands: K's 2 KJ (half u, instruction j), then V's CH, 1 KB each, lane by lane.
  auto operand = [&](int tile, int i) { return reinterpret_cast<u32x4*>(tiles + tile * kLds + i * 512 + lane * 8); };
  auto k_scale_dword = [&](int tile, int u) {
    return reinterpret_cast<uint32_t*>(tiles + tile * kLds + (2 * KJ + CH) * 512) + u * 64 + lane;
  };
  auto expand_tile = [&](int k) {
    const int t0 = (first + k * NS + sub) * kTile;
    if (does_k) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        arrange_k(w, u);
#pragma unroll
        for (int j = 0; j < KJ; ++j)
          *operand(sub, u * KJ + j) =
              __builtin_bit_cast(u32x4, expand<FMT>(w.kc[u][j], FMT == kINT ? 0.0f : k_scale(w, u, j)));
        if constexpr (FMT == kINT) *k_scale_dword(sub, u) = w.ks[u];
      }
    }
    if (does_v) {
      if (t0 < clear.lo || t0 + kTile > clear.hi) {
        if (clear_v(w, t0, p.lo, p.hi)) open = 1;
      }
      const VScales<FMT> vs = v_scales(w);
#pragma unroll
      for (int i = 0; i < RawT::kV; ++i)
        each<(CH < 8 ? CH / 2 : 4)>([&](auto bc) {
          constexpr int b = bc;
          u32x4 even, odd;
          expand_v<FMT, D, b>(w, vs, i, even, odd);
          *operand(sub, 2 * KJ + 8 * i + 2 * b) = even;
          *operand(sub, 2 * KJ + 8 * i + 2 * b + 1) = odd;
        });
    }
  };
  auto compute = [&](int tile, int t0) {
    f32x4 s[2][NQ];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct) s[u][ct] = f32x4{0, 0, 0, 0};
    // A wave among its matrix instructions goes before one among its exponentials: the other way
    // round, or without, the former wait for the latter (the prompts above: MXFP4 490 us with and 497
    // without, heads of 256 627 and 647, before K's operands were asked for ahead).
    __builtin_amdgcn_s_setprio(1);
    // K's operands, and what becomes of their products, in an order that the compiler, left to itself,
    // gives up when registers are short: read just before they are used they cost NVFP4 and INT4
    // 4 to 17% of the time.
    if constexpr (FMT == kINT && !kGroups) {
      each<KJ>([&](auto jc) {
        constexpr int j = jc;
        if constexpr (j % 2 == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bf16x8 kf = __builtin_bit_cast(bf16x8, *operand(tile, u * KJ + j));
          float sc[4];
          k_scales<KJ, j>(*k_scale_dword(tile, u), sc);
#pragma unroll
          for (int ct = 0; ct < NQ; ++ct) {
            f32x4 g = {qs[ct][j], qs[ct][j], qs[ct][j], qs[ct][j]};
#pragma unroll
            for (int t = 0; t < PLANES; ++t) g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[ct][t][j], g, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) s[u][ct][r] = __builtin_fmaf(sc[r], g[r], s[u][ct][r]);
          }
        }
      });
    } else {
      // The next operands are asked for before the instructions on these.
      u32x4 next[2] = {*operand(tile, 0), *operand(tile, KJ)};
      each<KJ>([&](auto jc) {
        constexpr int j = jc;
        const bf16x8 kf[2] = {__builtin_bit_cast(bf16x8, next[0]), __builtin_bit_cast(bf16x8, next[1])};
        if constexpr (j + 1 < KJ) {
          next[0] = *operand(tile, j + 1);
          next[1] = *operand(tile, KJ + j + 1);
        }
        if constexpr (!kGroups) __builtin_amdgcn_sched_barrier(0x76);  // of LDS and matrix instructions alone
        f32x4 g[2][NQ];  // INT4: sums over a group, all of them before the first one's scales
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int ct = 0; ct < NQ; ++ct) {
            f32x4& sum = kGroups ? g[u][ct] : s[u][ct];
            if constexpr (kGroups) sum = f32x4{qs[ct][j], qs[ct][j], qs[ct][j], qs[ct][j]};
#pragma unroll
            for (int t = 0; t < PLANES; ++t) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[u], qf[ct][t][j], sum, 0, 0, 0);
          }
        if constexpr (kGroups) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float sc[4];
            k_scales<KJ, j>(*k_scale_dword(tile, u), sc);
#pragma unroll
            for (int ct = 0; ct < NQ; ++ct)
#pragma unroll
              for (int r = 0; r < 4; ++r) s[u][ct][r] = __builtin_fmaf(sc[r], g[u][ct][r], s[u][ct][r]);
          }
        }
      });
    }
    __builtin_amdgcn_s_setprio(0);
    if (!(t0 >= clear.lo && t0 + kTile <= clear.hi)) mask_scores<NQ>(s, t0, lo, pos, a.window);
    u32x4 pf[NQ];
    softmax_step<FMT, NQ, CH>(s, scale, m, l, acc, pf);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const u32x4 vf = *operand(tile, 2 * KJ + j);
#pragma unroll
      for (int ct = 0; ct < NQ; ++ct) acc[j][ct] = add_pv<FMT>(vf, pf[ct], acc[j][ct]);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  for (int k = 0; k < stages; ++k) {
    expand_tile(k);
    load(k + 1);  // (behind the last one: a place in range)
    meet();
    for (int i = 0; i < NS; ++i) {
      const int t0 = (first + k * NS + i) * kTile;
      if (t0 < hi && t0 + kTile > lo) compute(i, t0);
    }
    meet();
  }
  if (__any(bad) && lane == 0) *any_bad = 1;
  if (open && lane == 0) *any_open = 1;
  __syncthreads();
  const bool nan = *any_bad != 0;
  uint32_t bad_rows[NQ] = {};
  if (uniform(*any_open)) spoiled<FMT, D, NC>(plan, wave * 16 * NQ, bad_rows);
  const float vg = FMT == kNV ? a.v_gs[0] : 1.0f / kVFactor<FMT>;
#pragma unroll
  for (int ct = 0; ct < NQ; ++ct) {
    l[ct] = column_sum(l[ct]);
    if (nan) l[ct] = __builtin_nanf("");
    const int col = c0 + 16 * ct + n, at = col - p.t * NC;
    if (col >= all) continue;
    const f32x4 f = row_factors(p.whole ? (l[ct] != 0.0f ? vg / l[ct] : 0.0f) : 1.0f, bad_rows[ct]);
    if (!p.whole && q == 0) {
      p.part[at] = m[ct];
      p.part[NC + at] = l[ct];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int ch = CH * (4 * q + r);
#pragma unroll
      for (int j = 0; j < CH; j += 4) {
        const f32x4 v = {acc[j][ct][r] * f[r], acc[j + 1][ct][r] * f[r], acc[j + 2][ct][r] * f[r], acc[j + 3][ct][r] * f[r]};
        if (p.whole) {
          *reinterpret_cast<u32x2*>(out_row(a, p, col, D) + ch + j) = u32x2{pack(cvt_bf16(v[0], v[1])), pack(cvt_bf16(v[2], v[3]))};
        } else {
          *reinterpret_cast<f32x4*>(p.part + 2 * NC + at * D + ch + j) = v;
        }
      }
    }
  }
}

template <int FMT, int D, int SHAPE, int PLANES>
__global__ __launch_bounds__(kThreads, kv_per_cu(SHAPE, D, FMT)) void kv4_attention_kernel(KvAttnArgs a) {
  constexpr int NC = kv_columns(SHAPE, D);
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ float stat[2][4][32];
  __shared__ PlanLds plan;
  const int w = blockIdx.x;
  const Seq first = seq_or_none(a, place_of(a));
  const Shares s = shares_of<NC, SHAPE>(a, plan, first);
  Place at;
  bool any;
  int several = 0, left = 0;  // units left of the run
  if (s.by_runs) {
    if (w >= a.runs) return;
    const int64_t begin = (int64_t)w * s.share;
    left = (int)(begin >= s.total ? 0 : s.total - begin < s.share ? s.total - begin : s.share);
    // A unit is a piece of one.
    any = left > 0 && find<NC>(a, plan, first, 1, (int)begin, at, several);
    at.slot = 2 * w;
  } else {
    any = find<NC>(a, plan, first, s.share, w, at, several);
  }
  // How many there are to join is written also where there is nothing at all.
  if (w == 0 && threadIdx.x == 0 && a.runs > 0) a.join[0].pieces = several;
  if (!any) return;
  for (;;) {
    KvJoin join = {at.pieces, at.slot, at.slot + 1, 1, 0, 0, at.s.start, at.h};
    bool listed = at.pieces > 1;
    if (s.by_runs) {
      at.take = at.units - at.off < left ? at.units - at.off : left;
      left -= at.take;
      // The rest of the item is at the beginnings of the runs behind.
      const int rest = at.units - at.off - at.take;
      join = KvJoin{rest > 0 ? (rest - 1) / s.share + 2 : 0, at.slot, 2 * w + 2, 2, 0, 0, at.s.start, at.h};
      listed = at.units > 1;
    }
    const int cols = at.s.count * a.group - at.t * NC;
    join.cols = cols < NC ? cols : NC;
    join.col0 = at.t * NC;
    const Span tokens = tokens_of<NC>(a, at);
    Piece p;
    p.b = at.b;
    p.h = at.h;
    p.t = at.t;
    p.s = at.s;
    p.lo = tokens.lo;
    p.hi = tokens.hi;
    p.whole = at.take == at.units;
    p.part = p.whole ? nullptr : a.part + (int64_t)at.slot * (NC * (D + 2));
    if (listed && at.off == 0 && threadIdx.x == 0) a.join[1 + at.rank] = join;
    // (Kept here rather than in registers.)
    if (threadIdx.x == 0) {
      plan.at = at;
      plan.left = left;
    }
    if constexpr (SHAPE == kKvPrompt) {
      attend_prompt<FMT, D, PLANES>(a, p, plan, lds);
    } else {
      attend<FMT, D, SHAPE, PLANES>(a, p, lds, stat);
    }
    __syncthreads();
    left = uniform(plan.left);
    if (left == 0) return;
    at.b = uniform(plan.at.b);
    at.h = uniform(plan.at.h);
    at.t = uniform(plan.at.t);
    at.units = uniform(plan.at.units);
    at.rank = uniform(plan.at.rank);
    at.s.start = uniform(plan.at.s.start);
    at.s.count = uniform(plan.at.s.count);
    at.s.len = uniform(plan.at.s.len);
    at.s.bad = uniform(plan.at.s.bad);
    next_item<NC>(a, at);
    // Only a run's last item can go on behind it.
    at.slot = 2 * w + 1;
    __syncthreads();  // LDS changes its use
  }
}

// The pieces of the items that have several: an item per blockIdx.x, its columns shared out
// over blockIdx.y.  D / 4 lanes take a row's channels, so that a workgroup reads 1024 / D rows
// at once: columns where there are few pieces, pieces of one column where there are many.
// 4.6 us behind 48 sequences' 192 items, 14.0 (62 MB read, 4.4 TB/s) behind the two prompts above.
constexpr int kFewPieces = 4;
template <int D, int SHAPE>
__global__ __launch_bounds__(kThreads) void kv4_join_kernel(KvAttnArgs a, int nv, float factor) {
  constexpr int NC = kv_columns(SHAPE, D), kLanes = D / 4, kAtOnce = kThreads / kLanes;
  __shared__ float row_m[kAtOnce], row_l[kAtOnce];
  __shared__ __attribute__((aligned(16))) float sums[kAtOnce][D];
  const int tid = threadIdx.x, mine = tid / kLanes, ch = tid % kLanes * 4;
  constexpr int64_t kPiece = NC * (D + 2);
  const float vg = nv ? a.v_gs[0] : factor;
  // (Both on their way at once.)
  KvJoin j = a.join[1 + blockIdx.x];
  const int count = a.join[0].pieces;
  for (int item = blockIdx.x; item < count;) {
    auto piece = [&](int i) {
      return a.part + (i == 0 ? (int64_t)j.first : (int64_t)j.next + (int64_t)(i - 1) * j.step) * kPiece;
    };
    auto out = [&](int c) {
      const int col = j.col0 + c, i = col / a.group;
      return a.out + ((int64_t)(j.start + i) * a.kv * a.group + j.head * a.group + col - i * a.group) * D;
    };
    // `several` of them from number i0 on, `by` apart, all on their way at once.
    auto add = [&](int c, int i0, int by, float& M, float& L, f32x4& v) {
      float m[kFewPieces], l[kFewPieces], next = M;
      f32x4 x[kFewPieces];
#pragma unroll
      for (int u = 0; u < kFewPieces; ++u) {
        const int i = i0 + u * by;
        const float* p = piece(i < j.pieces ? i : i0);
        m[u] = p[c];
        l[u] = p[NC + c];
        x[u] = *reinterpret_cast<const f32x4*>(p + 2 * NC + c * D + ch);
        next = fmaxf(next, m[u]);
      }
      const float f0 = __builtin_amdgcn_exp2f(M - next);
      M = next;
      L *= f0;
      v *= f0;
#pragma unroll
      for (int u = 0; u < kFewPieces; ++u) {
        const bool there = i0 + u * by < j.pieces;
        const float f = __builtin_amdgcn_exp2f(m[u] - M);
        L = there ? __builtin_fmaf(l[u], f, L) : L;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = there ? __builtin_fmaf(x[u][e], f, v[e]) : v[e];
      }
    };
    if (j.pieces > 1 && j.pieces <= kFewPieces) {
      for (int c = (int)blockIdx.y * kAtOnce + mine; c < j.cols; c += (int)gridDim.y * kAtOnce) {
        float M = -FLT_MAX, L = 0.0f;
        f32x4 v = {0, 0, 0, 0};
        add(c, 0, 1, M, L, v);
        const float g = L != 0.0f ? vg / L : 0.0f;
        *reinterpret_cast<u32x2*>(out(c) + ch) = u32x2{pack(cvt_bf16(v[0] * g, v[1] * g)), pack(cvt_bf16(v[2] * g, v[3] * g))};
      }
    } else if (j.pieces > 1) {
      for (int c = blockIdx.y; c < j.cols; c += gridDim.y) {
        float M = -FLT_MAX, L = 0.0f;
        f32x4 v = {0, 0, 0, 0};
        for (int i = mine; i < j.pieces; i += kFewPieces * kAtOnce) add(c, i, kAtOnce, M, L, v);
        *reinterpret_cast<f32x4*>(&sums[mine][ch]) = v;
        if (ch == 0) {
          row_m[mine] = M;
          row_l[mine] = L;
        }
        __syncthreads();
        if (tid < D) {
          float sum = 0.0f, all = 0.0f;
          M = row_m[0];
#pragma unroll
          for (int i = 1; i < kAtOnce; ++i) M = fmaxf(M, row_m[i]);
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const float f = __builtin_amdgcn_exp2f(row_m[i] - M);
            sum = __builtin_fmaf(sums[i][tid], f, sum);
            all = __builtin_fmaf(row_l[i], f, all);
          }
          out(c)[tid] = __builtin_bit_cast(uint16_t, (__bf16)(all != 0.0f ? sum * (vg / all) : 0.0f));
        }
        __syncthreads();
      }
    }
    item += gridDim.x;
    if (item < count) j = a.join[1 + item];
  }
}

template <int FMT, int D, int SHAPE, int PLANES>
hipError_t go(const KvAttnArgs& a, hipStream_t s) {
  hipError_t e = launch_lds(kv4_attention_kernel<FMT, D, SHAPE, PLANES>, dim3(a.workgroups), kThreads,
                            4 * lds_floats<FMT, D, SHAPE, PLANES>(), s, a);
  if (e != hipSuccess || a.runs == 0) return e;
  const int64_t columns = (int64_t)a.n * a.group / (a.B < a.n ? a.B : a.n);  // of a sequence, on average
  const int64_t most = kv_columns(SHAPE, D);
  // Enough workgroups to fill the chip, but at least as many as a pass over the columns takes
  // and at most one each.
  const int x = a.items < kKvJoins ? a.items : kKvJoins, cols = (int)(columns < most ? columns : most);
  const int pass = (cols * D + 4 * kThreads - 1) / (4 * kThreads), fill = (kKvFill + x - 1) / x;
  const int y = fill < pass ? pass : fill < cols ? fill : cols;
  hipLaunchKernelGGL((kv4_join_kernel<D, SHAPE>), dim3(x, y), dim3(kThreads), 0, s, a, FMT == kNV ? 1 : 0, 1.0f / kVFactor<FMT>);
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
