// The product of a few activation rows with rows of 4-bit weights, shared by
// the linear layer (wush_w4.hip) and the mixture of experts (wush_moe.hip).
// Device code only.
//
// v_mfma_f32_16x16x32_bf16 multiplies A = 16 tokens with B = 16 weight rows:
// D[m][n] with m = 4 (lane / 16) + i, n = lane % 16.  A few tokens leave
// most of A's rows unused (row m of D depends on row m of A alone, so unused rows
// hold copies of a valid token and are never stored); the matrix cores are
// still far from the limit.  The limit is the weights' way in, and behind it
// the vector instructions that turn codes into bf16.
//
// A workgroup has WN x WK waves: wave (wn, wk) owns R tiles of 16 weight rows
// and, of every chunk of K, its D steps of 128 elements.  R D = 4 units (16
// rows x 128 elements, 1 KB of codes) are in registers while the next four
// are on their way; the activations of a chunk come through LDS, where all waves
// of the same wk read them, one chunk ahead.  (Read from global memory they
// would share the weights' load counter, and each wait for them would drain the
// weights in flight.)  The WK sums meet in LDS at the end.
//
// A unit: lane (q = lane / 16, n) loads the 16 code bytes of row n, elements
// 32 q .. 32 q + 31, so the four lanes of a row read 64 contiguous bytes.
// MXFP4 and NVFP4 apply their scales to the elements; matrix instruction j takes
// elements 32 q + 8 j .. + 7 of every quarter q, and the activations from the
// same places.  INT4 applies its scale to sums over one group: a 4 x 4 transpose
// of dwords between the lane quarters (four lane-swap instructions) makes matrix
// instruction j cover group j of all 16 rows, elements 32 j + 8 q .. + 7.  The
// scales of four units come in one load, lane quarter u holding unit u's, and
// three lane swaps hand them round.
//
// Exactness.  E2M1 * 2^e and E2M1 * E4M3 have at most 6 significant bits, and
// the integers of INT4 have 4, so all of them are exact in bf16; the fp16
// scale of INT4 is applied in fp32 to each group's sum, NVFP4's tensor scale in
// fp32 to the result.  Products of bf16 are exact in the matrix cores, sums
// are fp32.  INT4's sums run over (code + 8) x and -8 x, whose rounding is relative to
// up to 23 |x| per element where the product itself may be smaller; they overflow
// where 15 sum |x| over a group does.
#ifndef WUSH_W4_CORE_H_
#define WUSH_W4_CORE_H_

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"

namespace wush {
namespace w4 {

constexpr int kMX = 0, kNV = 1, kINT = 2;
constexpr int kStep = 128;                          // elements of K per step

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Loads at the alignment that rows of odd lengths have (the hardware takes
// any; the type says what is known).
template <typename V>
__device__ __forceinline__ V load_unaligned(const void* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}

__device__ __forceinline__ uint32_t pack(bf16x2 v) { return __builtin_bit_cast(uint32_t, v); }

__device__ __forceinline__ bf16x2 cvt_bf16(float a, float b) {
  bf16x2 r;
  r[0] = (__bf16)a;
  r[1] = (__bf16)b;
  return r;
}

// One lane's share of R row tiles x D steps, as it is in memory.  With four
// units in all, lane quarter u holds the scales of unit u (row tile u / D, step
// u % D); otherwise every lane holds every unit's.
template <int FMT, int R, int D>
struct Raw {
  static constexpr int kUnits = R * D;
  static constexpr bool kShared = kUnits == 4;
  // Loads that it takes at least (two steps' scales of a row are neighbours, and may
  // come as one).
  static constexpr int kLoads = kUnits + (kShared ? 1 : R);
  u32x4 c[kUnits];
  u32x2 s[kShared ? 1 : kUnits];  // 4 E8M0 bytes, 8 E4M3 bytes or 4 fp16
};

template <int FMT>
__device__ __forceinline__ int64_t row_code_bytes(int64_t K) { return K / 2; }
template <int FMT>
__device__ __forceinline__ int64_t row_scale_bytes(int64_t K) { return FMT == kMX ? K / 32 : K / 16; }

template <int FMT>
__device__ __forceinline__ u32x2 load_scales(const uint8_t* sp, int64_t st) {
  if constexpr (FMT == kMX) {
    return u32x2{load_unaligned<uint32_t>(sp + 4 * st), 0};
  } else {
    return load_unaligned<u32x2>(sp + 8 * st);
  }
}

// A wave's R tiles: of each, the first row (the same in all lanes) and the lane's
// offset from there, to its 16 bytes of step 0; and the lane's scales.
template <int FMT, int R, int D>
struct Rows {
  const uint8_t* cp[R];
  uint32_t off[R];
  const uint8_t* sp[Raw<FMT, R, D>::kShared ? 1 : R];
};

// first(t): index of row tile t's first row; last(t): the last one it may read (rows
// past it stand for results that nobody stores).  K at most 2^27 keeps off
// within 32 bits.
template <int FMT, int R, int D, typename F, typename L>
__device__ __forceinline__ Rows<FMT, R, D> make_rows(const uint8_t* codes, const uint8_t* scales, int64_t K, F first,
                                                     L last) {
  const int n = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
  const auto clamped = [&](int t) {
    const int64_t room = last(t) - first(t);
    return (int)(n < room ? n : room);
  };
  Rows<FMT, R, D> o;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t at = first(r) * row_code_bytes<FMT>(K);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
    o.cp[r] = codes + (int64_t)(((uint64_t)hi << 32) | lo);
    o.off[r] = (uint32_t)(clamped(r) * row_code_bytes<FMT>(K) + 16 * q);
  }
  if constexpr (Raw<FMT, R, D>::kShared) {
    o.sp[0] = scales + (first(q / D) + clamped(q / D)) * row_scale_bytes<FMT>(K) + (FMT == kMX ? 4 : 8) * (q % D);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) o.sp[r] = scales + (first(r) + clamped(r)) * row_scale_bytes<FMT>(K);
  }
  return o;
}

// D whole steps from step st.
template <int FMT, int R, int D>
__device__ __forceinline__ void load_raw(Raw<FMT, R, D>& w, const Rows<FMT, R, D>& p, int64_t st) {
  using RawT = Raw<FMT, R, D>;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int d = 0; d < D; ++d) w.c[r * D + d] = load_unaligned<u32x4>(p.cp[r] + 64 * (st + d) + p.off[r]);
  if constexpr (RawT::kShared) {
    w.s[0] = load_scales<FMT>(p.sp[0], st);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < D; ++d) w.s[r * D + d] = load_scales<FMT>(p.sp[r], st + d);
  }
}

// D steps of which some reach past K, which is 128 or more: nothing is read past a
// row, and what is missing is zero once fix_tail has run.  The loads depend on no
// condition (their addresses do), so that fix_tail can be left until the weights are
// needed.
template <int FMT, int R, int D>
__device__ __forceinline__ void load_raw_tail(Raw<FMT, R, D>& w, const Rows<FMT, R, D>& p, int64_t st, int64_t K) {
  using RawT = Raw<FMT, R, D>;
  constexpr int kStepBytes = FMT == kMX ? 4 : 8;
  const int q = (threadIdx.x & 63) >> 4;
  const int64_t row_scales = row_scale_bytes<FMT>(K);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      // The lane's 16 bytes, or the row's last 16 if they reach past it.
      const int64_t last = K / 2 - 16 - 16 * q, at = 64 * (st + d);
      w.c[r * D + d] = load_unaligned<u32x4>(p.cp[r] + (at < last ? at : last) + p.off[r]);
    }
  // sp points at this step's bytes; not past the row's last kStepBytes.
  auto back = [&](int64_t step) {
    const int64_t over = kStepBytes * (step + 1) - row_scales;
    return over > 0 ? over : 0;
  };
  if constexpr (RawT::kShared) {
    w.s[0] = load_scales<FMT>(p.sp[0] - back(st + q % D), st);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < D; ++d) w.s[r * D + d] = load_scales<FMT>(p.sp[r] - back(st + d), st + d);
  }
}

// The only step, the wave's first, where K is less than 128.
template <int FMT, int R, int D>
__device__ __forceinline__ void load_raw_short(Raw<FMT, R, D>& w, const Rows<FMT, R, D>& p, int64_t K) {
  using RawT = Raw<FMT, R, D>;
  constexpr int kStepBytes = FMT == kMX ? 4 : 8;
  const int q = (threadIdx.x & 63) >> 4;
  const int64_t row_scales = row_scale_bytes<FMT>(K);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int64_t k = d * kStep + 32 * q;
      u32x4 c = {0, 0, 0, 0};
      if (k + 32 <= K) {
        c = load_unaligned<u32x4>(p.cp[r] + p.off[r]);
      } else if (FMT == kNV && k + 16 <= K) {
        const u32x2 h = load_unaligned<u32x2>(p.cp[r] + p.off[r]);
        c[0] = h[0];
        c[1] = h[1];
      }
      w.c[r * D + d] = c;
    }
  auto scales = [&](const uint8_t* sp, int d) {
    u32x2 s = {0, 0};
    if (d == 0) {
      for (int b = 0; b < row_scales; ++b) {
        const uint32_t v = (uint32_t)sp[b] << (8 * (b % 4));
        if (b < 4) {
          s[0] |= v;
        } else {
          s[1] |= v;
        }
      }
    }
    return s;
  };
  if constexpr (RawT::kShared) {
    w.s[0] = scales(p.sp[0], q % D);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < D; ++d) w.s[r * D + d] = scales(p.sp[r], d);
  }
}

// What load_raw_tail took from before its place: shifted there, zero behind it.
template <int FMT, int R, int D>
__device__ __forceinline__ void fix_tail(Raw<FMT, R, D>& w, int64_t st, int64_t K) {
  using RawT = Raw<FMT, R, D>;
  constexpr int kStepBytes = FMT == kMX ? 4 : 8;
  if (K < kStep) return;
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int64_t k = (st + d) * kStep + 32 * q;
      u32x4& c = w.c[r * D + d];
      const bool half = FMT == kNV && k + 16 == K;
      if (half) c = u32x4{c[2], c[3], 0, 0};
      if (k + 32 > K && !half) c = u32x4{0, 0, 0, 0};
    }
  auto fix = [&](u32x2 s, int64_t step) {
    const int64_t over = kStepBytes * (step + 1) - row_scale_bytes<FMT>(K);
    uint64_t v = ((uint64_t)s[1] << 32) | s[0];
    if (over >= kStepBytes) v = 0;
    else if (over > 0) v >>= 8 * over;
    return u32x2{(uint32_t)v, (uint32_t)(v >> 32)};
  };
  if constexpr (RawT::kShared) {
    w.s[0] = fix(w.s[0], st + q % D);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < D; ++d) w.s[r * D + d] = fix(w.s[r * D + d], st + d);
  }
}

// Dword j of the lane quarter q's chunk -> dword q of chunk j.
__device__ __forceinline__ void transpose4(u32x4& c) {
  const auto a = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
  const auto x = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto y = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  c = u32x4{x[0], x[1], y[0], y[1]};
}

// v of lane quarter u, in all quarters, as o[u].
__device__ __forceinline__ void hand_round(uint32_t v, uint32_t (&o)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const auto x = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
  const auto y = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
  o[0] = x[0];
  o[1] = x[1];
  o[2] = y[0];
  o[3] = y[1];
}

// What dword j of a lane's codes is multiplied with before (MXFP4, NVFP4) or
// after (INT4) the matrix instruction; s: the scales of the lane's row.
template <int FMT>
__device__ __forceinline__ float code_scale(const u32x2& s, int j, int q) {
  if constexpr (FMT == kMX) {
    // The E8M0 byte of group q is an fp32 exponent; the conversion reads
    // nothing else of its scale operand, and takes 0 for 2^-127 and 255 for NaN.
    return __uint_as_float(((s[0] >> (8 * q)) & 0xFFu) << 23);
  } else if constexpr (FMT == kNV) {
    // Dwords 0 and 1 are scale group 2 q, 2 and 3 are 2 q + 1.
    const uint32_t v = (q < 2 ? s[0] : s[1]) >> (16 * (q & 1));
    return j < 2 ? __builtin_amdgcn_cvt_f32_fp8(v, 0) : __builtin_amdgcn_cvt_f32_fp8(v, 1);
  } else {
    return __half2float(__ushort_as_half((uint16_t)(s[j >> 1] >> (16 * (j & 1)))));
  }
}

// Eight codes of one group as bf16 weights; INT4 as code + 8.
template <int FMT>
__device__ __forceinline__ bf16x8 expand(uint32_t d, float s) {
  u32x4 r;
  if constexpr (FMT == kMX) {
    r[0] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0));
    r[1] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1));
    r[2] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2));
    r[3] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3));
  } else if constexpr (FMT == kNV) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1);
    const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2);
    const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3);
    r[0] = pack(cvt_bf16(a[0] * s, a[1] * s));
    r[1] = pack(cvt_bf16(b[0] * s, b[1] * s));
    r[2] = pack(cvt_bf16(e[0] * s, e[1] * s));
    r[3] = pack(cvt_bf16(f[0] * s, f[1] * s));
  } else {
    // u = code + 8 in 0 .. 15 is, as an E4M3 byte, the number u * 2^-9 (up to
    // 7 as a subnormal, from 8 on with exponent 1); scaled by 2^9 the
    // conversion gives u.
    const uint32_t lo = (d & 0x0F0F0F0Fu) ^ 0x08080808u, hi = ((d >> 4) & 0x0F0F0F0Fu) ^ 0x08080808u;
    const uint32_t p0 = __builtin_amdgcn_perm(hi, lo, 0x05010400u);  // elements 0 .. 3
    const uint32_t p1 = __builtin_amdgcn_perm(hi, lo, 0x07030602u);  // elements 4 .. 7
    r[0] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, false));
    r[1] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, true));
    r[2] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, false));
    r[3] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, true));
  }
  return __builtin_bit_cast(bf16x8, r);
}

// The activations of a chunk in LDS: lines of bf16, one line per (term, token
// row).  One copy instruction writes a piece of 1 KB (64 lanes x 16 bytes).  Lines
// of 512 elements or more are whole pieces and 16 bytes more, which put the 16
// rows that a quarter wave reads at once on 16 different 16-byte groups of
// banks.  Two lines of 256 elements share a piece; there the second one's
// elements sit at their index ^ 64, for the same end.
template <int WIDTH>
struct Lines {
  static constexpr int kPerPiece = WIDTH >= 512 ? 1 : 2;            // lines per piece
  static constexpr int kPieces = WIDTH >= 512 ? WIDTH / 512 : 1;    // pieces per line
  static constexpr int kStride = WIDTH >= 512 ? WIDTH + 8 : 512 + 8;  // elements per kPerPiece lines
  static_assert(WIDTH == 256 || WIDTH % 512 == 0, "a line is half a piece or whole pieces");
  static __host__ __device__ __forceinline__ int at(int line) {
    return kPerPiece == 1 ? line * kStride : line / 2 * kStride + line % 2 * WIDTH;
  }
  static __device__ __forceinline__ int flip(int line) { return kPerPiece == 1 ? 0 : line % 2 * 64; }
  static __host__ __device__ __forceinline__ int groups(int lines) { return (lines + kPerPiece - 1) / kPerPiece; }
};

typedef __attribute__((address_space(3))) uint16_t lds_u16;
typedef const __attribute__((address_space(1))) uint16_t glb_u16;

// Global-to-LDS copy of 16 bytes per lane to LDS byte address dst (uniform;
// lane l writes at dst + 16 l), outside the compiler's view: it would wait for
// every copy in flight before any LDS read.  The copy takes its LDS base from
// M0, which nothing else in these kernels uses; between a scalar write of M0 and a
// load to LDS the hardware wants one wait state, which the compiler does not put
// inside a statement.  The statement has no outputs.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(glb_u16* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "memory", "m0");
}
#pragma clang diagnostic pop

// This wave's first copies have landed, given that at least N loads of
// weights were requested after them, and so have the others'.
template <int N>
__device__ __forceinline__ void arrive() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// This wave's copies have landed, given that at least N loads of weights were
// requested after them.
template <int N>
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// All of this wave's LDS reads are done, then the workgroup meets.  Loads
// and copies in flight stay in flight.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Where a lane reads its activations: of dword (MXFP4, NVFP4) or group (INT4) j
// of a step at x + at[j / 2] + kXJ * j.
template <int FMT>
constexpr int kXJ = FMT == kINT ? 32 : 8;
struct XAt {
  int at[2];
};

// acc += the wave's D steps.  x: the wave's first step in line 0 of the chunk; xo[t][p]:
// where the lane reads term p of its row of token tile t.
template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, typename A>
__device__ __forceinline__ void multiply(f32x4 (&acc)[R][NT], Raw<FMT, R, D>& w, A arrived, const uint16_t* x,
                                         const XAt (&xo)[NT][TERMS]) {
  const int q = (threadIdx.x & 63) >> 4;
  // The last weights asked for, wanted here.
  asm volatile("" : "+v"(w.s[Raw<FMT, R, D>::kShared ? 0 : R * D - 1][0]));
  arrived();
  u32x2 sc[R * D];
  if constexpr (Raw<FMT, R, D>::kShared) {
    uint32_t lo[4], hi[4] = {0, 0, 0, 0};
    hand_round(w.s[0][0], lo);
    if constexpr (FMT != kMX) hand_round(w.s[0][1], hi);
#pragma unroll
    for (int u = 0; u < 4; ++u) sc[u] = u32x2{lo[u], hi[u]};
  } else {
#pragma unroll
    for (int u = 0; u < R * D; ++u) sc[u] = w.s[u];
  }
  if constexpr (FMT == kINT) {
#pragma unroll
    for (int u = 0; u < R * D; ++u) transpose4(w.c[u]);
  }
  // INT4's codes come in as code + 8: the group's sum starts at
  // -8 sum x, which one more matrix instruction with a constant -8 gives in
  // every column.
  const uint32_t m8 = 0xC100C100u;  // bf16 -8, twice
  const bf16x8 minus8 = __builtin_bit_cast(bf16x8, (u32x4{m8, m8, m8, m8}));
  bf16x8 a[NT][TERMS], next[NT][TERMS];
  auto load_a = [&](bf16x8 (&to)[NT][TERMS], int i) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int p = 0; p < TERMS; ++p)
        to[t][p] = *reinterpret_cast<const bf16x8*>(x + xo[t][p].at[i % 4 / 2] + i / 4 * kStep + kXJ<FMT> * (i % 4));
  };
  load_a(a, 0);
#pragma unroll
  for (int i = 0; i < 4 * D; ++i) {  // dword or group j of step d
    const int d = i / 4, j = i % 4;
    if (i + 1 < 4 * D) load_a(next, i + 1);
    if constexpr (FMT == kINT) {
      f32x4 init[NT], sum[R][NT];
      float sc1[R];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        init[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < TERMS; ++p)
          init[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][p], minus8, init[t], 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        sc1[r] = code_scale<FMT>(sc[r * D + d], j, q);
        const bf16x8 b = expand<FMT>(w.c[r * D + d][j], 0.0f);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          sum[r][t] = init[t];
#pragma unroll
          for (int p = 0; p < TERMS; ++p)
            sum[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][p], b, sum[r][t], 0, 0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < (SPREAD ? 1 : 4); ++k) acc[r][t][k] = __builtin_fmaf(sc1[r], sum[r][t][k], acc[r][t][k]);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bf16x8 b = expand<FMT>(w.c[r * D + d][j], code_scale<FMT>(sc[r * D + d], j, q));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < TERMS; ++p)
            acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][p], b, acc[r][t], 0, 0, 0);
      }
    }
    // Expanding more than one dword ahead costs registers, and with them waves.
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int p = 0; p < TERMS; ++p) a[t][p] = next[t][p];
  }
  if constexpr (FMT == kINT) {
    // The sums are wanted here: left to itself the compiler moves the scales'
    // multiplications behind the branches that follow, and keeps every group's sum
    // until then.
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(acc[r][t]));
  }
}

constexpr int kBuffers = 3;  // activation chunks in LDS

// Waves per SIMD that the registers are cut for: four where the code fits 128
// without spilling, otherwise three (168), or two with several token tiles and for four
// row tiles of INT4 on three planes, which take 172.  (Those workgroups are eight
// waves: three waves per SIMD would be one workgroup per compute unit as well.)
template <int FMT, int R, int NT, int TERMS>
constexpr int min_waves() {
  return NT > 1 || (FMT == kINT && R == 4 && TERMS == 3) ? 2 : FMT == kMX || (FMT == kNV && TERMS == 1) ? 4 : 3;
}

// LDS of one workgroup in bytes: the activation buffers, or the sums that meet at
// the end, whichever is more.
template <int R, int D, int NT, int TERMS, int WN, int WK>
inline int64_t lds_bytes(int rows, int64_t K) {
  constexpr int kWidth = WK * D * kStep;
  const int64_t chunks = (K + kWidth - 1) / kWidth;
  const int64_t x = (chunks < kBuffers ? chunks : kBuffers) * 2 * Lines<kWidth>::groups(TERMS * rows) *
                    Lines<kWidth>::kStride;
  const int64_t red = 4 * (int64_t)WN * WK * R * 16 * rows;
  return x > red ? x : red;
}

// The workgroup's product of `rows` activation rows (at most 16 NT, or 4 where
// SPREAD) with its 16 R WN weight rows over all of K; wave wk * WN + wn takes
// its row tiles from p.  src(row): pointer to term 0 of an activation row, once
// ready() has run; terms are `plane` elements apart.  Afterwards group_sum gives
// the results.
//
// SPREAD: up to four tokens stand in rows 0, 4, 8 and 12 of A, so that each
// lane holds one result in the first component of D and INT4's scales cost one
// multiplication per instruction rather than four.
//
// A wave multiplies chunk c while the weights of chunk c + 1 are in flight.  Once
// chunk c's are there it asks for the activations of chunk c + 2 (from the cache,
// and into the buffer that chunk c - 1 left), after the chunk for the weights of
// chunk c + 2.  Loads complete in order: when in chunk c + 1 only these weights are
// still in flight (landed), the copies before them have arrived, and the barrier after
// chunk c + 1 tells the other waves.  That wait is written out, for the compiler does
// not see the copies: where its own waits leave nothing of chunk c + 1 to wait for, it
// has none there.  After the last whole chunk every wave waits for all that it asked
// for: a wave without a part in what remains loads no weights behind its copies of
// that.  (Asked for before the weights of chunk c + 1 were there, the copies would be
// waited for with them, at full latency.)
template <int FMT, int R, int D, int NT, int TERMS, bool SPREAD, int WN, int WK, typename P, typename F>
__device__ __forceinline__ void group_dot(uint16_t* lds, const Rows<FMT, R, D>& p, P ready, F src, int64_t plane,
                                          int rows, int64_t K) {
  constexpr int kSteps = WK * D, kWidth = kSteps * kStep, kWaves = WN * WK;
  static_assert(!SPREAD || NT == 1, "a spread tile is one tile");
  using Ln = Lines<kWidth>;
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wk = wave / WN;
  const int groups = Ln::groups(TERMS * rows), buffer = groups * Ln::kStride;
  const int chunks = (int)((K + kWidth - 1) / kWidth);
  const uint32_t base = (uint32_t)(uintptr_t)(lds_u16*)lds;

  f32x4 acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};
  XAt xo[NT][TERMS];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
      const int row = SPREAD ? n >> 2 : 16 * t + n;
      const int line = i * rows + (row < rows ? row : 0), f = Ln::flip(line);
      if (FMT == kINT) {  // element 32 j + 8 q, j = 0 .. 3
        xo[t][i].at[0] = Ln::at(line) + 8 * q + f;
        xo[t][i].at[1] = Ln::at(line) + 8 * q - f;
      } else {  // element 32 q + 8 j
        xo[t][i].at[0] = xo[t][i].at[1] = Ln::at(line) + ((32 * q) ^ f);
      }
    }

  // Elements past K are copies of the row's first ones: their weights are zero.
  auto copy_x = [&](int c) {
    const int total = groups * Ln::kPieces;
    for (int i = wave; i < total; i += kWaves) {
      const int group = i / Ln::kPieces, piece = i % Ln::kPieces;
      const int e = piece * 512 + lane * 8;  // element of the group
      int line = group * Ln::kPerPiece, pos = e;
      if (Ln::kPerPiece > 1) {
        if (line + e / kWidth < TERMS * rows) line += e / kWidth;
        pos = e % kWidth ^ Ln::flip(e / kWidth);
      }
      const int t = (TERMS > 1 && line >= rows) + (TERMS > 2 && line >= 2 * rows), row = line - t * rows;
      int64_t k = (int64_t)c * kWidth + pos;
      k = k + 8 <= K ? k : 0;
      copy16((glb_u16*)(src(row) + t * plane + k),
             __builtin_amdgcn_readfirstlane(base + 2 * (c % kBuffers * buffer + group * Ln::kStride + piece * 512)));
    }
  };

  const int full = (int)(K / kWidth);
  const int step0 = wk * D;
  const bool tail = full < chunks && ((int64_t)full * kSteps + step0) * kStep < K;  // this wave has a part of it
  const uint16_t* xw = lds + step0 * kStep;
  Raw<FMT, R, D> w0, w1;
  auto load = [&](Raw<FMT, R, D>& to, int c) { load_raw(to, p, (int64_t)c * kSteps + step0); };
  auto load_tail = [&](Raw<FMT, R, D>& to) {
    if (tail) load_raw_tail(to, p, (int64_t)full * kSteps + step0, K);
  };
  auto dot = [&](Raw<FMT, R, D>& w, int c) {
    const auto arrived = [&] {
      landed<Raw<FMT, R, D>::kLoads>();  // chunk c + 1's copies
      if (c + 2 < chunks) copy_x(c + 2);
    };
    multiply<FMT, R, D, NT, TERMS, SPREAD>(acc, w, arrived, xw + (c % kBuffers) * buffer, xo);
    meet();
  };
  auto dot_last = [&](Raw<FMT, R, D>& w) {  // of the whole chunks
    multiply<FMT, R, D, NT, TERMS, SPREAD>(acc, w, [] {}, xw + ((full - 1) % kBuffers) * buffer, xo);
    landed<0>();  // the copies of what remains; weights of it are wanted next
    meet();
  };
  auto dot_tail = [&](Raw<FMT, R, D>& w) {
    if (full == chunks) return;
    if (tail) {
      fix_tail(w, (int64_t)full * kSteps + step0, K);
      multiply<FMT, R, D, NT, TERMS, SPREAD>(acc, w, [] {}, xw + (full % kBuffers) * buffer, xo);
    }
    meet();
  };
  // The first weights need no activations, and are asked for before anything is
  // known of those.
  if (full > 0) {
    load(w0, 0);
  } else if (K >= kStep) {
    load_tail(w0);
  } else if (tail) {
    load_raw_short(w0, p, K);
  }
  ready();
  copy_x(0);
  if (chunks > 1) copy_x(1);
  // Two sets of registers in turn.  (The load behind the break stands on a condition:
  // the compiler gives it registers of its own and, where they become w1 at the loop's
  // end, waits for all that is in flight, so once in two chunks a wave's weights are not
  // asked for ahead.)  After the loop w0 holds chunk c and, unless that is the last
  // whole one, w1 chunk c + 1.
  int c = 0;
  if (full > 1) {
    load(w1, 1);
    arrive<R * D>();
    for (; c + 2 < full; c += 2) {
      dot(w0, c);
      load(w0, c + 2);
      dot(w1, c + 1);
      if (c + 3 >= full) {
        c += 2;
        break;
      }
      load(w1, c + 3);
    }
  } else {
    arrive<0>();
  }
  if (full > 0 && c + 1 == full) {
    load_tail(w1);
    dot_last(w0);
    dot_tail(w1);
  } else {
    if (full > 0) {
      dot(w0, c);
      load_tail(w0);
      dot_last(w1);
    }
    dot_tail(w0);
  }
  landed<0>();  // nothing is left on its way into what the sums take
  float* red = reinterpret_cast<float*>(lds) + wave * (R * 16 * rows);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < (SPREAD ? 1 : 4); ++i) {
        const int m = SPREAD ? q : 16 * t + 4 * q + i;
        if (m < rows) red[(r * rows + m) * 16 + n] = acc[r][t][i];
      }
  __syncthreads();
}

// Sum over wk of the product for weight row c (of 16 R WN) and token m.
template <int R, int WN, int WK>
__device__ __forceinline__ float group_sum(const uint16_t* lds, int c, int m, int rows) {
  const float* red = reinterpret_cast<const float*>(lds) + ((c >> 4) * rows + m) * 16 + (c & 15);
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < WK; ++k) v += red[k * (WN * R * 16 * rows)];
  return v;
}

// X' = T x per block of G channels in fp32, kept as a sum of bf16 planes:
// y = y0 + y1 (+ y2), each the rounding of what the planes before it left.
// Two planes hold 16 bits of y, three hold all 24.  A bf16 result gets two: they are
// off by 2^-17 of y, its own rounding by up to 2^-9, and the third plane, whose matrix
// instructions every weight meets, changes the error against 64 bits by less than one
// part in a thousand (1.655e-3 of the result's norm either way).  It would cost 17.0 ->
// 22.5 us for 4 tokens on 24576 x 4096 MXFP4, 38.6 -> 44.6 for one on 8192 x 28672 INT4 and,
// for the experts' h, 170 -> 184 for 64 tokens on 96 NVFP4 experts.  One wave: 32
// channels (panel) of 16 tokens from m0.
__device__ __forceinline__ void split_panel(const SplitArgs& a, int64_t panel, int64_t m0) {
  const int lane = threadIdx.x & 63, n = lane & 15, q = lane >> 4;
  const int64_t k0 = panel * 32, K = a.K;
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

// A launch with `lds` bytes of dynamic LDS (beyond 64 KB it has to be asked for).
template <typename Kernel, typename Args>
inline hipError_t launch_lds(Kernel kernel, dim3 grid, int threads, int64_t lds, hipStream_t s, const Args& a) {
  constexpr int64_t kLds = 163840;
  if (lds > kLds) return hipErrorInvalidConfiguration;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, grid, dim3(threads), (unsigned)lds, s, a);
  return hipGetLastError();
}

}  // namespace w4
}  // namespace wush

#endif  // WUSH_W4_CORE_H_
