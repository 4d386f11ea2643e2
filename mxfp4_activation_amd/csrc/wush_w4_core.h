// The wave-level product of a few activation rows with rows of 4-bit weights,
// shared by the linear layer (wush_w4.hip) and the mixture of experts
// (wush_moe.hip).  Device code only.
//
// One wave multiplies R tiles of 16 weight rows with NT tiles of 16 tokens
// on v_mfma_f32_16x16x32_bf16: A = activations (row m = token), B = weights
// (column n = weight row), D[m][n] with m = 4 (lane / 16) + i, n = lane % 16.
// A few tokens leave most of A's rows unused (row m of D depends on row m of A
// alone, so unused rows hold copies of a valid token and are never stored);
// the matrix cores are still far from the limit.  The limit is the weights'
// way in, and behind it the vector instructions that turn codes into bf16.
//
// A step is 128 elements of K: lane (q = lane / 16, n) loads the 16 code
// bytes of row n, elements 32 q .. 32 q + 31, so the four lanes of a row read
// 64 contiguous bytes.  A 4 x 4 transpose of dwords between the four
// lane quarters (four lane-swap instructions) then leaves in dword g elements
// 32 g + 8 q .. + 7: matrix instruction g covers exactly the group of 32
// elements g of all 16 rows, and the activations are read in their natural
// order.
//
// Exactness.  E2M1 * 2^e and E2M1 * E4M3 have at most 6 significant bits, and
// the integers of INT4 have 4, so all of them are exact in bf16; the fp16
// scale of INT4 is applied in fp32 to each group's sum, NVFP4's tensor scale in
// fp32 to the result.  Products of bf16 are exact in the matrix cores, sums
// are fp32.
#ifndef WUSH_W4_CORE_H_
#define WUSH_W4_CORE_H_

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wush {
namespace w4 {

constexpr int kMX = 0, kNV = 1, kINT = 2, kBF = 3;  // kBF: bf16 weights (the router)
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

// One lane's share of 16 rows x 128 elements as it is in memory.
template <int FMT>
struct Raw {
  u32x4 c;   // 32 codes
  u32x2 s;   // the row's scales of this step: 4 E8M0 bytes, 8 E4M3 bytes or 4 fp16
};
template <>
struct Raw<kBF> {
  u32x4 c[4];
};

template <int FMT>
__device__ __forceinline__ int64_t row_code_bytes(int64_t K) { return FMT == kBF ? 2 * K : K / 2; }
template <int FMT>
__device__ __forceinline__ int64_t row_scale_bytes(int64_t K) {
  return FMT == kMX ? K / 32 : FMT == kNV || FMT == kINT ? K / 16 : 0;
}

// A whole step: cp and sp point at the lane's row, st counts steps.
template <int FMT>
__device__ __forceinline__ void load_raw(Raw<FMT>& w, const uint8_t* cp, const uint8_t* sp, int64_t st, int q) {
  if constexpr (FMT == kBF) {
#pragma unroll
    for (int g = 0; g < 4; ++g) w.c[g] = load_unaligned<u32x4>(cp + 256 * st + 64 * g + 16 * q);
  } else {
    w.c = load_unaligned<u32x4>(cp + 64 * st + 16 * q);
    if constexpr (FMT == kMX) {
      w.s[0] = load_unaligned<uint32_t>(sp + 4 * st);
      w.s[1] = 0;
    } else {
      w.s = load_unaligned<u32x2>(sp + 8 * st);
    }
  }
}

// The last, partial step of a K that is no multiple of 128: nothing is read
// past the row, and what is missing is zero.
template <int FMT>
__device__ __forceinline__ void load_raw_tail(Raw<FMT>& w, const uint8_t* cp, const uint8_t* sp, int64_t st, int q,
                                              int K) {
  const int left = K - (int)st * kStep;  // 16 .. 112 elements
  if constexpr (FMT == kBF) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      w.c[g] = u32x4{0, 0, 0, 0};
      if (32 * g + 8 * q + 8 <= left) w.c[g] = load_unaligned<u32x4>(cp + 256 * st + 64 * g + 16 * q);
    }
  } else {
    w.c = u32x4{0, 0, 0, 0};
    if (32 * q + 32 <= left) {
      w.c = load_unaligned<u32x4>(cp + 64 * st + 16 * q);
    } else if (32 * q + 16 <= left) {
      const u32x2 h = load_unaligned<u32x2>(cp + 64 * st + 16 * q);
      w.c[0] = h[0];
      w.c[1] = h[1];
    }
    w.s = u32x2{0, 0};
    const int bytes = FMT == kMX ? left / 32 : left / 16;
#pragma unroll
    for (int b = 0; b < 7; ++b)
      if (b < bytes) w.s[b / 4] |= (uint32_t)sp[(FMT == kMX ? 4 : 8) * st + b] << (8 * (b % 4));
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

// What group g's codes are multiplied with before (MXFP4, NVFP4) or after
// (INT4) the matrix instruction.
template <int FMT>
__device__ __forceinline__ float group_scale(const Raw<FMT>& w, int g, int q) {
  if constexpr (FMT == kMX) {
    // The E8M0 byte is an fp32 exponent; the conversion reads nothing else
    // of its scale operand, and takes 0 for 2^-127 and 255 for NaN.
    return __uint_as_float(((w.s[0] >> (8 * g)) & 0xFFu) << 23);
  } else if constexpr (FMT == kNV) {
    // Elements 8 q .. 8 q + 7 of the 32 are in scale group 2 g + q / 2.
    const uint32_t v = w.s[g >> 1] >> (8 * (q >> 1));
    return g & 1 ? __builtin_amdgcn_cvt_f32_fp8(v, 2) : __builtin_amdgcn_cvt_f32_fp8(v, 0);
  } else if constexpr (FMT == kINT) {
    return __half2float(__ushort_as_half((uint16_t)(w.s[g >> 1] >> (16 * (g & 1)))));
  } else {
    return 1.0f;
  }
}

// Group g of the (transposed) codes as 8 bf16 weights; INT4 as code + 8.
template <int FMT>
__device__ __forceinline__ bf16x8 expand(const Raw<FMT>& w, int g, float s) {
  u32x4 r;
  if constexpr (FMT == kBF) {
    r = w.c[g];
  } else if constexpr (FMT == kMX) {
    const uint32_t d = w.c[g];
    r[0] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0));
    r[1] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1));
    r[2] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2));
    r[3] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3));
  } else if constexpr (FMT == kNV) {
    const uint32_t d = w.c[g];
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
    const uint32_t u = w.c[g] ^ 0x88888888u;
    const uint32_t lo = u & 0x0F0F0F0Fu, hi = (u >> 4) & 0x0F0F0F0Fu;
    const uint32_t p0 = __builtin_amdgcn_perm(hi, lo, 0x05010400u);  // elements 0 .. 3
    const uint32_t p1 = __builtin_amdgcn_perm(hi, lo, 0x07030602u);  // elements 4 .. 7
    r[0] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, false));
    r[1] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p0, 512.0f, true));
    r[2] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, false));
    r[3] = pack(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p1, 512.0f, true));
  }
  return __builtin_bit_cast(bf16x8, r);
}

// One step's products.  xp[t] points at the lane's token row of token tile t;
// TAIL: groups (of 8 elements) past K read nothing and count as zero.
template <int FMT, int R, int NT, int TERMS, bool TAIL>
__device__ __forceinline__ void step(f32x4 (&acc)[R][NT], Raw<FMT> (&w)[R], const uint16_t* const (&xp)[NT],
                                     int64_t plane, int64_t st, int q, int K) {
  bf16x8 x[4][NT][TERMS];
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int p = 0; p < TERMS; ++p) {
        const int64_t k = st * kStep + 32 * g + 8 * q;
        u32x4 v = {0, 0, 0, 0};
        if (!TAIL || k + 8 <= K) v = *reinterpret_cast<const u32x4*>(xp[t] + p * plane + k);
        x[g][t][p] = __builtin_bit_cast(bf16x8, v);
      }
  if constexpr (FMT != kBF) {
#pragma unroll
    for (int r = 0; r < R; ++r) transpose4(w[r].c);
  }
  // INT4's codes come in as code + 8: the group's sum starts at
  // -8 sum x, which one more matrix instruction with a constant -8 gives in
  // every column.
  const uint32_t m8 = 0xC100C100u;  // bf16 -8, twice
  const bf16x8 minus8 = __builtin_bit_cast(bf16x8, (u32x4{m8, m8, m8, m8}));
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    f32x4 init[NT];
    if constexpr (FMT == kINT) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        init[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < TERMS; ++p)
          init[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[g][t][p], minus8, init[t], 0, 0, 0);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float s = group_scale<FMT>(w[r], g, q);
      const bf16x8 b = expand<FMT>(w[r], g, s);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 c = FMT == kINT ? init[t] : acc[r][t];
#pragma unroll
        for (int p = 0; p < TERMS; ++p) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[g][t][p], b, c, 0, 0, 0);
        if constexpr (FMT == kINT) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(s, c[i], acc[r][t][i]);
        } else {
          acc[r][t] = c;
        }
      }
    }
  }
}

// acc += the product over steps first, first + every, ... below n_steps
// (ceil(K / 128)).  The next step's weights are on their way while this one's
// are multiplied.
template <int FMT, int R, int NT, int TERMS>
__device__ __forceinline__ void wave_dot(f32x4 (&acc)[R][NT], const uint8_t* const (&cp)[R],
                                         const uint8_t* const (&sp)[R], const uint16_t* const (&xp)[NT],
                                         int64_t plane, int K, int first, int every) {
  const int q = (threadIdx.x & 63) >> 4;
  const int whole = K / kStep;
  Raw<FMT> w[R];
  int st = first;
  if (st < whole) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_raw<FMT>(w[r], cp[r], sp[r], st, q);
  }
  while (st < whole) {
    Raw<FMT> nw[R];
    const int nx = st + every;
    // The last turn loads its own step once more, rather than branch.
    const int ld = nx < whole ? nx : st;
#pragma unroll
    for (int r = 0; r < R; ++r) load_raw<FMT>(nw[r], cp[r], sp[r], ld, q);
    step<FMT, R, NT, TERMS, false>(acc, w, xp, plane, st, q, K);
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = nw[r];
    st = nx;
  }
  if (st == whole && whole * kStep < K) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_raw_tail<FMT>(w[r], cp[r], sp[r], st, q, K);
    step<FMT, R, NT, TERMS, true>(acc, w, xp, plane, st, q, K);
  }
}

}  // namespace w4
}  // namespace wush

#endif  // WUSH_W4_CORE_H_
