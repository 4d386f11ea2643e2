// Penalties for repeated tokens, biases and grammar masks on rows of logits, in
// one pass.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_adjust.h"

namespace wush {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256, kEach = 8;  // neighbouring logits per thread and step

template <int TYPE>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if (TYPE == 0) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return TYPE == 1 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}
template <int TYPE>
__device__ __forceinline__ uint16_t narrow(float v) {
  return TYPE == 1 ? __builtin_bit_cast(uint16_t, (__bf16)v) : __half_as_ushort(__float2half_rn(v));
}
template <int TYPE>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if (TYPE == 0) {
    static_cast<float*>(p)[i] = v;
  } else {
    static_cast<uint16_t*>(p)[i] = narrow<TYPE>(v);
  }
}
template <int TYPE>
__device__ __forceinline__ void load_all(const void* p, int64_t i, float (&v)[kEach]) {
  if (TYPE == 0) {
    __builtin_memcpy(v, static_cast<const float*>(p) + i, sizeof(v));
  } else {
    uint16_t b[kEach];
    __builtin_memcpy(b, static_cast<const uint16_t*>(p) + i, sizeof(b));
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      v[k] = TYPE == 1 ? __uint_as_float((uint32_t)b[k] << 16) : __half2float(__ushort_as_half(b[k]));
  }
}
template <int TYPE>
__device__ __forceinline__ void store_all(void* p, int64_t i, const float (&v)[kEach]) {
  if (TYPE == 0) {
    __builtin_memcpy(static_cast<float*>(p) + i, v, sizeof(v));
  } else {
    uint16_t b[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) b[k] = narrow<TYPE>(v[k]);
    __builtin_memcpy(static_cast<uint16_t*>(p) + i, b, sizeof(b));
  }
}

// A thread's share of a row's list: the first kHeld entries were asked for when the kernel
// began, the others are read when they are wanted.
template <int HELD>
struct List {
  const int32_t* p;
  int64_t count;
  int32_t held[HELD][4];

  __device__ __forceinline__ void read(int64_t i, int32_t (&t)[4]) const {
    if (i + 4 <= count) {
      __builtin_memcpy(t, p + i, sizeof(t));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = i + k < count ? p[i + k] : -1;
    }
  }
  __device__ __forceinline__ List(const int32_t* list, int64_t n, int64_t row) : p(list + row * n), count(n) {
#pragma unroll
    for (int h = 0; h < HELD; ++h) read((int64_t)(h * kThreads + threadIdx.x) * 4, held[h]);
  }
  // f(token, place in the list) for the tokens in [v0, v0 + n).
  template <typename F>
  __device__ __forceinline__ void each(int64_t v0, int n, F f) const {
    const auto four = [&](const int32_t (&t)[4], int64_t i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t at = t[k] - v0;
        if (at >= 0 && at < n) f((int)at, i + k);
      }
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h) four(held[h], (int64_t)(h * kThreads + threadIdx.x) * 4);
    for (int64_t i = (int64_t)(HELD * kThreads + threadIdx.x) * 4; i < count; i += kThreads * 4) {
      int32_t t[4];
      read(i, t);
      four(t, i);
    }
  }
};

// A token's word in LDS: in the prompt, among the biases, and how often in the output.
constexpr uint32_t kAsked = 0x80000000u, kBiased = 0x40000000u;

// A workgroup takes CHUNK tokens of the vocabulary of one row.  It reads the row's lists
// (from the cache, after the first workgroup), marks and counts the chunk's tokens in LDS,
// and changes the logits in registers.  All that it can ask for is asked for before anything
// else: the logits, and the lists' first entries.  Counts are integers, and a token that is
// twice among the biases has them added up in the list's order, so nothing depends on the
// order of the atomics.
template <int TYPE, int CHUNK>
__global__ __launch_bounds__(kThreads) void adjust_kernel(AdjustArgs a) {
  constexpr int kSteps = CHUNK / (kThreads * kEach);
  __shared__ __attribute__((aligned(16))) uint32_t word[CHUNK];
  __shared__ __attribute__((aligned(16))) float bias[CHUNK];
  __shared__ int twice;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y, v0 = (int64_t)blockIdx.x * CHUNK;
  const int n = (int)(a.V - v0 < CHUNK ? a.V - v0 : CHUNK);
  const List<2> prompt(a.prompt, a.n_prompt, row);
  const List<1> output(a.output, a.n_output, row), biases(a.bias_ids, a.n_bias, row);
  float v[kSteps][kEach];
  uint32_t ok[kSteps];
  const int32_t* bits = a.allowed ? a.allowed + row * ((a.V + 31) / 32) : nullptr;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int i = (s * kThreads + tid) * kEach;
    if (i + kEach <= n) {
      load_all<TYPE>(a.in, row * a.ld_in + v0 + i, v[s]);
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k) v[s][k] = i + k < n ? load_one<TYPE>(a.in, row * a.ld_in + v0 + i + k) : 0.0f;
    }
    ok[s] = bits && i < n ? (uint32_t)bits[(v0 + i) >> 5] >> ((v0 + i) & 31) : 0xFFu;
  }
  const float rep = a.repetition ? a.repetition[row] : 1.0f;
  const float freq = a.frequency ? a.frequency[row] : 0.0f, pres = a.presence ? a.presence[row] : 0.0f;
  const bool marked = a.n_prompt > 0 || a.n_output > 0 || a.n_bias > 0;
  if (marked) {
    for (int i = tid * 4; i < CHUNK; i += kThreads * 4) *reinterpret_cast<u32x4*>(&word[i]) = u32x4{0, 0, 0, 0};
    if (tid == 0) twice = 0;
    __syncthreads();
    prompt.each(v0, n, [&](int t, int64_t) { atomicOr(&word[t], kAsked); });
    output.each(v0, n, [&](int t, int64_t) { atomicAdd(&word[t], 1u); });
    const float* values = a.bias + row * a.n_bias;
    biases.each(v0, n, [&](int t, int64_t i) {
      if (atomicOr(&word[t], kBiased) & kBiased) {
        twice = 1;
      } else {
        bias[t] = values[i];
      }
    });
    __syncthreads();
    if (twice) {
      for (int t = tid; t < n; t += kThreads) {
        if (!(word[t] & kBiased)) continue;
        float sum = 0.0f;
        bool any = false;
        for (int64_t j = 0; j < a.n_bias; ++j)
          if (biases.p[j] - v0 == t) {
            sum = any ? sum + values[j] : values[j];
            any = true;
          }
        bias[t] = sum;
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int i = (s * kThreads + tid) * kEach;
    if (i >= n) continue;
    const int64_t at = v0 + i;
    if (marked) {
      uint32_t w[kEach], any = 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        w[k] = word[i + k];
        any |= w[k];
      }
      if (any) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const uint32_t said = w[k] & ~kBiased, count = said & ~kAsked;
          float l = v[s][k];
          if (said) l = l > 0.0f ? l / rep : l * rep;
          if (count) l = l - freq * (float)count - pres;
          if (w[k] & kBiased) l += bias[i + k];
          v[s][k] = l;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) v[s][k] = (ok[s] >> k) & 1u ? v[s][k] : -__builtin_inff();
    if (i + kEach <= n) {
      store_all<TYPE>(a.out, row * a.ld_out + at, v[s]);
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (i + k < n) store_one<TYPE>(a.out, row * a.ld_out + at + k, v[s][k]);
    }
  }
}

// Chunks of 2048: 200 rows of 100003 fp32 logits take 44.6 us (3.6 TB/s), with 4096 54, for
// then half as many workgroups' loads are in flight; one row of 131072 bf16 logits 5.1 and 6.9.
template <int TYPE>
hipError_t go(const AdjustArgs& a, hipStream_t s) {
  constexpr int kChunk = 2048;
  const dim3 grid((unsigned)((a.V + kChunk - 1) / kChunk), (unsigned)a.R);
  hipLaunchKernelGGL((adjust_kernel<TYPE, kChunk>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t s) {
  if (a.type == 0) return go<0>(a, s);
  if (a.type == 1) return go<1>(a, s);
  return go<2>(a, s);
}

}  // namespace wush
