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

// f(token) for the tokens of a list that lie in [v0, v0 + n).
template <typename F>
__device__ __forceinline__ void each_token(const int32_t* list, int64_t count, int64_t v0, int n, F f) {
  for (int64_t i = (int64_t)threadIdx.x * 4; i < count; i += kThreads * 4) {
    int32_t t[4] = {-1, -1, -1, -1};
    if (i + 4 <= count) {
      __builtin_memcpy(t, list + i, sizeof(t));
    } else {
      for (int k = 0; k < (int)(count - i); ++k) t[k] = list[i + k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = t[k] - v0;
      if (at >= 0 && at < n) f((int)at);
    }
  }
}

constexpr uint32_t kAsked = 0x80000000u;  // in the prompt; below it, how often in the output

// A workgroup takes CHUNK tokens of the vocabulary of one row.  It reads the row's whole
// lists (from the cache, after the first workgroup) and keeps what falls into its chunk
// in LDS: how often a token was said, and its bias.  Then the logits pass through once.
// Counting with integers and adding a token's biases in the list's order makes the result
// independent of the order of the atomics.  Bound by the logits' way in and out.
template <int TYPE, int CHUNK>
__global__ __launch_bounds__(kThreads) void adjust_kernel(AdjustArgs a) {
  extern __shared__ uint32_t lds[];
  uint32_t* said = lds;
  uint32_t* times = lds + CHUNK;                                // a token's entries among the biases
  float* bias = reinterpret_cast<float*>(lds + 2 * CHUNK);
  const int64_t row = blockIdx.y, v0 = (int64_t)blockIdx.x * CHUNK;
  const int n = (int)(a.V - v0 < CHUNK ? a.V - v0 : CHUNK);
  const bool counted = a.n_prompt > 0 || a.n_output > 0, biased = a.n_bias > 0;
  if (counted)
    for (int i = threadIdx.x; i < n; i += kThreads) said[i] = 0;
  if (biased)
    for (int i = threadIdx.x; i < n; i += kThreads) {
      times[i] = 0;
      bias[i] = 0.0f;
    }
  __syncthreads();
  each_token(a.prompt + row * a.n_prompt, a.n_prompt, v0, n, [&](int t) { atomicOr(&said[t], kAsked); });
  each_token(a.output + row * a.n_output, a.n_output, v0, n, [&](int t) { atomicAdd(&said[t], 1u); });
  if (biased) {
    const int32_t* ids = a.bias_ids + row * a.n_bias;
    const float* values = a.bias + row * a.n_bias;
    each_token(ids, a.n_bias, v0, n, [&](int t) { atomicAdd(&times[t], 1u); });
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.n_bias; i += kThreads) {
      const int64_t t = ids[i] - v0;
      if (t < 0 || t >= n) continue;
      float sum = values[i];
      if (times[t] > 1) {
        bool first = true;
        for (int64_t j = 0; j < i && first; ++j) first = ids[j] != ids[i];
        if (!first) continue;
        for (int64_t j = i + 1; j < a.n_bias; ++j)
          if (ids[j] == ids[i]) sum += values[j];
      }
      bias[t] = sum;
    }
  }
  __syncthreads();
  const float rep = a.repetition ? a.repetition[row] : 1.0f;
  const float freq = a.frequency ? a.frequency[row] : 0.0f, pres = a.presence ? a.presence[row] : 0.0f;
  const int32_t* bits = a.allowed ? a.allowed + row * ((a.V + 31) / 32) : nullptr;
  const auto adjusted = [&](float l, int i, bool ok) {
    if (counted) {
      const uint32_t s = said[i];
      if (s) {
        l = l > 0.0f ? l / rep : l * rep;
        const uint32_t c = s & ~kAsked;
        if (c) l = l - freq * (float)c - pres;
      }
    }
    if (biased && times[i]) l += bias[i];
    return ok ? l : -__builtin_inff();
  };
  for (int i = threadIdx.x * kEach; i < n; i += kThreads * kEach) {
    const int64_t at = v0 + i;
    const uint32_t ok = bits ? (uint32_t)bits[at >> 5] >> (at & 31) : 0xFFu;
    if (i + kEach <= n) {
      float v[kEach];
      load_all<TYPE>(a.in, row * a.ld_in + at, v);
#pragma unroll
      for (int k = 0; k < kEach; ++k) v[k] = adjusted(v[k], i + k, (ok >> k) & 1u);
      store_all<TYPE>(a.out, row * a.ld_out + at, v);
    } else {
      for (int k = 0; k < n - i; ++k)
        store_one<TYPE>(a.out, row * a.ld_out + at + k,
                        adjusted(load_one<TYPE>(a.in, row * a.ld_in + at + k), i + k, (ok >> k) & 1u));
    }
  }
}

template <int TYPE, int CHUNK>
hipError_t go(const AdjustArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.V + CHUNK - 1) / CHUNK), (unsigned)a.R);
  const unsigned lds = a.n_bias > 0 ? 3 * CHUNK * 4 : CHUNK * 4;
  hipLaunchKernelGGL((adjust_kernel<TYPE, CHUNK>), grid, dim3(kThreads), lds, s, a);
  return hipGetLastError();
}

// Chunks as wide as leaves the chip about two workgroups per compute unit.
template <int TYPE>
hipError_t go_chunk(const AdjustArgs& a, hipStream_t s) {
  if (a.R * (a.V / 4096) >= 512) return go<TYPE, 4096>(a, s);
  if (a.R * (a.V / 2048) >= 256) return go<TYPE, 2048>(a, s);
  return go<TYPE, 512>(a, s);
}

}  // namespace

hipError_t launch_adjust(const AdjustArgs& a, hipStream_t s) {
  if (a.type == 0) return go_chunk<0>(a, s);
  if (a.type == 1) return go_chunk<1>(a, s);
  return go_chunk<2>(a, s);
}

}  // namespace wush
