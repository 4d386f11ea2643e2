// Log probabilities of given tokens, entropies and the largest entries of
// rows of logits, in one pass over the logits.
//
// With m = max l, S = sum e^(l - m) and U = sum e^(l - m) (l - m):
//   log p(t) = l_t - m - log S,   entropy = log S - U / S.
// Every thread keeps its own m, S and U over what it has read (rescaled when its
// maximum grows), so one read of the row suffices; the threads' triples, and where
// several workgroups share a row theirs, are joined by the same rule.
//
// The largest entries are kept as 64-bit keys (ordered value, then lower
// index first), which makes all keys distinct and ties well defined.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wush_w4.h"

namespace wush {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPerThread = 32;                       // elements per thread and batch
constexpr int kBatch = kThreads * kPerThread;        // elements per workgroup and batch
constexpr int kMaxSplits = 64;
// Candidates of one batch: at most `top` threads per wave hold any (see
// keep_largest), with 32 elements each, besides the entries kept so far.
constexpr int kMaxCandidates = kWaves * kLogprobMaxTop * kPerThread + kLogprobMaxTop;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

struct Triple {
  float m, s, u;
};

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// Differences of maxima stop here: their exponential is 0 long before, and
// their product with a sum stays finite (0 times infinity would be NaN).
constexpr float kFloor = -0x1p80f;

// a joined with b.  A triple without a maximum has s = u = 0, or s = NaN where
// a NaN was read.
__device__ __forceinline__ Triple join(Triple a, Triple b) {
  const float m = fmaxf(a.m, b.m);
  const float da = a.m == -kInf ? 0.0f : fmaxf(a.m - m, kFloor), db = b.m == -kInf ? 0.0f : fmaxf(b.m - m, kFloor);
  const float ea = exp_of(da), eb = exp_of(db);
  Triple r;
  r.m = m;
  r.s = a.s * ea + b.s * eb;
  r.u = ea * __builtin_fmaf(da, a.s, a.u) + eb * __builtin_fmaf(db, b.s, b.u);
  return r;
}

__device__ __forceinline__ Triple wave_join(Triple t) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    Triple o;
    o.m = __shfl_xor(t.m, d);
    o.s = __shfl_xor(t.s, d);
    o.u = __shfl_xor(t.u, d);
    t = join(t, o);
  }
  return t;
}

// Key of value v at index i; 0 for what never counts (-inf, NaN).
__device__ __forceinline__ uint64_t key_of(float v, uint32_t i) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return v > -kInf ? ((uint64_t)o << 32) | (0xFFFFFFFFu - i) : 0u;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

template <int TYPE>
struct Elem;
template <>
struct Elem<0> {
  static constexpr int kVec = 4, kBytes = 4;
  static __device__ __forceinline__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ float of(const u32x4& v, int i) { return __uint_as_float(v[i]); }
};
template <>
struct Elem<1> {
  static constexpr int kVec = 8, kBytes = 2;
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  }
  static __device__ __forceinline__ float of(const u32x4& v, int i) {
    return __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
  }
};
template <>
struct Elem<2> {
  static constexpr int kVec = 8, kBytes = 2;
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    return __half2float(__ushort_as_half(static_cast<const uint16_t*>(p)[i]));
  }
  static __device__ __forceinline__ float of(const u32x4& v, int i) {
    return __half2float(__ushort_as_half((uint16_t)(v[i >> 1] >> (16 * (i & 1)))));
  }
};

// The n-th largest (n >= 1) of the keys of the lanes with `in`, of which
// there are at least n: one bit of the key at a time.
__device__ __forceinline__ uint64_t nth_of_wave(uint64_t key, bool in, int n) {
  uint64_t live = __ballot(in);
  for (int b = 63; b >= 0 && __popcll(live) > 1; --b) {
    const uint64_t set = __ballot((key >> b) & 1u) & live;
    const int c = __popcll(set);
    if (c >= n) {
      live = set;
    } else {
      live &= ~set;
      n -= c;
    }
  }
  return __shfl((unsigned long long)key, __ffsll((unsigned long long)live) - 1);
}

struct TopState {
  uint64_t best[kLogprobMaxTop];  // sorted, 0 where there are fewer
  uint64_t wave_bound[kWaves];
  uint64_t cand[kMaxCandidates];
  int n;
};

// best <- the `top` largest of the n candidates, by counting for each how many are
// larger (keys are distinct).  All threads; `n` candidates are in place.
__device__ __forceinline__ void rank_candidates(TopState& t, int top) {
  const int n = t.n;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t k = t.cand[i];
    int larger = 0;
    for (int j = 0; j < n; ++j) larger += t.cand[j] > k;
    if (larger < top) t.best[larger] = k;
  }
  __syncthreads();
}

// One batch of the workgroup: thread's elements x[j] at index
// at + (j / VEC) * kThreads * VEC + j % VEC.
//
// Only what is larger than the worst entry kept counts.  Where a wave has at least
// `top` threads with such a maximum, its top-th largest thread maximum bounds the
// answer from below too: at least `top` elements reach it.  Under the largest
// such bound of the waves, at most `top` threads of any wave hold candidates.
template <int VEC>
__device__ __forceinline__ void keep_largest(TopState& t, const float (&x)[kPerThread], uint32_t at, float batch_max,
                                             int top) {
  const uint64_t worst = t.best[top - 1];
  const float worst_value = worst ? key_value(worst) : -kInf;
  // Later batches hold higher indices: an equal value does not enter.
  const bool in = batch_max > worst_value;
  if (!__syncthreads_or(in)) return;
  uint64_t mine = 0;
  if (in) {
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const uint64_t k = key_of(x[j], at + (uint32_t)((j / VEC) * kThreads * VEC + j % VEC));
      mine = k > mine ? k : mine;
    }
  }
  const uint64_t votes = __ballot(in);
  uint64_t bound = worst + 1;
  if (__popcll(votes) >= top) bound = nth_of_wave(mine, in, top);
  if ((threadIdx.x & 63) == 0) t.wave_bound[threadIdx.x >> 6] = bound;
  if (threadIdx.x < top) t.cand[threadIdx.x] = t.best[threadIdx.x];
  if (threadIdx.x == 0) t.n = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) bound = t.wave_bound[w] > bound ? t.wave_bound[w] : bound;
  if (mine >= bound) {
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const uint64_t k = key_of(x[j], at + (uint32_t)((j / VEC) * kThreads * VEC + j % VEC));
      if (k >= bound) t.cand[atomicAdd(&t.n, 1)] = k;
    }
  }
  __syncthreads();
  rank_candidates(t, top);
}

struct Finish {
  float m, log_s, entropy;
  bool none, bad;  // no finite logit; a NaN or +inf among them
};

__device__ __forceinline__ Finish finish(Triple t) {
  Finish f;
  f.m = t.m;
  f.bad = t.s != t.s;
  f.none = t.m == -kInf && !f.bad;
  f.log_s = __builtin_amdgcn_logf(t.s) * kLn2;
  f.entropy = f.none ? 0.0f : f.log_s - t.u / t.s;
  return f;
}

template <int TYPE>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, Triple t, const TopState* top) {
  const Finish f = finish(t);
  if (threadIdx.x == 0) {
    const int64_t id = a.targets[row];
    float lp = 0.0f;
    if (id >= a.V) {
      lp = __builtin_nanf("");
    } else if (id >= 0) {
      const float l =
          Elem<TYPE>::one(static_cast<const uint8_t*>(a.L) + row * a.ld * Elem<TYPE>::kBytes, id);
      lp = f.none ? -kInf : (l - f.m) - f.log_s;
    }
    a.logprob[row] = lp;
    a.entropy[row] = f.entropy;
  }
  if (top && (int)threadIdx.x < a.top) {
    const uint64_t k = top->best[threadIdx.x];
    const int64_t o = row * a.top + threadIdx.x;
    const bool there = k != 0 && !f.bad;
    a.top_ids[o] = there ? (int32_t)(0xFFFFFFFFu - (uint32_t)k) : -1;
    a.top_logprobs[o] = f.bad ? __builtin_nanf("") : there ? (key_value(k) - f.m) - f.log_s : -kInf;
  }
}

__device__ __forceinline__ Triple group_join(Triple t, Triple* lds) {
  t = wave_join(t);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = t;
  __syncthreads();
  t = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) t = join(t, lds[w]);
  return t;
}

template <bool TOP>
struct Shared {
  Triple part[kWaves];
};
template <>
struct Shared<true> {
  Triple part[kWaves];
  TopState top;
};

template <int TYPE, bool TOP>
__global__ __launch_bounds__(kThreads) void logprob_kernel(LogprobArgs a) {
  using El = Elem<TYPE>;
  constexpr int VEC = El::kVec, NV = kPerThread / VEC;
  __shared__ Shared<TOP> sh;
  const int64_t row = blockIdx.x / a.splits;
  const int split = blockIdx.x % a.splits;
  const uint8_t* L = static_cast<const uint8_t*>(a.L) + row * a.ld * El::kBytes;
  // Vectors on 16-byte boundaries: the first and the last may be partial.
  const int shift = (int)((reinterpret_cast<uintptr_t>(L) % 16) / El::kBytes);
  const int64_t V = a.V, n_vec = (V + shift + VEC - 1) / VEC;
  const int64_t batches = (n_vec + kThreads * NV - 1) / (kThreads * NV);
  const int64_t b0 = batches * split / a.splits, b1 = batches * (split + 1) / a.splits;
  if constexpr (TOP) {
    if ((int)threadIdx.x < kLogprobMaxTop) sh.top.best[threadIdx.x] = 0;
    __syncthreads();
  }
  Triple t = {-kInf, 0.0f, 0.0f};
  for (int64_t b = b0; b < b1; ++b) {
    const int64_t v0 = b * (kThreads * NV) + threadIdx.x;
    u32x4 raw[NV];
    float x[kPerThread];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t e = (v0 + j * kThreads) * VEC - shift;  // the vector's first element
      if (e >= 0 && e + VEC <= V) raw[j] = *reinterpret_cast<const u32x4*>(L + e * El::kBytes);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t e = (v0 + j * kThreads) * VEC - shift;
      const bool whole = e >= 0 && e + VEC <= V;
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j * VEC + i] = whole ? El::of(raw[j], i) : -kInf;
      if (!whole && e > -VEC && e < V) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (e + i >= 0 && e + i < V) x[j * VEC + i] = El::one(L, e + i);
      }
    }
    float bm = x[0];
#pragma unroll
    for (int j = 1; j < kPerThread; ++j) bm = fmaxf(bm, x[j]);
    if (bm > t.m) {
      const float d = t.m == -kInf ? 0.0f : fmaxf(t.m - bm, kFloor), e = exp_of(d);
      t.u = e * __builtin_fmaf(d, t.s, t.u);
      t.s *= e;
      t.m = bm;
    }
    const float m = t.m == -kInf ? 0.0f : t.m;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      // Masked: e = 0, and the floor keeps e d from being NaN.  NaN stays in e.
      const float d = x[j] - m, e = exp_of(d);
      t.s += e;
      t.u = __builtin_fmaf(e, fmaxf(d, kFloor), t.u);
    }
    if constexpr (TOP) keep_largest<VEC>(sh.top, x, (uint32_t)(v0 * VEC - shift), bm, a.top);
  }
  t = group_join(t, sh.part);
  const TopState* top = nullptr;
  if constexpr (TOP) top = &sh.top;
  if (a.splits == 1) {
    write_row<TYPE>(a, row, t, top);
  } else {
    if (threadIdx.x == 0) {
      float* p = a.part + 4 * (row * a.splits + split);
      p[0] = t.m;
      p[1] = t.s;
      p[2] = t.u;
    }
    if constexpr (TOP) {
      if ((int)threadIdx.x < a.top) a.keys[(row * a.splits + split) * a.top + threadIdx.x] = sh.top.best[threadIdx.x];
    }
  }
}

// Rows that several workgroups shared.
template <int TYPE, bool TOP>
__global__ __launch_bounds__(kThreads) void join_kernel(LogprobArgs a) {
  __shared__ Shared<TOP> sh;
  const int64_t row = blockIdx.x;
  Triple t = {-kInf, 0.0f, 0.0f};
  if ((int)threadIdx.x < a.splits) {
    const float* p = a.part + 4 * (row * a.splits + threadIdx.x);
    t = Triple{p[0], p[1], p[2]};
  }
  const TopState* top = nullptr;
  if constexpr (TOP) {
    const int n = a.splits * a.top;  // at most kMaxSplits * kLogprobMaxTop
    static_assert(kMaxSplits * kLogprobMaxTop <= kMaxCandidates, "the splits' entries must fit");
    for (int i = threadIdx.x; i < n; i += kThreads) sh.top.cand[i] = a.keys[row * n + i];
    if ((int)threadIdx.x < kLogprobMaxTop) sh.top.best[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.top.n = n;
    __syncthreads();
    rank_candidates(sh.top, a.top);
    top = &sh.top;
  }
  t = group_join(t, sh.part);
  write_row<TYPE>(a, row, t, top);
}

template <int TYPE, bool TOP>
hipError_t go(const LogprobArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((logprob_kernel<TYPE, TOP>), dim3((unsigned)(a.R * a.splits)), dim3(kThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((join_kernel<TYPE, TOP>), dim3((unsigned)a.R), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int logprob_splits(int64_t R, int64_t V, int) {
  const int64_t batches = (V + kBatch - 1) / kBatch;
  int64_t s = 1024 / (R > 0 ? R : 1);
  if (s > batches) s = batches;
  if (s > kMaxSplits) s = kMaxSplits;
  return s < 1 ? 1 : (int)s;
}

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s) {
  if (a.type == 0) return a.top ? go<0, true>(a, s) : go<0, false>(a, s);
  if (a.type == 1) return a.top ? go<1, true>(a, s) : go<1, false>(a, s);
  return a.top ? go<2, true>(a, s) : go<2, false>(a, s);
}

}  // namespace wush
