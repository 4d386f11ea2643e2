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
#include "wush_wave.h"

namespace wush {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = kLogprobThreads, kWaves = kThreads / 64;
constexpr int kWide = kLogprobWide, kNarrow = kLogprobNarrow;
// Candidates of one batch: at most `top` threads hold any (see keep_largest),
// besides the entries kept so far; padded for rank_candidates.
template <int PER>
constexpr int kMaxCandidates = kLogprobMaxTop * PER + kLogprobMaxTop + 8;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

struct Triple {
  float m, s, u;
};

// The product rounds once, so a probability is off by up to |d| roundings: 80 of them
// where it is 1e-35.
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

// Key of value v at index i, -0 like +0; 0 for what never counts (-inf, NaN).
__device__ __forceinline__ uint64_t key_of(float v, uint32_t i) {
  const uint32_t b = __float_as_uint(v + 0.0f);
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

// A bound that exactly n (>= 1) of the wave's keys reach, of which at least n are
// not 0 (those are distinct), by bisection between the smallest and the largest.
// Some eight halvings where values are spread, at most 64.
template <int K>
__device__ __forceinline__ uint64_t bound_of(const uint64_t (&key)[K], int n) {
  uint32_t most = 0, least = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const uint32_t word = (uint32_t)(key[i] >> 32);
    most = word > most ? word : most;
    least = key[i] != 0 && word < least ? word : least;
  }
  most = fold(most, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  least = fold(least, 0xFFFFFFFFu, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
  uint64_t lo = ((uint64_t)least << 32) + 1, hi = ((uint64_t)most << 32) + 0x100000000ull;  // n reach lo, none hi
  while (hi - lo > 1) {
    const uint64_t mid = lo + (hi - lo) / 2;
    int c = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) c += __popcll(__ballot(key[i] >= mid));
    if (c == n) return mid;
    if (c > n) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  return lo;
}

template <int PER>
struct TopState {
  uint64_t best[kLogprobMaxTop];  // sorted, 0 where there are fewer
  uint64_t largest[kThreads];     // of every thread
  __attribute__((aligned(16))) uint64_t cand[kMaxCandidates<PER>];
  int n;
};

// best <- the `top` largest of the t.n candidates, by counting for each how
// many are larger (keys are distinct, but for zeros, which all go last).  All
// threads; the candidates are in place.
template <int PER>
__device__ __forceinline__ void rank_candidates(TopState<PER>& t, int top) {
  constexpr int kStep = 8;
  const int n = t.n;
  if ((int)threadIdx.x < kStep) t.cand[n + threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t k = t.cand[i];
    int larger = 0;
    for (int j = 0; j < n; j += kStep) {
#pragma unroll
      for (int u = 0; u < kStep; ++u) larger += t.cand[j + u] > k;
    }
    if (larger < top) t.best[larger] = k;
  }
  __syncthreads();
}

// One batch of the workgroup: thread's elements x[j] at index
// at + (j / VEC) * kThreads * VEC + j % VEC.
//
// Only what is larger than the worst entry kept counts.  Where at least `top`
// threads have such a maximum, a bound that `top` of the threads' maxima reach bounds
// the answer from below too, and just these threads hold candidates.
template <int VEC, int PER>
__device__ __forceinline__ void keep_largest(TopState<PER>& t, const float (&x)[PER], uint32_t at, float batch_max,
                                             int top) {
  const uint64_t worst = t.best[top - 1];
  const float worst_value = worst ? key_value(worst) : -kInf;
  // Later batches hold higher indices: an equal value does not enter.
  const bool in = batch_max > worst_value;
  const int entering = __syncthreads_count(in);
  if (entering == 0) return;
  uint64_t mine = 0;
  if (in) {
    // The thread's first element of that value.
    int first = 0;
#pragma unroll
    for (int j = PER - 1; j >= 0; --j) first = x[j] == batch_max ? (j / VEC) * kThreads * VEC + j % VEC : first;
    mine = key_of(batch_max, at + (uint32_t)first);
  }
  // The entries kept so far, none before the first batch with any.
  const int kept = t.best[0] ? top : 0;
  if ((int)threadIdx.x < kept) t.cand[threadIdx.x] = t.best[threadIdx.x];
  if (threadIdx.x == 0) t.n = kept;
  uint64_t bound = worst + 1;
  if (entering >= top) {
    t.largest[threadIdx.x] = mine;
    __syncthreads();
    uint64_t all[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all[w] = t.largest[64 * w + (threadIdx.x & 63)];
    bound = bound_of<kWaves>(all, top);
  } else {
    __syncthreads();
  }
  // key >= bound, on the halves: the value first, then the lower index.
  const float least = bound > 1 ? key_value(bound) : -kInf;
  const uint32_t up_to = 0xFFFFFFFFu - (uint32_t)bound;
  const bool hold = mine >= bound;
  if (__ballot(hold) != 0) {
    uint64_t at_j[PER];  // lanes whose element j is a candidate
    int total = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint32_t i = at + (uint32_t)((j / VEC) * kThreads * VEC + j % VEC);
      at_j[j] = __ballot(hold && (x[j] > least || (x[j] == least && least > -kInf && i <= up_to)));
      total += __popcll(at_j[j]);
    }
    const int lane = threadIdx.x & 63;
    int to = 0;
    if (lane == 0) to = atomicAdd(&t.n, total);
    to = __builtin_amdgcn_readfirstlane(to);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (at_j[j] >> lane & 1)
        t.cand[to + __popcll(at_j[j] & ((1ull << lane) - 1))] =
            key_of(x[j], at + (uint32_t)((j / VEC) * kThreads * VEC + j % VEC));
      to += __popcll(at_j[j]);
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

template <int TYPE, typename Top>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, Triple t, const Top* top) {
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
  Triple w;
  w.m = wave_max(t.m);
  const float d = t.m == -kInf ? 0.0f : fmaxf(t.m - w.m, kFloor), e = exp_of(d);
  w.s = wave_sum(t.s * e);
  w.u = wave_sum(e * __builtin_fmaf(d, t.s, t.u));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = w;
  __syncthreads();
  t = lds[0];
#pragma unroll
  for (int k = 1; k < kWaves; ++k) t = join(t, lds[k]);
  return t;
}

template <bool TOP, int PER>
struct Shared {
  Triple part[kWaves];
};
template <int PER>
struct Shared<true, PER> {
  Triple part[kWaves];
  TopState<PER> top;
};

// One row, or one of its splits, per workgroup.  Bound by reading the logits where
// rows are many: 2048 x 65536 bf16 takes 56 us (4.8 TB/s, 94% of a copy's rate)
// without alternatives.  Few rows are bound by the way through one workgroup: 10.5 us
// for one row of 131072 on 64 workgroups with 20 alternatives, of which some 3.4 us are the
// choice (bisection 0.9, candidates 1.1, their order 0.5), then 4.5 us for the join.
// Many rows with alternatives are bound by the choice per batch of each row: 2048 x
// 65536 takes 59 us without, 96 with one and 152 with 20.
template <int TYPE, bool TOP, int PER>
__global__ __launch_bounds__(kThreads) void logprob_kernel(LogprobArgs a) {
  using El = Elem<TYPE>;
  constexpr int VEC = El::kVec, NV = PER / VEC;
  __shared__ Shared<TOP, PER> sh;
  const int64_t row = blockIdx.x;
  const int split = blockIdx.y;
  const uint8_t* L = static_cast<const uint8_t*>(a.L) + row * a.ld * El::kBytes;
  // Vectors on 16-byte boundaries: the first and the last may be partial.
  const int shift = (int)((reinterpret_cast<uintptr_t>(L) % 16) / El::kBytes);
  const int64_t V = a.V;
  constexpr uint32_t kVecs = kThreads * NV;  // vectors per batch
  const uint32_t n_vec = ((uint32_t)V + shift + VEC - 1) / VEC, batches = (n_vec + kVecs - 1) / kVecs;
  const uint32_t b0 = split * a.split_batches;
  const uint32_t b1 = split == a.splits - 1 ? batches : b0 + a.split_batches;
  if constexpr (TOP) {
    if ((int)threadIdx.x < kLogprobMaxTop) sh.top.best[threadIdx.x] = 0;
    __syncthreads();
  }
  Triple t = {-kInf, 0.0f, 0.0f};
  for (uint32_t b = b0; b < b1; ++b) {
    const int64_t v0 = (int64_t)b * kVecs + threadIdx.x;
    u32x4 raw[NV];
    float x[PER];
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
    for (int j = 1; j < PER; ++j) bm = fmaxf(bm, x[j]);
    if (bm > t.m) {
      const float d = t.m == -kInf ? 0.0f : fmaxf(t.m - bm, kFloor), e = exp_of(d);
      t.u = e * __builtin_fmaf(d, t.s, t.u);
      t.s *= e;
      t.m = bm;
    }
    const float m = t.m == -kInf ? 0.0f : t.m;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      // Masked: e = 0, and the floor keeps e d from being NaN.  NaN stays in e.
      const float d = x[j] - m, e = exp_of(d);
      t.s += e;
      t.u = __builtin_fmaf(e, fmaxf(d, kFloor), t.u);
    }
    if constexpr (TOP) keep_largest<VEC, PER>(sh.top, x, (uint32_t)(v0 * VEC - shift), bm, a.top);
  }
  t = group_join(t, sh.part);
  const TopState<PER>* top = nullptr;
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

// Rows that several workgroups shared.  Where there are `top` splits or more, a
// bound that `top` of their largest entries reach bounds the answer from below,
// and at most `top` splits hold candidates.
template <int TYPE, bool TOP>
__global__ __launch_bounds__(kThreads) void join_kernel(LogprobArgs a) {
  __shared__ Shared<TOP, kWide> sh;
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 63;
  Triple t = {-kInf, 0.0f, 0.0f};
  if ((int)threadIdx.x < a.splits) {
    const float* p = a.part + 4 * (row * a.splits + threadIdx.x);
    t = Triple{p[0], p[1], p[2]};
  }
  const TopState<kWide>* top = nullptr;
  if constexpr (TOP) {
    static_assert(kLogprobMaxSplits == 64, "one wave holds a row's splits");
    static_assert(kLogprobMaxTop * kLogprobMaxTop + 8 <= kMaxCandidates<kWide>, "the candidates must fit");
    const uint64_t* keys = a.keys + row * a.splits * a.top;
    const int n = a.splits * a.top;
    uint64_t bound = 1;
    if (a.splits >= a.top) {
      const uint64_t first[1] = {lane < a.splits ? keys[lane * a.top] : 0};
      if (__popcll(__ballot(first[0] != 0)) >= a.top) bound = bound_of<1>(first, a.top);
    }
    if ((int)threadIdx.x < kLogprobMaxTop) sh.top.best[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.top.n = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t k = keys[i];
      if (k >= bound) sh.top.cand[atomicAdd(&sh.top.n, 1)] = k;
    }
    __syncthreads();
    rank_candidates(sh.top, a.top);
    top = &sh.top;
  }
  t = group_join(t, sh.part);
  write_row<TYPE>(a, row, t, top);
}

template <int TYPE, bool TOP>
hipError_t go(const LogprobArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.R, (unsigned)a.splits);
  if (logprob_narrow(a.R, a.V)) {
    hipLaunchKernelGGL((logprob_kernel<TYPE, TOP, kNarrow>), grid, dim3(kThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL((logprob_kernel<TYPE, TOP, kWide>), grid, dim3(kThreads), 0, s, a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((join_kernel<TYPE, TOP>), dim3((unsigned)a.R), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s) {
  if (a.type == 0) return a.top ? go<0, true>(a, s) : go<0, false>(a, s);
  if (a.type == 1) return a.top ? go<1, true>(a, s) : go<1, false>(a, s);
  return a.top ? go<2, true>(a, s) : go<2, false>(a, s);
}

}  // namespace wush
