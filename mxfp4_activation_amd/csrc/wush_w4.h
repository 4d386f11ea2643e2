// Internal interface of the few-token kernels on 4-bit weights (wush_w4.hip,
// wush_moe.hip) and of the token log probabilities (wush_logprobs.hip) for
// their C-ABI layer (wush_decode_abi.cpp).  Not part of the public ABI.
#ifndef WUSH_W4_H_
#define WUSH_W4_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace wush {

// Activations as bf16 planes: plane t of row m starts at X + t * plane + m * ldx,
// and the operand is the sum of its planes (1, 2 or 3 of them).
struct Planes {
  const uint16_t* X;
  int64_t ldx;    // elements, a multiple of 8
  int64_t plane;  // elements
  int terms;
};

struct SplitArgs {
  const uint16_t* X;  // bf16 [M], row stride ldx
  int64_t ldx;
  const uint16_t* T;  // bf16 [K/G][G][G]
  uint16_t* out;      // [terms][M][K]
  int64_t M, K;
  int G, terms;
};

// Low-rank adapters of a batch: Y[m] += h[m] B[ids[m]]^T, h from launch_lora.  The product
// takes what it adds from delta, which launch_lora_expand writes, or for a few tokens
// forms it itself, which saves a launch.
// One lane then reads a result's whole row of B, which is slower than a launch of its own made
// for that where the rows are long or many.  N x rank, tokens: together, apart, us (MXFP4, K =
// 4096, 40 adapters): 4096 x 16, 16: 12.8, 16.2; 24576 x 16, 32: 29.2, 34.2; 24576 x 16, 64: 49.5,
// 50.0; 4096 x 32, 64: 18.3, 20.4; 24576 x 32, 16: 26.6, 27.7, and 32: 39.7, 37.8; 24576 x 64,
// 8: 25.2, 26.0, and 16: 38.1, 34.4; 4096 x 64, 64: 24.6, 22.7; 4096 x 128, 1: 10.4, 11.6;
// 4096 x 256, 1: 13.1, 12.4.  INT4 alike.
inline bool lora_together(int64_t M, int64_t N, int64_t rank) {
  return M <= 64 && rank <= (M <= 8 ? 128 : 32) && N * rank <= (3 << 22) / M;
}
constexpr int64_t kLoraChunk = 256;  // tokens that share a workspace
struct LoraArgs {
  const uint16_t* X;   // bf16 [M], row stride ldx
  int64_t ldx;
  const uint16_t* A;   // bf16 [E][rank][K]
  const uint16_t* B;   // bf16 [E][N][rank]
  const float* scale;  // [E] or null
  const int32_t* ids;  // [M]: negative, none; E or more, NaN
  float* h;            // [M][rank]: scale[ids[m]] A[ids[m]] x[m]
  float* delta;        // [M][N] or null
  int64_t M, K, E;
  int rank;            // a multiple of 8
};

struct LinearArgs {
  int fmt;
  Planes x;
  const uint8_t* codes;   // [N][K/2]
  const uint8_t* scales;  // [N][K/G]
  const float* gs;        // NVFP4 only
  void* Y;                // [M][N] fp32 or bf16
  int64_t M, N, K;
  bool bf16_out;
  LoraArgs lora;  // none if ids is null
};

// Mixture of experts over at most kMoeTokens tokens at a time.
constexpr int kMoeTokens = 64;
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int kRouterParts = 4;  // workgroups that share a row of the router

// Tokens of one expert that share a pass over its weights.
struct MoeTile {
  int expert, count;
  int16_t token[32], slot[32];  // slot: token * topk + place among its experts
};

struct MoeArgs {
  int fmt;
  const uint16_t* X;        // bf16 [M], row stride ldx
  int64_t ldx;
  const uint16_t* router;   // bf16 [E][H]
  const uint8_t* gu_codes;  // [E][2 I][H/2]: I gate rows, then I up rows
  const uint8_t* gu_scales;
  const float* gu_gs;       // [E], NVFP4 only
  const uint8_t* dn_codes;  // [E][H][I/2]
  const uint8_t* dn_scales;
  const float* dn_gs;
  const uint16_t* T_in;     // bf16 [H/G][G][G] or null
  const uint16_t* T_mid;    // bf16 [E][I/G][G][G] or null
  int M, E, topk;           // M <= kMoeTokens
  int64_t H, I;
  int renorm, terms;        // terms: planes of T_in X and of h
  bool bf16_out;
  void* Y;                  // [M][H]
  int32_t* ids;             // [M][topk]
  float* weights;           // [M][topk]
  // Workspace.
  uint16_t* xt;             // [terms][M][H], if T_in
  float* logits;            // [kRouterParts][M][E], to be summed
  uint16_t* h;              // [terms][M * topk][I]
  float* part;              // [M * topk][H]
  int32_t* n_tiles;
  MoeTile* tiles;           // [M * topk]
};

hipError_t launch_moe(const MoeArgs& a, hipStream_t s);

hipError_t launch_split(const SplitArgs& a, hipStream_t s);
hipError_t launch_linear_w4(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_w4_lora(const LinearArgs& a, hipStream_t s);  // where a.lora.ids is not null
// h of the adapters and, where t is not null, also what launch_split does.
hipError_t launch_lora(const LoraArgs& a, const SplitArgs* t, hipStream_t s);
hipError_t launch_lora_expand(const LoraArgs& a, int64_t N, hipStream_t s);

// Log probabilities, entropy and largest entries of rows of logits.
constexpr int kLogprobMaxTop = 32;

struct LogprobArgs {
  const void* L;           // [R][V], row stride ld elements
  int type;                // 0 fp32, 1 bf16, 2 fp16
  int64_t ld, R, V;
  const int64_t* targets;  // [R]
  int top;                 // 0 .. kLogprobMaxTop
  float* logprob;          // [R]
  float* entropy;          // [R]
  int32_t* top_ids;        // [R][top]
  float* top_logprobs;     // [R][top]
  int splits;              // workgroups per row
  int split_batches;       // batches of each but the last
  float* part;             // [R][splits][4], if splits > 1: max, sum, weighted sum
  uint64_t* keys;          // [R][splits][top], if splits > 1
};

// Elements per thread and batch: 32 where there are rows or batches enough to
// fill the chip, otherwise 8.
constexpr int kLogprobThreads = 256, kLogprobWide = 32, kLogprobNarrow = 8;
constexpr int kLogprobMaxSplits = 64;
// Workgroups that a launch should have.
constexpr int64_t kLogprobGroups = 1024;
inline bool logprob_narrow(int64_t R, int64_t V) {
  return R * ((V + kLogprobThreads * kLogprobWide - 1) / (kLogprobThreads * kLogprobWide)) < kLogprobGroups / 2;
}

// Workgroups per row (1: no workspace), and batches of each.
struct LogprobPlan {
  int splits, split_batches;
};
inline LogprobPlan logprob_plan(int64_t R, int64_t V) {
  const int64_t per = kLogprobThreads * (logprob_narrow(R, V) ? kLogprobNarrow : kLogprobWide);
  const int64_t batches = (V + per - 1) / per;
  int64_t s = kLogprobGroups / (R > 0 ? R : 1);
  if (s > batches) s = batches;
  if (s > kLogprobMaxSplits) s = kLogprobMaxSplits;
  if (s < 1) s = 1;
  // Whole batches per split; the last split also has the batch that an
  // unaligned row start may add.
  const int64_t each = (batches + s - 1) / s;
  return LogprobPlan{(int)((batches + each - 1) / each), (int)each};
}
hipError_t launch_logprobs(const LogprobArgs& a, hipStream_t s);

}  // namespace wush

#endif  // WUSH_W4_H_
