// Internal interface of the 4-bit key/value cache (wush_kv4.hip) and of the
// attention over it (wush_kv4_attention.h) for their C-ABI layer
// (wush_serving_abi.cpp).  Not part of the public ABI.
#ifndef WUSH_KV4_H_
#define WUSH_KV4_H_

#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace wush {

struct KvAppendSide {
  const uint16_t* X;  // bf16 [n][heads][D], row stride ld
  int64_t ld;         // elements, a multiple of 8
  const uint16_t* T;  // bf16 [heads][D/G][G][G] or null
  uint8_t* codes;     // [pages][heads][page][D/2]
  uint8_t* scales;    // [pages][heads][page][D/G]
  const float* gs;    // NVFP4 only
};

struct KvAppendArgs {
  int fmt;
  KvAppendSide side[2];  // keys, values
  const int64_t* slots;  // [n]: page * page size + place; outside the cache: not written
  int64_t n, pages;
  int heads, D, page_log2;
};

hipError_t launch_kv4_append(const KvAppendArgs& a, hipStream_t s);

// Attention.  A work item is one key head's queries of one sequence, as many
// columns (query, head of the group) as a workgroup holds; a unit is
// kKvUnit tokens of an item.
constexpr int kKvUnit = 128;

// Workspace: the number of items that may be in several pieces (in the first one's `pieces`),
// one of these for each, then the pieces.
struct KvJoin {
  int32_t pieces;             // of the item; 0: it is whole after all
  int32_t first, next, step;  // their places: first, next, next + step, ...
  int32_t cols, col0;         // columns, and the first one's place in the sequence
  int32_t start, head;        // row of the sequence's first query, key head
};

struct KvAttnArgs {
  int fmt;
  const uint16_t* q;  // bf16 [n][kv * group][D], row stride ldq
  int64_t ldq;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const float *k_gs, *v_gs;  // NVFP4 only
  const int32_t* table;      // [B][width], row stride ldt
  int64_t ldt;
  const int32_t* lengths;    // [B]
  const int32_t* q_start;    // [B + 1], or null: query b is sequence b's
  const uint16_t* T;         // bf16 [kv][D/G][G][G] or null
  uint16_t* out;             // bf16 [n][kv * group][D]
  KvJoin* join;              // [1 + items]
  float* part;               // [2 runs] pieces
  int B, n, kv, group, D, page_log2, width, pages;
  int window;                // 0: none
  float scale;               // of the scores, times log2 e
  int items, workgroups, runs;  // as in KvPlan
};

// How a call is cut: columns per workgroup, and the pieces that the device aims at.
enum { kKvNarrow, kKvWide, kKvPrompt };  // four waves share columns, the same with twice as many, waves have their own
// Tiles of 16 columns per wave: one where the results of two would not fit the registers.
constexpr int kv_tiles(int shape, int D) { return shape == kKvNarrow || D > 128 ? 1 : 2; }
constexpr int kv_columns(int shape, int D) { return 16 * kv_tiles(shape, D) * (shape == kKvPrompt ? 4 : 1); }
// Workgroups that the chip holds at a time, by the kernels' registers (INT4's scales take some).
constexpr int kv_resident(int shape, int D, int fmt) {
  return shape != kKvNarrow || D > 128 ? 512 : D == 128 ? (fmt == 2 ? 512 : 768) : fmt == 2 ? 768 : 1024;
}

// Workgroups per CU that the registers are cut for: as many as the units are shared out over, and
// for two tiles of narrow heads a third one, since items' last pieces come on top of them
// (16 sequences of up to 4000 tokens, 16 heads of 64, 20 columns: 24.8 us and 28.9).
constexpr int kv_per_cu(int shape, int D, int fmt) {
  return shape == kKvWide && D == 64 && fmt != 2 ? 3 : kv_resident(shape, D, fmt) / 256;
}

struct KvPlan {
  int shape;
  int runs;  // shares that the units are divided into; 0: every item is taken whole, without a workspace
  int64_t items, workgroups;  // at most
};

// Up to here an item is not worth cutting: tables of 512 tokens, 8 heads, us whole and cut: 1 sequence
// 8.3, 10.2; 8 8.4, 10.1; 128 20.8, 24.2.  Of 768: 9.6, 11.4; 9.8, 11.5; 29.0, 31.5.  Of 1024: 10.9,
// 9.9; 11.3, 10.4; 34.7, 39.3.  The host knows the table's width alone: a sequence of 500 tokens
// takes 8.2 in a table of 512 and 10.1 in one of 131072, with the shares and a join of nothing.
constexpr int64_t kKvWholeTokens = 512;

inline KvPlan kv_plan(int fmt, int64_t B, int64_t n, int64_t kv, int64_t group, int D, int64_t tokens) {
  KvPlan p;
  const int64_t columns = B > 0 ? n * group / B : 0;  // of a sequence, on average
  p.shape = columns <= 16 ? kKvNarrow : columns <= (D > 128 ? 32 : 64) ? (D > 128 ? kKvNarrow : kKvWide) : kKvPrompt;
  // Each sequence ends in a part of an item; sequences without queries have none.
  const int64_t seqs = B < n ? B : n;
  p.items = (n * group / kv_columns(p.shape, D) + seqs) * kv;
  const int64_t units = p.items * ((tokens + kKvUnit - 1) / kKvUnit + 1);
  const int64_t resident = kv_resident(p.shape, D, fmt);
  p.runs = (int)(tokens <= kKvWholeTokens ? 0 : units < resident ? units : resident);
  // Pieces of ceil(all units / runs) are at most runs and one more per item.
  p.workgroups = p.items + p.runs;
  return p;
}

constexpr int kKvJoins = 1024;  // items whose pieces are joined side by side, and
constexpr int kKvFill = 2048;   // workgroups that do it, where their columns allow

// Floats of one piece of an item: maxima, sums, results.
inline int64_t kv_piece(int shape, int D) { return (int64_t)kv_columns(shape, D) * (D + 2); }
// Bytes of the workspace in front of the pieces.
inline int64_t kv_join_bytes(const KvPlan& p) { return (1 + p.items) * (int64_t)sizeof(KvJoin); }
// Cut into pieces of a share, an item has less than 2 units / share of them, so all items together
// less than 2 runs; cut by runs, every run has at most two pieces of items that are not whole.
inline int64_t kv_workspace(const KvPlan& p, int D) {
  return p.runs ? kv_join_bytes(p) + 2 * (int64_t)p.runs * 4 * kv_piece(p.shape, D) : 0;
}

hipError_t launch_kv4_attention_mx(const KvAttnArgs& a, int shape, hipStream_t s);
hipError_t launch_kv4_attention_nv(const KvAttnArgs& a, int shape, hipStream_t s);
hipError_t launch_kv4_attention_int(const KvAttnArgs& a, int shape, hipStream_t s);

}  // namespace wush

#endif  // WUSH_KV4_H_
