// C-ABI layer of the decode entries around the 4-bit products: the cache of
// keys and values, attention over it.  Contract: include/wush.h.

#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/wush.h"
#include "wush_decode_checks.h"
#include "wush_kernels.h"
#include "wush_kv4.h"
#include "wush_w4.h"

namespace {

using wush::aligned;
using wush::check_device;
using wush::fail;
using wush::g_last_error;
using namespace wush::decode;

constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;

int log2_of(int64_t v) {
  int n = 0;
  while (((int64_t)1 << n) < v) ++n;
  return n;
}

wush_status check_cache(int fmt, int64_t heads, int64_t D, int64_t page, int64_t pages, const void* k_codes,
                        const void* k_scales, const float* k_global, const void* v_codes, const void* v_scales,
                        const float* v_global) {
  wush_status st = check_fmt(fmt, WUSH_OUT_BF16);
  if (st != WUSH_OK) return st;
  if (D != 64 && D != 128 && D != 256) return fail(WUSH_EUNSUPPORTED, "D must be 64, 128 or 256 (got %lld)", (long long)D);
  if (heads < 1 || heads > kMaxHeads) return fail(WUSH_EINVAL, "heads must be 1 .. %lld (got %lld)", (long long)kMaxHeads, (long long)heads);
  if (page < 16 || page > 65536 || (page & (page - 1)) != 0)
    return fail(WUSH_EINVAL, "page must be a power of two, 16 .. 65536 (got %lld)", (long long)page);
  if (pages < 0 || pages > INT32_MAX || pages > INT64_MAX / 256 / (page * heads))
    return fail(WUSH_EINVAL, "pages out of range (got %lld)", (long long)pages);
  if (pages == 0) return WUSH_OK;
  st = check_weights("key", fmt, k_codes, k_scales, k_global);
  if (st != WUSH_OK) return st;
  st = check_weights("value", fmt, v_codes, v_scales, v_global);
  if (st != WUSH_OK) return st;
  if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_scales, 16) || !aligned(v_scales, 16))
    return fail(WUSH_EALIGN, "the cache's codes and scales must be 16-byte aligned");
  return WUSH_OK;
}

}  // namespace

extern "C" {

wush_status wush_kv4_append(int fmt, const void* K, int64_t ldk, const void* V, int64_t ldv, const void* T_k,
                            const void* T_v, const int64_t* slots, int64_t n, int64_t heads, int64_t D, int64_t page,
                            int64_t pages, void* k_codes, void* k_scales, const float* k_global, void* v_codes,
                            void* v_scales, const float* v_global, hipStream_t stream) {
  g_last_error[0] = 0;
  wush_status st = check_cache(fmt, heads, D, page, pages, k_codes, k_scales, k_global, v_codes, v_scales, v_global);
  if (st != WUSH_OK) return st;
  if (n < 0) return fail(WUSH_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
  if (n == 0 || pages == 0) return WUSH_OK;
  if (n > kMaxTokens) return fail(WUSH_EINVAL, "n too large");
  st = check_rows(K, ldk, n, heads * D);
  if (st != WUSH_OK) return st;
  st = check_rows(V, ldv, n, heads * D);
  if (st != WUSH_OK) return st;
  if ((T_k && !aligned(T_k, 16)) || (T_v && !aligned(T_v, 16)))
    return fail(WUSH_EALIGN, "T_k and T_v must be 16-byte aligned");
  if (!slots) return fail(WUSH_EINVAL, "null slots");
  if (!aligned(slots, 8)) return fail(WUSH_EALIGN, "slots must be 8-byte aligned");
  const int64_t rows = pages * heads * page;
  const bool nv = fmt == wush::kNVFP4;
  const uint64_t bank = (uint64_t)heads * D * group_of(fmt) * 2;
  const Range ins[] = {{K, ((uint64_t)(n - 1) * (n > 1 ? ldk : 0) + heads * D) * 2},
                       {V, ((uint64_t)(n - 1) * (n > 1 ? ldv : 0) + heads * D) * 2},
                       {T_k, bank},
                       {T_v, bank},
                       {slots, (uint64_t)n * 8},
                       {nv ? k_global : nullptr, 4},
                       {nv ? v_global : nullptr, 4}};
  const Range outs[] = {{k_codes, code_bytes(rows, D)},
                        {k_scales, scale_bytes(fmt, rows, D)},
                        {v_codes, code_bytes(rows, D)},
                        {v_scales, scale_bytes(fmt, rows, D)}};
  if (any_overlap(outs, 4, ins, 7)) return fail(WUSH_EINVAL, "the cache's buffers must not overlap each other or an input");
  st = check_device();
  if (st != WUSH_OK) return st;

  wush::KvAppendArgs a{};
  a.fmt = fmt;
  a.side[0] = {static_cast<const uint16_t*>(K), n > 1 ? ldk : 0, static_cast<const uint16_t*>(T_k),
               static_cast<uint8_t*>(k_codes), static_cast<uint8_t*>(k_scales), k_global};
  a.side[1] = {static_cast<const uint16_t*>(V), n > 1 ? ldv : 0, static_cast<const uint16_t*>(T_v),
               static_cast<uint8_t*>(v_codes), static_cast<uint8_t*>(v_scales), v_global};
  a.slots = slots;
  a.n = n;
  a.pages = pages;
  a.heads = (int)heads;
  a.D = (int)D;
  a.page_log2 = log2_of(page);
  return launched(wush::launch_kv4_append(a, stream));
}

int64_t wush_kv4_attention_workspace(int64_t B, int64_t n, int64_t q_heads, int64_t heads, int64_t D, int64_t page,
                                     int64_t width) {
  if (B <= 0 || n <= 0 || heads <= 0 || q_heads <= 0 || q_heads % heads != 0 || page <= 0 || width <= 0) return 0;
  if (D != 64 && D != 128 && D != 256) return 0;
  if (B > kMaxTokens || n > kMaxTokens || heads > kMaxHeads || q_heads > kMaxHeads || width > kMaxTokens / page) return 0;
  const wush::KvPlan p = wush::kv_plan(B, n, heads, q_heads / heads, (int)D, page * width);
  return p.whole ? 0 : 4 * 2 * (int64_t)p.workgroups * wush::kv_piece(p.shape, (int)D);
}

wush_status wush_kv4_attention(int fmt, const void* Q, int64_t ldq, const void* T_q, const void* k_codes,
                               const void* k_scales, const float* k_global, const void* v_codes, const void* v_scales,
                               const float* v_global, const int32_t* block_table, int64_t ldt, int64_t width,
                               const int32_t* lengths, const int32_t* q_start, int64_t B, int64_t n, int64_t q_heads,
                               int64_t heads, int64_t D, int64_t page, int64_t pages, float scale, int64_t window,
                               void* out, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = 0;
  wush_status st = check_cache(fmt, heads, D, page, pages, k_codes, k_scales, k_global, v_codes, v_scales, v_global);
  if (st != WUSH_OK) return st;
  if (pages == 0) return fail(WUSH_EINVAL, "the cache has no pages");
  if (q_heads < heads || q_heads > kMaxHeads || q_heads % heads != 0)
    return fail(WUSH_EINVAL, "q_heads must be a multiple of heads, at most %lld (got %lld)", (long long)kMaxHeads, (long long)q_heads);
  if (B < 0 || n < 0) return fail(WUSH_EINVAL, "B and n must be >= 0");
  if (!q_start && B != n) return fail(WUSH_EINVAL, "without q_start every sequence has one query (B %lld, n %lld)", (long long)B, (long long)n);
  if (!(scale > 0.0f) || !(scale < INFINITY)) return fail(WUSH_EINVAL, "scale must be positive and finite");
  if (window < 0 || window > kMaxTokens) return fail(WUSH_EINVAL, "window must be 0 (none) .. 2^30 (got %lld)", (long long)window);
  if (width < 1 || width > kMaxTokens / page) return fail(WUSH_EINVAL, "width must be 1 .. 2^30 / page (got %lld)", (long long)width);
  if (B == 0 || n == 0) return WUSH_OK;
  if (B > kMaxTokens || n > kMaxTokens / q_heads) return fail(WUSH_EINVAL, "B or n too large for one launch");
  if (B > 1 && (ldt < width || ldt > kMaxTokens)) return fail(WUSH_EINVAL, "ldt must be width or more (got %lld)", (long long)ldt);
  st = check_rows(Q, ldq, n, q_heads * D);
  if (st != WUSH_OK) return st;
  if (T_q && !aligned(T_q, 16)) return fail(WUSH_EALIGN, "T_q must be 16-byte aligned");
  if (!block_table || !lengths || !out) return fail(WUSH_EINVAL, "null block_table, lengths or out");
  if (!aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(q_start, 4))
    return fail(WUSH_EALIGN, "block_table, lengths and q_start must be 4-byte aligned");
  if (!aligned(out, 16)) return fail(WUSH_EALIGN, "out must be 16-byte aligned");
  const wush::KvPlan plan = wush::kv_plan(B, n, heads, q_heads / heads, (int)D, page * width);
  // Items and units are counted in 32 bits.
  if (plan.items > INT32_MAX / ((plan.whole ? 1 : page * width / wush::kKvUnit) + 2))
    return fail(WUSH_EINVAL, "too many tokens for one launch");
  const int64_t need = wush_kv4_attention_workspace(B, n, q_heads, heads, D, page, width);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != WUSH_OK) return st;
  const int64_t rows = pages * heads * page;
  const bool nv = fmt == wush::kNVFP4;
  const Range ins[] = {{Q, ((uint64_t)(n - 1) * (n > 1 ? ldq : 0) + q_heads * D) * 2},
                       {T_q, (uint64_t)heads * D * group_of(fmt) * 2},
                       {k_codes, code_bytes(rows, D)},
                       {k_scales, scale_bytes(fmt, rows, D)},
                       {nv ? k_global : nullptr, 4},
                       {v_codes, code_bytes(rows, D)},
                       {v_scales, scale_bytes(fmt, rows, D)},
                       {nv ? v_global : nullptr, 4},
                       {block_table, ((uint64_t)(B - 1) * (B > 1 ? ldt : 0) + width) * 4},
                       {lengths, (uint64_t)B * 4},
                       {q_start, (uint64_t)(B + 1) * 4}};
  const Range outs[] = {{out, (uint64_t)n * q_heads * D * 2}, {workspace, (uint64_t)need}};
  if (any_overlap(outs, 2, ins, 11)) return fail(WUSH_EINVAL, "out and the workspace must not overlap each other or an input");
  st = check_device();
  if (st != WUSH_OK) return st;

  wush::KvAttnArgs a{};
  a.fmt = fmt;
  a.q = static_cast<const uint16_t*>(Q);
  a.ldq = n > 1 ? ldq : 0;
  a.k_codes = static_cast<const uint8_t*>(k_codes);
  a.k_scales = static_cast<const uint8_t*>(k_scales);
  a.v_codes = static_cast<const uint8_t*>(v_codes);
  a.v_scales = static_cast<const uint8_t*>(v_scales);
  a.k_gs = k_global;
  a.v_gs = v_global;
  a.table = block_table;
  a.ldt = B > 1 ? ldt : 0;
  a.lengths = lengths;
  a.q_start = q_start;
  a.T = static_cast<const uint16_t*>(T_q);
  a.out = static_cast<uint16_t*>(out);
  a.part = static_cast<float*>(workspace);
  a.B = (int)B;
  a.n = (int)n;
  a.kv = (int)heads;
  a.group = (int)(q_heads / heads);
  a.D = (int)D;
  a.page_log2 = log2_of(page);
  a.width = (int)width;
  a.pages = (int)pages;
  a.window = (int)window;
  a.scale = (float)(scale * 1.4426950408889634);  // the kernels take powers of two
  a.workgroups = plan.workgroups;
  a.whole = plan.whole;
  if (fmt == wush::kMXFP4) return launched(wush::launch_kv4_attention_mx(a, plan.shape, stream));
  if (fmt == wush::kNVFP4) return launched(wush::launch_kv4_attention_nv(a, plan.shape, stream));
  return launched(wush::launch_kv4_attention_int(a, plan.shape, stream));
}

}  // extern "C"
