// C-ABI layer of the decode entries around the 4-bit products: the cache of
// keys and values, attention over it, linear layers with low-rank adapters, and
// adjustments of logits.  Contract: include/wush.h.

#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/wush.h"
#include "wush_adjust.h"
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
constexpr int64_t kMaxLoraRows = 65535 * 16;
constexpr int64_t kMaxRank = 512;
constexpr int64_t kMaxAdjustRows = 65535;
constexpr int64_t kMaxOutputs = ((int64_t)1 << 30) - 1;  // a token's count in the kernel has 30 bits

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

struct LoraWorkspace {
  uint64_t h, delta, planes, total;
};

LoraWorkspace lora_workspace(int64_t M, int64_t N, int64_t K, int64_t rank, bool transform, int out_type) {
  const uint64_t c = (uint64_t)(M < wush::kLoraChunk ? M : wush::kLoraChunk);
  LoraWorkspace w;
  w.h = 0;
  w.delta = round16(c * rank * 4);
  w.planes = w.delta + (wush::lora_together(M, N, rank) ? 0 : round16(c * N * 4));
  w.total = w.planes + (transform ? 2 * terms_of(out_type) * c * K : 0);
  return w;
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

int64_t wush_kv4_attention_workspace(int fmt, int64_t B, int64_t n, int64_t q_heads, int64_t heads, int64_t D, int64_t page,
                                     int64_t width) {
  if (fmt < wush::kMXFP4 || fmt > wush::kINT4) return 0;
  if (B <= 0 || n <= 0 || heads <= 0 || q_heads <= 0 || q_heads % heads != 0 || page <= 0 || width <= 0) return 0;
  if (D != 64 && D != 128 && D != 256) return 0;
  if (B > kMaxTokens || n > kMaxTokens || heads > kMaxHeads || q_heads > kMaxHeads || width > kMaxTokens / page) return 0;
  const wush::KvPlan p = wush::kv_plan(fmt, B, n, heads, q_heads / heads, (int)D, page * width);
  return wush::kv_workspace(p, (int)D);
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
  // (The kernels take powers of two.)
  const float scale2 = (float)(scale * 1.4426950408889634);
  if (!(scale > 0.0f) || !(scale2 < INFINITY)) return fail(WUSH_EINVAL, "scale must be positive and finite");
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
  const wush::KvPlan plan = wush::kv_plan(fmt, B, n, heads, q_heads / heads, (int)D, page * width);
  // Items and units are counted in 32 bits.
  if (plan.items > INT32_MAX / 2 / (page * width / wush::kKvUnit + 2))
    return fail(WUSH_EINVAL, "too many tokens for one launch");
  const int64_t need = wush_kv4_attention_workspace(fmt, B, n, q_heads, heads, D, page, width);
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
  a.join = static_cast<wush::KvJoin*>(workspace);
  a.part = plan.runs ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + wush::kv_join_bytes(plan)) : nullptr;
  a.B = (int)B;
  a.n = (int)n;
  a.kv = (int)heads;
  a.group = (int)(q_heads / heads);
  a.D = (int)D;
  a.page_log2 = log2_of(page);
  a.width = (int)width;
  a.pages = (int)pages;
  a.window = (int)window;
  a.scale = scale2;
  a.workgroups = (int)plan.workgroups;
  a.runs = plan.runs;
  a.items = (int)plan.items;
  if (fmt == wush::kMXFP4) return launched(wush::launch_kv4_attention_mx(a, plan.shape, stream));
  if (fmt == wush::kNVFP4) return launched(wush::launch_kv4_attention_nv(a, plan.shape, stream));
  return launched(wush::launch_kv4_attention_int(a, plan.shape, stream));
}

int64_t wush_linear_w4_lora_workspace(int64_t M, int64_t N, int64_t K, int64_t rank, int transform, int out_type) {
  if (M <= 0 || N <= 0 || N > kMaxDim || K <= 0 || K > kMaxK || M > kMaxLoraRows || rank <= 0 || rank > kMaxRank) return 0;
  if (out_type != WUSH_OUT_F32 && out_type != WUSH_OUT_BF16) return 0;
  return (int64_t)lora_workspace(M, N, K, rank, transform != 0, out_type).total;
}

wush_status wush_linear_w4_lora(int fmt, const void* X, int64_t ldx, const void* T, const void* codes,
                                const void* scales, const float* global_scale, const void* A, const void* B,
                                const float* adapter_scale, const int32_t* ids, int64_t adapters, int64_t rank,
                                int64_t M, int64_t N, int64_t K, void* Y, int out_type, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = 0;
  wush_status st = check_fmt(fmt, out_type);
  if (st != WUSH_OK) return st;
  if (M < 0 || N < 0) return fail(WUSH_EINVAL, "M and N must be >= 0");
  st = check_width("K", K, fmt);
  if (st != WUSH_OK) return st;
  if (rank < 8 || rank > kMaxRank || rank % 8 != 0)
    return fail(WUSH_EINVAL, "rank must be a multiple of 8, 8 .. %lld (got %lld)", (long long)kMaxRank, (long long)rank);
  if (adapters < 0 || adapters > INT32_MAX) return fail(WUSH_EINVAL, "adapters out of range (got %lld)", (long long)adapters);
  if (M == 0 || N == 0) return WUSH_OK;
  if (N > kMaxDim) return fail(WUSH_EINVAL, "N too large");
  if (M > kMaxLoraRows) return fail(WUSH_EINVAL, "M too large for one launch");
  if (adapters > 0 && (adapters > INT64_MAX / 4 / rank / K || adapters > INT64_MAX / 4 / rank / N))
    return fail(WUSH_EINVAL, "adapters too large");
  st = check_rows(X, ldx, M, K);
  if (st != WUSH_OK) return st;
  st = check_weights("weight", fmt, codes, scales, global_scale);
  if (st != WUSH_OK) return st;
  if (T && !aligned(T, 16)) return fail(WUSH_EALIGN, "T must be 16-byte aligned");
  if (!Y || !ids || (adapters > 0 && (!A || !B))) return fail(WUSH_EINVAL, "null Y, ids, A or B");
  if (!aligned(Y, (uintptr_t)out_bytes_of(out_type))) return fail(WUSH_EALIGN, "Y must be aligned to its elements");
  if (!aligned(A, 16) || !aligned(B, 16)) return fail(WUSH_EALIGN, "A and B must be 16-byte aligned");
  if (!aligned(ids, 4) || !aligned(adapter_scale, 4)) return fail(WUSH_EALIGN, "ids and adapter_scale must be 4-byte aligned");
  const LoraWorkspace w = lora_workspace(M, N, K, rank, T != nullptr, out_type);
  const int64_t need = (int64_t)w.total;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != WUSH_OK) return st;
  const Range ins[] = {{X, ((uint64_t)(M - 1) * (M > 1 ? ldx : 0) + K) * 2},
                       {T, (uint64_t)K * group_of(fmt) * 2},
                       {codes, code_bytes(N, K)},
                       {scales, scale_bytes(fmt, N, K)},
                       {fmt == wush::kNVFP4 ? global_scale : nullptr, 4},
                       {A, (uint64_t)adapters * rank * K * 2},
                       {B, (uint64_t)adapters * rank * N * 2},
                       {adapter_scale, (uint64_t)adapters * 4},
                       {ids, (uint64_t)M * 4}};
  const Range outs[] = {{Y, (uint64_t)M * N * out_bytes_of(out_type)}, {workspace, (uint64_t)need}};
  if (any_overlap(outs, 2, ins, 9)) return fail(WUSH_EINVAL, "Y and the workspace must not overlap each other or an input");
  st = check_device();
  if (st != WUSH_OK) return st;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  wush::LinearArgs a{};
  a.fmt = fmt;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.gs = global_scale;
  a.N = N;
  a.K = K;
  a.bf16_out = out_type == WUSH_OUT_BF16;
  a.lora.ldx = M > 1 ? ldx : 0;
  a.lora.A = static_cast<const uint16_t*>(A);
  a.lora.B = static_cast<const uint16_t*>(B);
  a.lora.scale = adapter_scale;
  a.lora.h = reinterpret_cast<float*>(ws + w.h);
  a.lora.delta = wush::lora_together(M, N, rank) ? nullptr : reinterpret_cast<float*>(ws + w.delta);
  a.lora.K = K;
  a.lora.E = adapters;
  a.lora.rank = (int)rank;
  for (int64_t m0 = 0; m0 < M; m0 += wush::kLoraChunk) {
    const int64_t m = M - m0 < wush::kLoraChunk ? M - m0 : wush::kLoraChunk;
    a.M = a.lora.M = m;
    a.Y = static_cast<uint8_t*>(Y) + m0 * N * out_bytes_of(out_type);
    a.lora.X = static_cast<const uint16_t*>(X) + m0 * a.lora.ldx;
    a.lora.ids = ids + m0;
    a.x.X = a.lora.X;
    a.x.ldx = a.lora.ldx;
    a.x.plane = 0;
    a.x.terms = 1;
    wush::SplitArgs t{};
    if (T) {
      t.X = a.lora.X;
      t.ldx = a.lora.ldx;
      t.T = static_cast<const uint16_t*>(T);
      t.out = reinterpret_cast<uint16_t*>(ws + w.planes);
      t.M = m;
      t.K = K;
      t.G = group_of(fmt);
      t.terms = terms_of(out_type);
      a.x.X = t.out;
      a.x.ldx = K;
      a.x.plane = m * K;
      a.x.terms = t.terms;
    }
    st = launched(wush::launch_lora(a.lora, T ? &t : nullptr, stream));
    if (st == WUSH_OK && a.lora.delta) st = launched(wush::launch_lora_expand(a.lora, N, stream));
    if (st == WUSH_OK) st = launched(wush::launch_linear_w4(a, stream));
    if (st != WUSH_OK) return st;
  }
  return WUSH_OK;
}

wush_status wush_adjust_logits(const void* logits, int logit_type, int64_t ld, int64_t R, int64_t V,
                               const int32_t* prompt, int64_t n_prompt, const int32_t* output, int64_t n_output,
                               const float* repetition, const float* frequency, const float* presence,
                               const int32_t* bias_ids, const float* bias, int64_t n_bias, const int32_t* allowed,
                               void* out, int64_t ld_out, hipStream_t stream) {
  g_last_error[0] = 0;
  if (logit_type < WUSH_LOGITS_F32 || logit_type > WUSH_LOGITS_F16)
    return fail(WUSH_EINVAL, "unknown logit_type %d", logit_type);
  if (R < 0) return fail(WUSH_EINVAL, "R must be >= 0 (got %lld)", (long long)R);
  if (V < 1 || V > INT32_MAX) return fail(WUSH_EINVAL, "V must be 1 .. 2^31 - 1 (got %lld)", (long long)V);
  if (n_prompt < 0 || n_output < 0 || n_bias < 0 || n_prompt > INT32_MAX || n_output > INT32_MAX || n_bias > INT32_MAX)
    return fail(WUSH_EINVAL, "the lists' lengths must be 0 .. 2^31 - 1");
  if (n_output > kMaxOutputs) return fail(WUSH_EINVAL, "n_output must be less than 2^30 (got %lld)", (long long)n_output);
  if (R == 0) return WUSH_OK;
  if (R > kMaxAdjustRows) return fail(WUSH_EINVAL, "R too large for one launch");
  if (R > 1 && (ld < V || ld > ((int64_t)1 << 36) || ld_out < V || ld_out > ((int64_t)1 << 36)))
    return fail(WUSH_EINVAL, "ld and ld_out must be V or more (got %lld, %lld)", (long long)ld, (long long)ld_out);
  if (!logits || !out) return fail(WUSH_EINVAL, "null logits or out");
  if ((n_prompt > 0 && !prompt) || (n_output > 0 && !output) || (n_bias > 0 && (!bias_ids || !bias)))
    return fail(WUSH_EINVAL, "null list");
  const int eb = logit_type == WUSH_LOGITS_F32 ? 4 : 2;
  if (!aligned(logits, (uintptr_t)eb) || !aligned(out, (uintptr_t)eb))
    return fail(WUSH_EALIGN, "logits and out must be aligned to their elements");
  if (!aligned(prompt, 4) || !aligned(output, 4) || !aligned(repetition, 4) || !aligned(frequency, 4) ||
      !aligned(presence, 4) || !aligned(bias_ids, 4) || !aligned(bias, 4) || !aligned(allowed, 4))
    return fail(WUSH_EALIGN, "lists, penalties and masks must be 4-byte aligned");
  const bool in_place = out == logits && (R == 1 || ld_out == ld);
  const Range ins[] = {{in_place ? nullptr : logits, ((uint64_t)(R - 1) * (R > 1 ? ld : 0) + V) * eb},
                       {prompt, (uint64_t)R * n_prompt * 4},
                       {output, (uint64_t)R * n_output * 4},
                       {repetition, (uint64_t)R * 4},
                       {frequency, (uint64_t)R * 4},
                       {presence, (uint64_t)R * 4},
                       {bias_ids, (uint64_t)R * n_bias * 4},
                       {bias, (uint64_t)R * n_bias * 4},
                       {allowed, (uint64_t)R * ((V + 31) / 32) * 4}};
  const Range outs[] = {{out, ((uint64_t)(R - 1) * (R > 1 ? ld_out : 0) + V) * eb}};
  if (any_overlap(outs, 1, ins, 9)) return fail(WUSH_EINVAL, "out must be logits itself or not overlap an input");
  wush_status st = check_device();
  if (st != WUSH_OK) return st;

  wush::AdjustArgs a{};
  a.in = logits;
  a.out = out;
  a.type = logit_type;
  a.ld_in = R > 1 ? ld : 0;
  a.ld_out = R > 1 ? ld_out : 0;
  a.R = R;
  a.V = V;
  a.prompt = prompt;
  a.output = output;
  a.n_prompt = n_prompt;
  a.n_output = n_output;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_ids = bias_ids;
  a.bias = bias;
  a.n_bias = n_bias;
  a.allowed = allowed;
  return launched(wush::launch_adjust(a, stream));
}

}  // extern "C"
