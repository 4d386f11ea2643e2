// C-ABI layer of the few-token entries: linear layers and mixtures of experts
// on 4-bit weights, and token log probabilities.  Contract: include/wush.h.

#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/wush.h"
#include "wush_abi_common.h"
#include "wush_kernels.h"
#include "wush_w4.h"

namespace {

using wush::aligned;
using wush::check_device;
using wush::fail;
using wush::g_last_error;
using wush::overlap;

struct Range {
  const void* p;
  uint64_t n;
};

bool any_overlap(const Range* outs, int n_outs, const Range* ins, int n_ins) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return true;
    for (int j = i + 1; j < n_outs; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
  }
  return false;
}

int group_of(int fmt) { return fmt == wush::kNVFP4 ? 16 : 32; }
int scale_bytes_of(int fmt) { return fmt == wush::kINT4 ? 2 : 1; }
int out_bytes_of(int out_type) { return out_type == WUSH_OUT_F32 ? 4 : 2; }
// Planes of T x and of the experts' h (split_panel says why two do for bf16).
int terms_of(int out_type) { return out_type == WUSH_OUT_F32 ? 3 : 2; }

uint64_t round16(uint64_t n) { return (n + 15) / 16 * 16; }
uint64_t code_bytes(int64_t rows, int64_t K) { return (uint64_t)rows * K / 2; }
uint64_t scale_bytes(int fmt, int64_t rows, int64_t K) {
  return (uint64_t)rows * (K / group_of(fmt)) * scale_bytes_of(fmt);
}

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxK = (int64_t)1 << 27;
constexpr int64_t kMaxLogprobRows = (int64_t)1 << 24;

wush_status check_fmt(int fmt, int out_type) {
  if (fmt != wush::kMXFP4 && fmt != wush::kNVFP4 && fmt != wush::kINT4)
    return fail(WUSH_EUNSUPPORTED, "unknown format %d", fmt);
  if (out_type != WUSH_OUT_F32 && out_type != WUSH_OUT_BF16) return fail(WUSH_EINVAL, "unknown out_type %d", out_type);
  return WUSH_OK;
}

wush_status check_width(const char* name, int64_t K, int fmt) {
  if (K <= 0 || K > kMaxK || K % group_of(fmt) != 0)
    return fail(WUSH_EINVAL, "%s must be a positive multiple of %d, at most 2^27 (got %lld)", name, group_of(fmt),
                (long long)K);
  return WUSH_OK;
}

wush_status check_rows(const void* X, int64_t ldx, int64_t M, int64_t K) {
  if (!X) return fail(WUSH_EINVAL, "null X");
  if (M > 1 && (ldx < K || ldx > kMaxDim)) return fail(WUSH_EINVAL, "ldx must be K or more, at most 2^30 (got %lld)", (long long)ldx);
  if (!aligned(X, 16) || (M > 1 && ldx % 8 != 0))
    return fail(WUSH_EALIGN, "every row of X must be 16-byte aligned");
  return WUSH_OK;
}

wush_status check_weights(const char* name, int fmt, const void* codes, const void* scales, const float* gs) {
  if (!codes || !scales) return fail(WUSH_EINVAL, "null %s codes or scales", name);
  if (fmt == wush::kNVFP4 && !gs) return fail(WUSH_EINVAL, "NVFP4 needs %s's global_scale", name);
  if (!aligned(codes, 8)) return fail(WUSH_EALIGN, "%s codes must be 8-byte aligned", name);
  if (fmt == wush::kINT4 && !aligned(scales, 2)) return fail(WUSH_EALIGN, "%s scales must be 2-byte aligned", name);
  if (fmt == wush::kNVFP4 && !aligned(gs, 4)) return fail(WUSH_EALIGN, "%s global_scale must be 4-byte aligned", name);
  return WUSH_OK;
}

wush_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return WUSH_OK;
  if (!ws || have < need)
    return fail(WUSH_EINVAL, "workspace of %lld bytes needed (got %lld)", (long long)need, (long long)(ws ? have : 0));
  if (!aligned(ws, 16)) return fail(WUSH_EALIGN, "workspace must be 16-byte aligned");
  return WUSH_OK;
}

wush_status launched(hipError_t e) {
  return e == hipSuccess ? WUSH_OK : fail(WUSH_EHIP, "launch: %s", hipGetErrorString(e));
}

// Tokens of a mixture that share its five launches.
int64_t moe_chunk(int64_t M) { return M < wush::kMoeTokens ? M : wush::kMoeTokens; }

struct MoeWorkspace {
  uint64_t planes, h, part, logits, n_tiles, tiles, total;
};

MoeWorkspace moe_workspace(int64_t M, int64_t E, int topk, int64_t H, int64_t I, bool transform, int out_type) {
  const uint64_t c = (uint64_t)moe_chunk(M), terms = (uint64_t)terms_of(out_type), slots = c * topk;
  MoeWorkspace w;
  w.planes = 0;
  w.h = w.planes + (transform ? round16(terms * c * H * 2) : 0);
  w.part = w.h + round16(terms * slots * I * 2);
  w.logits = w.part + round16(slots * H * 4);
  w.n_tiles = w.logits + round16(wush::kRouterParts * c * E * 4);
  w.tiles = w.n_tiles + 16;
  // A tile holds at least one slot.
  w.total = w.tiles + slots * sizeof(wush::MoeTile);
  return w;
}

wush_status check_moe_shape(int64_t M, int64_t E, int topk, int64_t H, int64_t I) {
  if (M < 0) return fail(WUSH_EINVAL, "M must be >= 0 (got %lld)", (long long)M);
  if (E < 1 || E > wush::kMoeMaxExperts)
    return fail(WUSH_EINVAL, "E must be 1 .. %d (got %lld)", wush::kMoeMaxExperts, (long long)E);
  if (topk < 1 || topk > wush::kMoeMaxTopK || topk > E)
    return fail(WUSH_EINVAL, "topk must be 1 .. min(E, %d) (got %d)", wush::kMoeMaxTopK, topk);
  if (H > ((int64_t)1 << 24) || I > ((int64_t)1 << 24)) return fail(WUSH_EINVAL, "H and I must be at most 2^24");
  return WUSH_OK;
}

}  // namespace

extern "C" {

int64_t wush_linear_w4_workspace(int64_t M, int64_t K, int out_type) {
  if (M <= 0 || K <= 0 || K > kMaxK || M > INT64_MAX / 8 / K) return 0;
  return (int64_t)(2u * (uint64_t)terms_of(out_type) * (uint64_t)M * (uint64_t)K);
}

wush_status wush_linear_w4(int fmt, const void* X, int64_t ldx, const void* T, const void* codes, const void* scales,
                           const float* global_scale, int64_t M, int64_t N, int64_t K, void* Y, int out_type,
                           void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = 0;
  wush_status st = check_fmt(fmt, out_type);
  if (st != WUSH_OK) return st;
  if (M < 0 || N < 0) return fail(WUSH_EINVAL, "M and N must be >= 0");
  st = check_width("K", K, fmt);
  if (st != WUSH_OK) return st;
  if (M == 0 || N == 0) return WUSH_OK;
  if (N > kMaxDim) return fail(WUSH_EINVAL, "N too large");
  if (M > 65535 * 16) return fail(WUSH_EINVAL, "M too large for one launch");
  st = check_rows(X, ldx, M, K);
  if (st != WUSH_OK) return st;
  st = check_weights("weight", fmt, codes, scales, global_scale);
  if (st != WUSH_OK) return st;
  if (T && !aligned(T, 16)) return fail(WUSH_EALIGN, "T must be 16-byte aligned");
  if (!Y) return fail(WUSH_EINVAL, "null Y");
  if (!aligned(Y, (uintptr_t)out_bytes_of(out_type))) return fail(WUSH_EALIGN, "Y must be aligned to its elements");
  const int64_t need = T ? wush_linear_w4_workspace(M, K, out_type) : 0;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != WUSH_OK) return st;
  const Range ins[] = {{X, ((uint64_t)(M - 1) * (M > 1 ? ldx : 0) + K) * 2},
                       {T, (uint64_t)K * group_of(fmt) * 2},
                       {codes, code_bytes(N, K)},
                       {scales, scale_bytes(fmt, N, K)},
                       {fmt == wush::kNVFP4 ? global_scale : nullptr, 4}};
  const Range outs[] = {{Y, (uint64_t)M * N * out_bytes_of(out_type)}, {workspace, (uint64_t)need}};
  if (any_overlap(outs, 2, ins, 5)) return fail(WUSH_EINVAL, "Y and the workspace must not overlap each other or an input");
  st = check_device();
  if (st != WUSH_OK) return st;

  wush::LinearArgs a{};
  a.fmt = fmt;
  a.x.X = static_cast<const uint16_t*>(X);
  a.x.ldx = M > 1 ? ldx : 0;
  a.x.terms = 1;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.gs = global_scale;
  a.Y = Y;
  a.M = M;
  a.N = N;
  a.K = K;
  a.bf16_out = out_type == WUSH_OUT_BF16;
  if (T) {
    wush::SplitArgs t{};
    t.X = a.x.X;
    t.ldx = a.x.ldx;
    t.T = static_cast<const uint16_t*>(T);
    t.out = static_cast<uint16_t*>(workspace);
    t.M = M;
    t.K = K;
    t.G = group_of(fmt);
    t.terms = terms_of(out_type);
    st = launched(wush::launch_split(t, stream));
    if (st != WUSH_OK) return st;
    a.x.X = t.out;
    a.x.ldx = K;
    a.x.plane = M * K;
    a.x.terms = t.terms;
  }
  return launched(wush::launch_linear_w4(a, stream));
}

int64_t wush_moe_w4_workspace(int64_t M, int64_t E, int topk, int64_t H, int64_t I, int transform, int out_type) {
  if (M <= 0 || H <= 0 || I <= 0 || check_moe_shape(M, E, topk, H, I) != WUSH_OK) return 0;
  return (int64_t)moe_workspace(M, E, topk, H, I, transform != 0, out_type).total;
}

wush_status wush_moe_w4(int fmt, const void* X, int64_t ldx, const void* router, const void* gate_up_codes,
                        const void* gate_up_scales, const float* gate_up_global, const void* T_in,
                        const void* down_codes, const void* down_scales, const float* down_global, const void* T_mid,
                        int64_t M, int64_t E, int topk, int renormalize, int64_t H, int64_t I, void* Y, int out_type,
                        int32_t* ids, float* weights, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = 0;
  wush_status st = check_fmt(fmt, out_type);
  if (st != WUSH_OK) return st;
  st = check_moe_shape(M, E, topk, H, I);
  if (st != WUSH_OK) return st;
  st = check_width("H", H, fmt);
  if (st != WUSH_OK) return st;
  st = check_width("I", I, fmt);
  if (st != WUSH_OK) return st;
  if (M == 0) return WUSH_OK;
  if (M > ((int64_t)1 << 30)) return fail(WUSH_EINVAL, "M too large");
  st = check_rows(X, ldx, M, H);
  if (st != WUSH_OK) return st;
  if (!router) return fail(WUSH_EINVAL, "null router");
  if (!aligned(router, 16)) return fail(WUSH_EALIGN, "router must be 16-byte aligned");
  st = check_weights("gate_up", fmt, gate_up_codes, gate_up_scales, gate_up_global);
  if (st != WUSH_OK) return st;
  st = check_weights("down", fmt, down_codes, down_scales, down_global);
  if (st != WUSH_OK) return st;
  if ((T_in && !aligned(T_in, 16)) || (T_mid && !aligned(T_mid, 16)))
    return fail(WUSH_EALIGN, "T_in and T_mid must be 16-byte aligned");
  if (!Y || !ids || !weights) return fail(WUSH_EINVAL, "null Y, ids or weights");
  if (!aligned(Y, (uintptr_t)out_bytes_of(out_type)) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(WUSH_EALIGN, "Y, ids and weights must be aligned to their elements");
  const MoeWorkspace w = moe_workspace(M, E, topk, H, I, T_in != nullptr, out_type);
  st = check_workspace(workspace, workspace_bytes, (int64_t)w.total);
  if (st != WUSH_OK) return st;
  const int G = group_of(fmt);
  const bool nv = fmt == wush::kNVFP4;
  const Range ins[] = {{X, ((uint64_t)(M - 1) * (M > 1 ? ldx : 0) + H) * 2},
                       {router, (uint64_t)E * H * 2},
                       {gate_up_codes, code_bytes(E * 2 * I, H)},
                       {gate_up_scales, scale_bytes(fmt, E * 2 * I, H)},
                       {nv ? gate_up_global : nullptr, (uint64_t)E * 4},
                       {T_in, (uint64_t)H * G * 2},
                       {down_codes, code_bytes(E * H, I)},
                       {down_scales, scale_bytes(fmt, E * H, I)},
                       {nv ? down_global : nullptr, (uint64_t)E * 4},
                       {T_mid, (uint64_t)E * I * G * 2}};
  const Range outs[] = {{Y, (uint64_t)M * H * out_bytes_of(out_type)},
                        {ids, (uint64_t)M * topk * 4},
                        {weights, (uint64_t)M * topk * 4},
                        {workspace, w.total}};
  if (any_overlap(outs, 4, ins, 10))
    return fail(WUSH_EINVAL, "outputs and the workspace must not overlap each other or an input");
  st = check_device();
  if (st != WUSH_OK) return st;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  wush::MoeArgs a{};
  a.fmt = fmt;
  a.ldx = M > 1 ? ldx : 0;
  a.router = static_cast<const uint16_t*>(router);
  a.gu_codes = static_cast<const uint8_t*>(gate_up_codes);
  a.gu_scales = static_cast<const uint8_t*>(gate_up_scales);
  a.gu_gs = gate_up_global;
  a.dn_codes = static_cast<const uint8_t*>(down_codes);
  a.dn_scales = static_cast<const uint8_t*>(down_scales);
  a.dn_gs = down_global;
  a.T_mid = static_cast<const uint16_t*>(T_mid);
  a.E = (int)E;
  a.topk = topk;
  a.H = H;
  a.I = I;
  a.renorm = renormalize != 0;
  a.terms = terms_of(out_type);
  a.bf16_out = out_type == WUSH_OUT_BF16;
  a.T_in = static_cast<const uint16_t*>(T_in);
  a.xt = reinterpret_cast<uint16_t*>(ws + w.planes);
  a.h = reinterpret_cast<uint16_t*>(ws + w.h);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.logits = reinterpret_cast<float*>(ws + w.logits);
  a.n_tiles = reinterpret_cast<int32_t*>(ws + w.n_tiles);
  a.tiles = reinterpret_cast<wush::MoeTile*>(ws + w.tiles);
  for (int64_t m0 = 0; m0 < M; m0 += wush::kMoeTokens) {
    a.M = (int)moe_chunk(M - m0);
    a.X = static_cast<const uint16_t*>(X) + m0 * a.ldx;
    a.Y = static_cast<uint8_t*>(Y) + m0 * H * out_bytes_of(out_type);
    a.ids = ids + m0 * topk;
    a.weights = weights + m0 * topk;
    st = launched(wush::launch_moe(a, stream));
    if (st != WUSH_OK) return st;
  }
  return WUSH_OK;
}

int64_t wush_token_logprobs_workspace(int64_t R, int64_t V, int logit_type, int top) {
  if (R <= 0 || R > kMaxLogprobRows || V <= 0 || V > INT32_MAX) return 0;
  if (logit_type < 0 || logit_type > 2 || top < 0 || top > wush::kLogprobMaxTop) return 0;
  const int64_t s = wush::logprob_plan(R, V).splits;
  return s == 1 ? 0 : R * s * (16 + 8 * (int64_t)top);
}

wush_status wush_token_logprobs(const void* logits, int logit_type, int64_t ld, int64_t R, int64_t V,
                                const int64_t* targets, int top, float* logprob, float* entropy, int32_t* top_ids,
                                float* top_logprobs, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  g_last_error[0] = 0;
  if (logit_type < WUSH_LOGITS_F32 || logit_type > WUSH_LOGITS_F16)
    return fail(WUSH_EINVAL, "unknown logit_type %d", logit_type);
  if (R < 0) return fail(WUSH_EINVAL, "R must be >= 0 (got %lld)", (long long)R);
  if (V < 1 || V > INT32_MAX) return fail(WUSH_EINVAL, "V must be 1 .. 2^31 - 1 (got %lld)", (long long)V);
  if (top < 0 || top > wush::kLogprobMaxTop)
    return fail(WUSH_EINVAL, "top must be 0 .. %d (got %d)", wush::kLogprobMaxTop, top);
  if (R == 0) return WUSH_OK;
  if (R > kMaxLogprobRows) return fail(WUSH_EINVAL, "R too large for one launch");
  if (R > 1 && (ld < V || ld > ((int64_t)1 << 36))) return fail(WUSH_EINVAL, "ld must be V or more (got %lld)", (long long)ld);
  if (!logits || !targets || !logprob || !entropy) return fail(WUSH_EINVAL, "null pointer");
  if (top > 0 && (!top_ids || !top_logprobs)) return fail(WUSH_EINVAL, "null top_ids or top_logprobs");
  const int eb = logit_type == WUSH_LOGITS_F32 ? 4 : 2;
  if (!aligned(logits, (uintptr_t)eb)) return fail(WUSH_EALIGN, "logits must be aligned to their elements");
  if (!aligned(targets, 8)) return fail(WUSH_EALIGN, "targets must be 8-byte aligned");
  if (!aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
    return fail(WUSH_EALIGN, "outputs must be 4-byte aligned");
  const int64_t need = wush_token_logprobs_workspace(R, V, logit_type, top);
  wush_status st = check_workspace(workspace, workspace_bytes, need);
  if (st != WUSH_OK) return st;
  const Range ins[] = {{logits, ((uint64_t)(R - 1) * (R > 1 ? ld : 0) + V) * eb}, {targets, (uint64_t)R * 8}};
  const uint64_t nt = (uint64_t)R * top * 4;
  const Range outs[] = {{logprob, (uint64_t)R * 4},
                        {entropy, (uint64_t)R * 4},
                        {top > 0 ? top_ids : nullptr, nt},
                        {top > 0 ? top_logprobs : nullptr, nt},
                        {workspace, (uint64_t)need}};
  if (any_overlap(outs, 5, ins, 2))
    return fail(WUSH_EINVAL, "outputs and the workspace must not overlap each other or an input");
  st = check_device();
  if (st != WUSH_OK) return st;

  wush::LogprobArgs a{};
  a.L = logits;
  a.type = logit_type;
  a.ld = R > 1 ? ld : 0;
  a.R = R;
  a.V = V;
  a.targets = targets;
  a.top = top;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  const wush::LogprobPlan plan = wush::logprob_plan(R, V);
  a.splits = plan.splits;
  a.split_batches = plan.split_batches;
  // The keys first: they need 8-byte alignment whatever their number.
  a.keys = static_cast<uint64_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + (need ? R * a.splits * (int64_t)top * 8 : 0));
  return launched(wush::launch_logprobs(a, stream));
}

}  // extern "C"
