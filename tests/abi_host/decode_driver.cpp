// Host-side checks of the decode entries of the C ABI (include/wush.h), built
// with the sanitizers against stubs.cpp and decode_stubs.cpp.  It checks that:
//   * every malformed call returns its error code without making any HIP call
//     or launch;
//   * well-formed calls launch what they should, with all of a mixture's and of the
//     log probabilities' scratch inside the workspace that was asked for;
//   * the log probabilities' plan covers every batch of a row exactly once.
// Pointers are fake device addresses: nothing dereferences them.
#include <stdint.h>
#include <stdio.h>

#include "../../include/wush.h"
#include "decode_stubs.h"

static int g_fail = 0;

#define EXPECT(cond, ...)                                  \
  do {                                                     \
    if (!(cond)) {                                         \
      ++g_fail;                                            \
      fprintf(stderr, "FAIL %s:%d: ", __FILE__, __LINE__); \
      fprintf(stderr, __VA_ARGS__);                        \
      fprintf(stderr, "\n");                               \
    }                                                      \
  } while (0)

// A malformed call: the expected status, no HIP call, no launch.
#define REJECT(expr, status)                                                              \
  do {                                                                                    \
    const int h0 = g_hip_calls, l0 = g_launches;                                          \
    const wush_status st_ = (expr);                                                       \
    EXPECT(st_ == (status), "%s -> %d, want %d (%s)", #expr, (int)st_, (int)(status),     \
           wush_last_error());                                                            \
    EXPECT(g_hip_calls == h0 && g_launches == l0, "%s made a HIP call or launch", #expr); \
    EXPECT(wush_last_error()[0] != 0, "%s left no error text", #expr);                    \
  } while (0)

// A well-formed call: OK and exactly n launches.
#define ACCEPT(expr, n)                                                                           \
  do {                                                                                            \
    const int l0 = g_launches;                                                                    \
    const wush_status st_ = (expr);                                                               \
    EXPECT(st_ == WUSH_OK, "%s -> %d (%s)", #expr, (int)st_, wush_last_error());                  \
    EXPECT(g_launches - l0 == (n), "%s launched %d times, want %d", #expr, g_launches - l0, (n)); \
  } while (0)

static const uintptr_t A = (uintptr_t)1 << 40;  // aligned, far from the others
template <typename T = void>
static T* P(uintptr_t a) {
  return reinterpret_cast<T*>(a);
}

static void linear() {
  for (int fmt = 0; fmt < 3; ++fmt) {
    const int G = fmt == 1 ? 16 : 32;
    struct Call {
      int fmt;
      uintptr_t X = A, T = 0, c = 2 * A, s = 3 * A, g = 4 * A, Y = 5 * A, ws = 0;
      int64_t ldx, M = 3, N = 40, K, n = 0;
      int out = WUSH_OUT_BF16;
    };
    const auto call = [&](auto&& change) {
      Call k;
      k.fmt = fmt;
      k.ldx = k.K = 4 * G;
      change(k);
      return wush_linear_w4(k.fmt, P(k.X), k.ldx, P(k.T), P(k.c), P(k.s), P<float>(k.g), k.M, k.N, k.K, P(k.Y), k.out,
                            P(k.ws), k.n, nullptr);
    };
    ACCEPT(call([](Call&) {}), 1);
    ACCEPT(call([](Call& k) { k.M = 0; k.X = k.Y = 0; }), 0);
    ACCEPT(call([](Call& k) { k.N = 0; k.c = k.Y = 0; }), 0);
    ACCEPT(call([](Call& k) { k.M = 1; k.ldx = 0; }), 1);
    REJECT(call([](Call& k) { k.fmt = 3; }), WUSH_EUNSUPPORTED);
    REJECT(call([](Call& k) { k.fmt = -1; }), WUSH_EUNSUPPORTED);
    REJECT(call([](Call& k) { k.out = 2; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.M = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.M = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.N = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.N = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.K = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.K = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.K += 8; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldx = k.K - 8; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldx = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldx = k.K + 4; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.X = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.c = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.s = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.Y = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.X += 8; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.c += 4; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.Y += 1; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.T = 6 * A; }), WUSH_EINVAL);  // no workspace
    // The largest sizes that pass: sizes in bytes stay below 2^64.
    ACCEPT(call([](Call& k) {
             k.K = k.ldx = (int64_t)1 << 27;
             k.N = 1 << 20;
             k.M = 1 << 19;
             k.c = (uintptr_t)1 << 50;
             k.s = (uintptr_t)1 << 51;
             k.Y = (uintptr_t)1 << 53;
             k.X = (uintptr_t)1 << 54;
           }),
           1);
    for (int out = 0; out < 2; ++out)
      for (int64_t M : {1, 5, 64, 100}) {
        const int64_t n = wush_linear_w4_workspace(M, 4 * G, out);
        const auto with = [&](Call& k) {
          k.T = 6 * A;
          k.ws = 7 * A;
          k.M = M;
          k.n = n;
          k.out = out;
        };
        ACCEPT(call(with), 2);
        EXPECT(g_last_split.out == P<uint16_t>(7 * A) && g_last_linear.x.X == g_last_split.out, "planes");
        EXPECT(2 * g_last_split.terms * M * 4 * G <= n && g_last_linear.x.terms == g_last_split.terms, "planes' size");
        REJECT(call([&](Call& k) { with(k); k.n = n - 1; }), WUSH_EINVAL);
        REJECT(call([&](Call& k) { with(k); k.ws += 8; }), WUSH_EALIGN);
        REJECT(call([&](Call& k) { with(k); k.ws = k.X; }), WUSH_EINVAL);
        REJECT(call([&](Call& k) { with(k); k.ws = k.Y; }), WUSH_EINVAL);
        REJECT(call([&](Call& k) { with(k); k.T += 2; }), WUSH_EALIGN);
      }
    for (uintptr_t in : {A, 2 * A, 3 * A}) REJECT(call([&](Call& k) { k.Y = in; }), WUSH_EINVAL);
    if (fmt == 1) REJECT(call([](Call& k) { k.g = 0; }), WUSH_EINVAL);
    if (fmt == 1) REJECT(call([](Call& k) { k.g += 2; }), WUSH_EALIGN);
    if (fmt == 1) REJECT(call([](Call& k) { k.Y = k.g; }), WUSH_EINVAL);
    if (fmt == 2) REJECT(call([](Call& k) { k.s += 1; }), WUSH_EALIGN);
  }
  EXPECT(wush_linear_w4_workspace(0, 64, 0) == 0 && wush_linear_w4_workspace(-1, 64, 0) == 0, "no tokens");
  EXPECT(wush_linear_w4_workspace(INT64_MAX, 64, 0) == 0 && wush_linear_w4_workspace(1, INT64_MAX, 0) == 0, "too large");
}

static void mixture() {
  for (int fmt = 0; fmt < 3; ++fmt) {
    const int G = fmt == 1 ? 16 : 32;
    struct Call {
      uintptr_t X = A, r = 2 * A, gc = 3 * A, gs = 4 * A, gg = 5 * A, ti = 0, dc = 6 * A, ds = 7 * A, dg = 8 * A, tm = 0,
                Y = 9 * A, ids = 10 * A, w = 11 * A, ws = 12 * A;
      int64_t ldx, M = 3, E = 6, H, I, n = -1;
      int k = 2, out = WUSH_OUT_BF16;
    };
    const auto call = [&](auto&& change) {
      Call k;
      k.H = 4 * G;
      k.I = 3 * G;
      k.ldx = k.H;
      change(k);
      if (k.n < 0) k.n = wush_moe_w4_workspace(k.M, k.E, k.k, k.H, k.I, k.ti != 0, k.out);
      return wush_moe_w4(fmt, P(k.X), k.ldx, P(k.r), P(k.gc), P(k.gs), P<float>(k.gg), P(k.ti), P(k.dc), P(k.ds),
                         P<float>(k.dg), P(k.tm), k.M, k.E, k.k, 1, k.H, k.I, P(k.Y), k.out, P<int32_t>(k.ids),
                         P<float>(k.w), P(k.ws), k.n, nullptr);
    };
    ACCEPT(call([](Call&) {}), 1);
    ACCEPT(call([](Call& k) { k.M = 0; k.X = 0; }), 0);
    REJECT(call([](Call& k) { k.M = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.M = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.E = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.E = 1025; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.k = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.k = 7; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.E = 64; k.k = 33; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.H = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.I = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.H += 8; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.I += 8; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldx -= 8; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldx += 4; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.out = 7; }), WUSH_EINVAL);
    for (uintptr_t Call::*p : {&Call::X, &Call::r, &Call::gc, &Call::gs, &Call::dc, &Call::ds, &Call::Y, &Call::ids,
                               &Call::w, &Call::ws})
      REJECT(call([&](Call& k) { k.*p = 0; }), WUSH_EINVAL);
    for (uintptr_t Call::*p : {&Call::X, &Call::r, &Call::ws}) REJECT(call([&](Call& k) { k.*p += 8; }), WUSH_EALIGN);
    for (uintptr_t Call::*p : {&Call::gc, &Call::dc}) REJECT(call([&](Call& k) { k.*p += 4; }), WUSH_EALIGN);
    for (uintptr_t Call::*p : {&Call::ids, &Call::w}) REJECT(call([&](Call& k) { k.*p += 2; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.Y += 1; }), WUSH_EALIGN);
    for (uintptr_t Call::*p : {&Call::ti, &Call::tm}) REJECT(call([&](Call& k) { k.*p = 13 * A + 8; }), WUSH_EALIGN);
    for (uintptr_t Call::*o : {&Call::Y, &Call::ids, &Call::w, &Call::ws})
      for (uintptr_t Call::*i : {&Call::X, &Call::r, &Call::gc, &Call::gs, &Call::dc, &Call::ds})
        REJECT(call([&](Call& k) { k.*o = k.*i; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ids = k.w; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.Y = k.ws; }), WUSH_EINVAL);
    if (fmt == 1) REJECT(call([](Call& k) { k.gg = 0; }), WUSH_EINVAL);
    if (fmt == 1) REJECT(call([](Call& k) { k.dg = 0; }), WUSH_EINVAL);
    if (fmt == 2) REJECT(call([](Call& k) { k.ds += 1; }), WUSH_EALIGN);
    // All scratch lies in the workspace, one after the other, and all tokens are taken.
    for (int out = 0; out < 2; ++out)
      for (int t = 0; t < 2; ++t)
        for (int64_t M : {1, 2, 63, 64, 65, 128, 200})
          for (int64_t E : {1, 2, 15, 128, 1024})
            for (int topk : {1, 2, 32}) {
              if (topk > E) continue;
              const auto set = [&](Call& k) {
                k.M = M;
                k.E = E;
                k.k = topk;
                k.out = out;
                k.ti = t ? 13 * A : 0;
              };
              g_moe_tokens = 0;
              ACCEPT(call(set), (int)((M + 63) / 64));
              EXPECT(g_moe_tokens == M, "tokens");
              const auto& a = g_last_moe;
              const int64_t c = M < 64 ? M : 64, slots = c * topk;
              const int64_t n = wush_moe_w4_workspace(M, E, topk, a.H, a.I, t, out);
              uintptr_t at = 12 * A;
              const auto next = [&](const void* p, int64_t bytes) {
                EXPECT((uintptr_t)p >= at && (uintptr_t)p % 16 == 0, "scratch overlaps");
                at = (uintptr_t)p + bytes;
              };
              if (t) next(a.xt, 2 * a.terms * c * a.H);
              next(a.h, 2 * a.terms * slots * a.I);
              next(a.part, 4 * slots * a.H);
              next(a.logits, 4 * wush::kRouterParts * c * E);
              next(a.n_tiles, 4);
              next(a.tiles, slots * (int64_t)sizeof(wush::MoeTile));
              EXPECT(at <= 12 * A + n, "scratch past the workspace");
              REJECT(call([&](Call& k) { set(k); k.n = n - 1; }), WUSH_EINVAL);
            }
  }
  EXPECT(wush_moe_w4_workspace(0, 4, 2, 64, 64, 0, 0) == 0 && wush_moe_w4_workspace(4, 4, 5, 64, 64, 0, 0) == 0, "none");
}

static void logprobs() {
  struct Call {
    uintptr_t L = A, t = 2 * A, lp = 3 * A, en = 4 * A, ids = 5 * A, alt = 6 * A, ws = 7 * A;
    int type = 1, top = 5;
    int64_t ld = 100000, R = 3, V = 100000, n = -1;
  };
  const auto call = [&](auto&& change) {
    Call k;
    change(k);
    if (k.n < 0) k.n = wush_token_logprobs_workspace(k.R, k.V, k.type, k.top);
    return wush_token_logprobs(P(k.L), k.type, k.ld, k.R, k.V, P<int64_t>(k.t), k.top, P<float>(k.lp), P<float>(k.en),
                               P<int32_t>(k.ids), P<float>(k.alt), P(k.ws), k.n, nullptr);
  };
  ACCEPT(call([](Call&) {}), 1);
  ACCEPT(call([](Call& k) { k.R = 0; k.L = 0; }), 0);
  ACCEPT(call([](Call& k) { k.top = 0; k.ids = k.alt = 0; }), 1);
  REJECT(call([](Call& k) { k.type = 3; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.type = -1; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.R = -1; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.V = 0; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.V = (int64_t)1 << 31; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.top = 33; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.top = -1; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.ld = k.V - 1; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.ld = INT64_MAX; }), WUSH_EINVAL);
  for (uintptr_t Call::*p : {&Call::L, &Call::t, &Call::lp, &Call::en, &Call::ids, &Call::alt, &Call::ws})
    REJECT(call([&](Call& k) { k.*p = 0; }), WUSH_EINVAL);
  for (uintptr_t Call::*p : {&Call::L, &Call::t, &Call::lp, &Call::en, &Call::ids, &Call::alt, &Call::ws})
    REJECT(call([&](Call& k) { k.*p += 1; }), WUSH_EALIGN);
  for (uintptr_t Call::*o : {&Call::lp, &Call::en, &Call::ids, &Call::alt, &Call::ws})
    for (uintptr_t Call::*i : {&Call::L, &Call::t}) REJECT(call([&](Call& k) { k.*o = k.*i; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.ids = k.alt; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.n = wush_token_logprobs_workspace(k.R, k.V, k.type, k.top) - 1; }), WUSH_EINVAL);
  for (int64_t R : {1, 2, 3, 7, 64, 67, 511, 512, 1024, 1025, 5000})
    for (int64_t V : {1, 7, 2047, 2048, 2049, 8192, 50001, 131072, 200000, 10000000})
      for (int top : {0, 1, 32}) {
        const int64_t n = wush_token_logprobs_workspace(R, V, 1, top);
        ACCEPT(call([&](Call& k) { k.R = R; k.V = k.ld = V; k.top = top; }), 1);
        const auto& a = g_last_logprobs;
        const int64_t per = 256 * (wush::logprob_narrow(R, V) ? 8 : 32), batches = (V + per - 1) / per;
        EXPECT(a.splits >= 1 && a.splits <= 64 && a.split_batches >= 1, "plan");
        EXPECT((int64_t)(a.splits - 1) * a.split_batches < batches && (int64_t)a.splits * a.split_batches >= batches,
               "the splits cover %lld batches with %d x %d", (long long)batches, a.splits, a.split_batches);
        EXPECT((a.splits == 1) == (n == 0), "workspace of one workgroup per row");
        if (n == 0) continue;
        const uintptr_t end = (uintptr_t)a.keys + 8 * R * a.splits * top;
        EXPECT((uintptr_t)a.keys == 7 * A && (uintptr_t)a.part == end && end + 16 * R * a.splits == 7 * A + n, "scratch");
      }
  // More rows than a call takes.
  for (int64_t R : {((int64_t)1 << 24) + 1, (int64_t)1 << 50, INT64_MAX}) {
    EXPECT(wush_token_logprobs_workspace(R, INT32_MAX, 0, 32) == 0, "too many rows");
    REJECT(call([&](Call& k) { k.R = R; }), WUSH_EINVAL);
  }
  EXPECT(wush_token_logprobs_workspace(0, 9, 0, 0) == 0 && wush_token_logprobs_workspace(4, 0, 0, 0) == 0, "none");
}

int main() {
  linear();
  mixture();
  logprobs();
  if (g_fail) {
    fprintf(stderr, "%d failures\n", g_fail);
    return 1;
  }
  printf("decode abi host checks passed\n");
  return 0;
}
