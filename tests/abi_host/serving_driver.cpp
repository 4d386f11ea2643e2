// Host-side checks of the C ABI's entries for the cache, attention, adapters and
// logits (include/wush.h), built with the sanitizers against stubs.cpp,
// decode_stubs.cpp and serving_stubs.cpp: every malformed call returns its error code
// without any HIP call or launch, and well-formed calls launch what they should, with
// all scratch inside the workspace that was asked for.  Pointers are fake device
// addresses: nothing dereferences them.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/wush.h"
#include "serving_stubs.h"

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


struct Cache {
  uintptr_t kc = 10 * A, ks = 11 * A, kg = 12 * A, vc = 13 * A, vs = 14 * A, vg = 15 * A;
  int64_t heads = 2, D = 128, page = 16, pages = 9;
};

static void append() {
  for (int fmt = 0; fmt < 3; ++fmt) {
    struct Call : Cache {
      int fmt;
      uintptr_t K = A, V = 2 * A, Tk = 0, Tv = 0, slots = 3 * A;
      int64_t ldk = 256, ldv = 256, n = 3;
    };
    const auto call = [&](auto&& change) {
      Call k;
      k.fmt = fmt;
      change(k);
      return wush_kv4_append(k.fmt, P(k.K), k.ldk, P(k.V), k.ldv, P(k.Tk), P(k.Tv), P<int64_t>(k.slots), k.n, k.heads, k.D,
                             k.page, k.pages, P(k.kc), P(k.ks), P<float>(k.kg), P(k.vc), P(k.vs), P<float>(k.vg), nullptr);
    };
    ACCEPT(call([](Call&) {}), 1);
    EXPECT(g_last_append.page_log2 == 4 && g_last_append.heads == 2 && g_last_append.D == 128, "append's sizes");
    ACCEPT(call([](Call& k) { k.Tk = 4 * A; }), 1);
    EXPECT(g_last_append.side[0].T && !g_last_append.side[1].T, "append's transforms");
    ACCEPT(call([](Call& k) { k.n = 0; k.K = k.V = k.slots = 0; }), 0);
    ACCEPT(call([](Call& k) { k.pages = 0; k.kc = k.vs = 0; }), 0);
    ACCEPT(call([](Call& k) { k.n = 1; k.ldk = k.ldv = 0; }), 1);
    REJECT(call([](Call& k) { k.fmt = 3; }), WUSH_EUNSUPPORTED);
    for (int64_t D : {0, 32, 96, 192, 512}) REJECT(call([&](Call& k) { k.D = D; }), WUSH_EUNSUPPORTED);
    for (int64_t p : {0, 8, 24, 131072, -16}) REJECT(call([&](Call& k) { k.page = p; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.heads = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.heads = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.pages = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.pages = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.n = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.n = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.K = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.V = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.slots = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.kc = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.vs = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldk = 248; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldv = 260; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.K += 8; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.Tv = 4 * A + 8; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.slots += 4; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.vc += 8; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.ks += 8; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.kc = k.K; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.vc = k.kc; }), WUSH_EINVAL);
    if (fmt == 1) {
      REJECT(call([](Call& k) { k.kg = 0; }), WUSH_EINVAL);
      REJECT(call([](Call& k) { k.vg += 2; }), WUSH_EALIGN);
      REJECT(call([](Call& k) { k.kg = k.ks; }), WUSH_EINVAL);
    } else {
      ACCEPT(call([](Call& k) { k.kg = k.vg = 0; }), 1);
    }
  }
}

static void attention() {
  for (int fmt = 0; fmt < 3; ++fmt) {
    struct Call : Cache {
      int fmt;
      uintptr_t Q = A, T = 0, table = 3 * A, lengths = 4 * A, start = 0, out = 5 * A, ws = 6 * A;
      int64_t ldq = 1024, ldt = 50, width = 50, B = 3, n = 3, hq = 8, window = 0, bytes = -1;
      float scale = 0.1f;
    };
    const auto call = [&](auto&& change) {
      Call k;
      k.fmt = fmt;
      change(k);
      if (k.bytes < 0) k.bytes = wush_kv4_attention_workspace(k.fmt, k.B, k.n, k.hq, k.heads, k.D, k.page, k.width);
      return wush_kv4_attention(k.fmt, P(k.Q), k.ldq, P(k.T), P(k.kc), P(k.ks), P<float>(k.kg), P(k.vc), P(k.vs),
                                P<float>(k.vg), P<int32_t>(k.table), k.ldt, k.width, P<int32_t>(k.lengths),
                                P<int32_t>(k.start), k.B, k.n, k.hq, k.heads, k.D, k.page, k.pages, k.scale, k.window,
                                P(k.out), P(k.ws), k.bytes, nullptr);
    };
    ACCEPT(call([](Call&) {}), 1);
    EXPECT(g_last_attention.group == 4 && g_last_shape == wush::kKvNarrow, "attention's columns");
    EXPECT(g_last_attention.workgroups >= g_last_attention.runs && g_last_attention.runs > 0, "attention's runs");
    ACCEPT(call([](Call& k) { k.B = k.n = 0; k.Q = k.out = 0; }), 0);
    ACCEPT(call([](Call& k) { k.width = k.ldt = 2; k.ws = 0; k.bytes = 0; }), 1);  // short: no workspace
    EXPECT(g_last_attention.runs == 0 && !g_last_attention.part, "a short call's workspace");
    ACCEPT(call([](Call& k) { k.start = 7 * A; k.n = 300; }), 1);
    EXPECT(g_last_shape == wush::kKvPrompt, "a prompt's shape");
    ACCEPT(call([](Call& k) { k.start = 7 * A; k.n = 12; }), 1);
    EXPECT(g_last_shape == wush::kKvNarrow, "drafted tokens' shape");
    // Scratch for any sizes lies inside the workspace, and ends where it does.
    for (int64_t D : {64, 128, 256})
      for (int64_t B : {1, 7, 900})
        for (int64_t per : {1, 9, 400})
          for (int64_t width : {33, 5000}) {
            const int64_t need = wush_kv4_attention_workspace(fmt, B, B * per, 8, 2, D, 16, width);
            ACCEPT(call([&](Call& k) {
                     k.start = 7 * A;
                     k.B = B;
                     k.n = B * per;
                     k.D = D;
                     k.width = k.ldt = width;
                     k.ldq = 8 * D;
                   }),
                   1);
            const auto& a = g_last_attention;
            const uintptr_t end = (uintptr_t)a.part + 2 * (uintptr_t)a.runs * 4 * wush::kv_piece(g_last_shape, (int)D);
            EXPECT((uintptr_t)a.join == 6 * A && end == 6 * A + (uintptr_t)need, "workspace of %lld x %lld", (long long)B, (long long)per);
            EXPECT((uintptr_t)a.part % 16 == 0, "pieces' alignment");
          }
    REJECT(call([](Call& k) { k.fmt = -1; }), WUSH_EUNSUPPORTED);
    REJECT(call([](Call& k) { k.D = 96; }), WUSH_EUNSUPPORTED);
    REJECT(call([](Call& k) { k.page = 48; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.pages = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.hq = 7; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.hq = 1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.hq = 8192; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.n = 4; }), WUSH_EINVAL);  // without q_start
    REJECT(call([](Call& k) { k.B = k.n = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.n = k.B = INT64_MAX; k.bytes = 0; }), WUSH_EINVAL);
    for (float s : {0.0f, -1.0f, INFINITY, NAN}) REJECT(call([&](Call& k) { k.scale = s; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.window = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.window = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.width = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.width = k.ldt = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldt = 49; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.width = k.ldt = (int64_t)1 << 25; k.B = k.n = 1 << 14; k.bytes = 0; }), WUSH_EINVAL);
    for (uintptr_t Call::*p : {&Call::Q, &Call::table, &Call::lengths, &Call::out, &Call::ws})
      REJECT(call([&](Call& k) { k.*p = 0; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldq = 1016; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.ldq = 1028; }), WUSH_EALIGN);
    for (uintptr_t Call::*p : {&Call::Q, &Call::out, &Call::ws}) REJECT(call([&](Call& k) { k.*p += 8; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.T = 8 * A + 8; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.table += 2; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.start = 7 * A + 2; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.bytes = wush_kv4_attention_workspace(k.fmt, 3, 3, 8, 2, 128, 16, 50) - 1; }), WUSH_EINVAL);
    for (uintptr_t in : {A, 3 * A, 4 * A, 10 * A, 14 * A}) {
      REJECT(call([&](Call& k) { k.out = in; }), WUSH_EINVAL);
      REJECT(call([&](Call& k) { k.ws = in; }), WUSH_EINVAL);
    }
    REJECT(call([](Call& k) { k.ws = k.out; }), WUSH_EINVAL);
    if (fmt == 1) REJECT(call([](Call& k) { k.vg = 0; }), WUSH_EINVAL);
  }
  EXPECT(wush_kv4_attention_workspace(3, 1, 1, 8, 2, 128, 16, 50) == 0, "workspace of a bad format");
  EXPECT(wush_kv4_attention_workspace(0, -1, 1, 8, 2, 128, 16, 50) == 0, "workspace of a bad batch");
  EXPECT(wush_kv4_attention_workspace(0, 1, 1, 8, 3, 128, 16, 50) == 0, "workspace of bad heads");
  EXPECT(wush_kv4_attention_workspace(0, INT64_MAX, INT64_MAX, 8, 2, 128, INT64_MAX, INT64_MAX) == 0, "workspace of huge sizes");
}

static void lora() {
  for (int fmt = 0; fmt < 3; ++fmt) {
    const int G = fmt == 1 ? 16 : 32;
    struct Call {
      int fmt;
      uintptr_t X = A, T = 0, c = 2 * A, s = 3 * A, g = 4 * A, a = 5 * A, b = 6 * A, e = 7 * A, ids = 8 * A, Y = 9 * A,
                ws = 10 * A;
      int64_t ldx, E = 4, r = 16, M = 3, N = 40, K, n = -1;
      int out = WUSH_OUT_BF16;
    };
    const auto call = [&](auto&& change) {
      Call k;
      k.fmt = fmt;
      k.ldx = k.K = 4 * G;
      change(k);
      if (k.n < 0) k.n = wush_linear_w4_lora_workspace(k.M, k.N, k.K, k.r, k.T != 0, k.out);
      return wush_linear_w4_lora(k.fmt, P(k.X), k.ldx, P(k.T), P(k.c), P(k.s), P<float>(k.g), P(k.a), P(k.b), P<float>(k.e),
                                 P<int32_t>(k.ids), k.E, k.r, k.M, k.N, k.K, P(k.Y), k.out, P(k.ws), k.n, nullptr);
    };
    ACCEPT(call([](Call&) {}), 2);
    EXPECT(!g_last_linear.lora.delta && g_last_linear.lora.ids, "few tokens add in the product");
    ACCEPT(call([](Call& k) { k.M = 0; k.X = k.Y = 0; }), 0);
    ACCEPT(call([](Call& k) { k.N = 0; k.Y = 0; }), 0);
    ACCEPT(call([](Call& k) { k.E = 0; k.a = k.b = 0; }), 2);
    ACCEPT(call([](Call& k) { k.e = 0; }), 2);
    for (int out = 0; out < 2; ++out)
      for (int64_t M : {1, 8, 9, 64, 256, 257, 1000})
        for (int t = 0; t < 2; ++t) {
          const int64_t need = wush_linear_w4_lora_workspace(M, 40, 4 * G, 16, t, out), c = M < 256 ? M : 256;
          const int chunks = (int)((M + 255) / 256);
          g_lora_tokens = 0;
          ACCEPT(call([&](Call& k) { k.M = M; k.out = out; k.T = t ? 11 * A : 0; }), chunks * (M > 64 ? 3 : 2));
          EXPECT(g_lora_tokens == M, "tokens of the chunks");
          const uintptr_t h = (uintptr_t)g_last_lora.h, d = (uintptr_t)g_last_lora.delta, end = 10 * A + (uintptr_t)need;
          EXPECT(h == 10 * A && h + c * 16 * 4 <= (d ? d : end), "h");
          EXPECT((M > 64) == (d != 0), "delta");
          if (t) {
            const uintptr_t p = (uintptr_t)g_last_split.out;
            EXPECT(p % 16 == 0 && p >= (d ? d + c * 40 * 4 : h + c * 64) && p + (out ? 2 : 3) * c * 4 * G * 2 == end, "planes");
          } else {
            EXPECT(!d || d + c * 40 * 4 <= end, "delta's end");
          }
        }
    REJECT(call([](Call& k) { k.fmt = 3; }), WUSH_EUNSUPPORTED);
    REJECT(call([](Call& k) { k.out = 5; }), WUSH_EINVAL);
    for (int64_t r : {0, 4, 12, 520, -8}) REJECT(call([&](Call& k) { k.r = r; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.E = -1; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.E = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.M = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.N = INT64_MAX; }), WUSH_EINVAL);
    REJECT(call([](Call& k) { k.K = 8; }), WUSH_EINVAL);
    for (uintptr_t Call::*p : {&Call::X, &Call::c, &Call::s, &Call::a, &Call::b, &Call::ids, &Call::Y, &Call::ws})
      REJECT(call([&](Call& k) { k.*p = 0; }), WUSH_EINVAL);
    for (uintptr_t Call::*p : {&Call::X, &Call::a, &Call::b, &Call::ws}) REJECT(call([&](Call& k) { k.*p += 8; }), WUSH_EALIGN);
    for (uintptr_t Call::*p : {&Call::ids, &Call::e}) REJECT(call([&](Call& k) { k.*p += 2; }), WUSH_EALIGN);
    REJECT(call([](Call& k) { k.n = wush_linear_w4_lora_workspace(k.M, k.N, k.K, k.r, 0, k.out) - 1; }), WUSH_EINVAL);
    for (uintptr_t in : {A, 2 * A, 5 * A, 6 * A, 7 * A, 8 * A}) {
      REJECT(call([&](Call& k) { k.Y = in; }), WUSH_EINVAL);
      REJECT(call([&](Call& k) { k.ws = in; }), WUSH_EINVAL);
    }
    REJECT(call([](Call& k) { k.ws = k.Y; }), WUSH_EINVAL);
    if (fmt == 1) REJECT(call([](Call& k) { k.g = 0; }), WUSH_EINVAL);
  }
  EXPECT(wush_linear_w4_lora_workspace(INT64_MAX, 8, 8, 8, 1, 0) == 0, "workspace of huge sizes");
  EXPECT(wush_linear_w4_lora_workspace(1, 8, 32, 8, 1, 7) == 0, "workspace of a bad type");
}

static void adjust() {
  struct Call {
    uintptr_t L = A, p = 2 * A, o = 3 * A, rep = 4 * A, f = 5 * A, pr = 6 * A, bi = 7 * A, b = 8 * A, m = 9 * A, out = 10 * A;
    int t = 0;
    int64_t ld = 100, R = 4, V = 100, np = 5, no = 6, nb = 7, ldo = 100;
  };
  const auto call = [&](auto&& change) {
    Call k;
    change(k);
    return wush_adjust_logits(P(k.L), k.t, k.ld, k.R, k.V, P<int32_t>(k.p), k.np, P<int32_t>(k.o), k.no, P<float>(k.rep),
                              P<float>(k.f), P<float>(k.pr), P<int32_t>(k.bi), P<float>(k.b), k.nb, P<int32_t>(k.m),
                              P(k.out), k.ldo, nullptr);
  };
  ACCEPT(call([](Call&) {}), 1);
  ACCEPT(call([](Call& k) { k.R = 0; k.L = k.out = 0; }), 0);
  ACCEPT(call([](Call& k) { k.p = k.o = k.rep = k.f = k.pr = k.bi = k.b = k.m = 0; k.np = k.no = k.nb = 0; }), 1);
  ACCEPT(call([](Call& k) { k.out = k.L; }), 1);
  ACCEPT(call([](Call& k) { k.R = 1; k.ld = k.ldo = 0; k.out = k.L; }), 1);
  for (int t : {-1, 3}) REJECT(call([&](Call& k) { k.t = t; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.R = -1; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.R = 65536; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.V = 0; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.V = INT64_MAX; }), WUSH_EINVAL);
  for (int64_t Call::*n : {&Call::np, &Call::no, &Call::nb}) {
    REJECT(call([&](Call& k) { k.*n = -1; }), WUSH_EINVAL);
    REJECT(call([&](Call& k) { k.*n = INT64_MAX; }), WUSH_EINVAL);
  }
  REJECT(call([](Call& k) { k.ld = 99; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.ldo = 99; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.ldo = INT64_MAX; }), WUSH_EINVAL);
  for (uintptr_t Call::*p : {&Call::L, &Call::p, &Call::o, &Call::bi, &Call::b, &Call::out})
    REJECT(call([&](Call& k) { k.*p = 0; }), WUSH_EINVAL);
  for (uintptr_t Call::*p : {&Call::L, &Call::p, &Call::o, &Call::rep, &Call::f, &Call::pr, &Call::bi, &Call::b, &Call::m, &Call::out})
    REJECT(call([&](Call& k) { k.*p += 2; }), WUSH_EALIGN);
  REJECT(call([](Call& k) { k.t = 1; k.L += 1; }), WUSH_EALIGN);
  for (uintptr_t Call::*p : {&Call::p, &Call::o, &Call::rep, &Call::f, &Call::pr, &Call::bi, &Call::b, &Call::m})
    REJECT(call([&](Call& k) { k.out = k.*p; }), WUSH_EINVAL);
  REJECT(call([](Call& k) { k.out = k.L; k.ldo = 104; }), WUSH_EINVAL);  // in place, other strides
  REJECT(call([](Call& k) { k.out = k.L + 4; }), WUSH_EINVAL);
}

int main() {
  append();
  attention();
  lora();
  adjust();
  if (g_fail) {
    fprintf(stderr, "%d failures\n", g_fail);
    return 1;
  }
  printf("serving abi host checks passed\n");
  return 0;
}
