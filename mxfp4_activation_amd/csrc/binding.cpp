// The wrappers of the entries around the 4-bit products (kv4.py, decode.py) and of dequant, by
// which a cache is read back, in native code, for the calls on one token, whose time is the host's: the same checks,
// outputs and workspaces, in about a microsecond where Python takes ten.
//
// Every function returns its result; an int, the status of a library call that
// failed; or None for a call that is not plainly right, which the Python wrapper then takes
// and refuses with its reasons.  The library's entries come in by address, from the one
// that Python has loaded.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/wush.h"

namespace {

decltype(&wush_kv4_append) f_append;
decltype(&wush_kv4_attention) f_attention;
decltype(&wush_kv4_attention_workspace) f_attention_workspace;
decltype(&wush_linear_w4_lora) f_lora;
decltype(&wush_linear_w4_lora_workspace) f_lora_workspace;
decltype(&wush_adjust_logits) f_adjust;
decltype(&wush_dequant) f_dequant;

using at::ScalarType;
using at::Tensor;
typedef std::initializer_list<int64_t> Sizes;

// What a call has come to: plain tensors of the current device, or not.
struct Call {
  int device = -1;
  bool ok = true;

  // A plain tensor, or null.
  const Tensor* tensor(PyObject* o) {
    if (ok && !THPVariable_CheckExact(o)) ok = false;
    return ok ? &THPVariable_Unpack(o) : nullptr;
  }
  // The call's first tensor settles its device.
  const Tensor* first(PyObject* o, ScalarType type, int64_t dim) {
    const Tensor* t = tensor(o);
    if (!ok) return nullptr;
    if (!t->is_cuda() || t->scalar_type() != type || t->dim() != dim) {
      ok = false;
      return nullptr;
    }
    device = t->get_device();
    if (device != c10::hip::current_device()) ok = false;
    return ok ? t : nullptr;
  }
  void* address(PyObject* o, ScalarType type, Sizes sizes) {
    const Tensor* t = tensor(o);
    if (!ok) return nullptr;
    if (t->scalar_type() != type || !t->is_cuda() || t->get_device() != device || t->sizes() != at::IntArrayRef(sizes) ||
        !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* maybe(PyObject* o, ScalarType type, Sizes sizes) { return o == Py_None ? nullptr : address(o, type, sizes); }
  // A tensor scale: one element of any shape, for NVFP4.
  const float* global(PyObject* o, int fmt) {
    if (fmt != 1) return nullptr;
    const Tensor* t = tensor(o);
    if (ok && (t->scalar_type() != at::kFloat || t->numel() != 1 || !t->is_cuda() || t->get_device() != device)) ok = false;
    return ok ? static_cast<const float*>(t->data_ptr()) : nullptr;
  }
  int64_t integer(PyObject* o) {
    const int64_t v = PyLong_CheckExact(o) ? PyLong_AsLongLong(o) : (ok = false, 0);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int format(PyObject* o) {
    if (PyUnicode_Check(o)) {
      if (PyUnicode_CompareWithASCIIString(o, "mxfp4") == 0) return 0;
      if (PyUnicode_CompareWithASCIIString(o, "nvfp4") == 0) return 1;
      if (PyUnicode_CompareWithASCIIString(o, "int4") == 0) return 2;
    }
    ok = false;
    return 0;
  }
};

int group_of(int fmt) { return fmt == 1 ? 16 : 32; }
ScalarType scale_type(int fmt) { return fmt == 2 ? at::kHalf : at::kByte; }
hipStream_t stream_of(int device) { return c10::hip::getCurrentHIPStream(device).stream(); }

Tensor workspace(int64_t n, const Tensor& like) { return n ? at::empty({n}, like.options().dtype(at::kByte)) : Tensor(); }
void* data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// f() without Python's lock, which other threads may want: allocations and launches can wait for
// the device, and for a host callback that needs the lock.
template <typename F>
auto unlocked(F f) {
  struct Lock {
    PyThreadState* state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return f();
}

PyObject* answer(wush_status st, const Tensor& t) {
  if (st != WUSH_OK) return PyLong_FromLong(st);
  return THPVariable_Wrap(t);
}
PyObject* answer(wush_status st, PyObject* o) {
  if (st != WUSH_OK) return PyLong_FromLong(st);
  Py_INCREF(o);
  return o;
}

// Rows [heads][D], contiguous, of a bf16 tensor [n, heads, D].
bool plain_rows(const Tensor& t) {
  return t.size(0) == 0 || ((t.size(2) == 1 || t.stride(2) == 1) && (t.size(1) == 1 || t.stride(1) == t.size(2)));
}

struct Cache {
  void *kc, *ks, *vc, *vs;
  const float *kg, *vg;
  int64_t pages, heads, page;
};
Cache cache_of(Call& c, int fmt, int64_t D, PyObject* const* a) {
  Cache k{};
  const Tensor* codes = c.tensor(a[0]);
  if (!c.ok || codes->dim() != 4) {
    c.ok = false;
    return k;
  }
  k.pages = codes->size(0);
  k.heads = codes->size(1);
  k.page = codes->size(2);
  const int64_t G = group_of(fmt);
  k.kc = c.address(a[0], at::kByte, {k.pages, k.heads, k.page, D / 2});
  k.ks = c.address(a[1], scale_type(fmt), {k.pages, k.heads, k.page, D / G});
  k.vc = c.address(a[2], at::kByte, {k.pages, k.heads, k.page, D / 2});
  k.vs = c.address(a[3], scale_type(fmt), {k.pages, k.heads, k.page, D / G});
  k.kg = c.global(a[4], fmt);
  k.vg = c.global(a[5], fmt);
  return k;
}

// (fmt, k, v, k_codes, k_scales, v_codes, v_scales, k_global, v_global, slots, T_k, T_v)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t count) {
  Call c;
  if (count != 12) Py_RETURN_NONE;
  const int fmt = c.format(a[0]);
  const Tensor* k = c.first(a[1], at::kBFloat16, 3);
  const Tensor* v = c.tensor(a[2]);
  if (!c.ok || v->scalar_type() != at::kBFloat16 || v->sizes() != k->sizes() || !v->is_cuda() || v->get_device() != c.device ||
      !plain_rows(*k) || !plain_rows(*v))
    Py_RETURN_NONE;
  const int64_t n = k->size(0), heads = k->size(1), D = k->size(2), G = group_of(fmt);
  const Cache e = cache_of(c, fmt, D, a + 3);
  const void* slots = c.address(a[9], at::kLong, {n});
  const void* tk = c.maybe(a[10], at::kBFloat16, {heads, D / G, G, G});
  const void* tv = c.maybe(a[11], at::kBFloat16, {heads, D / G, G, G});
  if (!c.ok || e.heads != heads) Py_RETURN_NONE;
  const wush_status st = unlocked([&] {
    return f_append(fmt, k->data_ptr(), k->stride(0), v->data_ptr(), v->stride(0), tk, tv, static_cast<const int64_t*>(slots), n,
                    heads, D, e.page, e.pages, e.kc, e.ks, e.kg, e.vc, e.vs, e.vg, stream_of(c.device));
  });
  return PyLong_FromLong(st);
}

// (fmt, q, k_codes, k_scales, v_codes, v_scales, k_global, v_global, block_table, lengths, q_start, scale, window, T_q, out)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t count) {
  Call c;
  if (count != 15) Py_RETURN_NONE;
  const int fmt = c.format(a[0]);
  const Tensor* q = c.first(a[1], at::kBFloat16, 3);
  if (!c.ok || !plain_rows(*q)) Py_RETURN_NONE;
  const int64_t n = q->size(0), hq = q->size(1), D = q->size(2), G = group_of(fmt);
  const Cache e = cache_of(c, fmt, D, a + 2);
  const Tensor* table = c.tensor(a[8]);
  if (!c.ok || table->scalar_type() != at::kInt || table->dim() != 2 || !table->is_cuda() || table->get_device() != c.device ||
      (table->size(1) > 1 && table->stride(1) != 1))
    Py_RETURN_NONE;
  const int64_t B = table->size(0), width = table->size(1);
  const void* lengths = c.address(a[9], at::kInt, {B});
  const void* start = c.maybe(a[10], at::kInt, {B + 1});
  double scale = 0.0;
  if (a[11] != Py_None) {
    if (!PyFloat_CheckExact(a[11])) Py_RETURN_NONE;
    scale = PyFloat_AS_DOUBLE(a[11]);
  } else {
    scale = D == 64 ? 0.125 : D == 256 ? 0.0625 : 0.08838834764831845;
  }
  const int64_t window = c.integer(a[12]);
  const void* T = c.maybe(a[13], at::kBFloat16, {e.heads, D / G, G, G});
  void* given = c.maybe(a[14], at::kBFloat16, {n, hq, D});
  if (!c.ok || (D != 64 && D != 128 && D != 256)) Py_RETURN_NONE;
  const int64_t nw = f_attention_workspace(fmt, B, n, hq, e.heads, D, e.page, width);
  Tensor out;
  const wush_status st = unlocked([&] {
    if (!given) out = at::empty({n, hq, D}, q->options());
    const Tensor ws = workspace(nw, *q);
    return f_attention(fmt, q->data_ptr(), q->stride(0), T, e.kc, e.ks, e.kg, e.vc, e.vs, e.vg,
                       static_cast<const int32_t*>(table->data_ptr()), table->stride(0), width, static_cast<const int32_t*>(lengths),
                       static_cast<const int32_t*>(start), B, n, hq, e.heads, D, e.page, e.pages, (float)scale, window,
                       given ? given : out.data_ptr(), data(ws), nw, stream_of(c.device));
  });
  return given ? answer(st, a[14]) : answer(st, out);
}

// (fmt, x, codes, scales, A, B, adapter scale, ids, T, global_scale, fp32 result, out)
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t count) {
  Call c;
  if (count != 12) Py_RETURN_NONE;
  const int fmt = c.format(a[0]);
  const Tensor* x = c.first(a[1], at::kBFloat16, 2);
  const Tensor* codes = c.tensor(a[2]);
  const Tensor* A = c.tensor(a[4]);
  if (!c.ok || codes->dim() != 2 || A->dim() != 3 || (x->size(1) > 1 && x->stride(1) != 1)) Py_RETURN_NONE;
  const int64_t M = x->size(0), K = x->size(1), N = codes->size(0), E = A->size(0), rank = A->size(1), G = group_of(fmt);
  const void* pc = c.address(a[2], at::kByte, {N, K / 2});
  const void* ps = c.address(a[3], scale_type(fmt), {N, K / G});
  const void* pa = c.address(a[4], at::kBFloat16, {E, rank, K});
  const void* pb = c.address(a[5], at::kBFloat16, {E, N, rank});
  const void* pe = c.maybe(a[6], at::kFloat, {E});
  const void* ids = c.address(a[7], at::kInt, {M});
  const void* T = c.maybe(a[8], at::kBFloat16, {K / G, G, G});
  const float* g = c.global(a[9], fmt);
  const bool f32 = a[10] == Py_True;
  const ScalarType type = f32 ? at::kFloat : at::kBFloat16;
  void* given = c.maybe(a[11], type, {M, N});
  if (!c.ok) Py_RETURN_NONE;
  const int ot = f32 ? WUSH_OUT_F32 : WUSH_OUT_BF16;
  const int64_t nw = f_lora_workspace(M, N, K, rank, T != nullptr, ot);
  Tensor out;
  const wush_status st = unlocked([&] {
    if (!given) out = at::empty({M, N}, x->options().dtype(type));
    const Tensor ws = workspace(nw, *x);
    return f_lora(fmt, x->data_ptr(), x->stride(0), T, pc, ps, g, pa, pb, static_cast<const float*>(pe),
                  static_cast<const int32_t*>(ids), E, rank, M, N, K, given ? given : out.data_ptr(), ot, data(ws), nw,
                  stream_of(c.device));
  });
  return given ? answer(st, a[11]) : answer(st, out);
}

// (logits, prompt, output, repetition, frequency, presence, bias_ids, bias, allowed, out)
PyObject* adjust(PyObject*, PyObject* const* a, Py_ssize_t count) {
  Call c;
  if (count != 10) Py_RETURN_NONE;
  const Tensor* l = c.tensor(a[0]);
  if (!c.ok) Py_RETURN_NONE;
  const ScalarType type = l->scalar_type();
  const int lt = type == at::kFloat ? WUSH_LOGITS_F32 : type == at::kBFloat16 ? WUSH_LOGITS_BF16 : WUSH_LOGITS_F16;
  if ((lt == WUSH_LOGITS_F16 && type != at::kHalf) || !c.first(a[0], type, 2)) Py_RETURN_NONE;
  const int64_t R = l->size(0), V = l->size(1);
  if (V > 1 && l->stride(1) != 1) Py_RETURN_NONE;
  const auto list = [&](PyObject* o, int64_t& n) -> const int32_t* {
    n = 0;
    if (o == Py_None) return nullptr;
    const Tensor* t = c.tensor(o);
    if (!c.ok || t->dim() != 2) {
      c.ok = false;
      return nullptr;
    }
    n = t->size(1);
    return static_cast<const int32_t*>(c.address(o, at::kInt, {R, n}));
  };
  int64_t np, no, nb;
  const int32_t *p = list(a[1], np), *o = list(a[2], no), *bi = list(a[6], nb);
  const void* rep = c.maybe(a[3], at::kFloat, {R});
  const void* freq = c.maybe(a[4], at::kFloat, {R});
  const void* pres = c.maybe(a[5], at::kFloat, {R});
  const void* b = c.maybe(a[7], at::kFloat, {R, nb});
  const void* m = c.maybe(a[8], at::kInt, {R, (V + 31) / 32});
  if (!c.ok || (a[6] == Py_None) != (a[7] == Py_None)) Py_RETURN_NONE;
  const Tensor* given = a[9] == Py_None ? nullptr : c.tensor(a[9]);
  if (!c.ok || (given && (given->scalar_type() != type || given->sizes() != l->sizes() || !given->is_cuda() ||
                          given->get_device() != c.device || (V > 1 && given->stride(1) != 1))))
    Py_RETURN_NONE;
  Tensor fresh;
  const wush_status st = unlocked([&] {
    if (!given) fresh = at::empty({R, V}, l->options());
    const Tensor& out = given ? *given : fresh;
    return f_adjust(l->data_ptr(), lt, l->stride(0), R, V, p, np, o, no, static_cast<const float*>(rep),
                    static_cast<const float*>(freq), static_cast<const float*>(pres), bi, static_cast<const float*>(b), nb,
                    static_cast<const int32_t*>(m), out.data_ptr(), out.stride(0), stream_of(c.device));
  });
  return given ? answer(st, a[9]) : answer(st, fresh);
}

// (fmt, codes, scales, global_scale, out)
PyObject* dequant(PyObject*, PyObject* const* a, Py_ssize_t count) {
  Call c;
  if (count != 5) Py_RETURN_NONE;
  const int fmt = c.format(a[0]);
  const Tensor* codes = c.first(a[1], at::kByte, 2);
  if (!c.ok || !codes->is_contiguous()) Py_RETURN_NONE;
  const int64_t M = codes->size(0), K = codes->size(1) * 2;
  const void* scales = c.address(a[2], scale_type(fmt), {M, K / group_of(fmt)});
  const float* g = c.global(a[3], fmt);
  void* given = c.maybe(a[4], at::kFloat, {M, K});
  if (!c.ok) Py_RETURN_NONE;
  Tensor out;
  const wush_status st = unlocked([&] {
    if (!given) out = at::empty({M, K}, codes->options().dtype(at::kFloat));
    return f_dequant(fmt, codes->data_ptr(), scales, g, M, K, static_cast<float*>(given ? given : out.data_ptr()),
                     stream_of(c.device));
  });
  return given ? answer(st, a[4]) : answer(st, out);
}

// Functions above, with C++ exceptions (an allocation that fails, say) as Python's.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  return F(self, a, count);
  END_HANDLE_TH_ERRORS
}

// bind({name: address}) of the library's entries.
PyObject* bind(PyObject*, PyObject* entries) {
  const auto take = [&](const char* name, auto& f) {
    PyObject* v = PyDict_GetItemString(entries, name);
    void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
    if (!p && !PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "%s", name);
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p);
    return p != nullptr;
  };
  if (take("wush_kv4_append", f_append) && take("wush_kv4_attention", f_attention) &&
      take("wush_kv4_attention_workspace", f_attention_workspace) && take("wush_linear_w4_lora", f_lora) &&
      take("wush_linear_w4_lora_workspace", f_lora_workspace) && take("wush_adjust_logits", f_adjust) &&
      take("wush_dequant", f_dequant))
    Py_RETURN_NONE;
  return nullptr;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(append), FAST(attention), FAST(lora), FAST(adjust), FAST(dequant),
                         {"bind", bind, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// Its `built_for` is what _lib.built_for() gave when it was compiled.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
