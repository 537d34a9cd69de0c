// torch_calls.cpp - the short way from torch tensors to the C ABI.
//
// A small call's time is the host's: with its argument checks in Python and
// its outputs allocated from there, a decode step of 10 us of GPU time took 24
// us.  This module does the same for a call that is as the documentation wants
// it: every tensor a contiguous CUDA tensor of the right type and shape on the
// current device, the workspace given, the current stream.  It checks exactly
// that, allocates the outputs and calls the library.  Anything else, an error
// of the library too, returns None, and the Python function of the same name
// runs its own checks, raises what is to be raised or makes the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "fa_kvcache.h"
#include "fa_prefix.h"
#include "fa_rope.h"
#include "fa_window.h"

namespace {

using at::ScalarType;
using at::Tensor;

// The library's functions, bound once by the Python module (which may have
// loaded the checked build).
struct {
  decltype(&fa_fwd_window) fwd_window;
  decltype(&fa_fwd_varlen_window) fwd_varlen_window;
  decltype(&fa_fwd_paged_window) fwd_paged_window;
  decltype(&fa_decode_paged_window) decode_paged_window;
  decltype(&fa_bwd_window) bwd_window;
  decltype(&fa_bwd_varlen_window) bwd_varlen_window;
  decltype(&fa_cache_append_fp8) cache_append_fp8;
  decltype(&fa_decode_paged_fp8) decode_paged_fp8;
  decltype(&fa_fwd_paged_fp8) fwd_paged_fp8;
  decltype(&fa_rope) rope;
  decltype(&fa_rope_bwd) rope_bwd;
  decltype(&fa_cache_append_rope) cache_append_rope;
  decltype(&fa_cache_append_rope_fp8) cache_append_rope_fp8;
  decltype(&fa_decode_paged_prefix) decode_paged_prefix;
} lib;

// One call's arguments.  Every getter clears `ok` when its argument is not as
// the call wants it; the caller looks at `ok` before it uses any of them.
struct Args {
  PyObject *const *v;
  int n;   // arguments
  int at = 0;
  bool ok = true;
  int dev = -1;

  PyObject *next() { return v[at++]; }

  // a plain contiguous CUDA tensor of this type and rank on the call's device
  // (that of the first tensor, which has to be current)
  const Tensor *tensor(ScalarType type, int dim) {
    PyObject *o = next();
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.scalar_type() != type || t.dim() != dim ||
        !t.is_contiguous())
      return fail();
    if (dev < 0) {
      dev = t.get_device();
      if (dev != c10::cuda::current_device()) return fail();
    }
    return t.get_device() == dev ? &t : fail();
  }
  const Tensor *tensor(ScalarType type, at::IntArrayRef shape) {
    const Tensor *t = tensor(type, static_cast<int>(shape.size()));
    return t && t->sizes() == shape ? t : fail();
  }
  // e4m3 codes, as such or as bytes
  const Tensor *codes(int dim) {
    PyObject *o = v[at];
    if (!THPVariable_CheckExact(o)) return fail();
    const ScalarType type = THPVariable_Unpack(o).scalar_type();
    return tensor(type == ScalarType::Byte ? type : ScalarType::Float8_e4m3fn, dim);
  }
  // a tensor that the call does not read, or None
  const Tensor *unread(ScalarType type, at::IntArrayRef shape) {
    if (v[at] != Py_None) return tensor(type, shape);
    ++at;
    return nullptr;
  }
  // the workspace, the last argument: asked for before there are outputs, so that
  // a call without one, which is made from Python, allocates nothing here
  const Tensor *workspace() {
    const int here = at;
    at = n - 1;
    const Tensor *t = tensor(ScalarType::Byte, 1);
    at = here;
    return t;
  }
  // the caller's tensor of this type and shape, or a new one
  Tensor output(ScalarType type, at::IntArrayRef shape) {
    if (v[at] == Py_None) {
      ++at;
      return ok ? at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev)) : Tensor();
    }
    const Tensor *t = tensor(type, shape);
    return t ? *t : Tensor();
  }
  int integer(long lo, long hi) {
    PyObject *o = next();
    if (!ok || !PyLong_CheckExact(o)) return fail_int();
    int over = 0;
    const long x = PyLong_AsLongAndOverflow(o, &over);
    if (over || x < lo || x > hi) return fail_int();
    return static_cast<int>(x);
  }
  // a softmax scale, or None for 1 / sqrt(d)
  float scale(int64_t d) {
    PyObject *o = next();
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    if (!PyFloat_CheckExact(o)) return ok = false, 0.f;
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
  }
  float number() {
    PyObject *o = next();
    if (!PyFloat_CheckExact(o)) return ok = false, 0.f;
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
  }
  bool flag() {
    PyObject *o = next();
    if (o != Py_True && o != Py_False) ok = false;
    return o == Py_True;
  }
  fa_stream_t stream() const {
    return reinterpret_cast<fa_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
  }

 private:
  const Tensor *fail() { return ok = false, nullptr; }
  int fail_int() { return ok = false, 0; }
};

const auto kBf16 = ScalarType::BFloat16;
const auto kInt = ScalarType::Int;
const auto kF32 = ScalarType::Float;

void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
int size(const Tensor *t, int i) { return static_cast<int>(t->size(i)); }
const int32_t *ints(const Tensor *t) { return static_cast<const int32_t *>(t->data_ptr()); }
float *floats(const Tensor *t) { return static_cast<float *>(t->data_ptr()); }
float *floats(const Tensor &t) { return static_cast<float *>(ptr(t)); }

// sizes that the C arguments take
bool small(const Tensor *t) {
  for (int64_t s : t->sizes())
    if (s > INT_MAX) return false;
  return true;
}

PyObject *wrap(const Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject *results(int rc, const Tensor &a, const Tensor &b) {
  if (rc != FA_OK) Py_RETURN_NONE;
  PyObject *x = wrap(a), *y = wrap(b);
  PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

PyObject *results(int rc, const Tensor &a, const Tensor &b, const Tensor &c) {
  if (rc != FA_OK) Py_RETURN_NONE;
  PyObject *x = wrap(a), *y = wrap(b), *z = wrap(c);
  PyObject *r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  Py_XDECREF(z);
  return r;
}

// the log-sum-exp of a call: the caller's, or a new one if it is wanted
Tensor lse_output(Args &a, at::IntArrayRef shape, bool want) {
  if (a.v[a.at] == Py_None && !want) return ++a.at, Tensor();
  return a.output(kF32, shape);
}

// The body of a call: `n` arguments, None where something is not as it should
// be or throws (the Python function then finds out what).
template <typename Body>
PyObject *call(PyObject *const *v, Py_ssize_t given, Py_ssize_t n, Body body) {
  if (given != n) Py_RETURN_NONE;
  try {
    Args a{v, static_cast<int>(n)};
    return body(a);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

#define NEED(condition)            \
  do {                             \
    if (!(condition)) Py_RETURN_NONE; \
  } while (0)

// q, k, v, window, sinks, scale, want_lse, out, lse
PyObject *fwd_window(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 9, [](Args &a) -> PyObject * {
    const Tensor *q = a.tensor(kBf16, 4), *k = a.tensor(kBf16, 4), *w = a.tensor(kBf16, 4);
    NEED(a.ok && small(q) && k->sizes() == w->sizes() && k->size(0) == q->size(0) &&
         k->size(1) == q->size(1) && k->size(3) == q->size(3) && k->size(2) <= INT_MAX);
    const int window = a.integer(1, INT_MAX), sinks = a.integer(0, INT_MAX);
    const float scale = a.scale(q->size(3));
    const bool want = a.flag();
    NEED(a.ok);
    const Tensor out = a.output(kBf16, q->sizes());
    const Tensor lse = lse_output(a, {q->size(0), q->size(2), q->size(1)}, want);
    NEED(a.ok);
    return results(lib.fwd_window(ptr(q), ptr(k), ptr(w), ptr(out), floats(lse), size(q, 0),
                                  size(q, 2), size(k, 2), size(q, 1), size(q, 3), scale, window,
                                  sinks, a.stream()),
                   out, lse);
  });
}

// q, k, v, cu_seqlens, max_seqlen, window, sinks, scale, want_lse, out, lse
PyObject *fwd_varlen_window(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 11, [](Args &a) -> PyObject * {
    const Tensor *q = a.tensor(kBf16, 3), *k = a.tensor(kBf16, 3), *w = a.tensor(kBf16, 3);
    const Tensor *cu = a.tensor(kInt, 1);
    NEED(a.ok && small(q) && k->sizes() == w->sizes() && k->size(0) == q->size(0) &&
         k->size(2) == q->size(2) && k->size(1) <= INT_MAX && cu->numel() >= 1 && small(cu));
    const int longest = a.integer(INT_MIN, INT_MAX);
    const int window = a.integer(1, INT_MAX), sinks = a.integer(0, INT_MAX);
    const float scale = a.scale(q->size(2));
    const bool want = a.flag();
    NEED(a.ok);
    const Tensor out = a.output(kBf16, q->sizes());
    const Tensor lse = lse_output(a, {q->size(1), q->size(0)}, want);
    NEED(a.ok);
    return results(lib.fwd_varlen_window(ptr(q), ptr(k), ptr(w), ptr(out), floats(lse), ints(cu),
                                         size(cu, 0) - 1, size(q, 0), longest, size(q, 1),
                                         size(k, 1), size(q, 2), scale, window, sinks, a.stream()),
                   out, lse);
  });
}

// q, k_pool, v_pool, block_table, ctx_lens, cu_seqlens_q, max_seqlen_q,
// max_ctx_len, window, sinks, scale, want_lse, out, lse
PyObject *fwd_paged_window(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 14, [](Args &a) -> PyObject * {
    const Tensor *q = a.tensor(kBf16, 3), *k = a.tensor(kBf16, 4), *w = a.tensor(kBf16, 4);
    const Tensor *table = a.tensor(kInt, 2), *ctx = a.tensor(kInt, 1), *cu = a.tensor(kInt, 1);
    NEED(a.ok && small(q) && small(k) && small(table) && k->sizes() == w->sizes() &&
         k->size(3) == q->size(2) && ctx->size(0) == table->size(0) &&
         cu->size(0) == table->size(0) + 1);
    const int longest = a.integer(INT_MIN, INT_MAX), most = a.integer(INT_MIN, INT_MAX);
    const int window = a.integer(1, INT_MAX), sinks = a.integer(0, INT_MAX);
    const float scale = a.scale(q->size(2));
    const bool want = a.flag();
    NEED(a.ok);
    const Tensor out = a.output(kBf16, q->sizes());
    const Tensor lse = lse_output(a, {q->size(1), q->size(0)}, want);
    NEED(a.ok);
    return results(
        lib.fwd_paged_window(ptr(q), ptr(k), ptr(w), ints(table), size(table, 1), ints(ctx),
                             ints(cu), size(table, 0), size(q, 0), longest, most, size(q, 1),
                             size(k, 2), size(q, 2), size(k, 1), size(k, 0), scale, window, sinks,
                             ptr(out), floats(lse), a.stream()),
        out, lse);
  });
}

// q, k_pool, v_pool, block_table, ctx_lens, max_ctx_len, window, sinks, scale,
// want_lse, out, lse, workspace
PyObject *decode_paged_window(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 13, [](Args &a) -> PyObject * {
    const Tensor *q = a.tensor(kBf16, 3), *k = a.tensor(kBf16, 4), *w = a.tensor(kBf16, 4);
    const Tensor *table = a.tensor(kInt, 2), *ctx = a.tensor(kInt, 1);
    NEED(a.ok && small(q) && small(k) && small(table) && k->sizes() == w->sizes() &&
         k->size(3) == q->size(2) && table->size(0) == q->size(0) && ctx->size(0) == q->size(0));
    const int most = a.integer(INT_MIN, INT_MAX);
    const int window = a.integer(1, INT_MAX), sinks = a.integer(0, INT_MAX);
    const float scale = a.scale(q->size(2));
    const bool want = a.flag();
    const Tensor *ws = a.workspace();
    NEED(a.ok);
    const Tensor out = a.output(kBf16, q->sizes());
    const Tensor lse = lse_output(a, {q->size(0), q->size(1)}, want);
    NEED(a.ok);
    return results(
        lib.decode_paged_window(ptr(q), ptr(k), ptr(w), ints(table), size(table, 1), ints(ctx),
                                most, size(q, 0), size(q, 1), size(k, 2), size(q, 2), size(k, 1),
                                size(k, 0), scale, window, sinks, ptr(out), floats(lse), ptr(ws),
                                static_cast<size_t>(ws->numel()), a.stream()),
        out, lse);
  });
}

// q, k, v, out, lse, dout, window, sinks, scale, dq, dk, dv, workspace
PyObject *bwd_window(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 13, [](Args &a) -> PyObject * {
    const Tensor *q = a.tensor(kBf16, 4), *k = a.tensor(kBf16, 4), *w = a.tensor(kBf16, 4);
    NEED(a.ok && small(q) && k->sizes() == w->sizes() && k->size(0) == q->size(0) &&
         k->size(1) == q->size(1) && k->size(3) == q->size(3) && k->size(2) <= INT_MAX);
    const Tensor *out = a.unread(kBf16, q->sizes());
    const Tensor *lse = a.tensor(kF32, {q->size(0), q->size(2), q->size(1)});
    const Tensor *dout = a.tensor(kBf16, q->sizes());
    const int window = a.integer(1, INT_MAX), sinks = a.integer(0, INT_MAX);
    const float scale = a.scale(q->size(3));
    const Tensor *ws = a.workspace();
    NEED(a.ok);
    const Tensor dq = a.output(kBf16, q->sizes()), dk = a.output(kBf16, k->sizes());
    const Tensor dv = a.output(kBf16, k->sizes());
    NEED(a.ok);
    return results(lib.bwd_window(ptr(q), ptr(k), ptr(w), ptr(out), floats(lse), ptr(dout), ptr(dq),
                                  ptr(dk), ptr(dv), size(q, 0), size(q, 2), size(k, 2), size(q, 1),
                                  size(q, 3), scale, window, sinks, ptr(ws),
                                  static_cast<size_t>(ws->numel()), a.stream()),
                   dq, dk, dv);
  });
}

// q, k, v, out, lse, dout, cu_seqlens, max_seqlen, window, sinks, scale, dq,
// dk, dv, workspace
PyObject *bwd_varlen_window(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 15, [](Args &a) -> PyObject * {
    const Tensor *q = a.tensor(kBf16, 3), *k = a.tensor(kBf16, 3), *w = a.tensor(kBf16, 3);
    NEED(a.ok && small(q) && k->sizes() == w->sizes() && k->size(0) == q->size(0) &&
         k->size(2) == q->size(2) && k->size(1) <= INT_MAX);
    const Tensor *out = a.unread(kBf16, q->sizes());
    const Tensor *lse = a.tensor(kF32, {q->size(1), q->size(0)});
    const Tensor *dout = a.tensor(kBf16, q->sizes()), *cu = a.tensor(kInt, 1);
    const int longest = a.integer(INT_MIN, INT_MAX);
    const int window = a.integer(1, INT_MAX), sinks = a.integer(0, INT_MAX);
    const float scale = a.scale(q->size(2));
    const Tensor *ws = a.workspace();
    NEED(a.ok && cu->numel() >= 1 && small(cu));
    const Tensor dq = a.output(kBf16, q->sizes()), dk = a.output(kBf16, k->sizes());
    const Tensor dv = a.output(kBf16, k->sizes());
    NEED(a.ok);
    return results(
        lib.bwd_varlen_window(ptr(q), ptr(k), ptr(w), ptr(out), floats(lse), ptr(dout), ptr(dq),
                              ptr(dk), ptr(dv), ints(cu), size(cu, 0) - 1, size(q, 0), longest,
                              size(q, 1), size(k, 1), size(q, 2), scale, window, sinks, ptr(ws),
                              static_cast<size_t>(ws->numel()), a.stream()),
        dq, dk, dv);
  });
}

// the 8-bit cache's tensors: k_pool, v_pool, k_scale, v_scale
struct Cache {
  const Tensor *k, *v, *k_scale, *v_scale;
  explicit Cache(Args &a) {
    k = a.codes(4);
    v = a.codes(4);
    k_scale = a.tensor(kF32, 2);
    v_scale = a.tensor(kF32, 2);
    if (!a.ok) return;
    a.ok = small(k) && k->scalar_type() == v->scalar_type() && k->sizes() == v->sizes() &&
           k_scale->size(0) == k->size(0) && k_scale->size(1) == k->size(2) &&
           v_scale->sizes() == k_scale->sizes();
  }
};

// a cache call's window and sinks: none, or a window with or without sinks
bool cache_window(Args &a, int &window, int &sinks) {
  window = a.integer(0, INT_MAX);
  sinks = a.integer(0, INT_MAX);
  return a.ok && (window > 0 || sinks == 0);
}

// rows [T, Hkv, d] whose tokens may lie apart
const Tensor *token_rows(Args &a, const Cache &c) {
  PyObject *o = a.next();
  if (!a.ok || !THPVariable_CheckExact(o)) return a.ok = false, nullptr;
  const Tensor &t = THPVariable_Unpack(o);
  a.ok = t.defined() && t.is_cuda() && t.get_device() == a.dev && t.scalar_type() == kBf16 &&
         t.dim() == 3 && t.numel() > 0 && t.size(0) <= INT_MAX && t.size(1) == c.k->size(2) &&
         t.size(2) == c.k->size(3) && t.stride(2) == 1 && t.stride(1) == t.size(2) &&
         (t.size(0) == 1 || (t.stride(0) >= t.size(1) * t.size(2) && t.stride(0) % 8 == 0));
  return a.ok ? &t : nullptr;
}

// k_pool, v_pool, k_scale, v_scale, k, v, block_table, ctx_lens, cu_seqlens,
// max_new
PyObject *cache_append_fp8(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 10, [](Args &a) -> PyObject * {
    const Cache c(a);
    const Tensor *k = token_rows(a, c), *w = token_rows(a, c);
    const Tensor *table = a.tensor(kInt, 2), *ctx = a.tensor(kInt, 1), *cu = a.tensor(kInt, 1);
    const int most = a.integer(INT_MIN, INT_MAX);
    NEED(a.ok && k->size(0) == w->size(0) && small(table) && ctx->size(0) == table->size(0) &&
         cu->size(0) == table->size(0) + 1);
    const int64_t row = k->size(1) * k->size(2);
    const int rc = lib.cache_append_fp8(
        ptr(k), ptr(w), k->size(0) == 1 ? row : k->stride(0), w->size(0) == 1 ? row : w->stride(0),
        ptr(c.k), ptr(c.v), floats(c.k_scale), floats(c.v_scale), ints(table), size(table, 1),
        ints(ctx), ints(cu), size(table, 0), size(k, 0), most, size(c.k, 2), size(c.k, 3),
        size(c.k, 1), size(c.k, 0), a.stream());
    NEED(rc == FA_OK);
    Py_RETURN_TRUE;
  });
}

// k_pool, v_pool, k_scale, v_scale, q, block_table, ctx_lens, max_ctx_len,
// window, sinks, scale, want_lse, out, lse, workspace
PyObject *decode_paged_fp8(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 15, [](Args &a) -> PyObject * {
    const Cache c(a);
    const Tensor *q = a.tensor(kBf16, 3), *table = a.tensor(kInt, 2), *ctx = a.tensor(kInt, 1);
    NEED(a.ok && small(q) && small(table) && c.k->size(3) == q->size(2) &&
         table->size(0) == q->size(0) && ctx->size(0) == q->size(0));
    const int most = a.integer(INT_MIN, INT_MAX);
    int window, sinks;
    NEED(cache_window(a, window, sinks));
    const float scale = a.scale(q->size(2));
    const bool want = a.flag();
    const Tensor *ws = a.workspace();
    NEED(a.ok);
    const Tensor out = a.output(kBf16, q->sizes());
    const Tensor lse = lse_output(a, {q->size(0), q->size(1)}, want);
    NEED(a.ok);
    return results(
        lib.decode_paged_fp8(ptr(q), ptr(c.k), ptr(c.v), floats(c.k_scale), floats(c.v_scale),
                             ints(table), size(table, 1), ints(ctx), most, size(q, 0), size(q, 1),
                             size(c.k, 2), size(q, 2), size(c.k, 1), size(c.k, 0), scale, window,
                             sinks, ptr(out), floats(lse), ptr(ws),
                             static_cast<size_t>(ws->numel()), a.stream()),
        out, lse);
  });
}

// k_pool, v_pool, k_scale, v_scale, q, block_table, ctx_lens, cu_seqlens_q,
// max_seqlen_q, max_ctx_len, window, sinks, scale, want_lse, out, lse
PyObject *fwd_paged_fp8(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 16, [](Args &a) -> PyObject * {
    const Cache c(a);
    const Tensor *q = a.tensor(kBf16, 3), *table = a.tensor(kInt, 2), *ctx = a.tensor(kInt, 1);
    const Tensor *cu = a.tensor(kInt, 1);
    NEED(a.ok && small(q) && small(table) && c.k->size(3) == q->size(2) &&
         ctx->size(0) == table->size(0) && cu->size(0) == table->size(0) + 1);
    const int longest = a.integer(INT_MIN, INT_MAX), most = a.integer(INT_MIN, INT_MAX);
    int window, sinks;
    NEED(cache_window(a, window, sinks));
    const float scale = a.scale(q->size(2));
    const bool want = a.flag();
    NEED(a.ok);
    const Tensor out = a.output(kBf16, q->sizes());
    const Tensor lse = lse_output(a, {q->size(1), q->size(0)}, want);
    NEED(a.ok);
    return results(
        lib.fwd_paged_fp8(ptr(q), ptr(c.k), ptr(c.v), floats(c.k_scale), floats(c.v_scale),
                          ints(table), size(table, 1), ints(ctx), ints(cu), size(table, 0),
                          size(q, 0), longest, most, size(q, 1), size(c.k, 2), size(q, 2),
                          size(c.k, 1), size(c.k, 0), scale, window, sinks, ptr(out), floats(lse),
                          a.stream()),
        out, lse);
  });
}

// Rows [lead.., heads, d] of bf16 whose tokens may lie apart (heads or d below
// 0: any), on the call's device; `stride` is their distance.
struct Rows {
  const Tensor *t = nullptr;
  int64_t stride = 0;
  Rows() = default;
  Rows(Args &a, at::IntArrayRef lead, int64_t heads, int64_t d) {
    PyObject *o = a.next();
    a.ok = a.ok && THPVariable_CheckExact(o);
    if (!a.ok) return;
    const Tensor &x = THPVariable_Unpack(o);
    const int64_t n = x.dim() - 2;
    a.ok = x.defined() && x.is_cuda() && x.scalar_type() == kBf16 && (n == 1 || n == 2) &&
           x.numel() > 0 && small(&x) && (heads < 0 || x.size(n) == heads) &&
           (d < 0 || x.size(n + 1) == d) && (lead.empty() || x.sizes().slice(0, n) == lead) &&
           x.stride(n + 1) == 1 && (x.size(n) == 1 || x.stride(n) == x.size(n + 1));
    if (!a.ok) return;
    if (a.dev < 0) {
      a.dev = x.get_device();
      a.ok = a.dev == c10::cuda::current_device();
    } else {
      a.ok = x.get_device() == a.dev;
    }
    const int64_t row = x.size(n) * x.size(n + 1);
    stride = x.size(n - 1) > 1 ? x.stride(n - 1) : n == 2 && x.size(0) > 1 ? x.stride(0) : row;
    a.ok = a.ok && stride >= row && stride % 8 == 0 &&
           (n == 1 || x.size(0) == 1 || x.stride(0) == stride * x.size(1));
    if (a.ok) t = &x;
  }
  int heads() const { return t ? static_cast<int>(t->size(t->dim() - 2)) : 0; }
};

// The caller's rows like x's, or new ones; `keep` holds them.
Rows rows_like(Args &a, const Rows &x, Tensor &keep) {
  Rows r;
  if (a.v[a.at] == Py_None) {
    ++a.at;
    if (!a.ok || !x.t) return r;
    keep = at::empty(x.t->sizes(), at::TensorOptions().dtype(kBf16).device(at::kCUDA, a.dev));
    r.stride = static_cast<int64_t>(x.heads()) * x.t->size(x.t->dim() - 1);
    r.t = &keep;
    return r;
  }
  if (!x.t) return a.ok = false, r;
  const int64_t n = x.t->dim() - 2;
  r = Rows(a, x.t->sizes().slice(0, n), x.t->size(n), x.t->size(n + 1));
  if (a.ok) keep = *r.t;
  return r;
}

// fp64 [rot_dim / 2]; rot is rot_dim
const double *frequencies(Args &a, int64_t d, int &rot) {
  const Tensor *t = a.tensor(ScalarType::Double, 1);
  rot = t && t->numel() > 0 && 2 * t->numel() <= d ? static_cast<int>(2 * t->numel()) : 0;
  a.ok = a.ok && rot > 0;
  return a.ok ? static_cast<const double *>(t->data_ptr()) : nullptr;
}

// q, k, inv_freq, positions, factor, interleaved, q_out, k_out
PyObject *turn(PyObject *const *v, Py_ssize_t given, decltype(&fa_rope) f) {
  return call(v, given, 8, [f](Args &a) -> PyObject * {
    const Rows q(a, {}, -1, -1);
    NEED(a.ok);
    const int64_t n = q.t->dim() - 2, d = q.t->size(n + 1);
    const at::IntArrayRef lead = q.t->sizes().slice(0, n);
    Rows k;
    if (a.v[a.at] == Py_None)
      ++a.at;
    else
      k = Rows(a, lead, -1, d);
    int rot;
    const double *freq = frequencies(a, d, rot);
    const Tensor *pos = a.unread(kInt, lead);
    const float factor = a.number();
    const bool interleaved = a.flag();
    const int64_t tokens = n == 2 ? lead[0] * lead[1] : lead[0];
    NEED(a.ok && tokens <= INT_MAX);
    Tensor keep_q, keep_k;
    const Rows qo = rows_like(a, q, keep_q), ko = rows_like(a, k, keep_k);
    NEED(a.ok);
    return results(f(ptr(q.t), ptr(k.t), q.stride, k.stride, ptr(qo.t), ptr(ko.t), qo.stride,
                     ko.stride, freq, rot, factor, interleaved, pos ? ints(pos) : nullptr,
                     static_cast<int>(lead[n - 1]), static_cast<int>(tokens), q.heads(), k.heads(),
                     static_cast<int>(d), a.stream()),
                   keep_q, keep_k);
  });
}
PyObject *rope(PyObject *, PyObject *const *v, Py_ssize_t given) { return turn(v, given, lib.rope); }
PyObject *rope_bwd(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return turn(v, given, lib.rope_bwd);
}

// What a write with rotation takes behind its pools: q, k, v, inv_freq,
// block_table, ctx_lens, cu_seqlens, max_new, factor, interleaved, q_out.
struct Write {
  Rows q, k, v, qo;
  Tensor keep;
  const double *freq = nullptr;
  int rot = 0, most = 0;
  const Tensor *table, *ctx, *cu;
  float factor = 1.f;
  bool interleaved = false;
  Write(Args &a, const Tensor *pool) {
    if (!a.ok) return;
    const int64_t Hkv = pool->size(2), d = pool->size(3);
    if (a.v[a.at] == Py_None)
      ++a.at;
    else
      q = Rows(a, {}, -1, d);
    k = Rows(a, {}, Hkv, d);
    v = Rows(a, {}, Hkv, d);
    if (!a.ok) return;
    a.ok = k.t->dim() == 3 && v.t->dim() == 3 && v.t->size(0) == k.t->size(0) &&
           (!q.t || (q.t->dim() == 3 && q.t->size(0) == k.t->size(0)));
    if (a.v[a.at] == Py_None)
      ++a.at;
    else
      freq = frequencies(a, d, rot);
    table = a.tensor(kInt, 2);
    ctx = a.tensor(kInt, 1);
    cu = a.tensor(kInt, 1);
    most = a.integer(INT_MIN, INT_MAX);
    factor = a.number();
    interleaved = a.flag();
    if (!a.ok) return;
    a.ok = small(table) && ctx->size(0) == table->size(0) && cu->size(0) == table->size(0) + 1;
    qo = rows_like(a, q, keep);
  }
  // the queries, or True where there are none
  PyObject *result(int rc) const {
    NEED(rc == FA_OK);
    if (!q.t) Py_RETURN_TRUE;
    return wrap(keep);
  }
};

// k_pool, v_pool, then a Write's
PyObject *cache_append_rope(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 13, [](Args &a) -> PyObject * {
    const Tensor *kp = a.tensor(kBf16, 4), *vp = a.tensor(kBf16, 4);
    NEED(a.ok && small(kp) && kp->sizes() == vp->sizes());
    const Write w(a, kp);
    NEED(a.ok);
    return w.result(lib.cache_append_rope(
        ptr(w.q.t), ptr(w.k.t), ptr(w.v.t), w.q.stride, w.k.stride, w.v.stride, ptr(w.qo.t),
        w.qo.stride, w.freq, w.rot, w.factor, w.interleaved, ptr(kp), ptr(vp), ints(w.table),
        size(w.table, 1), ints(w.ctx), ints(w.cu), size(w.table, 0), size(w.k.t, 0), w.most,
        w.q.heads(), size(kp, 2), size(kp, 3), size(kp, 1), size(kp, 0), a.stream()));
  });
}

// k_pool, v_pool, k_scale, v_scale, then a Write's
PyObject *cache_append_rope_fp8(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 15, [](Args &a) -> PyObject * {
    const Cache c(a);
    NEED(a.ok);
    const Write w(a, c.k);
    NEED(a.ok && w.freq);
    return w.result(lib.cache_append_rope_fp8(
        ptr(w.q.t), ptr(w.k.t), ptr(w.v.t), w.q.stride, w.k.stride, w.v.stride, ptr(w.qo.t),
        w.qo.stride, w.freq, w.rot, w.factor, w.interleaved, ptr(c.k), ptr(c.v), floats(c.k_scale),
        floats(c.v_scale), ints(w.table), size(w.table, 1), ints(w.ctx), ints(w.cu),
        size(w.table, 0), size(w.k.t, 0), w.most, w.q.heads(), size(c.k, 2), size(c.k, 3),
        size(c.k, 1), size(c.k, 0), a.stream()));
  });
}

// q, k_pool, v_pool, block_table, ctx_lens, cu_groups, prefix_lens,
// max_prefix_len, max_own_len, scale, want_lse, out, lse, workspace
PyObject *decode_paged_prefix(PyObject *, PyObject *const *v, Py_ssize_t given) {
  return call(v, given, 14, [](Args &a) -> PyObject * {
    const Tensor *q = a.tensor(kBf16, 3), *k = a.tensor(kBf16, 4), *w = a.tensor(kBf16, 4);
    const Tensor *table = a.tensor(kInt, 2), *ctx = a.tensor(kInt, 1);
    const Tensor *cu = a.tensor(kInt, 1), *pre = a.tensor(kInt, 1);
    NEED(a.ok && small(q) && small(k) && small(table) && small(pre) && k->sizes() == w->sizes() &&
         k->size(3) == q->size(2) && table->size(0) == q->size(0) && ctx->size(0) == q->size(0) &&
         cu->size(0) == pre->size(0) + 1);
    const int most = a.integer(INT_MIN, INT_MAX), most_own = a.integer(INT_MIN, INT_MAX);
    const float scale = a.scale(q->size(2));
    const bool want = a.flag();
    const Tensor *ws = a.workspace();
    NEED(a.ok);
    const Tensor out = a.output(kBf16, q->sizes());
    const Tensor lse = lse_output(a, {q->size(0), q->size(1)}, want);
    NEED(a.ok);
    return results(
        lib.decode_paged_prefix(ptr(q), ptr(k), ptr(w), ints(table), size(table, 1), ints(ctx),
                                ints(cu), ints(pre), size(pre, 0), most, most_own, size(q, 0),
                                size(q, 1), size(k, 2), size(q, 2), size(k, 1), size(k, 0), scale,
                                ptr(out), floats(lse), ptr(ws), static_cast<size_t>(ws->numel()),
                                a.stream()),
        out, lse);
  });
}

// the library's functions' addresses, in the order of `lib`
PyObject *bind(PyObject *, PyObject *const *v, Py_ssize_t given) {
  constexpr Py_ssize_t kCalls = sizeof(lib) / sizeof(void *);
  if (given != kCalls) {
    PyErr_SetString(PyExc_TypeError, "bind takes one address per call");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < kCalls; ++i) {
    void *address = PyLong_AsVoidPtr(v[i]);
    if (address == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
    reinterpret_cast<void **>(&lib)[i] = address;
  }
  Py_RETURN_NONE;
}

#define METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),
                         METHOD(fwd_window),
                         METHOD(fwd_varlen_window),
                         METHOD(fwd_paged_window),
                         METHOD(decode_paged_window),
                         METHOD(bwd_window),
                         METHOD(bwd_varlen_window),
                         METHOD(cache_append_fp8),
                         METHOD(decode_paged_fp8),
                         METHOD(fwd_paged_fp8),
                         METHOD(rope),
                         METHOD(rope_bwd),
                         METHOD(cache_append_rope),
                         METHOD(cache_append_rope_fp8),
                         METHOD(decode_paged_prefix),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
