// The calls of ops.py for ordinary arguments, as a CPython extension: the checks of the Python
// functions over at::Tensor, and the C entry point.  A call that is not plainly in order (a check that fails, a
// tensor of another device, a refusal of the entry point) returns None with nothing
// enqueued; the Python function then repeats it with its own checks and messages.  A launch
// that fails raises MokError here: part of the call may be enqueued, so it is not repeated.
//
// The entry points' addresses come from the library that _lib.py has loaded (bind), the
// current device and stream from torch's own functions.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <vector>

#include "../../include/mok.h"

namespace {

struct Entries {
  decltype(&mok_permute) permute;
  decltype(&mok_permute_bwd) permute_bwd;
  decltype(&mok_unpermute) unpermute;
  decltype(&mok_unpermute_bwd) unpermute_bwd;
  decltype(&mok_quantize_mx4) quantize_mx4;
  decltype(&mok_dequantize_mx4) dequantize_mx4;
  decltype(&mok_grouped_mx4) grouped_mx4;
} g_fn;
struct MoreEntries {
  decltype(&mok_grouped_mm) grouped_mm;
  decltype(&mok_grouped_mm_bwd_rows) grouped_mm_bwd_rows;
  decltype(&mok_grouped_mm_bwd_weights) grouped_mm_bwd_weights;
  decltype(&mok_quantize_mx8) quantize_mx8;
  decltype(&mok_dequantize_mx8) dequantize_mx8;
  decltype(&mok_swiglu_mx8) swiglu_mx8;
  decltype(&mok_swiglu_mx8_bwd) swiglu_mx8_bwd;
  decltype(&mok_grouped_mm_workspace) grouped_mm_workspace;
} g_more;  // null until bind_more
PyObject* g_device = nullptr;  // torch: the current device's index
PyObject* g_stream = nullptr;  // torch: the current raw stream of a device index

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A call's device and checks; ok turns false with the first that fails.
struct Call {
  bool ok = true;
  c10::Device dev{c10::kCPU};

  explicit Call(const at::Tensor* t) {
    if (!t || !t->is_cuda()) {
      ok = false;
      return;
    }
    dev = t->device();
  }
  bool on_device(const at::Tensor* t) {
    return ok = ok && t && t->device() == dev && t->layout() == c10::kStrided;
  }
  // The stream, where the tensors' device is the current one.
  bool stream(void** st) {
    if (!ok) return false;
    PyObject* d = PyObject_CallNoArgs(g_device);
    const long index = d ? PyLong_AsLong(d) : -1;
    PyObject* s = d && index == dev.index() ? PyObject_CallOneArg(g_stream, d) : nullptr;
    Py_XDECREF(d);
    if (s) *st = PyLong_AsVoidPtr(s);
    ok = s != nullptr && !PyErr_Occurred();
    Py_XDECREF(s);
    PyErr_Clear();
    return ok;
  }
};

struct Span {
  const char *lo, *hi;
};
Span span(const at::Tensor& t, int64_t elems) {
  const char* p = static_cast<const char*>(t.data_ptr());
  return {p, p + elems * t.element_size()};
}
bool apart(const Span& a, std::initializer_list<Span> others) {
  for (const Span& b : others)
    if (a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi) return false;
  return true;
}

struct Matrix {
  void* p;
  int64_t rows, cols, ld;
  Span s;
};
// A matrix with contiguous rows; of an output they may not overlap.
bool matrix(Call& c, const at::Tensor* t, Matrix* m, bool write) {
  if (!c.on_device(t) || t->dim() != 2) return c.ok = false;
  m->rows = t->size(0);
  m->cols = t->size(1);
  m->ld = m->rows <= 1 ? m->cols : t->stride(0);
  // (the entry points take the sizes of a row as 32 bits)
  if (m->cols > INT32_MAX) return c.ok = false;
  if ((m->rows > 0 && m->cols > 1 && t->stride(1) != 1) || (write && m->ld < m->cols) || m->ld < 0) return c.ok = false;
  m->s = span(*t, m->rows && m->cols ? (m->rows - 1) * m->ld + m->cols : 0);
  m->p = t->data_ptr();
  return true;
}
// A tensor [..., cols] as the matrix of its rows: a matrix, or contiguous.
bool rows_of(Call& c, const at::Tensor* t, Matrix* m, bool write) {
  if (t && t->dim() == 2) return matrix(c, t, m, write);
  if (!c.on_device(t) || t->dim() < 1 || !t->is_contiguous() || t->size(-1) == 0 ||
      t->size(-1) > INT32_MAX)
    return c.ok = false;
  m->cols = m->ld = t->size(-1);
  m->rows = t->numel() / m->cols;
  m->s = span(*t, t->numel());
  m->p = t->data_ptr();
  return true;
}
bool flat(Call& c, const at::Tensor* t, at::IntArrayRef shape, c10::ScalarType type, Span* s) {
  if (!c.on_device(t) || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous())
    return c.ok = false;
  *s = span(*t, t->numel());
  return true;
}
int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOK_TYPE_BF16;
    case at::kHalf: return MOK_TYPE_FP16;
    case at::kFloat: return MOK_TYPE_FP32;
    default: return -1;
  }
}
template <typename T>
T* at_ptr(const Span& s) { return reinterpret_cast<T*>(const_cast<char*>(s.lo)); }

PyObject* none() { Py_RETURN_NONE; }
// What a call gives that entry point `fn` returned `code` for, other than MOK_OK.
PyObject* refused(const char* fn, mok_status_t code) {
  if (code != MOK_E_LAUNCH) return none();
  PyObject* lib = PyImport_ImportModule("mixture_experts_layer_mok_amd._lib");
  PyObject* cls = lib ? PyObject_GetAttrString(lib, "MokError") : nullptr;
  PyObject* err = cls ? PyObject_CallFunction(cls, "si", fn, int(code)) : nullptr;
  if (err) PyErr_SetObject(cls, err);
  Py_XDECREF(err);
  Py_XDECREF(cls);
  Py_XDECREF(lib);
  return nullptr;
}
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}
// A graph that saved an output passed in finds it changed.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
// The output passed in (borrowed) or, for None, one made here; null where it is neither.
struct Output {
  at::Tensor made;
  const at::Tensor* t = nullptr;
  PyObject* o;
  template <typename F>
  Output(PyObject* given, F make) : o(given) {
    if (given == Py_None) {
      made = make();
      t = &made;
    } else {
      t = tensor(given);
    }
  }
  PyObject* result() const {
    if (o == Py_None) return THPVariable_Wrap(made);
    written(*t);
    return same(o);
  }
};

PyObject* do_permute(PyObject* const* a) {
  const at::Tensor *x = tensor(a[0]), *pos = tensor(a[1]), *out = tensor(a[2]);
  Call c(x);
  Matrix mx, mo, mp;
  if (!matrix(c, x, &mx, false) || !matrix(c, out, &mo, true) || !matrix(c, pos, &mp, false)) return none();
  const int ty = type_of(*x);
  void* st;
  if (ty < 0 || out->scalar_type() != x->scalar_type() || pos->scalar_type() != at::kInt ||
      !pos->is_contiguous() || mp.rows != mx.rows || mo.cols != mx.cols || !apart(mo.s, {mx.s, mp.s}) ||
      !c.stream(&st))
    return none();
  const auto s = g_fn.permute(ty, mx.p, mx.ld, at_ptr<int32_t>(mp.s), mp.rows, int32_t(mp.cols),
                              int32_t(mx.cols), mo.p, mo.ld, mo.rows, st);
  if (s != MOK_OK) return refused("mok_permute", s);
  written(*out);
  return same(a[2]);
}

// rows, pos, weights (None: without), out
PyObject* do_sum(PyObject* const* a, bool weighted) {
  const at::Tensor *rows = tensor(a[0]), *pos = tensor(a[1]), *w = weighted ? tensor(a[2]) : nullptr;
  Call c(rows);
  Matrix mr, mp, mo;
  Span sw = {nullptr, nullptr};
  if (!matrix(c, rows, &mr, false) || !matrix(c, pos, &mp, false)) return none();
  const int ty = type_of(*rows);
  if (ty < 0 || pos->scalar_type() != at::kInt || !pos->is_contiguous() ||
      (weighted && !flat(c, w, {mp.rows, mp.cols}, at::kFloat, &sw)))
    return none();
  void* st;
  if (!c.stream(&st)) return none();
  Output out(a[3], [&] { return at::empty({mp.rows, mr.cols}, rows->options().requires_grad(false)); });
  if (!matrix(c, out.t, &mo, true) || out.t->scalar_type() != rows->scalar_type() || mo.rows != mp.rows ||
      mo.cols != mr.cols || !apart(mo.s, {mr.s, mp.s, sw}))
    return none();
  const auto s = weighted ? g_fn.unpermute(ty, mr.p, mr.ld, mr.rows, at_ptr<int32_t>(mp.s), at_ptr<float>(sw),
                                           mp.rows, int32_t(mp.cols), int32_t(mr.cols), mo.p, mo.ld, st)
                          : g_fn.permute_bwd(ty, mr.p, mr.ld, mr.rows, at_ptr<int32_t>(mp.s), mp.rows,
                                             int32_t(mp.cols), int32_t(mr.cols), mo.p, mo.ld, st);
  return s == MOK_OK ? out.result() : refused(weighted ? "mok_unpermute" : "mok_permute_bwd", s);
}

// dy, rows, pos, weights, d_rows, d_weights
PyObject* do_unpermute_bwd(PyObject* const* a) {
  const at::Tensor *dy = tensor(a[0]), *rows = tensor(a[1]), *pos = tensor(a[2]), *w = tensor(a[3]),
                   *d_rows = tensor(a[4]);
  Call c(rows);
  Matrix my, mr, mp, md;
  Span sw, sdw;
  if (!matrix(c, rows, &mr, false) || !matrix(c, dy, &my, false) || !matrix(c, pos, &mp, false) ||
      !matrix(c, d_rows, &md, true) || !flat(c, w, {mp.rows, mp.cols}, at::kFloat, &sw))
    return none();
  const int ty = type_of(*rows);
  void* st;
  if (ty < 0 || dy->scalar_type() != rows->scalar_type() || d_rows->scalar_type() != rows->scalar_type() ||
      pos->scalar_type() != at::kInt || !pos->is_contiguous() || my.rows != mp.rows || my.cols != mr.cols ||
      md.rows != mr.rows || md.cols != mr.cols || !c.stream(&st))
    return none();
  Output dw(a[5], [&] { return at::empty({mp.rows, mp.cols}, w->options().requires_grad(false)); });
  if (!flat(c, dw.t, {mp.rows, mp.cols}, at::kFloat, &sdw) || !apart(md.s, {my.s, mr.s, mp.s, sw}) ||
      !apart(sdw, {my.s, mr.s, mp.s, sw, md.s}))
    return none();
  const auto s = g_fn.unpermute_bwd(ty, my.p, my.ld, mr.p, mr.ld, mr.rows, at_ptr<int32_t>(mp.s),
                                    at_ptr<float>(sw), mp.rows, int32_t(mp.cols), int32_t(mr.cols), md.p, md.ld,
                                    at_ptr<float>(sdw), st);
  if (s != MOK_OK) return refused("mok_unpermute_bwd", s);
  written(*d_rows);
  PyObject* r = dw.result();
  return r ? Py_BuildValue("(ON)", a[4], r) : nullptr;
}

// The element type that a torch dtype names; Undefined where it is none.
at::ScalarType dtype_of(PyObject* o) {
  return THPDtype_Check(o) ? reinterpret_cast<THPDtype*>(o)->scalar_type : at::ScalarType::Undefined;
}

std::vector<int64_t> with_last(const at::Tensor& t, int64_t last) {
  std::vector<int64_t> s = t.sizes().vec();
  s.back() = last;
  return s;
}

// src, codes, scales; PER: elements a byte of codes
template <int PER>
PyObject* do_quantize(PyObject* const* a) {
  const auto fn = PER == 2 ? g_fn.quantize_mx4 : g_more.quantize_mx8;
  if (!fn) return none();
  const at::Tensor* src = tensor(a[0]);
  Call c(src);
  Matrix ms, mc, mq;
  void* st;
  if (!rows_of(c, src, &ms, false) || ms.cols == 0 || ms.cols % 32) return none();
  const int ty = type_of(*src);
  if (ty < 0 || !c.stream(&st)) return none();
  const auto u8 = src->options().dtype(at::kByte).requires_grad(false);
  Output codes(a[1], [&] { return at::empty(with_last(*src, ms.cols / PER), u8); });
  Output scales(a[2], [&] { return at::empty(with_last(*src, ms.cols / 32), u8); });
  if (!rows_of(c, codes.t, &mc, true) || !rows_of(c, scales.t, &mq, true) ||
      codes.t->scalar_type() != at::kByte || scales.t->scalar_type() != at::kByte || mc.rows != ms.rows ||
      mq.rows != ms.rows || mc.cols != ms.cols / PER || mq.cols != ms.cols / 32 || !apart(mc.s, {ms.s}) ||
      !apart(mq.s, {ms.s, mc.s}))
    return none();
  const auto s = fn(ty, ms.p, ms.ld, ms.rows, int32_t(ms.cols), static_cast<uint8_t*>(mc.p), mc.ld,
                    static_cast<uint8_t*>(mq.p), mq.ld, st);
  if (s != MOK_OK) return refused(PER == 2 ? "mok_quantize_mx4" : "mok_quantize_mx8", s);
  PyObject *x = codes.result(), *y = scales.result();
  return x && y ? Py_BuildValue("(NN)", x, y) : nullptr;
}

// codes, scales, dtype (of an output made here), out
template <int PER>
PyObject* do_dequantize(PyObject* const* a) {
  const auto fn = PER == 2 ? g_fn.dequantize_mx4 : g_more.dequantize_mx8;
  if (!fn) return none();
  const at::Tensor *codes = tensor(a[0]), *scales = tensor(a[1]);
  Call c(codes);
  Matrix mc, mq, mo;
  void* st;
  const at::ScalarType type = dtype_of(a[2]);
  if (!rows_of(c, codes, &mc, false) || !rows_of(c, scales, &mq, false) || mc.cols > INT32_MAX / PER ||
      (a[3] == Py_None && type == at::ScalarType::Undefined) || !c.stream(&st))
    return none();
  Output out(a[3], [&] { return at::empty(with_last(*codes, PER * mc.cols), codes->options().dtype(type)); });
  if (!rows_of(c, out.t, &mo, true)) return none();
  const int ty = type_of(*out.t);
  if (ty < 0 || codes->scalar_type() != at::kByte || scales->scalar_type() != at::kByte || mc.cols == 0 ||
      mc.cols % (32 / PER) || mq.cols != mc.cols / (32 / PER) || mo.cols != PER * mc.cols || mq.rows != mc.rows ||
      mo.rows != mc.rows || !apart(mo.s, {mc.s, mq.s}))
    return none();
  const auto s = fn(static_cast<uint8_t*>(mc.p), mc.ld, static_cast<uint8_t*>(mq.p), mq.ld, mc.rows,
                    int32_t(mo.cols), ty, mo.p, mo.ld, st);
  return s == MOK_OK ? out.result() : refused(PER == 2 ? "mok_dequantize_mx4" : "mok_dequantize_mx8", s);
}

// a, a_scales, offsets, b, b_scales, dtype (of an output made here), out
PyObject* do_grouped(PyObject* const* v) {
  const at::Tensor *a = tensor(v[0]), *as = tensor(v[1]), *off = tensor(v[2]), *b = tensor(v[3]),
                   *bs = tensor(v[4]);
  Call c(a);
  Matrix ma, mas, mo;
  Span so, sb, sbs;
  if (!c.on_device(b) || b->dim() != 3) return none();
  const int64_t E = b->size(0), N = b->size(1), half = b->size(2), K = 2 * half;
  if (half == 0 || half % 16 || !matrix(c, a, &ma, false) || !matrix(c, as, &mas, false) ||
      !flat(c, b, {E, N, half}, at::kByte, &sb) || !flat(c, bs, {E, N, K / 32}, at::kByte, &sbs) ||
      !flat(c, off, {E + 1}, at::kInt, &so))
    return none();
  void* st;
  const at::ScalarType type = dtype_of(v[5]);
  if ((v[6] == Py_None && type != at::kBFloat16 && type != at::kFloat) || !c.stream(&st)) return none();
  Output out(v[6], [&] { return at::empty({ma.rows, N}, a->options().dtype(type)); });
  if (!matrix(c, out.t, &mo, true)) return none();
  const int ty = type_of(*out.t);
  if ((ty != MOK_TYPE_BF16 && ty != MOK_TYPE_FP32) || a->scalar_type() != at::kByte ||
      as->scalar_type() != at::kByte || (ma.cols != half && ma.cols != K) || mas.rows != ma.rows ||
      mas.cols != K / 32 || mo.rows != ma.rows || mo.cols != N || E > INT32_MAX || N > INT32_MAX ||
      K > INT32_MAX || !apart(mo.s, {ma.s, mas.s, so, sb, sbs}))
    return none();
  const auto s = g_fn.grouped_mx4(ma.cols == half ? MOK_MX_E2M1 : MOK_MX_E4M3, static_cast<uint8_t*>(ma.p),
                                  ma.ld, static_cast<uint8_t*>(mas.p), mas.ld, ma.rows, at_ptr<int32_t>(so),
                                  int32_t(E), at_ptr<uint8_t>(sb), at_ptr<uint8_t>(sbs), int32_t(N),
                                  int32_t(K), ty, mo.p, mo.ld, st);
  return s == MOK_OK ? out.result() : refused("mok_grouped_mx4", s);
}

// A flag; what has no truth value turns the call down.
bool flag(Call& c, PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) {
    PyErr_Clear();
    c.ok = false;
  }
  return t > 0;
}
bool half_type(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }

// A product's workspace, undefined where it needs none.
struct Workspace {
  at::Tensor t;
  size_t bytes = 0;
  Workspace(int32_t which, int64_t rows, int64_t E, int64_t N, int64_t K, const at::Tensor& like) {
    if (g_more.grouped_mm_workspace(which, rows, int32_t(E), int32_t(N), int32_t(K), &bytes) != MOK_OK) bytes = 0;
    if (bytes) t = at::empty({int64_t(bytes)}, like.options().dtype(at::kByte).requires_grad(false));
  }
  void* p() const { return bytes ? t.data_ptr() : nullptr; }
};

// rows (a or d_out), offsets, b, dtype (of an output made here; None: b's), out
template <bool FORWARD>
PyObject* do_product(PyObject* const* v) {
  const auto fn = FORWARD ? g_more.grouped_mm : g_more.grouped_mm_bwd_rows;
  const at::Tensor *r = tensor(v[0]), *off = tensor(v[1]), *b = tensor(v[2]);
  Call c(r);
  Matrix mr, mo;
  Span so, sb;
  if (!fn || !c.on_device(b) || b->dim() != 3) return none();
  const int64_t E = b->size(0), N = b->size(1), K = b->size(2);
  const at::ScalarType held = b->scalar_type();
  const at::ScalarType type = v[3] == Py_None ? held : dtype_of(v[3]);
  void* st;
  if (!half_type(held) || E > INT32_MAX || N > INT32_MAX || K > INT32_MAX || !matrix(c, r, &mr, false) ||
      !flat(c, b, {E, N, K}, held, &sb) || !flat(c, off, {E + 1}, at::kInt, &so) || r->scalar_type() != held ||
      mr.cols != (FORWARD ? K : N) || (v[4] == Py_None && type != held && type != at::kFloat) || !c.stream(&st))
    return none();
  const int64_t cols = FORWARD ? N : K;
  Output out(v[4], [&] { return at::empty({mr.rows, cols}, r->options().dtype(type).requires_grad(false)); });
  if (!matrix(c, out.t, &mo, true) || (out.t->scalar_type() != held && out.t->scalar_type() != at::kFloat) ||
      mo.rows != mr.rows || mo.cols != cols || !apart(mo.s, {mr.s, so, sb}))
    return none();
  const Workspace ws(FORWARD ? 0 : 1, mr.rows, E, N, K, *r);
  const auto s = fn(type_of(*r), mr.p, mr.ld, mr.rows, at_ptr<int32_t>(so), int32_t(E), at_ptr<void>(sb), int32_t(N),
                    int32_t(K), type_of(*out.t), mo.p, mo.ld, ws.p(), ws.bytes, st);
  return s == MOK_OK ? out.result() : refused(FORWARD ? "mok_grouped_mm" : "mok_grouped_mm_bwd_rows", s);
}

// d_out, a, offsets, a_scales (None: a is not in 8 bits), dtype (of an output made here), out, accumulate
PyObject* do_product_weights(PyObject* const* v) {
  const at::Tensor *d = tensor(v[0]), *a = tensor(v[1]), *off = tensor(v[2]),
                   *as = v[3] == Py_None ? nullptr : tensor(v[3]);
  Call c(d);
  Matrix md, ma, ms = {nullptr, 0, 0, 0, {nullptr, nullptr}};
  Span so, sb;
  const bool add = flag(c, v[6]);
  if (!g_more.grouped_mm_bwd_weights || (v[3] != Py_None && !as) || !matrix(c, d, &md, false) ||
      !matrix(c, a, &ma, false) || (as && !matrix(c, as, &ms, false)) || !c.on_device(off) || off->dim() != 1)
    return none();
  const int64_t E = off->size(0) - 1, N = md.cols, K = ma.cols;
  const at::ScalarType held = d->scalar_type(), type = dtype_of(v[4]);
  void* st;
  if (!half_type(held) || a->scalar_type() != (as ? at::kByte : held) || ma.rows != md.rows || E < 1 ||
      E > INT32_MAX || !flat(c, off, {E + 1}, at::kInt, &so) ||
      (as && (as->scalar_type() != at::kByte || K % 32 || ms.rows != md.rows || ms.cols != K / 32)) ||
      (v[5] == Py_None && (add || (type != held && type != at::kFloat))) || !c.stream(&st))
    return none();
  Output out(v[5], [&] { return at::empty({E, N, K}, d->options().dtype(type).requires_grad(false)); });
  if (!out.t) return none();
  const at::ScalarType made = out.t->scalar_type();
  if ((made != at::kFloat && (add || made != held)) || !flat(c, out.t, {E, N, K}, made, &sb) ||
      !apart(sb, {md.s, ma.s, so, ms.s}))
    return none();
  if (N > INT32_MAX || K > INT32_MAX) return none();
  const Workspace ws(2, md.rows, E, N, K, *d);
  const auto s = g_more.grouped_mm_bwd_weights(
      type_of(*d), md.p, md.ld, ma.p, ma.ld, static_cast<uint8_t*>(ms.p), ms.ld, md.rows, at_ptr<int32_t>(so),
      int32_t(E), int32_t(N), int32_t(K), type_of(*out.t), at_ptr<void>(sb), add, ws.p(), ws.bytes, st);
  return s == MOK_OK ? out.result() : refused("mok_grouped_mm_bwd_weights", s);
}

// The offsets whose last says how many rows there are, or None; false where they are neither.
bool covered(Call& c, PyObject* o, Span* s, int32_t* groups) {
  *s = {nullptr, nullptr};
  *groups = 0;
  if (o == Py_None) return c.ok;
  const at::Tensor* t = tensor(o);
  if (!c.on_device(t) || t->dim() != 1 || t->size(0) < 2 || t->size(0) > INT32_MAX ||
      !flat(c, t, t->sizes(), at::kInt, s))
    return c.ok = false;
  *groups = int32_t(t->size(0) - 1);
  return true;
}

// ab, offsets, h, codes, scales
PyObject* do_swiglu(PyObject* const* v) {
  const at::Tensor* ab = tensor(v[0]);
  Call c(ab);
  Matrix ma, mh, mc, mq;
  Span so;
  int32_t groups;
  void* st;
  if (!g_more.swiglu_mx8 || !matrix(c, ab, &ma, false) || ma.cols == 0 || ma.cols % 64 ||
      !covered(c, v[1], &so, &groups))
    return none();
  const int ty = type_of(*ab);
  if (ty < 0 || !c.stream(&st)) return none();
  const int64_t n = ma.rows, I = ma.cols / 2;
  const auto u8 = ab->options().dtype(at::kByte).requires_grad(false);
  Output h(v[2], [&] { return at::empty({n, I}, ab->options().requires_grad(false)); });
  Output codes(v[3], [&] { return at::empty({n, 2 * I}, u8); });
  Output scales(v[4], [&] { return at::empty({n, I / 16}, u8); });
  if (!matrix(c, h.t, &mh, true) || !matrix(c, codes.t, &mc, true) || !matrix(c, scales.t, &mq, true) ||
      h.t->scalar_type() != ab->scalar_type() || codes.t->scalar_type() != at::kByte ||
      scales.t->scalar_type() != at::kByte || mh.rows != n || mh.cols != I || mc.rows != n || mc.cols != 2 * I ||
      mq.rows != n || mq.cols != I / 16 || !apart(mh.s, {ma.s, so}) || !apart(mc.s, {ma.s, so, mh.s}) ||
      !apart(mq.s, {ma.s, so, mh.s, mc.s}))
    return none();
  const auto s = g_more.swiglu_mx8(ty, ma.p, ma.ld, n, int32_t(I), at_ptr<int32_t>(so), groups, mh.p, mh.ld,
                                   static_cast<uint8_t*>(mc.p), mc.ld, static_cast<uint8_t*>(mq.p), mq.ld, st);
  if (s != MOK_OK) return refused("mok_swiglu_mx8", s);
  PyObject *x = h.result(), *y = codes.result(), *z = scales.result();
  return x && y && z ? Py_BuildValue("(NNN)", x, y, z) : nullptr;
}

// dh, codes, scales, offsets, d_ab, h, with_h
PyObject* do_swiglu_bwd(PyObject* const* v) {
  const at::Tensor *dh = tensor(v[0]), *codes = tensor(v[1]), *scales = tensor(v[2]);
  Call c(dh);
  Matrix md, mc, mq, ma, mh = {nullptr, 0, 0, 0, {nullptr, nullptr}};
  Span so;
  int32_t groups;
  void* st;
  const bool with_h = flag(c, v[6]);
  if (!g_more.swiglu_mx8_bwd || !matrix(c, dh, &md, false) || !matrix(c, codes, &mc, false) ||
      !matrix(c, scales, &mq, false) || md.cols == 0 || md.cols % 32 || !covered(c, v[3], &so, &groups))
    return none();
  const int64_t n = md.rows, I = md.cols;
  const int ty = type_of(*dh);
  if (ty < 0 || codes->scalar_type() != at::kByte || scales->scalar_type() != at::kByte || mc.rows != n ||
      mc.cols != 2 * I || mq.rows != n || mq.cols != I / 16 || !c.stream(&st))
    return none();
  const auto as = dh->options().requires_grad(false);
  Output d_ab(v[4], [&] { return at::empty({n, 2 * I}, as); });
  if (!matrix(c, d_ab.t, &ma, true) || d_ab.t->scalar_type() != dh->scalar_type() || ma.rows != n ||
      ma.cols != 2 * I || !apart(ma.s, {md.s, mc.s, mq.s, so}))
    return none();
  // (without h, a tensor of no elements that is not returned)
  Output h(v[5], [&] { return at::empty({with_h ? n : 0, I}, as); });
  if (with_h && (!matrix(c, h.t, &mh, true) || h.t->scalar_type() != dh->scalar_type() || mh.rows != n ||
                 mh.cols != I || !apart(mh.s, {md.s, mc.s, mq.s, so, ma.s})))
    return none();
  const auto s = g_more.swiglu_mx8_bwd(ty, md.p, md.ld, static_cast<uint8_t*>(mc.p), mc.ld,
                                       static_cast<uint8_t*>(mq.p), mq.ld, n, int32_t(I), at_ptr<int32_t>(so),
                                       groups, ma.p, ma.ld, with_h ? mh.p : nullptr, mh.ld, st);
  if (s != MOK_OK) return refused("mok_swiglu_mx8_bwd", s);
  PyObject *x = d_ab.result(), *y = with_h ? h.result() : same(Py_None);
  return x && y ? Py_BuildValue("(NN)", x, y) : nullptr;
}

// A call with `want` arguments; a C++ exception (a tensor without strides or storage) is a
// call that is not plainly in order.
template <int WANT, PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != WANT || !g_stream) return none();
  try {
    PyObject* r = F(a);
    if (!r && !PyErr_Occurred()) return none();
    return r;
  } catch (...) {
    PyErr_Clear();
    return none();
  }
}
PyObject* f_permute_bwd(PyObject* const* a) {
  PyObject* v[4] = {a[0], a[1], Py_None, a[2]};
  return do_sum(v, false);
}
PyObject* f_unpermute(PyObject* const* a) { return do_sum(a, true); }

// bind(current device, current raw stream, addresses of the entry points in the order of Entries)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9 || !PyCallable_Check(a[0]) || !PyCallable_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "bind: two functions and seven addresses are wanted");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[2 + i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
      return nullptr;
    }
  g_fn = {reinterpret_cast<decltype(g_fn.permute)>(p[0]),
          reinterpret_cast<decltype(g_fn.permute_bwd)>(p[1]),
          reinterpret_cast<decltype(g_fn.unpermute)>(p[2]),
          reinterpret_cast<decltype(g_fn.unpermute_bwd)>(p[3]),
          reinterpret_cast<decltype(g_fn.quantize_mx4)>(p[4]),
          reinterpret_cast<decltype(g_fn.dequantize_mx4)>(p[5]),
          reinterpret_cast<decltype(g_fn.grouped_mx4)>(p[6])};
  Py_XDECREF(g_device);
  Py_XDECREF(g_stream);
  g_device = same(a[0]);
  g_stream = same(a[1]);
  return none();
}

// bind_more(addresses of the entry points in the order of MoreEntries)
PyObject* bind_more(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind_more: eight addresses are wanted");
    return nullptr;
  }
  void* p[8];
  for (int i = 0; i < 8; ++i)
    if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind_more: a null address");
      return nullptr;
    }
  g_more = {reinterpret_cast<decltype(g_more.grouped_mm)>(p[0]),
            reinterpret_cast<decltype(g_more.grouped_mm_bwd_rows)>(p[1]),
            reinterpret_cast<decltype(g_more.grouped_mm_bwd_weights)>(p[2]),
            reinterpret_cast<decltype(g_more.quantize_mx8)>(p[3]),
            reinterpret_cast<decltype(g_more.dequantize_mx8)>(p[4]),
            reinterpret_cast<decltype(g_more.swiglu_mx8)>(p[5]),
            reinterpret_cast<decltype(g_more.swiglu_mx8_bwd)>(p[6]),
            reinterpret_cast<decltype(g_more.grouped_mm_workspace)>(p[7])};
  return none();
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}
PyMethodDef g_methods[] = {
    {"bind", method<bind>(), METH_FASTCALL, nullptr},
    {"permute", method<entry<3, do_permute>>(), METH_FASTCALL, nullptr},
    {"permute_backward", method<entry<3, f_permute_bwd>>(), METH_FASTCALL, nullptr},
    {"unpermute", method<entry<4, f_unpermute>>(), METH_FASTCALL, nullptr},
    {"unpermute_backward", method<entry<6, do_unpermute_bwd>>(), METH_FASTCALL, nullptr},
    {"quantize_mx4", method<entry<3, do_quantize<2>>>(), METH_FASTCALL, nullptr},
    {"dequantize_mx4", method<entry<4, do_dequantize<2>>>(), METH_FASTCALL, nullptr},
    {"grouped_mx4", method<entry<7, do_grouped>>(), METH_FASTCALL, nullptr},
    {"bind_more", method<bind_more>(), METH_FASTCALL, nullptr},
    {"grouped_mm", method<entry<5, do_product<true>>>(), METH_FASTCALL, nullptr},
    {"grouped_mm_backward_rows", method<entry<5, do_product<false>>>(), METH_FASTCALL, nullptr},
    {"grouped_mm_backward_weights", method<entry<7, do_product_weights>>(), METH_FASTCALL, nullptr},
    {"quantize_mx8", method<entry<3, do_quantize<1>>>(), METH_FASTCALL, nullptr},
    {"dequantize_mx8", method<entry<4, do_dequantize<1>>>(), METH_FASTCALL, nullptr},
    {"swiglu_mx8", method<entry<5, do_swiglu>>(), METH_FASTCALL, nullptr},
    {"swiglu_mx8_backward", method<entry<7, do_swiglu_bwd>>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers it is compiled against, the only one that it fits.
PyMODINIT_FUNC PyInit__fast() {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "torch_version", MOK_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
