// The plain case of the gradient operators' Python calls without the interpreter's share of the
// argument checks, allocations and ctypes conversions, which cost more than the launch of a small
// call (one row through the norm: 16 us a call with them, 7 without).
//
// Plain: exact torch tensors on the current device, contiguous, of supported and matching types and
// shapes, outputs to be allocated, the current stream. Each function returns None for any other
// call and for one that the C ABI refuses; gradients.py then checks it in full and reports.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/muon.h"

namespace {

struct Calls {
  decltype(&muon_embedding) embedding;
  decltype(&muon_embedding_grad) embedding_grad;
  decltype(&muon_embedding_grad_workspace) embedding_grad_workspace;
  decltype(&muon_rms_norm) rms_norm;
  decltype(&muon_rms_norm_grad) rms_norm_grad;
  decltype(&muon_rms_norm_grad_workspace) rms_norm_grad_workspace;
  decltype(&muon_checkpoint_store) checkpoint_store;
  decltype(&muon_checkpoint_restore) checkpoint_restore;
  decltype(&muon_weight_grad) weight_grad;
  decltype(&muon_weight_grad_workspace) weight_grad_workspace;
} calls;

using at::ScalarType;
using at::Tensor;

struct Ctx {
  int dev;
  muon_stream_t stream;
};

int code(ScalarType t) { return t == ScalarType::BFloat16 ? MUON_BF16 : t == ScalarType::Float ? MUON_FP32 : -1; }

// The tensor behind a Python object if it is plain (on the current device, contiguous), else null.
const Tensor* plain(PyObject* o, int dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.get_device() == dev && t.dim() >= 1 && t.is_contiguous() ? &t : nullptr;
}

Ctx context() {
  const auto s = c10::cuda::getCurrentCUDAStream();
  return {s.device_index(), reinterpret_cast<muon_stream_t>(s.stream())};
}

Tensor empty(at::IntArrayRef shape, ScalarType t, int dev) {
  return at::detail::empty_cuda(shape, t, c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)dev), std::nullopt);
}

c10::SmallVector<int64_t, 8> with_last(at::IntArrayRef shape, int64_t last) {
  c10::SmallVector<int64_t, 8> v(shape.begin(), shape.end());
  v.back() = last;
  return v;
}

PyObject* none() { Py_RETURN_NONE; }

// A dtype argument: the tensor's own where it is None; false if it is no dtype.
bool dtype_or(PyObject* o, ScalarType own, ScalarType* out) {
  if (o == Py_None) {
    *out = own;
    return true;
  }
  if (!THPDtype_Check(o)) return false;
  *out = reinterpret_cast<THPDtype*>(o)->scalar_type;
  return true;
}

bool number(PyObject* o, double* v) {
  *v = PyFloat_AsDouble(o);
  if (*v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// A truth value; -1 if it has none (the full path then meets the error again and raises it).
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) PyErr_Clear();
  return v;
}

int token_bits(const Tensor& t) { return t.scalar_type() == ScalarType::Long ? 64 : t.scalar_type() == ScalarType::Int ? 32 : 0; }

#define NONE_IF(cond) \
  do {                \
    if (cond) return none(); \
  } while (0)
#define BEGIN(n)          \
  NONE_IF(nargs != (n)); \
  try {
#define END                     \
  } catch (const std::exception& e) { \
    return none(); /* allocation: the full path reports it */ \
  }

// embedding(tokens, table, scale, out_dtype) -> out
PyObject* embedding(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  BEGIN(4)
  const Ctx c = context();
  const Tensor *t = plain(args[0], c.dev), *e = plain(args[1], c.dev);
  double scale;
  NONE_IF(!t || !e || e->dim() != 2 || !number(args[2], &scale));
  ScalarType od;
  const int bits = token_bits(*t), ec = code(e->scalar_type());
  NONE_IF(!bits || ec < 0 || !dtype_or(args[3], e->scalar_type(), &od) || code(od) < 0);
  c10::SmallVector<int64_t, 8> shape(t->sizes().begin(), t->sizes().end());
  const int64_t dim = e->size(1);
  shape.push_back(dim);
  Tensor out = empty(shape, od, c.dev);
  NONE_IF(calls.embedding(t->data_ptr(), bits, t->numel(), e->data_ptr(), (muon_dtype_t)ec, dim, e->size(0), dim, (float)scale,
                          out.data_ptr(), (muon_dtype_t)code(od), dim, c.stream) != MUON_OK);
  return THPVariable_Wrap(std::move(out));
  END
}

// embedding_grad(tokens, dy, vocab, scale, grad or None, grad_dtype, accumulate) -> grad
PyObject* embedding_grad(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  BEGIN(7)
  const Ctx c = context();
  const Tensor *t = plain(args[0], c.dev), *d = plain(args[1], c.dev);
  double scale;
  NONE_IF(!t || !d || !PyLong_CheckExact(args[2]) || !number(args[3], &scale));
  const int64_t vocab = PyLong_AsLongLong(args[2]), dim = d->sizes().back(), n = t->numel();
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return none();
  }
  NONE_IF(d->sizes().slice(0, d->dim() - 1) != t->sizes() || vocab < 1);
  const int bits = token_bits(*t), dc = code(d->scalar_type()), acc = truth(args[6]);
  NONE_IF(!bits || dc < 0 || acc < 0);
  Tensor grad;
  if (args[4] == Py_None) {
    ScalarType gd;
    NONE_IF(acc || !dtype_or(args[5], d->scalar_type(), &gd) || code(gd) < 0);
    grad = empty({vocab, dim}, gd, c.dev);
  } else {
    const Tensor* g = plain(args[4], c.dev);
    NONE_IF(!g || args[5] != Py_None || g->dim() != 2 || g->size(0) != vocab || g->size(1) != dim || code(g->scalar_type()) < 0);
    grad = *g;
  }
  const int64_t bytes = calls.embedding_grad_workspace(n, vocab, dim);
  NONE_IF(bytes < 0);
  Tensor ws = empty({bytes}, ScalarType::Byte, c.dev);
  NONE_IF(calls.embedding_grad(t->data_ptr(), bits, n, d->data_ptr(), (muon_dtype_t)dc, dim, vocab, dim, (float)scale,
                               grad.data_ptr(), (muon_dtype_t)code(grad.scalar_type()), dim, acc, ws.data_ptr(), bytes,
                               c.stream) != MUON_OK);
  return THPVariable_Wrap(std::move(grad));
  END
}

PyObject* item(Tensor& t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : none(); }

// rms_norm(x, weight, residual or None, eps, output, checkpoint) -> (y, h, rstd, q, scales), with None for what is not made
PyObject* rms_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  BEGIN(6)
  const Ctx c = context();
  const Tensor *x = plain(args[0], c.dev), *w = plain(args[1], c.dev);
  double eps;
  NONE_IF(!x || !w || !number(args[3], &eps));
  const int64_t dim = x->sizes().back(), blocks = (dim + 31) / 32;
  const int xc = code(x->scalar_type()), wc = code(w->scalar_type()), output = truth(args[4]),
            checkpoint = truth(args[5]);
  NONE_IF(xc < 0 || wc < 0 || w->dim() != 1 || w->size(0) != dim || dim < 1 || output < 0 || checkpoint < 0 || (!output && !checkpoint));
  const Tensor* r = nullptr;
  Tensor h, y, q, s;
  int rc = 0;
  if (args[2] != Py_None) {
    r = plain(args[2], c.dev);
    NONE_IF(!r || r->sizes() != x->sizes());
    rc = code(r->scalar_type());
    NONE_IF(rc < 0);
    h = empty(r->sizes(), r->scalar_type(), c.dev);
  }
  if (output) y = empty(x->sizes(), x->scalar_type(), c.dev);
  Tensor rstd = empty(x->sizes().slice(0, x->dim() - 1), ScalarType::Float, c.dev);
  if (checkpoint) {
    q = empty(x->sizes(), ScalarType::Float8_e4m3fn, c.dev);
    s = empty(with_last(x->sizes(), blocks), ScalarType::Float8_e8m0fnu, c.dev);
  }
  auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  NONE_IF(calls.rms_norm(x->data_ptr(), (muon_dtype_t)xc, dim, r ? r->data_ptr() : nullptr, (muon_dtype_t)rc, dim, w->data_ptr(),
                         (muon_dtype_t)wc, x->numel() / dim, dim, (float)eps, ptr(h), dim, ptr(y), dim, ptr(q), dim, ptr(s), blocks,
                         static_cast<float*>(rstd.data_ptr()), c.stream) != MUON_OK);
  PyObject* out = PyTuple_New(5);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, item(y));
  PyTuple_SET_ITEM(out, 1, item(h));
  PyTuple_SET_ITEM(out, 2, item(rstd));
  PyTuple_SET_ITEM(out, 3, item(q));
  PyTuple_SET_ITEM(out, 4, item(s));
  return out;
  END
}

// rms_norm_grad(dy, h, weight, rstd, dh or None) -> (dx, dweight)
PyObject* rms_norm_grad(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  BEGIN(5)
  const Ctx c = context();
  const Tensor *d = plain(args[0], c.dev), *h = plain(args[1], c.dev), *w = plain(args[2], c.dev), *r = plain(args[3], c.dev);
  NONE_IF(!d || !h || !w || !r || d->sizes() != h->sizes() || r->scalar_type() != ScalarType::Float);
  const int64_t dim = h->sizes().back();
  const int dc = code(d->scalar_type()), hc = code(h->scalar_type()), wc = code(w->scalar_type());
  NONE_IF(dc < 0 || hc < 0 || wc < 0 || dim < 1 || w->dim() != 1 || w->size(0) != dim ||
          r->sizes() != h->sizes().slice(0, h->dim() - 1));
  const Tensor* g = nullptr;
  if (args[4] != Py_None) {
    g = plain(args[4], c.dev);
    NONE_IF(!g || g->sizes() != h->sizes() || g->scalar_type() != h->scalar_type());
  }
  const int64_t rows = h->numel() / dim, bytes = calls.rms_norm_grad_workspace(rows, dim);
  NONE_IF(bytes < 0);
  Tensor dx = empty(h->sizes(), h->scalar_type(), c.dev), dw = empty({dim}, ScalarType::Float, c.dev);
  Tensor ws = empty({bytes}, ScalarType::Byte, c.dev);
  NONE_IF(calls.rms_norm_grad(d->data_ptr(), (muon_dtype_t)dc, dim, h->data_ptr(), (muon_dtype_t)hc, dim, w->data_ptr(),
                              (muon_dtype_t)wc, static_cast<const float*>(r->data_ptr()), g ? g->data_ptr() : nullptr, dim, rows,
                              dim, dx.data_ptr(), dim, static_cast<float*>(dw.data_ptr()), 0, ws.data_ptr(), bytes,
                              c.stream) != MUON_OK);
  PyObject* out = PyTuple_New(2);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, item(dx));
  PyTuple_SET_ITEM(out, 1, item(dw));
  return out;
  END
}

// checkpoint_store(x) -> (q, scales)
PyObject* checkpoint_store(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  BEGIN(1)
  const Ctx c = context();
  const Tensor* x = plain(args[0], c.dev);
  NONE_IF(!x);
  const int64_t dim = x->sizes().back(), blocks = (dim + 31) / 32;
  const int xc = code(x->scalar_type());
  NONE_IF(xc < 0 || dim < 1);
  Tensor q = empty(x->sizes(), ScalarType::Float8_e4m3fn, c.dev);
  Tensor s = empty(with_last(x->sizes(), blocks), ScalarType::Float8_e8m0fnu, c.dev);
  NONE_IF(calls.checkpoint_store(x->data_ptr(), (muon_dtype_t)xc, dim, x->numel() / dim, dim, q.data_ptr(), dim, s.data_ptr(), blocks,
                                 c.stream) != MUON_OK);
  PyObject* out = PyTuple_New(2);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, item(q));
  PyTuple_SET_ITEM(out, 1, item(s));
  return out;
  END
}

// The two tensors of a checkpoint, or false.
bool checkpoint_of(PyObject* qo, PyObject* so, int dev, const Tensor** q, const Tensor** s) {
  *q = plain(qo, dev);
  *s = plain(so, dev);
  if (!*q || !*s || (*q)->scalar_type() != ScalarType::Float8_e4m3fn || (*s)->scalar_type() != ScalarType::Float8_e8m0fnu) return false;
  const auto a = (*q)->sizes(), b = (*s)->sizes();
  const size_t n = a.size() - 1;
  return a.size() == b.size() && a.back() >= 1 && b.back() == (a.back() + 31) / 32 && a.slice(0, n) == b.slice(0, n);
}

// checkpoint_restore(q, scales, dtype) -> x
PyObject* checkpoint_restore(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  BEGIN(3)
  const Ctx c = context();
  const Tensor *q, *s;
  ScalarType od;
  NONE_IF(!checkpoint_of(args[0], args[1], c.dev, &q, &s) || args[2] == Py_None || !dtype_or(args[2], ScalarType::BFloat16, &od) ||
          code(od) < 0);
  const int64_t dim = q->sizes().back();
  Tensor x = empty(q->sizes(), od, c.dev);
  NONE_IF(calls.checkpoint_restore(q->data_ptr(), dim, s->data_ptr(), s->sizes().back(), q->numel() / dim, dim, x.data_ptr(),
                                   (muon_dtype_t)code(od), dim, c.stream) != MUON_OK);
  return THPVariable_Wrap(std::move(x));
  END
}

// weight_grad(dy, q, scales, grad or None, grad_dtype, accumulate) -> grad
PyObject* weight_grad(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  BEGIN(6)
  const Ctx c = context();
  const Tensor *d = plain(args[0], c.dev), *q, *s;
  NONE_IF(!d || !checkpoint_of(args[1], args[2], c.dev, &q, &s));
  const int64_t n = d->sizes().back(), k = q->sizes().back();
  const int dc = code(d->scalar_type()), acc = truth(args[5]);
  NONE_IF(dc < 0 || n < 1 || acc < 0 || d->dim() != q->dim() || d->sizes().slice(0, d->dim() - 1) != q->sizes().slice(0, q->dim() - 1));
  Tensor grad;
  if (args[3] == Py_None) {
    ScalarType gd;
    NONE_IF(acc || !dtype_or(args[4], d->scalar_type(), &gd) || code(gd) < 0);
    grad = empty({n, k}, gd, c.dev);
  } else {
    const Tensor* g = plain(args[3], c.dev);
    NONE_IF(!g || args[4] != Py_None || g->dim() != 2 || g->size(0) != n || g->size(1) != k || code(g->scalar_type()) < 0);
    grad = *g;
  }
  const int64_t rows = d->numel() / n, bytes = calls.weight_grad_workspace(rows, n, k, (muon_dtype_t)dc);
  NONE_IF(bytes < 0);
  Tensor ws = empty({bytes}, ScalarType::Byte, c.dev);
  NONE_IF(calls.weight_grad(d->data_ptr(), (muon_dtype_t)dc, n, q->data_ptr(), k, s->data_ptr(), s->sizes().back(), rows, n, k,
                            grad.data_ptr(), (muon_dtype_t)code(grad.scalar_type()), k, acc, ws.data_ptr(), bytes,
                            c.stream) != MUON_OK);
  return THPVariable_Wrap(std::move(grad));
  END
}

// bind(addresses of the C calls, in the order of Calls)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  void* p[sizeof(Calls) / sizeof(void*)];
  if (nargs != (Py_ssize_t)(sizeof(p) / sizeof(p[0]))) {
    PyErr_SetString(PyExc_TypeError, "bind takes the address of each call");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < nargs; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  memcpy(&calls, p, sizeof(calls));
  return none();
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),          METHOD(embedding),        METHOD(embedding_grad),     METHOD(rms_norm),
                         METHOD(rms_norm_grad), METHOD(checkpoint_store), METHOD(checkpoint_restore), METHOD(weight_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_plain", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__plain() { return PyModule_Create(&module); }
