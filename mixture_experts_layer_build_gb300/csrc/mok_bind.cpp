// mok_bind.cpp -- the norm, dropout and feed-forward calls of the Python binding: checks, outputs and the C call in one
// step.
//
// At small sizes the host is what bounds these calls: three tensors made one by one from Python and a call with eleven
// arguments through ctypes took 15.3 us for a norm kernel of 1.6, now 6.4.  Each function returns its tensors in a
// tuple (feed-forward: an empty one); the mok_status as an int when the library refuses; None when a tensor is not
// what it has to be, which the caller then names.
#include <Python.h>

#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mok.h"

namespace {

using at::Tensor;

// A tensor argument, or nullptr for None; false when it is neither.
bool tensor_arg(PyObject* o, const Tensor** t) {
  *t = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return true;
}

bool plain(const Tensor& t) { return t.is_cuda() && t.is_contiguous(); }
bool plain(const Tensor& t, at::ScalarType type) { return plain(t) && t.scalar_type() == type; }
bool like(const Tensor& t, const Tensor& other, at::ScalarType type) {
  return plain(t, type) && t.sizes() == other.sizes();
}
bool vec(const Tensor& t, int64_t n, at::ScalarType type) { return plain(t, type) && t.dim() == 1 && t.size(0) == n; }

// mok_dtype of a residual stream, or -1.
int stream_type(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? MOK_DT_BF16 : t.scalar_type() == at::kFloat ? MOK_DT_FP32 : -1;
}

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
void* current_stream(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }
Tensor make(at::IntArrayRef shape, const Tensor& on, at::ScalarType type) {
  return at::empty(shape, on.options().dtype(type).requires_grad(false));
}

// Whether every tensor that is there is on `device`: its address goes to a kernel there.
bool all_on(c10::Device device, std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts)
    if (t && t->device() != device) return false;
  return true;
}

// Dropout's arguments, and the device that holds the generator's state.
struct PlacedDropout {
  mok_dropout d;
  int32_t device;
};
// False when they are on another device than `device`.
bool drop_arg(PyObject* o, c10::Device device, const mok_dropout** drop) {
  *drop = nullptr;
  if (o == Py_None) return true;
  const PlacedDropout* p = static_cast<const PlacedDropout*>(PyLong_AsVoidPtr(o));
  if (!p) return true;  // (the caller sees the error)
  *drop = &p->d;
  return p->device == device.index();
}

PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
template <size_t N>
PyObject* wrap_all(const Tensor (&t)[N]) {
  PyObject* r = PyTuple_New(N);
  for (size_t i = 0; r && i < N; ++i) {
    PyObject* o = wrap(t[i]);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// Runs f() with x's device current and Python's lock free: an allocation or a launch may wait for the GPU (memory to be
// freed, a full queue), and what the GPU waits for may need another thread.
template <class F>
int on_device(const Tensor& x, F&& f) {
  struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
  };
  const c10::cuda::CUDAGuard guard(x.device());
  const Unlocked unlocked;
  return f();
}

template <class F>
PyObject* guarded(F&& f) {  // no C++ exception leaves (an allocation may fail)
  try {
    return f();
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    Py_XDECREF(torch);
    if (type) PyErr_SetString(type, e.what());  // (else the lookup's error stands)
    Py_XDECREF(type);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (x, weight, eps, residual, dropout, bf16, mx) -> (h or None: x, y, q, s, rstd)
PyObject* rmsnorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *x, *w, *res;
    if (n != 7 || !tensor_arg(a[0], &x) || !tensor_arg(a[1], &w) || !tensor_arg(a[3], &res) || !x || !w || x->dim() != 2)
      Py_RETURN_NONE;
    const int64_t T = x->size(0), H = x->size(1);
    const Tensor& stream = res ? *res : *x;
    const int st = stream_type(stream);
    if (st < 0 || !plain(*x, at::kBFloat16) || !like(stream, *x, stream.scalar_type()) || !vec(*w, H, at::kBFloat16) ||
        !all_on(x->device(), {w, res}) || H > INT32_MAX)
      Py_RETURN_NONE;
    const double eps = PyFloat_AsDouble(a[2]);
    const mok_dropout* drop;
    if (!drop_arg(a[4], x->device(), &drop)) Py_RETURN_NONE;
    const int bf16 = PyObject_IsTrue(a[5]), mx = PyObject_IsTrue(a[6]);
    if (PyErr_Occurred()) return nullptr;
    Tensor out[5];
    const int rc = on_device(*x, [&] {
      if (res || drop) out[0] = make({T, H}, *x, stream.scalar_type());
      if (bf16) out[1] = make({T, H}, *x, at::kBFloat16);
      if (mx) {
        out[2] = make({T, H}, *x, at::kByte);
        out[3] = make({T, H / 32}, *x, at::kByte);
      }
      out[4] = make({T}, *x, at::kFloat);
      const mok_norm_shape shape{T, static_cast<int32_t>(H), st, static_cast<float>(eps)};
      return mok_rmsnorm_forward(&shape, x->data_ptr(), ptr(res), drop, w->data_ptr(), ptr(out[0]), ptr(out[1]),
                                 static_cast<uint8_t*>(ptr(out[2])), static_cast<uint8_t*>(ptr(out[3])),
                                 static_cast<float*>(ptr(out[4])), current_stream(*x));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (h, rstd, weight, dy, dres, dropout) -> (dh, dx or None: dh, dweight)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *h, *rstd, *w, *dy, *dres;
    if (n != 6 || !tensor_arg(a[0], &h) || !tensor_arg(a[1], &rstd) || !tensor_arg(a[2], &w) || !tensor_arg(a[3], &dy) ||
        !tensor_arg(a[4], &dres) || !h || !rstd || !w || !dy || h->dim() != 2)
      Py_RETURN_NONE;
    const int64_t T = h->size(0), H = h->size(1);
    const int st = stream_type(*h);
    if (st < 0 || !plain(*h) || !vec(*rstd, T, at::kFloat) || !vec(*w, H, at::kBFloat16) ||
        !like(*dy, *h, at::kBFloat16) || (dres && !like(*dres, *h, h->scalar_type())) ||
        !all_on(h->device(), {rstd, w, dy, dres}) || H > INT32_MAX)
      Py_RETURN_NONE;
    const mok_dropout* drop;
    if (!drop_arg(a[5], h->device(), &drop)) Py_RETURN_NONE;
    if (PyErr_Occurred()) return nullptr;
    const mok_norm_shape shape{T, static_cast<int32_t>(H), st, 0.0f};
    const size_t bytes = mok_rmsnorm_workspace_bytes(&shape);
    if (!bytes) return PyLong_FromLong(MOK_ERR_INVALID_ARG);
    Tensor out[3];
    const int rc = on_device(*h, [&] {
      out[0] = make({T, H}, *h, h->scalar_type());
      if (drop || st != MOK_DT_BF16) out[1] = make({T, H}, *h, at::kBFloat16);
      out[2] = make({H}, *h, at::kFloat);
      const Tensor ws = make({static_cast<int64_t>(bytes)}, *h, at::kByte);
      return mok_rmsnorm_backward(&shape, h->data_ptr(), static_cast<const float*>(rstd->data_ptr()), w->data_ptr(),
                                  dy->data_ptr(), ptr(dres), drop, ptr(out[0]), ptr(out[1]),
                                  static_cast<float*>(ptr(out[2])), ws.data_ptr(), bytes, current_stream(*h));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (x, dropout, residual, out) -> (out,)
PyObject* dropout_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *x, *res, *given;
    if (n != 4 || !tensor_arg(a[0], &x) || !tensor_arg(a[2], &res) || !tensor_arg(a[3], &given) || !x) Py_RETURN_NONE;
    const Tensor& stream = res ? *res : *x;
    const int st = stream_type(stream);
    if (st < 0 || !plain(*x, at::kBFloat16) || !like(stream, *x, stream.scalar_type()) ||
        (given && !like(*given, *x, stream.scalar_type())) || !all_on(x->device(), {res, given}))
      Py_RETURN_NONE;
    const mok_dropout* drop;
    if (!drop_arg(a[1], x->device(), &drop)) Py_RETURN_NONE;
    if (PyErr_Occurred()) return nullptr;
    Tensor out[1];
    const int rc = on_device(*x, [&] {
      out[0] = given ? *given : make(x->sizes(), *x, stream.scalar_type());
      return mok_dropout_forward(x->numel(), st, drop, x->data_ptr(), ptr(res), ptr(out[0]), current_stream(*x));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (dout, dropout, dx) -> (dx,)
PyObject* dropout_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *dout, *given;
    if (n != 3 || !tensor_arg(a[0], &dout) || !tensor_arg(a[2], &given) || !dout) Py_RETURN_NONE;
    const int st = stream_type(*dout);
    if (st < 0 || !plain(*dout) || (given && !like(*given, *dout, at::kBFloat16)) ||
        !all_on(dout->device(), {given}))
      Py_RETURN_NONE;
    const mok_dropout* drop;
    if (!drop_arg(a[1], dout->device(), &drop)) Py_RETURN_NONE;
    if (PyErr_Occurred()) return nullptr;
    Tensor out[1];
    const int rc = on_device(*dout, [&] {
      out[0] = given ? *given : make(dout->sizes(), *dout, at::kBFloat16);
      return mok_dropout_backward(dout->numel(), st, drop, dout->data_ptr(), ptr(out[0]), current_stream(*dout));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

bool mat(const Tensor& t, int64_t rows, int64_t cols) {
  return plain(t, at::kBFloat16) && t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
}

// (device, shape, out, ctx, ctx bytes, save, status: the plan's index, addresses and sizes, x, w_gate, w_up, w_down,
// residual, stream or None: the current one of x's device) -> ()
PyObject* ffn_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *x, *wg, *wu, *wd, *res;
    if (n != 13 || !tensor_arg(a[7], &x) || !tensor_arg(a[8], &wg) || !tensor_arg(a[9], &wu) || !tensor_arg(a[10], &wd) ||
        !tensor_arg(a[11], &res) || !x || !wg || !wu || !wd)
      Py_RETURN_NONE;
    const long device = PyLong_AsLong(a[0]);
    const mok_ffn_shape* s = static_cast<const mok_ffn_shape*>(PyLong_AsVoidPtr(a[1]));
    void* out = PyLong_AsVoidPtr(a[2]);
    void* ctx = PyLong_AsVoidPtr(a[3]);
    const size_t bytes = PyLong_AsSize_t(a[4]);
    const long save = PyLong_AsLong(a[5]);
    uint32_t* status = static_cast<uint32_t*>(PyLong_AsVoidPtr(a[6]));
    if (PyErr_Occurred()) return nullptr;
    if (!mat(*x, s->T, s->H) || !mat(*wg, s->I, s->H) || !mat(*wu, s->I, s->H) || !mat(*wd, s->H, s->I) ||
        (res && !mat(*res, s->T, s->H)) || x->device().index() != device || !all_on(x->device(), {wg, wu, wd, res}))
      Py_RETURN_NONE;
    void* stream = a[12] == Py_None ? current_stream(*x) : PyLong_AsVoidPtr(a[12]);
    if (PyErr_Occurred()) return nullptr;
    const int rc = on_device(*x, [&] {
      return mok_ffn_forward(s, x->data_ptr(), wg->data_ptr(), wu->data_ptr(), wd->data_ptr(), ptr(res), out, ctx, bytes,
                             static_cast<int32_t>(save), status, stream);
    });
    return rc ? PyLong_FromLong(rc) : PyTuple_New(0);
  });
}

// (device, shape, ctx, ctx bytes, gradients, ws, ws bytes, status: the plan's index, addresses and sizes, x, w_gate, w_up,
// w_down, dy, dx_add, stream or None: the current one of x's device) -> ()
PyObject* ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *x, *wg, *wu, *wd, *dy, *add;
    if (n != 15 || !tensor_arg(a[8], &x) || !tensor_arg(a[9], &wg) || !tensor_arg(a[10], &wu) || !tensor_arg(a[11], &wd) ||
        !tensor_arg(a[12], &dy) || !tensor_arg(a[13], &add) || !x || !wg || !wu || !wd || !dy)
      Py_RETURN_NONE;
    const long device = PyLong_AsLong(a[0]);
    const mok_ffn_shape* s = static_cast<const mok_ffn_shape*>(PyLong_AsVoidPtr(a[1]));
    const void* ctx = PyLong_AsVoidPtr(a[2]);
    const size_t ctx_bytes = PyLong_AsSize_t(a[3]);
    const mok_ffn_grads* plan = static_cast<const mok_ffn_grads*>(PyLong_AsVoidPtr(a[4]));
    void* ws = PyLong_AsVoidPtr(a[5]);
    const size_t ws_bytes = PyLong_AsSize_t(a[6]);
    uint32_t* status = static_cast<uint32_t*>(PyLong_AsVoidPtr(a[7]));
    if (PyErr_Occurred()) return nullptr;
    if (!mat(*x, s->T, s->H) || !mat(*wg, s->I, s->H) || !mat(*wu, s->I, s->H) || !mat(*wd, s->H, s->I) ||
        !mat(*dy, s->T, s->H) || (add && !mat(*add, s->T, s->H)) || x->device().index() != device ||
        !all_on(x->device(), {wg, wu, wd, dy, add}))
      Py_RETURN_NONE;
    void* stream = a[14] == Py_None ? current_stream(*x) : PyLong_AsVoidPtr(a[14]);
    if (PyErr_Occurred()) return nullptr;
    mok_ffn_grads g = *plan;
    g.dx_add = ptr(add);
    const int rc = on_device(*x, [&] {
      return mok_ffn_backward(s, x->data_ptr(), wg->data_ptr(), wu->data_ptr(), wd->data_ptr(), ctx, ctx_bytes,
                              dy->data_ptr(), &g, ws, ws_bytes, status, stream);
    });
    return rc ? PyLong_FromLong(rc) : PyTuple_New(0);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<rmsnorm_forward>("rmsnorm_forward"), method<rmsnorm_backward>("rmsnorm_backward"),
                         method<dropout_forward>("dropout_forward"), method<dropout_backward>("dropout_backward"),
                         method<ffn_forward>("ffn_forward"), method<ffn_backward>("ffn_backward"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_mok_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mok_bind() {
  PyObject* m = PyModule_Create(&module_def);
  if (m && PyModule_AddStringConstant(m, "built_for", MOK_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
