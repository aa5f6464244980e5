// mok_bind.cpp -- the norm, dropout, feed-forward, routed-row and 8-bit calls of the Python binding: checks, outputs and
// the C call in one step.
//
// At small sizes the host is what bounds these calls: three tensors made one by one from Python and a call with eleven
// arguments through ctypes took 15.3 us for a norm kernel of 1.6, now 6.4.  Each function returns its tensors in a
// tuple (feed-forward: an empty one); the mok_status as an int when the library refuses; None when a tensor is not
// what it has to be, which the caller then names.
#include <Python.h>

#include <initializer_list>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
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

// ---- routed rows and 8-bit products ----

// The address of a mok_schedule and the index of the device that holds its tables; nullptr (with an error set) when it
// is none.
struct PlacedSchedule {
  const mok_schedule* s;
  long device;
};
bool sched_arg(PyObject* addr, PyObject* device, PlacedSchedule* p) {
  p->s = static_cast<const mok_schedule*>(PyLong_AsVoidPtr(addr));
  p->device = PyLong_AsLong(device);
  return p->s && !PyErr_Occurred();
}
bool rows_of(const Tensor& t, int64_t rows, int64_t cols, at::ScalarType type) {
  return plain(t, type) && t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
}

int64_t up_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t blocks(int64_t n) { return (n + 127) / 128; }

// `make` from the allocator itself: the dispatcher is most of the 1.2 us that an allocation adds to a call's host time.
Tensor make_raw(at::IntArrayRef shape, const Tensor& on, at::ScalarType type) {
  if (at::globalContext().deterministicAlgorithms()) return make(shape, on, type);  // (which may fill what nobody writes)
  int64_t n = static_cast<int64_t>(c10::elementSize(type));
  for (int64_t k : shape) n *= k;
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(c10::Storage::use_byte_size_t(), n, c10::cuda::CUDACachingAllocator::get(), /*resizable=*/true),
      c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

// Codes and scales of one matrix, each in a storage of its own: torch saves no storage that tensors of two types share.
void make_fp8(at::IntArrayRef q, at::IntArrayRef s, const Tensor& on, Tensor* tq, Tensor* ts) {
  *tq = make_raw(q, on, at::kByte);
  *ts = make_raw(s, on, at::kFloat);
}

// Codes [.., rows, ld] and scales as one matrix; false where they do not go together.
bool fp8_arg(PyObject* q, PyObject* s, PyObject* cols, bool block, int batch_dims, const Tensor** tq, const Tensor** ts,
             mok_fp8_matrix* m) {
  if (!tensor_arg(q, tq) || !tensor_arg(s, ts) || !*tq || !*ts) return false;
  const Tensor &c = **tq, &f = **ts;
  m->cols = PyLong_AsLongLong(cols);
  if (PyErr_Occurred()) return false;
  const int d = 2 + batch_dims;
  if (c.dim() != d || f.dim() != d || !plain(c) || !plain(f, at::kFloat) || f.device() != c.device()) return false;
  if (c.scalar_type() != at::kByte && c.scalar_type() != at::kFloat8_e4m3fn) return false;
  m->rows = c.size(d - 2);
  m->ld = c.size(d - 1);
  m->batch = batch_dims ? static_cast<int32_t>(c.size(0)) : 1;
  m->scaling = block ? MOK_FP8_BLOCKS : MOK_FP8_ROWS;
  if (batch_dims && f.size(0) != c.size(0)) return false;
  const int64_t r = block ? blocks(m->rows) : blocks(m->cols), k = block ? blocks(m->cols) : up_to(m->rows, 4);
  if (f.size(d - 2) != r || f.size(d - 1) != k) return false;
  m->q = static_cast<const uint8_t*>(c.data_ptr());
  m->s = static_cast<const float*>(f.data_ptr());
  return true;
}

// (schedule, device, x, out) -> (out,): one row per routed row from one per token (`to_rows`), or the other way
template <mok_status (*CALL)(const mok_schedule*, const void*, int32_t, void*, void*), bool TO_ROWS>
PyObject* move_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    PlacedSchedule p;
    const Tensor *x, *given;
    if (n != 4 || !sched_arg(a[0], a[1], &p) || !tensor_arg(a[2], &x) || !tensor_arg(a[3], &given) || !x || x->dim() != 2) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    const int64_t W = x->size(1), from = TO_ROWS ? p.s->shape.T : p.s->rpad_max, to = TO_ROWS ? p.s->rpad_max : p.s->shape.T;
    if (!rows_of(*x, from, W, at::kBFloat16) || (given && !rows_of(*given, to, W, at::kBFloat16)) ||
        x->device().index() != p.device || !all_on(x->device(), {given}) || W > INT32_MAX)
      Py_RETURN_NONE;
    Tensor out[1];
    const int rc = on_device(*x, [&] {
      out[0] = given ? *given : make({to, W}, *x, at::kBFloat16);
      return CALL(p.s, x->data_ptr(), static_cast<int32_t>(W), ptr(out[0]), current_stream(*x));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (schedule, device, rows, dout, drows) -> (drows, dweights)
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    PlacedSchedule p;
    const Tensor *rows, *dout, *given;
    if (n != 5 || !sched_arg(a[0], a[1], &p) || !tensor_arg(a[2], &rows) || !tensor_arg(a[3], &dout) ||
        !tensor_arg(a[4], &given) || !rows || !dout || rows->dim() != 2) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    const int64_t W = rows->size(1), R = p.s->rpad_max;
    if (!rows_of(*rows, R, W, at::kBFloat16) || !rows_of(*dout, p.s->shape.T, W, at::kBFloat16) ||
        (given && !rows_of(*given, R, W, at::kBFloat16)) || rows->device().index() != p.device ||
        !all_on(rows->device(), {dout, given}) || W > INT32_MAX)
      Py_RETURN_NONE;
    Tensor out[2];
    const int rc = on_device(*rows, [&] {
      out[0] = given ? *given : make({R, W}, *rows, at::kBFloat16);
      out[1] = make({p.s->shape.T, p.s->shape.K}, *rows, at::kFloat);
      return mok_combine_backward(p.s, rows->data_ptr(), dout->data_ptr(), static_cast<int32_t>(W), ptr(out[0]),
                                  static_cast<float*>(ptr(out[1])), current_stream(*rows));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (x, rows, transposed, schedule or 0, device, gather) -> (q, s, qt, st)
PyObject* fp8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor* x;
    if (n != 6 || !tensor_arg(a[0], &x) || !x || x->dim() != 2) Py_RETURN_NONE;
    const int rows = PyObject_IsTrue(a[1]), cols = PyObject_IsTrue(a[2]);
    const mok_schedule* s = static_cast<const mok_schedule*>(PyLong_AsVoidPtr(a[3]));
    const long device = PyLong_AsLong(a[4]), gather = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) return nullptr;
    const int64_t C = x->size(1), R = s ? s->rpad_max : x->size(0);
    if (!rows_of(*x, s && gather ? s->shape.T : R, C, at::kBFloat16) || (s && x->device().index() != device) ||
        C > INT32_MAX)
      Py_RETURN_NONE;
    Tensor out[4];
    const int rc = on_device(*x, [&] {
      if (rows) make_fp8({R, up_to(C, 16)}, {blocks(C), up_to(R, 4)}, *x, &out[0], &out[1]);
      if (cols) make_fp8({C, up_to(R, 16)}, {blocks(R), up_to(C, 4)}, *x, &out[2], &out[3]);
      uint8_t *q = static_cast<uint8_t*>(ptr(out[0])), *qt = static_cast<uint8_t*>(ptr(out[2]));
      float *f = static_cast<float*>(ptr(out[1])), *ft = static_cast<float*>(ptr(out[3]));
      if (s)
        return mok_fp8_quantize_routed(s, static_cast<int32_t>(gather), x->data_ptr(), static_cast<int32_t>(C), q, f, qt, ft,
                                       current_stream(*x));
      return mok_fp8_quantize(x->data_ptr(), R, static_cast<int32_t>(C), q, f, qt, ft, current_stream(*x));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (w, rows, transposed) -> (q, s, qt, st)
PyObject* fp8_quantize_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor* x;
    if (n != 3 || !tensor_arg(a[0], &x) || !x || !plain(*x, at::kBFloat16) || (x->dim() != 2 && x->dim() != 3)) Py_RETURN_NONE;
    const int rows = PyObject_IsTrue(a[1]), cols = PyObject_IsTrue(a[2]);
    if (PyErr_Occurred()) return nullptr;
    const bool many = x->dim() == 3;
    const int64_t B = many ? x->size(0) : 1, R = x->size(many), C = x->size(many + 1);
    if (C > INT32_MAX || B > INT32_MAX) Py_RETURN_NONE;
    Tensor out[4];
    const int rc = on_device(*x, [&] {
      auto pair = [&](int64_t r, int64_t c, int i) {
        if (many) make_fp8({B, r, up_to(c, 16)}, {B, blocks(r), blocks(c)}, *x, &out[i], &out[i + 1]);
        else make_fp8({r, up_to(c, 16)}, {blocks(r), blocks(c)}, *x, &out[i], &out[i + 1]);
      };
      if (rows) pair(R, C, 0);
      if (cols) pair(C, R, 2);
      return mok_fp8_quantize_blocks(x->data_ptr(), static_cast<int32_t>(B), R, static_cast<int32_t>(C),
                                     static_cast<uint8_t*>(ptr(out[0])), static_cast<float*>(ptr(out[1])),
                                     static_cast<uint8_t*>(ptr(out[2])), static_cast<float*>(ptr(out[3])),
                                     current_stream(*x));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

bool status_arg(PyObject* o, const Tensor** t) {
  return tensor_arg(o, t) && (!*t || (plain(**t, at::kInt) && (*t)->numel() == 1));
}

// (a.q, a.s, a.cols, b.q, b.s, b.cols, b.block, out, f32, status) -> (out,)
PyObject* fp8_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *aq, *as, *bq, *bs, *given, *status;
    mok_fp8_matrix ma{}, mb{};
    if (n != 10 || !fp8_arg(a[0], a[1], a[2], false, 0, &aq, &as, &ma) ||
        !fp8_arg(a[3], a[4], a[5], PyObject_IsTrue(a[6]), 0, &bq, &bs, &mb) || !tensor_arg(a[7], &given) ||
        !status_arg(a[9], &status)) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    const at::ScalarType type = PyObject_IsTrue(a[8]) ? at::kFloat : at::kBFloat16;
    if ((given && !rows_of(*given, ma.rows, mb.rows, type)) || !all_on(aq->device(), {bq, given, status})) Py_RETURN_NONE;
    Tensor out[1];
    const int rc = on_device(*aq, [&] {
      out[0] = given ? *given : make({ma.rows, mb.rows}, *aq, type);
      return mok_fp8_matmul(&ma, &mb, ptr(out[0]), type == at::kFloat ? MOK_DT_FP32 : MOK_DT_BF16,
                            static_cast<uint32_t*>(ptr(status)), current_stream(*aq));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (x, w.q, w.s, w.cols, out, status) -> (out,)
PyObject* fp8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const Tensor *x, *wq, *ws, *given, *status;
    mok_fp8_matrix w{};
    if (n != 6 || !tensor_arg(a[0], &x) || !x || x->dim() != 2 || !fp8_arg(a[1], a[2], a[3], true, 0, &wq, &ws, &w) ||
        !tensor_arg(a[4], &given) || !status_arg(a[5], &status)) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    const int64_t M = x->size(0);
    if (!rows_of(*x, M, w.cols, at::kBFloat16) || (given && !rows_of(*given, M, w.rows, at::kBFloat16)) ||
        !all_on(x->device(), {wq, given, status}))
      Py_RETURN_NONE;
    const size_t bytes = mok_fp8_linear_workspace_bytes(M, w.cols);
    if (!bytes)  // rows or columns that the call refuses: it says how
      return PyLong_FromLong(mok_fp8_linear(x->data_ptr(), M, &w, nullptr, nullptr, 0, nullptr, nullptr));
    Tensor out[1];
    const int rc = on_device(*x, [&] {
      out[0] = given ? *given : make({M, w.rows}, *x, at::kBFloat16);
      const Tensor scratch = bytes > 256 ? make({static_cast<int64_t>(bytes)}, *x, at::kByte) : Tensor();  // else not used
      return mok_fp8_linear(x->data_ptr(), M, &w, ptr(out[0]), ptr(scratch), bytes,
                            static_cast<uint32_t*>(ptr(status)), current_stream(*x));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (schedule, device, a.q, a.s, a.cols, w.q, w.s, w.cols, out) -> (out,)
PyObject* fp8_grouped_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    PlacedSchedule p;
    const Tensor *aq, *as, *wq, *ws, *given;
    mok_fp8_matrix ma{}, w{};
    if (n != 9 || !sched_arg(a[0], a[1], &p) || !fp8_arg(a[2], a[3], a[4], false, 0, &aq, &as, &ma) ||
        !fp8_arg(a[5], a[6], a[7], true, 1, &wq, &ws, &w) || !tensor_arg(a[8], &given)) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    if (ma.rows != p.s->rpad_max || w.batch != p.s->shape.E || (given && !rows_of(*given, ma.rows, w.rows, at::kBFloat16)) ||
        aq->device().index() != p.device || !all_on(aq->device(), {wq, given}))
      Py_RETURN_NONE;
    Tensor out[1];
    const int rc = on_device(*aq, [&] {
      out[0] = given ? *given : make({ma.rows, w.rows}, *aq, at::kBFloat16);
      return mok_fp8_grouped_matmul(p.s, &ma, &w, ptr(out[0]), current_stream(*aq));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

// (schedule, device, a.q, a.s, a.cols, b.q, b.s, b.cols, out, f32) -> (out,)
PyObject* fp8_grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    PlacedSchedule p;
    const Tensor *aq, *as, *bq, *bs, *given;
    mok_fp8_matrix ma{}, mb{};
    if (n != 10 || !sched_arg(a[0], a[1], &p) || !fp8_arg(a[2], a[3], a[4], false, 0, &aq, &as, &ma) ||
        !fp8_arg(a[5], a[6], a[7], false, 0, &bq, &bs, &mb) || !tensor_arg(a[8], &given)) {
      if (PyErr_Occurred()) return nullptr;
      Py_RETURN_NONE;
    }
    const at::ScalarType type = PyObject_IsTrue(a[9]) ? at::kFloat : at::kBFloat16;
    const int64_t E = p.s->shape.E;
    if (aq->device().index() != p.device || !all_on(aq->device(), {bq, given}) ||
        (given && (!plain(*given, type) || given->dim() != 3 || given->size(0) != E || given->size(1) != ma.rows ||
                   given->size(2) != mb.rows)))
      Py_RETURN_NONE;
    Tensor out[1];
    const int rc = on_device(*aq, [&] {
      out[0] = given ? *given : make({E, ma.rows, mb.rows}, *aq, type);
      return mok_fp8_grouped_wgrad(p.s, &ma, &mb, ptr(out[0]), type == at::kFloat ? MOK_DT_FP32 : MOK_DT_BF16,
                                   current_stream(*aq));
    });
    return rc ? PyLong_FromLong(rc) : wrap_all(out);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<rmsnorm_forward>("rmsnorm_forward"), method<rmsnorm_backward>("rmsnorm_backward"),
                         method<dropout_forward>("dropout_forward"), method<dropout_backward>("dropout_backward"),
                         method<ffn_forward>("ffn_forward"), method<ffn_backward>("ffn_backward"),
                         method<move_rows<mok_dispatch, true>>("dispatch"),
                         method<move_rows<mok_dispatch_backward, false>>("dispatch_backward"),
                         method<move_rows<mok_combine, false>>("combine"), method<combine_backward>("combine_backward"),
                         method<fp8_quantize>("fp8_quantize"), method<fp8_quantize_blocks>("fp8_quantize_blocks"),
                         method<fp8_matmul>("fp8_matmul"), method<fp8_linear>("fp8_linear"),
                         method<fp8_grouped_matmul>("fp8_grouped_matmul"), method<fp8_grouped_wgrad>("fp8_grouped_wgrad"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_mok_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mok_bind() {
  PyObject* m = PyModule_Create(&module_def);
  if (m && PyModule_AddStringConstant(m, "built_for", MOK_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
