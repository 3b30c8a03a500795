// binding.cpp -- the Python side of the short calls: norm, dropout, rows as
// e4m3 numbers and the linear product (include/tps.h), as a CPython extension.
//
// These calls take a few microseconds on the GPU; views of six or seven
// tensors and three or four allocations cost several times that in Python (a
// norm of 64 rows 39 us, with 5.6 us of kernel).  Here a call takes its tensors
// from their C++ objects, makes its outputs with ATen and calls the library
// through the addresses that init() was given, those of the build that api.py
// has loaded.  No computation: argument marshalling only.
//
// Every function returns what its wrapper in api.py returns, or an int, the
// library's status, where that is not TPS_OK; it raises where an argument is
// not what a view can be made of.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <optional>

#include "tps.h"

namespace {

using at::Tensor;

struct Entries {
  decltype(&tps_rmsnorm_fwd) rmsnorm_fwd;
  decltype(&tps_rmsnorm_bwd) rmsnorm_bwd;
  decltype(&tps_rmsnorm_workspace_bytes) rmsnorm_workspace_bytes;
  decltype(&tps_dropout_fwd) dropout_fwd;
  decltype(&tps_dropout_bwd) dropout_bwd;
  decltype(&tps_quantize_e4m3) quantize_e4m3;
  decltype(&tps_linear_fwd) linear_fwd;
  decltype(&tps_linear_bwd) linear_bwd;
  decltype(&tps_linear_workspace_bytes) linear_workspace_bytes;
};
Entries f = {};

struct Raised {};  // a Python error is set
[[noreturn]] void raise(PyObject* type, const char* what) {
  PyErr_SetString(type, what);
  throw Raised();
}

// The tensor of an argument, nullptr for None.
const Tensor* tensor(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "expected a torch.Tensor");
  return &THPVariable_Unpack(o);
}

// Collects the tensors of a call: all on the current GPU, where the kernels
// are going to run.
struct Call {
  int device = -1;
  bool cpu = false, several = false;
  void on(const Tensor* t) {
    if (t == nullptr) return;
    if (!t->is_cuda()) {
      cpu = true;
      return;
    }
    const int d = t->get_device();
    if (device >= 0 && d != device) several = true;
    device = d;
  }
  void check() const {
    if (cpu) raise(PyExc_ValueError, "tensors must live on the GPU (no CPU path)");
    if (several) raise(PyExc_ValueError, "tensors on different GPUs");
    if (device >= 0 && device != static_cast<int>(c10::cuda::current_device()))
      raise(PyExc_ValueError, "tensors on another GPU than the current one");
  }
  void* stream() const {
    return device < 0 ? nullptr : c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  }
};

// A view of a tensor; `p()` is NULL for none.
struct View {
  tps_tensor t;
  bool some = false;
  const tps_tensor* p() const { return some ? &t : nullptr; }
};
int dtype_of(at::ScalarType s, bool codes) {
  switch (s) {
    case at::kFloat: return TPS_F32;
    case at::kBFloat16: return TPS_BF16;
    case at::kInt: return TPS_I32;
    case at::kLong: return TPS_I64;
    case at::kFloat8_e4m3fn:
      if (codes) return TPS_E4M3;
      [[fallthrough]];
    default: PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(s)); throw Raised();
  }
}
enum Form { AS_IS, ROWS, FLAT };  // ROWS: a vector is one row; FLAT: a contiguous tensor is a vector
View view(const Tensor* x, Form form = AS_IS, bool codes = false) {
  View v;
  if (x == nullptr) return v;
  v.some = true;
  v.t.data = x->data_ptr();
  v.t.dtype = dtype_of(x->scalar_type(), codes);
  const int64_t n = x->dim();
  if (form == FLAT && n != 1 && x->is_contiguous()) {
    v.t.ndim = 1;
    v.t.shape[0] = x->numel();
    v.t.stride[0] = 1;
    return v;
  }
  if (n < 1 || n > 4) raise(PyExc_ValueError, "shape");
  const int add = form == ROWS && n == 1 ? 1 : 0;
  v.t.ndim = static_cast<int32_t>(n) + add;
  if (add) {
    v.t.shape[0] = 1;
    v.t.stride[0] = x->size(0) * x->stride(0);
  }
  for (int64_t i = 0; i < n; ++i) {
    v.t.shape[i + add] = x->size(i);
    v.t.stride[i + add] = x->stride(i);
  }
  return v;
}

// Without the dispatcher, a third of an allocation's time.
Tensor make(c10::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
at::ScalarType type_of(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) raise(PyExc_TypeError, "expected a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
// The entries of `out` (a sequence of n tensors or None).
struct Given {
  PyObject* seq = nullptr;
  Given(PyObject* o, Py_ssize_t n) {
    if (o == Py_None) return;
    seq = PySequence_Fast(o, "out: a sequence of tensors");
    if (seq == nullptr) throw Raised();
    if (PySequence_Fast_GET_SIZE(seq) != n) {
      Py_DECREF(seq);
      raise(PyExc_ValueError, "out: another number of tensors");
    }
  }
  ~Given() { Py_XDECREF(seq); }
  explicit operator bool() const { return seq != nullptr; }
  std::optional<Tensor> at(Py_ssize_t i) const {
    const Tensor* t = tensor(PySequence_Fast_GET_ITEM(seq, i));
    return t == nullptr ? std::nullopt : std::optional<Tensor>(*t);
  }
};
const Tensor* ptr(const std::optional<Tensor>& t) { return t.has_value() ? &*t : nullptr; }
// The caller's tensors hold something else now: what an eager graph saved of them is
// not what it computed with, and its backward pass raises instead of using it.
// (Inference tensors have no such count, and no graph saves them.)
template <class... T>
void written(const T&... given) {
  auto one = [](const Tensor* t) {
    if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
  };
  (one(ptr(given)), ...);
}
PyObject* wrap(const std::optional<Tensor>& t) { return t.has_value() ? THPVariable_Wrap(*t) : Py_NewRef(Py_None); }
template <class... T>
PyObject* tuple_of(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(t));
  if (r == nullptr) throw Raised();
  Py_ssize_t i = 0;
  bool ok = true;
  auto put = [&](const std::optional<Tensor>& x) {
    PyObject* o = wrap(x);
    ok = ok && o != nullptr;
    PyTuple_SET_ITEM(r, i++, o);
  };
  (put(t), ...);
  if (!ok) {
    Py_DECREF(r);
    throw Raised();
  }
  return r;
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised();
  return x;
}
uint64_t word(PyObject* o) {
  const unsigned long long x = PyLong_AsUnsignedLongLongMask(o);
  if (x == static_cast<unsigned long long>(-1) && PyErr_Occurred()) throw Raised();
  return x;
}
int integer(PyObject* o) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  return static_cast<int>(x);
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised();
  return x != 0;
}
// p, seed (a number or one int64 on the GPU) and site.
tps_dropout dropout_of(PyObject* p, PyObject* seed, PyObject* site, Call* call) {
  tps_dropout d = {};
  d.p = number(p);
  d.site = word(site);
  if (THPVariable_Check(seed)) {
    const Tensor& t = THPVariable_Unpack(seed);
    if (t.scalar_type() != at::kLong || t.numel() != 1) raise(PyExc_ValueError, "seed: one int64");
    call->on(&t);
    d.seed_ptr = static_cast<const int64_t*>(t.data_ptr());
  } else {
    d.seed = word(seed);
  }
  return d;
}

// A workspace that the caller gave.
void given_room(const Tensor& w) {
  if (!w.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
}

// Runs the library's call without the interpreter's lock.
template <class F>
int run(F&& body) {
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = body();
  Py_END_ALLOW_THREADS;
  return rc;
}

c10::IntArrayRef leading(const Tensor& x) { return x.sizes().slice(0, x.dim() - 1); }
void has_rows(const Tensor* x) {
  if (x == nullptr) raise(PyExc_TypeError, "expected a torch.Tensor");
  if (x->dim() < 1) raise(PyExc_ValueError, "shape");
}

// (x, weight, residual, eps, dropout, seed, site, out_dtype, out)
PyObject* rmsnorm_fwd(PyObject* const* a) {
  Call call;
  const Tensor *x = tensor(a[0]), *w = tensor(a[1]), *res = tensor(a[2]);
  has_rows(x);
  const double eps = number(a[3]);
  const tps_dropout d = dropout_of(a[4], a[5], a[6], &call);
  const bool dropped = d.p != 0.0;
  for (const Tensor* t : {x, w, res}) call.on(t);
  call.check();
  std::optional<Tensor> y, scale, h, rstd;
  if (const Given out(a[8], 4); out) {
    y = out.at(0);
    scale = out.at(1);
    h = out.at(2);
    rstd = out.at(3);
    for (const auto* t : {&y, &scale, &h, &rstd}) call.on(ptr(*t));
    call.check();
  } else {
    const at::ScalarType type = type_of(a[7], x->scalar_type());
    y = make(x->sizes(), type, *x);
    if (type == at::kFloat8_e4m3fn) scale = make(leading(*x), at::kFloat, *x);
    if (res != nullptr || dropped) h = make(x->sizes(), (res != nullptr ? res : x)->scalar_type(), *x);
    rstd = make(leading(*x), at::kFloat, *x);
  }
  const View vx = view(x, ROWS), vr = view(res, ROWS), vw = view(w), vh = view(ptr(h), ROWS), vy = view(ptr(y), ROWS, true);
  const View vs = view(ptr(scale), FLAT), vd = view(ptr(rstd), FLAT);
  void* stream = call.stream();
  const int rc = run([&] {
    return f.rmsnorm_fwd(vx.p(), vr.p(), vw.p(), eps, dropped ? &d : nullptr, vh.p(), vy.p(), vs.p(), vd.p(), stream);
  });
  if (rc != TPS_OK) return PyLong_FromLong(rc);
  if (a[8] != Py_None) written(y, scale, h, rstd);
  return tuple_of(y, scale, h, rstd);
}

// (dy, h, weight, rstd, dh, dropout, seed, site, x_dtype, want_dweight, workspace, out)
PyObject* rmsnorm_bwd(PyObject* const* a) {
  Call call;
  const Tensor *dy = tensor(a[0]), *h = tensor(a[1]), *w = tensor(a[2]), *rstd = tensor(a[3]), *dh = tensor(a[4]);
  const Tensor* ws = tensor(a[10]);
  has_rows(dy);
  has_rows(h);
  const tps_dropout d = dropout_of(a[5], a[6], a[7], &call);
  const bool dropped = d.p != 0.0;
  for (const Tensor* t : {dy, h, w, rstd, dh, ws}) call.on(t);
  call.check();
  std::optional<Tensor> dx, dres, dw;
  bool one = false;  // dx is dres
  if (const Given out(a[11], 3); out) {
    dx = out.at(0);
    dres = out.at(1);
    dw = out.at(2);
    for (const auto* t : {&dx, &dres, &dw}) call.on(ptr(*t));
    call.check();
    one = dx.has_value() && dres.has_value() && !dropped && dx->is_same(*dres);
  } else {
    const at::ScalarType type = type_of(a[8], h->scalar_type());
    dres = make(h->sizes(), h->scalar_type(), *h);
    one = !dropped && type == h->scalar_type();
    dx = one ? *dres : make(h->sizes(), type, *h);
    if (truth(a[9])) dw = make({h->size(-1)}, at::kFloat, *h);
  }
  const int64_t width = h->size(-1);
  size_t bytes = 0;
  std::optional<Tensor> room;
  void* at_room = nullptr;
  if (ws != nullptr) {
    given_room(*ws);
    at_room = ws->data_ptr();
    bytes = ws->nbytes();
  } else if (dw.has_value()) {
    bytes = f.rmsnorm_workspace_bytes(width > 0 ? h->numel() / width : 0, width);
    room = make({static_cast<int64_t>(bytes)}, at::kByte, *h);
    at_room = room->data_ptr();
  }
  const View vy = view(dy, ROWS), vh = view(h, ROWS), vw = view(w), vr = view(rstd, FLAT), vu = view(dh, ROWS);
  const View vs = view(ptr(dres), ROWS), vx = one ? View() : view(ptr(dx), ROWS), vd = view(ptr(dw));
  void* stream = call.stream();
  const int rc = run([&] {
    return f.rmsnorm_bwd(vy.p(), vh.p(), vw.p(), vr.p(), vu.p(), dropped ? &d : nullptr, vs.p(), vx.p(), vd.p(), at_room,
                         bytes, stream);
  });
  if (rc != TPS_OK) return PyLong_FromLong(rc);
  if (a[11] != Py_None) written(dx, dres, dw);
  if (!one) return tuple_of(dx, dres, dw);
  PyObject* t = wrap(dres);  // one object for both
  PyObject* u = t == nullptr ? nullptr : wrap(dw);
  PyObject* r = u == nullptr ? nullptr : PyTuple_Pack(3, t, t, u);
  Py_XDECREF(t);
  Py_XDECREF(u);
  if (r == nullptr) throw Raised();
  return r;
}

// (x, p, seed, site, residual, out, backward)
PyObject* dropout(PyObject* const* a) {
  Call call;
  const Tensor *x = tensor(a[0]), *res = tensor(a[4]), *given = tensor(a[5]);
  has_rows(x);
  const tps_dropout d = dropout_of(a[1], a[2], a[3], &call);
  for (const Tensor* t : {x, res, given}) call.on(t);
  call.check();
  const std::optional<Tensor> y = given != nullptr ? *given : make(x->sizes(), x->scalar_type(), *x);
  const View vx = view(x, ROWS), vr = view(res, ROWS), vy = view(ptr(y), ROWS);
  const bool back = truth(a[6]);
  void* stream = call.stream();
  const int rc = run([&] {
    return back ? f.dropout_bwd(vx.p(), &d, vy.p(), stream) : f.dropout_fwd(vx.p(), vr.p(), &d, vy.p(), stream);
  });
  if (rc != TPS_OK) return PyLong_FromLong(rc);
  if (given != nullptr) written(y);
  return wrap(y);
}

// (x, out)
PyObject* quantize_e4m3(PyObject* const* a) {
  Call call;
  const Tensor* x = tensor(a[0]);
  has_rows(x);
  call.on(x);
  call.check();
  std::optional<Tensor> q, scale;
  if (const Given out(a[1], 2); out) {
    q = out.at(0);
    scale = out.at(1);
    call.on(ptr(q));
    call.on(ptr(scale));
    call.check();
  } else {
    q = make(x->sizes(), at::kFloat8_e4m3fn, *x);
    scale = make(leading(*x), at::kFloat, *x);
  }
  const View vx = view(x, ROWS), vq = view(ptr(q), ROWS, true), vs = view(ptr(scale), FLAT);
  void* stream = call.stream();
  const int rc = run([&] { return f.quantize_e4m3(vx.p(), vq.p(), vs.p(), stream); });
  if (rc != TPS_OK) return PyLong_FromLong(rc);
  if (a[1] != Py_None) written(q, scale);
  return tuple_of(q, scale);
}

// Runs body(workspace, bytes) with the caller's workspace, or with the least that
// may do: a call that needs more is refused before any launch and run again.  A few
// fp32 rows mostly need none; then comes the size for aligned operands, and at last
// the one that holds all of them laid out.
constexpr int64_t kFewRows = 8;
template <class F>
int with_room(const Tensor* ws, const Tensor& x, int64_t T, int64_t K, int64_t N, int backward, F&& body) {
  if (ws != nullptr) {
    given_room(*ws);
    void* p = ws->data_ptr();
    const size_t n = ws->nbytes();
    return run([&] { return body(p, n); });
  }
  const int own = dtype_of(x.scalar_type(), true);
  const size_t aligned = f.linear_workspace_bytes(T, K, N, own, backward);
  const size_t laid = own == TPS_BF16 ? f.linear_workspace_bytes(T, K, N, TPS_F32, backward) : aligned;
  const bool few = own == TPS_F32 && !backward && T <= kFewRows;
  int rc = TPS_ERR_WORKSPACE;
  std::optional<size_t> had;
  for (const size_t n : {few ? size_t(0) : aligned, aligned, laid}) {
    if (rc != TPS_ERR_WORKSPACE) break;
    if (had.has_value() && n <= *had) continue;
    std::optional<Tensor> room;
    if (n > 0) room = make({static_cast<int64_t>(n)}, at::kByte, x);
    void* p = n > 0 ? room->data_ptr() : nullptr;
    rc = run([&] { return body(p, n); });
    had = n;
  }
  return rc;
}
struct Sizes {
  int64_t T, K, N;
};
Sizes sizes_of(const Tensor* x, const Tensor* W, int layout) {
  has_rows(x);
  if (W == nullptr) raise(PyExc_TypeError, "expected a torch.Tensor");
  if (W->dim() != 2) raise(PyExc_ValueError, "shape");
  const int64_t K = x->size(-1);
  return {K > 0 ? x->numel() / K : 0, K, W->size(layout == TPS_W_IN_OUT ? 1 : 0)};
}

// (x, W, bias, residual, act, layout, x_scale, w_scale, want_pre, out_dtype, workspace, out)
PyObject* linear_fwd(PyObject* const* a) {
  Call call;
  const Tensor *x = tensor(a[0]), *W = tensor(a[1]), *bias = tensor(a[2]), *res = tensor(a[3]);
  const Tensor *xs = tensor(a[6]), *wsc = tensor(a[7]), *ws = tensor(a[10]);
  const int act = integer(a[4]), layout = integer(a[5]);
  const Sizes s = sizes_of(x, W, layout);
  for (const Tensor* t : {x, W, bias, res, xs, wsc, ws}) call.on(t);
  call.check();
  std::optional<Tensor> y, z;
  if (const Given out(a[11], 2); out) {
    y = out.at(0);
    z = out.at(1);
    call.on(ptr(y));
    call.on(ptr(z));
    call.check();
  } else {
    const at::ScalarType type =
        type_of(a[9], x->scalar_type() == at::kFloat8_e4m3fn ? at::kBFloat16 : x->scalar_type());
    c10::SmallVector<int64_t, 4> shape(x->sizes().begin(), x->sizes().end());
    shape.back() = s.N;
    y = make(shape, type, *x);
    if (truth(a[8])) z = make(shape, type, *x);
  }
  const View vx = view(x, ROWS, true), vw = view(W, AS_IS, true), vb = view(bias), vr = view(res, ROWS);
  const View v1 = view(xs, FLAT), v2 = view(wsc, FLAT), vz = view(ptr(z), ROWS), vy = view(ptr(y), ROWS);
  void* stream = call.stream();
  const int rc = with_room(ws, *x, s.T, s.K, s.N, 0, [&](void* p, size_t n) {
    return f.linear_fwd(vx.p(), vw.p(), vb.p(), vr.p(), act, layout, v1.p(), v2.p(), vz.p(), vy.p(), p, n, stream);
  });
  if (rc != TPS_OK) return PyLong_FromLong(rc);
  if (a[11] != Py_None) written(y, z);
  return tuple_of(y, z);
}

// (x, W, dy, pre, act, layout, want_dx, want_dw, want_dbias, grad_dtype, workspace, out)
PyObject* linear_bwd(PyObject* const* a) {
  Call call;
  const Tensor *x = tensor(a[0]), *W = tensor(a[1]), *dy = tensor(a[2]), *pre = tensor(a[3]), *ws = tensor(a[10]);
  const int act = integer(a[4]), layout = integer(a[5]);
  const Sizes s = sizes_of(x, W, layout);
  for (const Tensor* t : {x, W, dy, pre, ws}) call.on(t);
  call.check();
  std::optional<Tensor> dx, dw, db;
  if (const Given out(a[11], 3); out) {
    dx = out.at(0);
    dw = out.at(1);
    db = out.at(2);
    for (const auto* t : {&dx, &dw, &db}) call.on(ptr(*t));
    call.check();
  } else {
    const at::ScalarType type = type_of(a[9], at::kFloat);
    if (truth(a[6])) dx = make(x->sizes(), type, *x);
    if (truth(a[7])) dw = make(W->sizes(), type, *x);
    if (truth(a[8])) db = make({s.N}, type, *x);
  }
  const View vx = view(x, ROWS), vw = view(W), vy = view(dy, ROWS), vz = view(pre, ROWS);
  const View v1 = view(ptr(dx), ROWS), v2 = view(ptr(dw)), v3 = view(ptr(db));
  void* stream = call.stream();
  const int rc = with_room(ws, *x, s.T, s.K, s.N, 1, [&](void* p, size_t n) {
    return f.linear_bwd(vx.p(), vw.p(), vy.p(), vz.p(), act, layout, v1.p(), v2.p(), v3.p(), p, n, stream);
  });
  if (rc != TPS_OK) return PyLong_FromLong(rc);
  if (a[11] != Py_None) written(dx, dw, db);
  return tuple_of(dx, dw, db);
}

// Addresses of the library's entry points, in the order of Entries.
PyObject* init(PyObject* const* a) {
  void* p[sizeof(Entries) / sizeof(void*)];
  for (size_t i = 0; i < sizeof(p) / sizeof(p[0]); ++i) p[i] = reinterpret_cast<void*>(word(a[i]));
  static_assert(sizeof(p) == sizeof(Entries), "one address each");
  memcpy(&f, p, sizeof(f));
  return Py_NewRef(Py_None);
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  HANDLE_TH_ERRORS  // ATen's exceptions, running out of memory among them, as torch raises them
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<init, sizeof(Entries) / sizeof(void*)>("init"),
    method<rmsnorm_fwd, 9>("rmsnorm_fwd"),
    method<rmsnorm_bwd, 12>("rmsnorm_bwd"),
    method<dropout, 7>("dropout"),
    method<quantize_e4m3, 2>("quantize_e4m3"),
    method<linear_fwd, 12>("linear_fwd"),
    method<linear_bwd, 12>("linear_bwd"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
