// binding.cpp - Python binding of the operators around the MLP (norm, 8-bit
// checkpoints, ragged products) on torch tensors.
//
// These calls take 2 to 5 us on the device at their smallest, and a binding in
// Python took 12 to 20 us for one: a microsecond and a half for each output that
// it allocated, as much again for its checks and for turning nineteen arguments
// into C values.  Here a call checks its tensors, allocates its outputs and calls
// the C entry point of include/mxmlp.h on the tensors' device and its current
// stream in one go (4 to 7 us).  Refusals raise MxError with the status and text
// that the C entry gives, allocation failures torch's own error; no C++ exception
// leaves a function.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string>
#include <utility>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxmlp.h"

namespace {

PyObject* g_error = nullptr;  // MxError

struct Refusal {
  int status;
  std::string text;
};

[[noreturn]] void refuse(std::string text) { throw Refusal{MX_ERR_INVALID_ARG, std::move(text)}; }

void check(int rc) {
  if (rc) throw Refusal{rc, std::string(mx_status_string(rc)) + ": " + mx_last_error()};
}

template <class F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal& r) {
    PyObject* e = PyObject_CallFunction(g_error ? g_error : PyExc_RuntimeError, "is", r.status, r.text.c_str());
    if (e) {
      PyErr_SetObject((PyObject*)Py_TYPE(e), e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

// A contiguous CUDA tensor of the type, on the first tensor's device.
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType type, const at::Tensor* first = nullptr) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  if (first && t.device() != first->device()) refuse(std::string(name) + " must be on the same device");
  return t;
}

const at::Tensor& need(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Tensor* first) {
  const at::Tensor& t = need(o, name, type, first);
  if (t.sizes() != shape)
    refuse(std::string(name) + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  return t;
}

const at::Tensor& matrix(PyObject* o, const char* name, const at::Tensor* first = nullptr) {
  const at::Tensor& t = need(o, name, at::kBFloat16, first);
  if (t.dim() != 2) refuse(std::string(name) + " must be a matrix, got " + shape_text(t.sizes()));
  return t;
}

// From the caching allocator without the dispatcher's rounds (1.2 us an output with
// them, 0.8 without).
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The device of a call's tensors, made current, and its current stream, with
// the interpreter's lock released: an allocation or a launch may wait for the
// device, and other threads run meanwhile.  finish() takes the lock back and
// turns a status into a refusal.
struct On {
  c10::cuda::CUDAGuard guard;
  void* stream;
  PyThreadState* thread;  // last: what may throw comes before it
  explicit On(const at::Tensor& t)
      : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()),
        thread(PyEval_SaveThread()) {}
  void finish(int rc) {
    lock();
    check(rc);
  }
  ~On() { lock(); }
  On(const On&) = delete;
  On& operator=(const On&) = delete;

 private:
  void lock() {
    if (thread) PyEval_RestoreThread(thread);
    thread = nullptr;
  }
};

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

template <class... T>
PyObject* tuple_of(const T&... t) {
  PyObject* items[] = {wrap(t)...};
  PyObject* out = PyTuple_New(sizeof...(T));
  bool ok = out != nullptr;
  for (size_t i = 0; i < sizeof...(T); ++i) {
    ok = ok && items[i];
    if (out && items[i]) PyTuple_SET_ITEM(out, i, items[i]);
    else Py_XDECREF(items[i]);
  }
  if (!ok) {
    Py_XDECREF(out);
    return nullptr;
  }
  return out;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("expected a whole number");
  }
  return v;
}

int small_integer(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return (int)v;
}

bool truth(PyObject* o, const char* name) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) {
    PyErr_Clear();
    refuse(std::string(name) + " must be true or false");
  }
  return t == 1;
}

void arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse("wrong number of arguments");
}

at::Tensor scales(int64_t rows, int64_t cols, int layout, const at::Tensor& like) {
  const int64_t s = cols / 32;
  return empty({layout == MX_SCALE_MMA ? (rows + 127) / 128 * ((s + 3) / 4) * 512 : rows * s}, at::kByte, like);
}

// ckpt8_save(x) -> (codes, scales)
PyObject* py_ckpt8_save(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 1);
    const at::Tensor& x = matrix(a[0], "x");
    On on(x);
    const int64_t rows = x.size(0), cols = x.size(1);
    at::Tensor codes = empty({rows, cols}, at::kChar, x), sc = empty({rows, cols / 32}, at::kByte, x);
    on.finish(mx_ckpt8_save(ptr(x), rows, cols, ptr(codes), ptr(sc), on.stream));
    return tuple_of(codes, sc);
  });
}

// The two tensors of a checkpoint of a [rows, cols] matrix (-1: whatever codes has).
void checkpoint(PyObject* codes, PyObject* sc, int64_t rows, int64_t cols, const char* name, const at::Tensor* first,
                const at::Tensor** c, const at::Tensor** s) {
  *c = &need(codes, name, at::kChar, first);
  *s = &need(sc, name, at::kByte, *c);
  if ((*c)->dim() != 2) refuse(std::string(name) + " must hold a matrix");
  if (rows < 0) rows = (*c)->size(0), cols = (*c)->size(1);
  const int64_t want[2] = {rows, cols}, want_s[2] = {rows, cols / 32};
  if ((*c)->sizes() != at::IntArrayRef(want) || (*s)->sizes() != at::IntArrayRef(want_s))
    refuse(std::string(name) + " must be a checkpoint of a " + shape_text(want) + " matrix, got " +
           shape_text((*c)->sizes()) + " with scales " + shape_text((*s)->sizes()));
}

// ckpt8_load(codes, scales) -> x
PyObject* py_ckpt8_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 2);
    const at::Tensor *c, *s;
    checkpoint(a[0], a[1], -1, -1, "ck", nullptr, &c, &s);
    On on(*c);
    at::Tensor x = empty(c->sizes(), at::kBFloat16, *c);
    on.finish(mx_ckpt8_load(ptr(*c), ptr(*s), c->size(0), c->size(1), ptr(x), on.stream));
    return wrap(x);
  });
}

// swiglu_ckpt8_fwd(h13) -> (y, codes, scales)
PyObject* py_swiglu_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 1);
    const at::Tensor& h13 = matrix(a[0], "h13");
    const int64_t M = h13.size(0), h2 = h13.size(1), h = h2 / 2;
    if (h2 % 64)
      throw Refusal{MX_ERR_UNSUPPORTED, "h13 must have 2h columns with h a multiple of 32, got " + std::to_string(h2)};
    On on(h13);
    at::Tensor y = empty({M, h}, at::kBFloat16, h13), codes = empty({M, h2}, at::kChar, h13);
    at::Tensor sc = empty({M, h2 / 32}, at::kByte, h13);
    on.finish(mx_swiglu_ckpt8_fwd(ptr(h13), M, h, ptr(y), ptr(codes), ptr(sc), on.stream));
    return tuple_of(y, codes, sc);
  });
}

// swiglu_ckpt8_bwd(dy, codes, scales, want_y) -> (dh13, y or None)
PyObject* py_swiglu_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 4);
    const at::Tensor& dy = matrix(a[0], "dy");
    const int64_t M = dy.size(0), h = dy.size(1);
    const at::Tensor *c, *s;
    checkpoint(a[1], a[2], M, 2 * h, "ck", &dy, &c, &s);
    const bool want_y = truth(a[3], "y");
    On on(dy);
    at::Tensor dh13 = empty({M, 2 * h}, at::kBFloat16, dy), y;
    if (want_y) y = empty({M, h}, at::kBFloat16, dy);
    on.finish(mx_swiglu_ckpt8_bwd(ptr(dy), ptr(*c), ptr(*s), M, h, ptr(dh13), ptr(y), on.stream));
    return tuple_of(dh13, y);
  });
}

// add_rmsnorm_fwd(x, w, residual, eps, y, axis, layout, scale_mode, ckpt)
//   -> (r, rstd, y, q_row, s_row, q_col, s_col, codes, scales), None where not asked for; r: the sum, or x
PyObject* py_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 9);
    const at::Tensor& x = matrix(a[0], "x");
    const int64_t M = x.size(0), d = x.size(1);
    const at::Tensor& w = need(a[1], "w", at::kBFloat16, {d}, &x);
    const at::Tensor* residual = a[2] == Py_None ? nullptr : &need(a[2], "residual", at::kBFloat16, x.sizes(), &x);
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("eps must be a number");
    }
    const bool want_y = truth(a[4], "y"), ckpt = truth(a[8], "ckpt");
    const int axis = small_integer(a[5], "axis"), layout = small_integer(a[6], "layout");
    const int mode = small_integer(a[7], "scale_mode");
    On on(x);
    at::Tensor r, y, q_row, s_row, q_col, s_col, codes, sc;
    if (residual) r = empty({M, d}, at::kBFloat16, x);
    at::Tensor rstd = empty({M}, at::kFloat, x);
    if (want_y) y = empty({M, d}, at::kBFloat16, x);
    if (axis & MX_ROW) {
      q_row = empty({M, d}, at::kByte, x);
      s_row = scales(M, d, layout, x);
    }
    if (axis & MX_COL) {
      q_col = empty({d, M}, at::kByte, x);
      s_col = scales(d, M, layout, x);
    }
    if (ckpt) {
      codes = empty({M, d}, at::kChar, x);
      sc = empty({M, d / 32}, at::kByte, x);
    }
    on.finish(mx_add_rmsnorm_fwd(ptr(x), residual ? ptr(*residual) : nullptr, ptr(w), M, d, (float)eps, ptr(r),
                                 (float*)ptr(rstd), ptr(y), axis, layout, mode, ptr(q_row), ptr(s_row),
                                 ptr(q_col), ptr(s_col), ptr(codes), ptr(sc), on.stream));
    return tuple_of(residual ? r : x, rstd, y, q_row, s_row, q_col, s_col, codes, sc);
  });
}

// add_rmsnorm_bwd(dy, r, codes, scales, rstd, w, dres) -> (dx, dw); r, or codes and scales, and dres may be None
PyObject* py_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 7);
    const at::Tensor& dy = matrix(a[0], "dy");
    const int64_t M = dy.size(0), d = dy.size(1);
    const at::Tensor *r = nullptr, *c = nullptr, *s = nullptr;
    if (a[2] == Py_None) r = &need(a[1], "saved", at::kBFloat16, dy.sizes(), &dy);
    else checkpoint(a[2], a[3], M, d, "saved", &dy, &c, &s);
    const at::Tensor& rstd = need(a[4], "rstd", at::kFloat, {M}, &dy);
    const at::Tensor& w = need(a[5], "w", at::kBFloat16, {d}, &dy);
    const at::Tensor* dres = a[6] == Py_None ? nullptr : &need(a[6], "dres", at::kBFloat16, dy.sizes(), &dy);
    On on(dy);
    at::Tensor dx = empty({M, d}, at::kBFloat16, dy), dw = empty({d}, at::kBFloat16, dy);
    at::Tensor ws = empty({(int64_t)mx_add_rmsnorm_bwd_workspace(M, d) + 16}, at::kByte, dy);
    on.finish(mx_add_rmsnorm_bwd(ptr(dy), r ? ptr(*r) : nullptr, c ? ptr(*c) : nullptr, s ? ptr(*s) : nullptr,
                                 (const float*)ptr(rstd), ptr(w), dres ? ptr(*dres) : nullptr, M, d, ptr(dx), ptr(dw),
                                 ptr(ws), on.stream));
    return tuple_of(dx, dw);
  });
}

// ragged(mode, a, b, offs, err) -> c; err: an error word's tensor, or None
PyObject* py_ragged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 5);
    const int mode = small_integer(a[0], "mode");
    const at::Tensor& t = matrix(a[1], mode == MX_RAGGED_FWD ? "x" : "dout");
    const at::Tensor& offs = need(a[3], "offs", at::kInt, &t);
    void* err = a[4] == Py_None ? nullptr : ptr(need(a[4], "err", at::kInt, {1}, &t));
    const int64_t M = t.size(0), E = offs.numel();
    if (E < 1 || E > 1024) refuse("E must be in [1, 1024], got " + std::to_string(E));  // before dw is allocated
    int64_t N, K;
    const at::Tensor* b;
    at::Tensor c;
    if (mode == MX_RAGGED_WGRAD) {
      b = &matrix(a[2], "x", &t);
      if (b->size(0) != M)
        refuse("dout and x must have the same rows, got " + std::to_string(M) + " and " + std::to_string(b->size(0)));
      N = t.size(1);
      K = b->size(1);
    } else {
      b = &need(a[2], "w", at::kBFloat16, &t);
      if (b->dim() != 3 || b->size(0) != E)
        refuse("w must be [E, N, K] with E = " + std::to_string(E) + ", got " + shape_text(b->sizes()));
      N = b->size(1);
      K = b->size(2);
      const int64_t cols = mode == MX_RAGGED_FWD ? K : N;
      if (t.size(1) != cols)
        refuse(std::string(mode == MX_RAGGED_FWD ? "x" : "dout") + " must have " + std::to_string(cols) + " columns, got " +
               std::to_string(t.size(1)));
    }
    On on(t);
    if (mode == MX_RAGGED_WGRAD) c = empty({E, N, K}, at::kBFloat16, t);
    else c = empty({M, mode == MX_RAGGED_FWD ? N : K}, at::kBFloat16, t);
    on.finish(mx_ragged_mm(mode, ptr(t), ptr(*b), M, N, K, (const int32_t*)ptr(offs), (int32_t)E, ptr(c),
                           (int32_t*)err, on.stream));
    return wrap(c);
  });
}

// set_error(MxError)
PyObject* py_set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  Py_INCREF(cls);
  g_error = cls;
  Py_RETURN_NONE;
}

#define MX_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {{"set_error", py_set_error, METH_O, nullptr},
                           {"ckpt8_save", MX_FAST(py_ckpt8_save)},
                           {"ckpt8_load", MX_FAST(py_ckpt8_load)},
                           {"swiglu_ckpt8_fwd", MX_FAST(py_swiglu_fwd)},
                           {"swiglu_ckpt8_bwd", MX_FAST(py_swiglu_bwd)},
                           {"add_rmsnorm_fwd", MX_FAST(py_norm_fwd)},
                           {"add_rmsnorm_bwd", MX_FAST(py_norm_bwd)},
                           {"ragged", MX_FAST(py_ragged)},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
