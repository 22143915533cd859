// binding.cpp - Python binding of the operators around the MLP (norm, 8-bit
// checkpoints, ragged products, routing, FP8 with 128-blocks) on torch tensors.
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

// A router's logits: a matrix of bf16 or fp32.
const at::Tensor& logits_of(PyObject* o, const at::Tensor* first = nullptr) {
  const bool wide = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kFloat;
  const at::Tensor& t = need(o, "logits", wide ? at::kFloat : at::kBFloat16, first);
  if (t.dim() != 2) refuse("logits must be a matrix, got " + shape_text(t.sizes()));
  return t;
}

int float_type(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? MX_FP32 : MX_BF16; }

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return (float)v;
}

int32_t* error_word(PyObject* o, const at::Tensor& first) {
  return o == Py_None ? nullptr : (int32_t*)ptr(need(o, "err", at::kInt, {1}, &first));
}

// Experts of a matrix of logits, as the C entries take them.
int32_t experts_of(const at::Tensor& logits) {
  const int64_t E = logits.size(1);
  if (E < 1 || E > 1024) refuse("E must be in [1, 1024], got " + std::to_string(E));
  return (int32_t)E;
}

// Refused before an output of that width is allocated.
int32_t top_k(PyObject* o, int64_t E) {
  const int k = small_integer(o, "k");
  if (k < 1 || k > 32 || k > E) refuse("k must be in [1, 32] and at most E, got " + std::to_string(k));
  return k;
}

// moe_route(logits, k, score, bias, groups, top_groups, renorm, scale) -> (ids, weights)
PyObject* py_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 8);
    const at::Tensor& l = logits_of(a[0]);
    const int64_t T = l.size(0);
    const int32_t E = experts_of(l), k = top_k(a[1], E);
    const int score = small_integer(a[2], "score"), groups = small_integer(a[4], "groups");
    const at::Tensor* bias = a[3] == Py_None ? nullptr : &need(a[3], "bias", at::kFloat, {(int64_t)E}, &l);
    const int top = small_integer(a[5], "top_groups");
    const bool renorm = truth(a[6], "renorm");
    const float scale = number(a[7], "scale");
    On on(l);
    at::Tensor ids = empty({T, k}, at::kInt, l), w = empty({T, k}, at::kFloat, l);
    on.finish(mx_moe_route(ptr(l), float_type(l), T, E, k, score, bias ? (const float*)ptr(*bias) : nullptr, groups, top, renorm,
                           scale, (int32_t*)ptr(ids), (float*)ptr(w), on.stream));
    return tuple_of(ids, w);
  });
}

// moe_route_bwd(dweights, logits, ids, score, renorm, scale, err) -> dlogits
PyObject* py_route_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 7);
    const at::Tensor& l = logits_of(a[1]);
    const int64_t T = l.size(0);
    const int32_t E = experts_of(l);
    const at::Tensor& dw = need(a[0], "dweights", at::kFloat, &l);
    if (dw.dim() != 2 || dw.size(0) != T) refuse("dweights must be [" + std::to_string(T) + ", k], got " + shape_text(dw.sizes()));
    const int64_t k = dw.size(1);
    if (k < 1 || k > 32) refuse("k must be in [1, 32], got " + std::to_string(k));
    const at::Tensor& ids = need(a[2], "ids", at::kInt, dw.sizes(), &l);
    const int score = small_integer(a[3], "score");
    const bool renorm = truth(a[4], "renorm");
    const float scale = number(a[5], "scale");
    int32_t* err = error_word(a[6], l);
    On on(l);
    at::Tensor d = empty(l.sizes(), l.scalar_type(), l);
    on.finish(mx_moe_route_bwd((const float*)ptr(dw), ptr(l), float_type(l), (const int32_t*)ptr(ids), T, E, (int32_t)k, score,
                               renorm, scale, ptr(d), err, on.stream));
    return wrap(d);
  });
}

// token_group(expert_of, E, err) -> (offs, row_dst, row_src)
PyObject* py_token_group(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 3);
    const at::Tensor& ids = need(a[0], "expert_of", at::kInt);
    const int E = small_integer(a[1], "E");
    if (E < 1 || E > 1024) refuse("E must be in [1, 1024], got " + std::to_string(E));
    int32_t* err = error_word(a[2], ids);
    const int64_t R = ids.numel();
    On on(ids);
    at::Tensor offs = empty({E}, at::kInt, ids), dst = empty({R}, at::kInt, ids), src = empty({R}, at::kInt, ids);
    at::Tensor ws;
    if (const int64_t bytes = (int64_t)mx_token_group_workspace(R, E)) ws = empty({bytes}, at::kByte, ids);
    on.finish(mx_token_group((const int32_t*)ptr(ids), R, E, (int32_t*)ptr(offs), (int32_t*)ptr(dst), (int32_t*)ptr(src), ptr(ws),
                             err, on.stream));
    return tuple_of(offs, dst, src);
  });
}

// moe_combine(rows, row_dst, weights, k, add, err) -> out; weights or k, and add, may be None
PyObject* py_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 6);
    const at::Tensor& rows = matrix(a[0], "rows");
    const at::Tensor& dst = need(a[1], "row_dst", at::kInt, &rows);
    const at::Tensor* w = a[2] == Py_None ? nullptr : &need(a[2], "weights", at::kFloat, &rows);
    if (w && w->dim() != 2) refuse("weights must be [T, k], got " + shape_text(w->sizes()));
    if (!w && a[3] == Py_None) refuse("k is needed without weights");
    const int64_t k = a[3] == Py_None ? w->size(1) : small_integer(a[3], "k");
    if (k < 1 || k > 32) refuse("k must be in [1, 32], got " + std::to_string(k));
    if (dst.numel() % k) refuse("row_dst must hold k numbers a token, got " + std::to_string(dst.numel()));
    const int64_t T = dst.numel() / k, d = rows.size(1);
    if (w) need(a[2], "weights", at::kFloat, {T, k}, &rows);
    const at::Tensor* add = a[4] == Py_None ? nullptr : &need(a[4], "add", at::kBFloat16, {T, d}, &rows);
    int32_t* err = error_word(a[5], rows);
    On on(rows);
    at::Tensor out = empty({T, d}, at::kBFloat16, rows);
    on.finish(mx_moe_combine(ptr(rows), rows.size(0), d, (const int32_t*)ptr(dst), T, (int32_t)k, w ? (const float*)ptr(*w) : nullptr,
                             add ? ptr(*add) : nullptr, ptr(out), err, on.stream));
    return wrap(out);
  });
}

// moe_combine_bwd(dout, rows, row_dst, row_src, weights, err) -> (drows, dweights)
PyObject* py_combine_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 6);
    const at::Tensor& dout = matrix(a[0], "dout");
    const int64_t T = dout.size(0), d = dout.size(1);
    const at::Tensor& rows = matrix(a[1], "rows", &dout);
    if (rows.size(1) != d) refuse("rows must have " + std::to_string(d) + " columns, got " + shape_text(rows.sizes()));
    const at::Tensor& w = need(a[4], "weights", at::kFloat, &dout);
    if (w.dim() != 2 || w.size(0) != T) refuse("weights must be [" + std::to_string(T) + ", k], got " + shape_text(w.sizes()));
    const int64_t k = w.size(1);
    const at::Tensor& dst = need(a[2], "row_dst", at::kInt, &dout);
    if (dst.numel() != T * k) refuse("row_dst must hold " + std::to_string(T * k) + " numbers, got " + std::to_string(dst.numel()));
    const at::Tensor& src = need(a[3], "row_src", at::kInt, {rows.size(0)}, &dout);
    if (k < 1 || k > 32) refuse("k must be in [1, 32], got " + std::to_string(k));
    int32_t* err = error_word(a[5], dout);
    On on(dout);
    at::Tensor drows = empty(rows.sizes(), at::kBFloat16, dout), dw = empty({T, k}, at::kFloat, dout);
    on.finish(mx_moe_combine_bwd(ptr(dout), ptr(rows), rows.size(0), d, (const int32_t*)ptr(dst), (const int32_t*)ptr(src), T,
                                 (int32_t)k, (const float*)ptr(w), ptr(drows), (float*)ptr(dw), err, on.stream));
    return tuple_of(drows, dw);
  });
}

// fp8_block_quantize(x, src, div, err) -> (codes, scales); src may be None
PyObject* py_fp8_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 4);
    const at::Tensor& x = matrix(a[0], "x");
    const at::Tensor* src = a[1] == Py_None ? nullptr : &need(a[1], "src", at::kInt, &x);
    const int div = small_integer(a[2], "div");
    int32_t* err = error_word(a[3], x);
    const int64_t rows = src ? src->numel() : x.size(0), cols = x.size(1);
    On on(x);
    at::Tensor codes = empty({rows, cols}, at::kByte, x), sc = empty({(cols + 127) / 128, rows}, at::kFloat, x);
    on.finish(mx_fp8_block_quantize(ptr(x), x.size(0), cols, src ? (const int32_t*)ptr(*src) : nullptr, rows, div, ptr(codes),
                                    (float*)ptr(sc), err, on.stream));
    return tuple_of(codes, sc);
  });
}

// fp8_block_quantize_weight(w, transposed) -> (codes, codes_t or None, scales)
PyObject* py_fp8_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 2);
    const at::Tensor& w = need(a[0], "w", at::kBFloat16);
    if (w.dim() != 2 && w.dim() != 3) refuse("w must be [N, K] or [E, N, K], got " + shape_text(w.sizes()));
    const bool transposed = truth(a[1], "transposed"), batch = w.dim() == 3;
    const int64_t E = batch ? w.size(0) : 1, N = w.size(-2), K = w.size(-1), nb = (N + 127) / 128, kb = (K + 127) / 128;
    On on(w);
    at::Tensor codes = empty(w.sizes(), at::kByte, w), codes_t, sc;
    if (batch) {
      if (transposed) codes_t = empty({E, K, N}, at::kByte, w);
      sc = empty({E, nb, kb}, at::kFloat, w);
    } else {
      if (transposed) codes_t = empty({K, N}, at::kByte, w);
      sc = empty({nb, kb}, at::kFloat, w);
    }
    on.finish(mx_fp8_block_quantize_weight(ptr(w), E, N, K, ptr(codes), ptr(codes_t), (float*)ptr(sc), on.stream));
    return tuple_of(codes, codes_t, sc);
  });
}

// fp8_block_mm(mode, codes, scales, w_codes, w_scales, offs, err) -> c; w_codes: the transposed ones for the input gradient; offs
// may be None: dense
PyObject* py_fp8_mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] {
    arguments(n, 7);
    const int mode = small_integer(a[0], "mode");
    const bool fwd = mode == MX_RAGGED_FWD;
    const char* name = fwd ? "x" : "dout";
    const at::Tensor& t = need(a[1], name, at::kByte);
    if (t.dim() != 2) refuse(std::string(name) + " must hold a matrix, got " + shape_text(t.sizes()));
    const int64_t M = t.size(0), C = t.size(1);
    const at::Tensor& st = need(a[2], "the scales of the rows", at::kFloat, {(C + 127) / 128, M}, &t);
    const at::Tensor& w = need(a[3], "w", at::kByte, &t);
    const at::Tensor* offs = a[5] == Py_None ? nullptr : &need(a[5], "offs", at::kInt, &t);
    const int64_t E = offs ? offs->numel() : 1;
    if (E < 1 || E > 1024) refuse("E must be in [1, 1024], got " + std::to_string(E));
    if ((w.dim() != 3 || w.size(0) != E) && (offs || w.dim() != 2))
      refuse("w must hold " + std::string(offs ? "[" + std::to_string(E) + ", N, K]" : "[N, K] or [1, N, K]") + ", got codes " +
             shape_text(w.sizes()));
    const int64_t F = w.size(-2);
    if (w.size(-1) != C) refuse(std::string(name) + " must have " + std::to_string(w.size(-1)) + " columns, got " + std::to_string(C));
    const int64_t N = fwd ? F : C, K = fwd ? C : F, nb = (N + 127) / 128, kb = (K + 127) / 128;
    const at::Tensor& sw = w.dim() == 3 ? need(a[4], "the scales of w", at::kFloat, {E, nb, kb}, &t)
                                        : need(a[4], "the scales of w", at::kFloat, {nb, kb}, &t);
    int32_t* err = error_word(a[6], t);
    On on(t);
    at::Tensor c = empty({M, F}, at::kBFloat16, t);
    on.finish(mx_fp8_block_mm(mode, ptr(t), (const float*)ptr(st), ptr(w), (const float*)ptr(sw), M, N, K,
                              offs ? (const int32_t*)ptr(*offs) : nullptr, (int32_t)E, ptr(c), err, on.stream));
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
                           {"moe_route", MX_FAST(py_route)},
                           {"moe_route_bwd", MX_FAST(py_route_bwd)},
                           {"token_group", MX_FAST(py_token_group)},
                           {"moe_combine", MX_FAST(py_combine)},
                           {"moe_combine_bwd", MX_FAST(py_combine_bwd)},
                           {"fp8_block_quantize", MX_FAST(py_fp8_rows)},
                           {"fp8_block_quantize_weight", MX_FAST(py_fp8_weight)},
                           {"fp8_block_mm", MX_FAST(py_fp8_mm)},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
