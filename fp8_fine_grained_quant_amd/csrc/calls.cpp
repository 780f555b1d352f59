// The Python calls of the MoE routing operators and of gradient clipping: what
// stands between a call and the library's entry point (argument checks,
// allocation of outputs, the current stream) in native code.  Their kernels on
// a decode step take 2 us, a launch 3 us; with that part in Python a call took
// 13 to 16 us (57 us for the clipping of 60 tensors), and so took every call
// whose kernels are shorter than that.
//
// Each function takes its arguments by position.  Outputs given as None are
// allocated; a stream given as None is torch's current one.  A call that
// allocates and is to run on another stream is made once more with that one as
// torch's current stream, so that the caching allocator hands memory freed at
// the call's end only to later work of that stream.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <initializer_list>
#include <limits>
#include <string>
#include <vector>

#include "fp8q.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Library {
  decltype(&fp8q_moe_route) moe_route;
  decltype(&fp8q_moe_route_bwd) moe_route_bwd;
  decltype(&fp8q_moe_sort) moe_sort;
  decltype(&fp8q_moe_sort_workspace) moe_sort_workspace;
  decltype(&fp8q_moe_dispatch) moe_dispatch;
  decltype(&fp8q_moe_dispatch_bwd) moe_dispatch_bwd;
  decltype(&fp8q_moe_combine) moe_combine;
  decltype(&fp8q_moe_combine_bwd) moe_combine_bwd;
  decltype(&fp8q_grad_clip) grad_clip;
  decltype(&fp8q_grad_clip_workspace) grad_clip_workspace;
} lib;
PyObject *current_device, *current_stream, *raise_status, *score_code, *on_stream;  // Python callables

// ------------------------------------------------------------------ arguments
[[noreturn]] void refuse(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw python_error();
}

std::string name_of(ScalarType t) { return std::string("torch.") + torch::getTHPDtype(t)->name; }

std::string text_of(at::IntArrayRef sizes) {
  std::string s = "(";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + (sizes[i] < 0 ? "any" : std::to_string(sizes[i]));
  return s + ")";
}

const Tensor* optional(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(what) + ": expected a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* what) {
  const Tensor* t = optional(o, what);
  if (!t) refuse(PyExc_ValueError, std::string(what) + " is required");
  return *t;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int small(PyObject* o) {  // out of range stays out of range
  const int64_t v = integer(o);
  return v < 0 ? -1 : v > std::numeric_limits<int>::max() ? std::numeric_limits<int>::max() : (int)v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
int score_of(PyObject* o) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "softmax") == 0) return FP8Q_SOFTMAX;
    if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0) return FP8Q_SIGMOID;
  }
  THPObjectPtr r(PyObject_CallFunctionObjArgs(score_code, o, nullptr));  // refuses
  if (!r) throw python_error();
  return small(r.get());
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// Shape (-1: any) and type of an operand that the library reads or writes
// through a raw pointer.
void expect(const Tensor* t, at::IntArrayRef sizes, ScalarType type, const char* what) {
  if (!t) refuse(PyExc_ValueError, std::string(what) + " is required");
  if (t->scalar_type() != type)
    refuse(PyExc_TypeError, std::string(what) + ": dtype " + name_of(t->scalar_type()) + ", expected " + name_of(type));
  bool ok = t->dim() == (int64_t)sizes.size();
  for (size_t i = 0; ok && i < sizes.size(); ++i) ok = sizes[i] < 0 || t->size((int64_t)i) == sizes[i];
  if (!ok)
    refuse(PyExc_ValueError, std::string(what) + ": shape " + text_of(t->sizes()) + ", expected " + text_of(sizes));
}
void matrix(const Tensor& t, const char* what) {
  if (t.dim() != 2) refuse(PyExc_ValueError, std::string(what) + ": shape " + text_of(t.sizes()) + ", expected 2-D");
}

// A [T, k] map, ids or weights.
void expect_map(const Tensor& t, int64_t tokens, const char* what) {
  if (t.dim() != 2 || (tokens >= 0 && t.size(0) != tokens))
    refuse(PyExc_ValueError, std::string(what) + ": shape " + text_of(t.sizes()) + ", expected [" +
                                 (tokens < 0 ? "T" : std::to_string(tokens)) + ", k]");
  if (t.scalar_type() != at::kInt)
    refuse(PyExc_TypeError, std::string(what) + ": dtype " + name_of(t.scalar_type()) + ", expected torch.int32");
}

fp8q_dtype type_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return FP8Q_BF16;
  if (t.scalar_type() == at::kFloat) return FP8Q_F32;
  refuse(PyExc_TypeError, "unsupported dtype " + name_of(t.scalar_type()));
}

[[noreturn]] void refuse_place() { refuse(PyExc_ValueError, "fp8q works on GPU tensors only"); }
[[noreturn]] void refuse_devices(c10::Device a, c10::Device b) {
  refuse(PyExc_ValueError, "tensors on " + a.str() + " and " + b.str() + ", expected one device");
}
// Tensors on one GPU, which is the result.
c10::Device on_gpu(std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts)
    if (t && !t->is_cuda()) refuse_place();
  const c10::Device device = (*ts.begin())->device();
  for (const Tensor* t : ts)
    if (t && t->device() != device) refuse_devices(device, t->device());
  return device;
}
void dense(std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts)
    if (t && !t->is_contiguous())
      refuse(PyExc_ValueError, "ids, maps, weights, offsets, biases, workspaces and gradients must be contiguous");
}

// Row stride of a matrix whose rows are contiguous.
int64_t stride(const Tensor& t) {
  if (t.size(1) > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "expected a 2-D tensor with contiguous rows");
  return t.size(0) > 1 ? t.stride(0) : std::max(t.size(1), t.stride(0));
}

template <class T>
T* data(const Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
template <class T>
T* data(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }

// What at::empty calls behind its dispatch, which is half of its 0.85 us.
Tensor make(at::IntArrayRef sizes, ScalarType type, c10::Device device) {
  return at::detail::empty_cuda(sizes, type, device, std::nullopt);
}
Tensor make(at::IntArrayRef sizes, ScalarType type, const Tensor& like) { return make(sizes, type, like.device()); }
// `given`, or a new tensor that `own` keeps.
const Tensor& given_or(const Tensor* given, Tensor& own, at::IntArrayRef sizes, ScalarType type, const Tensor& like) {
  if (given) return *given;
  own = make(sizes, type, like);
  return own;
}

// ---------------------------------------------------------------------- calls
hipStream_t handle_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return static_cast<hipStream_t>(p);
}
// The stream to launch on, given as None, a torch stream or a pointer as a
// number of any kind.  A launch is on the current device, which must be the
// tensors' own (index -1: there are none).
hipStream_t stream_of(PyObject* o, c10::Device device) {
  THPObjectPtr current(PyObject_CallNoArgs(current_device));
  if (!current) throw python_error();
  if (const int64_t at = integer(current.get()); device.index() >= 0 && at != device.index())
    refuse(PyExc_ValueError,
           "tensors on " + device.str() + ", but the current device is cuda:" + std::to_string(at));
  if (o != Py_None) {
    if (PyLong_Check(o)) return handle_of(o);
    THPObjectPtr handle(PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream")
                                                                 : PyNumber_Long(o));
    if (!handle) throw python_error();
    return handle_of(handle.get());
  }
  THPObjectPtr handle(PyObject_CallFunctionObjArgs(current_stream, current.get(), nullptr));
  if (!handle) throw python_error();
  return handle_of(handle.get());
}

// The call of `name` with these arguments but the last, the stream, which is
// torch's current one meanwhile.
PyObject* again_on(const char* name, PyObject* const* a, Py_ssize_t n) {
  THPObjectPtr args(PyTuple_New(n - 1));
  if (!args) throw python_error();
  for (Py_ssize_t i = 0; i + 1 < n; ++i) {
    Py_INCREF(a[i]);
    PyTuple_SET_ITEM(args.get(), i, a[i]);
  }
  PyObject* r = PyObject_CallFunction(on_stream, "sOO", name, args.get(), a[n - 1]);
  if (!r) throw python_error();
  return r;
}

void check(fp8q_status status, const char* name) {
  if (status == FP8Q_OK) return;
  THPObjectPtr r(PyObject_CallFunction(raise_status, "is", (int)status, name));
  throw python_error();
}

// The library's call without the interpreter's lock, as a foreign call has it;
// the lock comes back also where a tensor has no memory to point to and throws.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F>
fp8q_status unlocked(F f) {
  Unlocked guard;
  return f();
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

PyObject* pack(std::initializer_list<PyObject*> items) {
  THPObjectPtr t(PyTuple_New((Py_ssize_t)items.size()));
  bool ok = t.get() != nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (ok && o) PyTuple_SET_ITEM(t.get(), i++, o);
    else {
      ok = false;
      Py_XDECREF(o);
    }
  }
  if (!ok) throw python_error();
  return t.release();
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// logits, k, score, bias, renormalize, scale, ids, weights, stream
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 9);
  if (a[6] == Py_None && a[n - 1] != Py_None) return again_on("moe_route", a, n);
  const int score = score_of(a[2]), renorm = truth(a[4]);
  const float scale = (float)real(a[5]);
  const Tensor &logits = tensor(a[0], "logits");
  const Tensor *bias = optional(a[3], "bias"), *ids = optional(a[6], "ids"), *weights = optional(a[7], "weights");
  matrix(logits, "logits");
  const int64_t tokens = logits.size(0), experts = logits.size(1);
  int k = small(a[1]);
  if (ids) {
    expect_map(*ids, tokens, "ids");
    k = (int)std::min<int64_t>(ids->size(1), std::numeric_limits<int>::max());
    expect(weights, {tokens, k}, at::kFloat, "weights");
  }
  if (bias) expect(bias, {experts}, at::kFloat, "bias");
  const c10::Device device = on_gpu({&logits, ids, weights, bias});
  dense({ids, weights, bias});
  const fp8q_dtype type = type_of(logits);
  const int64_t ld = stride(logits);
  if (k < 1 || k > 32) check(FP8Q_ERR_SHAPE, "fp8q_moe_route");
  Tensor own_ids, own_weights;
  const Tensor& i = given_or(ids, own_ids, {tokens, k}, at::kInt, logits);
  const Tensor& w = given_or(weights, own_weights, {tokens, k}, at::kFloat, logits);
  const hipStream_t st = stream_of(a[8], device);
  check(unlocked([&] {
          return lib.moe_route(data<void>(logits), type, tokens, experts, ld, k, score, data<float>(bias), renorm,
                               scale, data<int32_t>(i), data<float>(w), st);
        }),
        "fp8q_moe_route");
  if (ids) return none();
  return pack({THPVariable_Wrap(own_ids), THPVariable_Wrap(own_weights)});
  END_HANDLE_TH_ERRORS
}

// dweights, logits, ids, score, renormalize, scale, dlogits, stream
PyObject* moe_route_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  if (a[6] == Py_None && a[n - 1] != Py_None) return again_on("moe_route_bwd", a, n);
  const int score = score_of(a[3]), renorm = truth(a[4]);
  const float scale = (float)real(a[5]);
  const Tensor &dweights = tensor(a[0], "dweights"), &logits = tensor(a[1], "logits"), &ids = tensor(a[2], "ids");
  const Tensor* dlogits = optional(a[6], "dlogits");
  matrix(logits, "logits");
  const int64_t tokens = logits.size(0), experts = logits.size(1);
  expect_map(ids, tokens, "ids");
  const int k = (int)std::min<int64_t>(ids.size(1), std::numeric_limits<int>::max());
  expect(&dweights, {tokens, k}, at::kFloat, "dweights");
  if (dlogits) expect(dlogits, {tokens, experts}, logits.scalar_type(), "dlogits");
  const c10::Device device = on_gpu({&dweights, &logits, &ids, dlogits});
  dense({&dweights, &ids});
  const fp8q_dtype type = type_of(logits);
  Tensor own;
  const Tensor& d = given_or(dlogits, own, {tokens, experts}, logits.scalar_type(), logits);
  const int64_t ld = stride(logits), ld_d = stride(d);
  const hipStream_t st = stream_of(a[7], device);
  check(unlocked([&] {
          return lib.moe_route_bwd(data<float>(dweights), data<void>(logits), type, tokens, experts, ld,
                                   data<int32_t>(ids), k, score, renorm, scale, data<void>(d), ld_d, st);
        }),
        "fp8q_moe_route_bwd");
  return dlogits ? none() : THPVariable_Wrap(own);
  END_HANDLE_TH_ERRORS
}

// ids, experts, cover, offsets, dst, src, workspace, stream; with offsets None
// all are allocated, else src and workspace may be missing
PyObject* moe_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 8);
  if (a[3] == Py_None && a[n - 1] != Py_None) return again_on("moe_sort", a, n);
  const Tensor& ids = tensor(a[0], "ids");
  const Tensor *offsets = optional(a[3], "offsets"), *dst = optional(a[4], "dst"), *src = optional(a[5], "src"),
               *ws = optional(a[6], "workspace");
  expect_map(ids, -1, "ids");
  const int64_t tokens = ids.size(0), k = ids.size(1), pairs = ids.numel(), experts = integer(a[1]);
  if (offsets) {
    expect(offsets, {experts + 1}, at::kInt, "offsets");
    expect(dst, {tokens, k}, at::kInt, "dst");
    if (src) expect(src, {pairs}, at::kInt, "src");
    if (ws) expect(ws, {-1}, at::kByte, "workspace");
  }
  const c10::Device device = on_gpu({&ids, offsets, dst, src, ws});
  dense({&ids, offsets, dst, src, ws});
  const int cover = truth(a[2]);
  Tensor own_offsets, own_dst, own_src, own_ws;
  if (!offsets) {
    const int64_t need = lib.moe_sort_workspace(pairs, experts);
    if (need < 0)
      refuse(PyExc_ValueError, std::to_string(pairs) + " pairs, " + std::to_string(experts) +
                                   " experts: out of range (at most 1024 experts)");
    offsets = &given_or(nullptr, own_offsets, {experts + 1}, at::kInt, ids);
    dst = &given_or(nullptr, own_dst, {tokens, k}, at::kInt, ids);
    src = &given_or(nullptr, own_src, {pairs}, at::kInt, ids);
    if (need) ws = &given_or(nullptr, own_ws, {need}, at::kByte, ids);
  }
  const hipStream_t st = stream_of(a[7], device);
  check(unlocked([&] {
          return lib.moe_sort(data<int32_t>(ids), pairs, experts, cover, data<int32_t>(offsets), data<int32_t>(dst),
                              data<int32_t>(src), data<void>(ws), ws ? ws->numel() : 0, st);
        }),
        "fp8q_moe_sort");
  if (!own_offsets.defined()) return none();
  return pack({THPVariable_Wrap(own_offsets), THPVariable_Wrap(own_dst), THPVariable_Wrap(own_src)});
  END_HANDLE_TH_ERRORS
}

// Expert rows, their codes and scales as outputs: given, or those that `want`
// names (1: rows, 2: codes) allocated.
struct RowOutputs {
  const Tensor *rows, *q, *scale;
  Tensor own_rows, own_q, own_scale;

  RowOutputs(PyObject* r, PyObject* c, PyObject* s)
      : rows(optional(r, "rows")), q(optional(c, "q")), scale(optional(s, "scale")) {}
  void expect_all(int64_t m, int64_t cols, ScalarType type) {
    if (rows) expect(rows, {m, cols}, type, "rows");
    if (q || scale) {
      expect(q, {m, cols}, at::kByte, "q");
      expect(scale, {m, (cols + 127) / 128}, at::kFloat, "scale");
    }
  }
  // Rows and codes in rows a multiple of 64 bytes apart: the quantizers and the
  // grouped products take them as they are, and they are written in whole
  // segments.
  static Tensor spaced(int64_t m, int64_t cols, int64_t bytes, ScalarType type, const Tensor& like) {
    const int64_t step = 64 / bytes, ld = (cols + step - 1) / step * step;
    const Tensor t = make({m, ld}, type, like);
    return ld == cols ? t : t.narrow(1, 0, cols);
  }
  void allocate(int want, int64_t m, int64_t cols, const Tensor& like) {
    if (want & 1) {
      own_rows = spaced(m, cols, (int64_t)like.element_size(), like.scalar_type(), like);
      rows = &own_rows;
    }
    if (want & 2) {
      own_q = spaced(m, cols, 1, at::kByte, like);
      q = &own_q;
      scale = &given_or(nullptr, own_scale, {m, (cols + 127) / 128}, at::kFloat, like);
    }
  }
  int64_t ld_rows() const { return rows ? stride(*rows) : 0; }
  int64_t ld_q() const { return q ? stride(*q) : 0; }
  int64_t ld_scale() const { return scale ? stride(*scale) : 0; }
};
PyObject* wrap_or_none(const Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : none(); }

// x, dst, rows, q, scale, want, stream; with want None the outputs are given
PyObject* moe_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 7);
  if (a[5] != Py_None && a[n - 1] != Py_None) return again_on("moe_dispatch", a, n);
  const Tensor &x = tensor(a[0], "x"), &dst = tensor(a[1], "dst");
  RowOutputs out(a[2], a[3], a[4]);
  matrix(x, "x");
  const int64_t tokens = x.size(0), cols = x.size(1);
  expect_map(dst, tokens, "dst");
  const int64_t k = dst.size(1), m = tokens * k;
  out.expect_all(m, cols, x.scalar_type());
  const c10::Device device = on_gpu({&x, &dst, out.rows, out.q, out.scale});
  dense({&dst});
  const fp8q_dtype type = type_of(x);
  if (a[5] != Py_None) out.allocate(small(a[5]), m, cols, x);
  const int64_t ld = stride(x), ld_r = out.ld_rows(), ld_q = out.ld_q(), ld_s = out.ld_scale();
  const hipStream_t st = stream_of(a[6], device);
  check(unlocked([&] {
          return lib.moe_dispatch(data<void>(x), type, tokens, cols, ld, data<int32_t>(dst), (int)k,
                                  data<void>(out.rows), ld_r, data<uint8_t>(out.q), ld_q, data<float>(out.scale),
                                  ld_s, st);
        }),
        "fp8q_moe_dispatch");
  if (a[5] == Py_None) return none();
  return pack({wrap_or_none(out.own_rows), wrap_or_none(out.own_q), wrap_or_none(out.own_scale)});
  END_HANDLE_TH_ERRORS
}

// drows, dst, dx, stream
PyObject* moe_dispatch_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 4);
  if (a[2] == Py_None && a[n - 1] != Py_None) return again_on("moe_dispatch_bwd", a, n);
  const Tensor &drows = tensor(a[0], "drows"), &dst = tensor(a[1], "dst");
  const Tensor* dx = optional(a[2], "dx");
  matrix(drows, "drows");
  expect_map(dst, -1, "dst");
  const int64_t tokens = dst.size(0), k = dst.size(1), cols = drows.size(1);
  expect(&drows, {tokens * k, cols}, drows.scalar_type(), "drows");
  if (dx) expect(dx, {tokens, cols}, drows.scalar_type(), "dx");
  const c10::Device device = on_gpu({&drows, &dst, dx});
  dense({&dst});
  const fp8q_dtype type = type_of(drows);
  Tensor own;
  const Tensor& y = given_or(dx, own, {tokens, cols}, drows.scalar_type(), drows);
  const int64_t ld = stride(drows), ld_y = stride(y);
  const hipStream_t st = stream_of(a[3], device);
  check(unlocked([&] {
          return lib.moe_dispatch_bwd(data<void>(drows), type, tokens, cols, ld, data<int32_t>(dst), (int)k,
                                      data<void>(y), ld_y, st);
        }),
        "fp8q_moe_dispatch_bwd");
  return dx ? none() : THPVariable_Wrap(own);
  END_HANDLE_TH_ERRORS
}

// yp, dst, weights, y, stream
PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 5);
  if (a[3] == Py_None && a[n - 1] != Py_None) return again_on("moe_combine", a, n);
  const Tensor &yp = tensor(a[0], "yp"), &dst = tensor(a[1], "dst"), &weights = tensor(a[2], "weights");
  const Tensor* out = optional(a[3], "y");
  matrix(yp, "yp");
  expect_map(dst, -1, "dst");
  const int64_t tokens = dst.size(0), k = dst.size(1), cols = yp.size(1);
  expect(&yp, {tokens * k, cols}, yp.scalar_type(), "yp");
  expect(&weights, {tokens, k}, at::kFloat, "weights");
  if (out) expect(out, {tokens, cols}, yp.scalar_type(), "y");
  const c10::Device device = on_gpu({&yp, &dst, &weights, out});
  dense({&dst, &weights});
  const fp8q_dtype type = type_of(yp);
  Tensor own;
  const Tensor& y = given_or(out, own, {tokens, cols}, yp.scalar_type(), yp);
  const int64_t ld = stride(yp), ld_y = stride(y);
  const hipStream_t st = stream_of(a[4], device);
  check(unlocked([&] {
          return lib.moe_combine(data<void>(yp), type, tokens, cols, ld, data<int32_t>(dst), (int)k,
                                 data<float>(weights), data<void>(y), ld_y, st);
        }),
        "fp8q_moe_combine");
  return out ? none() : THPVariable_Wrap(own);
  END_HANDLE_TH_ERRORS
}

// dy, yp, dst, weights, dweights, rows, q, scale, want, stream; with dweights
// None it is allocated with the outputs that `want` names
PyObject* moe_combine_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 10);
  if (a[4] == Py_None && a[n - 1] != Py_None) return again_on("moe_combine_bwd", a, n);
  const Tensor &dy = tensor(a[0], "dy"), &yp = tensor(a[1], "yp"), &dst = tensor(a[2], "dst"),
               &weights = tensor(a[3], "weights");
  const Tensor* dweights = optional(a[4], "dweights");
  RowOutputs out(a[5], a[6], a[7]);
  matrix(dy, "dy");
  const int64_t tokens = dy.size(0), cols = dy.size(1);
  expect_map(dst, tokens, "dst");
  const int64_t k = dst.size(1), m = tokens * k;
  expect(&yp, {m, cols}, dy.scalar_type(), "yp");
  expect(&weights, {tokens, k}, at::kFloat, "weights");
  if (dweights) expect(dweights, {tokens, k}, at::kFloat, "dweights");
  out.expect_all(m, cols, dy.scalar_type());
  const c10::Device device = on_gpu({&dy, &yp, &dst, &weights, dweights, out.rows, out.q, out.scale});
  dense({&dst, &weights, dweights});
  const fp8q_dtype type = type_of(dy);
  if (!dweights) out.allocate(small(a[8]), m, cols, dy);
  Tensor own;
  const Tensor& dw = given_or(dweights, own, {tokens, k}, at::kFloat, dy);
  const int64_t ld = stride(dy), ld_p = stride(yp), ld_r = out.ld_rows(), ld_q = out.ld_q(), ld_s = out.ld_scale();
  const hipStream_t st = stream_of(a[9], device);
  check(unlocked([&] {
          return lib.moe_combine_bwd(data<void>(dy), data<void>(yp), type, tokens, cols, ld, ld_p, data<int32_t>(dst),
                                     (int)k, data<float>(weights), data<void>(out.rows), ld_r, data<uint8_t>(out.q),
                                     ld_q, data<float>(out.scale), ld_s, data<float>(dw), st);
        }),
        "fp8q_moe_combine_bwd");
  if (dweights) return none();
  return pack({wrap_or_none(out.own_rows), wrap_or_none(out.own_q), wrap_or_none(out.own_scale),
               THPVariable_Wrap(own)});
  END_HANDLE_TH_ERRORS
}

// grads, out, max_norm, norm, workspace, stream (grads, out: sequences; out
// None: in place); with norm None it and the workspace are allocated
PyObject* grad_clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  if (a[3] == Py_None && a[n - 1] != Py_None) return again_on("grad_clip", a, n);
  // tuples of the caller's lists, which other code may change before the launch
  auto fixed = [](PyObject* o, const char* text) {
    THPObjectPtr items(PySequence_Fast(o, text));
    THPObjectPtr t(items ? PySequence_Tuple(items.get()) : nullptr);
    if (!t) throw python_error();
    return t;
  };
  THPObjectPtr grads = fixed(a[0], "grads: expected a sequence of tensors");
  THPObjectPtr outs = fixed(a[1] == Py_None ? grads.get() : a[1], "out: expected a sequence of tensors");
  const Py_ssize_t tensors = PyTuple_GET_SIZE(grads.get());
  if (PyTuple_GET_SIZE(outs.get()) != tensors)
    refuse(PyExc_ValueError, "out: " + std::to_string(PyTuple_GET_SIZE(outs.get())) + " tensors for " +
                                 std::to_string(tensors) + " gradients");
  const Tensor *norm = optional(a[3], "norm"), *ws = optional(a[4], "workspace");
  ScalarType type = at::kFloat;
  const Tensor* abroad = nullptr;
  bool gpu = true;
  c10::Device device(c10::kCUDA);
  for (Py_ssize_t i = 0; i < tensors; ++i) {
    const Tensor &g = tensor(PyTuple_GET_ITEM(grads.get(), i), "grads"),
                 &o = tensor(PyTuple_GET_ITEM(outs.get(), i), "out");
    if (i == 0) {
      type = o.scalar_type();
      device = g.device();
    }
    if (g.scalar_type() != at::kFloat || o.scalar_type() != type)
      refuse(PyExc_TypeError, "gradients of " + name_of(g.scalar_type()) + " to " + name_of(o.scalar_type()) +
                                  ", expected torch.float32 to " + name_of(type));
    if (g.sizes() != o.sizes())
      refuse(PyExc_ValueError, "out: shape " + text_of(o.sizes()) + " for a gradient of " + text_of(g.sizes()));
    if (!g.is_contiguous() || !o.is_contiguous())
      refuse(PyExc_ValueError, "gradients and their outputs must be contiguous");
    gpu = gpu && g.is_cuda() && o.is_cuda();
    if (g.device() != device) abroad = &g;
    if (o.device() != device) abroad = &o;
  }
  if (norm) {
    expect(norm, {}, at::kFloat, "norm");
    expect(ws, {-1}, at::kByte, "workspace");
    dense({ws});
    const c10::Device at = on_gpu({norm, ws});
    if (tensors == 0) device = at;
    if (gpu && at != device) refuse_devices(device, at);
  }
  if (!gpu) refuse_place();
  if (abroad) refuse_devices(device, abroad->device());
  if (type != at::kFloat && type != at::kBFloat16) refuse(PyExc_TypeError, "unsupported dtype " + name_of(type));
  const double max_norm = real(a[2]);
  Tensor own_norm, own_ws;
  if (!norm) {
    own_norm = make({}, at::kFloat, device);
    own_ws = make({lib.grad_clip_workspace(tensors)}, at::kByte, device);
    norm = &own_norm;
    ws = &own_ws;
  }
  const hipStream_t st = stream_of(a[5], device);
  std::vector<fp8q_grad> table((size_t)tensors);
  for (Py_ssize_t i = 0; i < tensors; ++i) {
    const Tensor& g = THPVariable_Unpack(PyTuple_GET_ITEM(grads.get(), i));
    table[(size_t)i] = {data<float>(g), data<void>(THPVariable_Unpack(PyTuple_GET_ITEM(outs.get(), i))),
                        g.numel()};
  }
  check(unlocked([&] {
          return lib.grad_clip(table.data(), tensors, type == at::kBFloat16 ? FP8Q_BF16 : FP8Q_F32, max_norm,
                               data<void>(ws), ws->numel(), data<float>(norm), st);
        }),
        "fp8q_grad_clip");
  return own_norm.defined() ? THPVariable_Wrap(own_norm) : none();
  END_HANDLE_TH_ERRORS
}

// {name: address}, current_device, current_stream, raise_status, score_code, on_stream
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count(n, 6);
  auto find = [&](auto& f, const char* name) {
    PyObject* o = PyDict_GetItemString(a[0], name);
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
    if (!p) refuse(PyExc_ValueError, std::string("no address of ") + name);
    f = reinterpret_cast<std::decay_t<decltype(f)>>(p);
  };
  find(lib.moe_route, "fp8q_moe_route");
  find(lib.moe_route_bwd, "fp8q_moe_route_bwd");
  find(lib.moe_sort, "fp8q_moe_sort");
  find(lib.moe_sort_workspace, "fp8q_moe_sort_workspace");
  find(lib.moe_dispatch, "fp8q_moe_dispatch");
  find(lib.moe_dispatch_bwd, "fp8q_moe_dispatch_bwd");
  find(lib.moe_combine, "fp8q_moe_combine");
  find(lib.moe_combine_bwd, "fp8q_moe_combine_bwd");
  find(lib.grad_clip, "fp8q_grad_clip");
  find(lib.grad_clip_workspace, "fp8q_grad_clip_workspace");
  PyObject** const slots[] = {&current_device, &current_stream, &raise_status, &score_code, &on_stream};
  for (int i = 0; i < 5; ++i) {
    Py_INCREF(a[1 + i]);
    Py_XDECREF(*slots[i]);
    *slots[i] = a[1 + i];
  }
  return none();
  END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),         FAST(moe_route),    FAST(moe_route_bwd),   FAST(moe_sort),
                         FAST(moe_dispatch), FAST(moe_dispatch_bwd), FAST(moe_combine), FAST(moe_combine_bwd),
                         FAST(grad_clip),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
