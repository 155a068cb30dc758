// Python entry of the operators around the routed experts: tensor checks, output tensors and the current stream in
// C++, then one call of the C ABI.  The same marshalling in Python cost 19-28 us a call (five tensors, 20 to 28
// ctypes arguments), several times what the smallest of these operators take on the device.
//
// Functions take positional arguments only (their Python wrappers in _binding.py have the names and defaults),
// raise TypeError / ValueError for what the tensors get wrong, and hand any other status to a callable given to
// init(), which raises.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "../../include/w4a8moe.h"

namespace {

PyObject* g_raise = nullptr;  // called with a status that is not W4A8_OK; raises

struct Bad {  // a Python exception type and its text, thrown inside a call
  PyObject* type;
  std::string text;
};

[[noreturn]] void type_error(const std::string& t) { throw Bad{PyExc_TypeError, t}; }
[[noreturn]] void value_error(const std::string& t) { throw Bad{PyExc_ValueError, t}; }

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + (t.dim() == 1 ? ",)" : ")");
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
  if (t.layout() != at::kStrided) type_error(std::string(name) + " must be a dense tensor");
  return t;
}

int dtype_id(at::ScalarType t) {
  return t == at::kBFloat16 ? W4A8_DTYPE_BF16 : t == at::kHalf ? W4A8_DTYPE_F16 : t == at::kFloat ? W4A8_DTYPE_F32 : -1;
}
const char* dtype_name(at::ScalarType t) { return c10::toString(t); }

void need_dtype(const at::Tensor& t, const char* name, at::ScalarType a, at::ScalarType b) {
  if (t.scalar_type() != a && t.scalar_type() != b)
    type_error(std::string(name) + " must be one of (" + dtype_name(a) +
               (a == b ? "" : std::string(", ") + dtype_name(b)) + "), got " + dtype_name(t.scalar_type()));
}
void need_device(const at::Tensor& t, const char* name, const at::Device& dev) {
  if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
}

struct Mat {
  const void* p = nullptr;
  int64_t ld = 0, rows = 0, cols = 0;
  at::ScalarType dtype = at::kFloat;
};

// a matrix with contiguous rows and any row stride
Mat mat(const at::Tensor& t, const char* name, const at::Device& dev) {
  need_device(t, name, dev);
  if (t.dim() != 2) value_error(std::string(name) + " must have 2 dimensions");
  Mat m;
  m.rows = t.size(0);
  m.cols = t.size(1);
  const int64_t rs = t.stride(0);
  if (t.stride(1) != 1 && m.cols > 1) value_error(std::string(name) + " must have contiguous rows");
  if (m.rows > 1 && rs < m.cols)
    value_error(std::string(name) + " has overlapping rows (row stride " + std::to_string(rs) + ", " +
                std::to_string(m.cols) + " columns)");
  m.p = t.data_ptr();
  m.ld = rs > m.cols ? rs : m.cols > 1 ? m.cols : 1;
  m.dtype = t.scalar_type();
  return m;
}
void need_shape(const Mat& m, const char* name, int64_t rows, int64_t cols) {
  if (m.rows != rows || m.cols != cols)
    value_error(std::string(name) + " must have shape (" + std::to_string(rows) + ", " + std::to_string(cols) +
                "), got (" + std::to_string(m.rows) + ", " + std::to_string(m.cols) + ")");
}

// a contiguous vector of n elements, or None
const void* vec(PyObject* o, const char* name, const at::Device& dev, int64_t n, at::ScalarType a, at::ScalarType b,
                at::ScalarType* got) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = cuda_tensor(o, name);
  need_device(t, name, dev);
  need_dtype(t, name, a, b);
  if (t.dim() != 1 || t.size(0) != n)
    value_error(std::string(name) + " must have shape (" + std::to_string(n) + ",), got " + shape_of(t));
  if (n > 1 && t.stride(0) != 1) value_error(std::string(name) + " must be contiguous");
  if (got) *got = t.scalar_type();
  return t.data_ptr();
}

at::Tensor empty(int64_t rows, int64_t cols, at::ScalarType dt, const at::Device& dev) {
  return at::Tensor(at::detail::empty_cuda({rows, cols}, dt, dev, std::nullopt));
}

int64_t as_int(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Bad{nullptr, ""};
  return v;
}
int as_i32(PyObject* o) {
  const int64_t v = as_int(o);
  if (v != static_cast<int32_t>(v)) value_error("integer argument out of range: " + std::to_string(v));
  return static_cast<int>(v);
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Bad{nullptr, ""};
  return static_cast<float>(v);
}
bool as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Bad{nullptr, ""};
  return v != 0;
}
bool as_dtype(PyObject* o, const char* name, at::ScalarType* out) {  // false for None
  if (o == Py_None) return false;
  if (!THPDtype_Check(o)) type_error(std::string(name) + " must be a torch.dtype");
  *out = reinterpret_cast<THPDtype*>(o)->scalar_type;
  return true;
}

// Runs f, turning what it throws into a Python exception; f returns a new reference.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  try {
    if (got != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
    at::AutoDispatchBelowADInplaceOrView no_autograd;  // outputs carry no gradient
    return f();
  } catch (const Bad& b) {
    if (b.type) PyErr_SetString(b.type, b.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* oom = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_SetString(oom ? oom : PyExc_RuntimeError, e.what_without_backtrace());
    Py_XDECREF(oom);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

void check(int status) {
  if (status == W4A8_OK) return;
  PyObject* r = g_raise ? PyObject_CallFunction(g_raise, "i", status) : nullptr;
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "status %d", status);
  throw Bad{nullptr, ""};
}

PyObject* py_init(PyObject*, PyObject* arg) {
  Py_INCREF(arg);
  Py_XSETREF(g_raise, arg);
  Py_RETURN_NONE;
}

// (logits, k, bias, score, n_group, topk_group, group_top, renormalize, scale) -> (ids, weights)
PyObject* py_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& lt = cuda_tensor(a[0], "logits");
    const at::Device dev = lt.device();
    const Mat l = mat(lt, "logits", dev);
    if (dtype_id(l.dtype) < 0) type_error(std::string("logits must be bf16, f16 or fp32, got ") + dtype_name(l.dtype));
    const int k = as_i32(a[1]);
    const void* bias = vec(a[2], "bias", dev, l.cols, at::kFloat, at::kFloat, nullptr);
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t cols = k > 0 ? k : 0;
    at::Tensor ids = empty(l.rows, cols, at::kInt, dev), w = empty(l.rows, cols, at::kFloat, dev);
    check(moe_route_grouped_topk(l.p, dtype_id(l.dtype), l.ld, l.rows, l.cols, k, as_i32(a[3]),
                                 static_cast<const float*>(bias), as_i32(a[4]), as_i32(a[5]), as_i32(a[6]),
                                 as_bool(a[7]), as_float(a[8]), static_cast<int32_t*>(ids.data_ptr()),
                                 static_cast<float*>(w.data_ptr()), c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    PyObject* pi = THPVariable_Wrap(std::move(ids));
    PyObject* pw = THPVariable_Wrap(std::move(w));
    PyObject* r = pi && pw ? PyTuple_Pack(2, pi, pw) : nullptr;
    Py_XDECREF(pi);
    Py_XDECREF(pw);
    return r;
  });
}

// (f, residual, post, w_post, b_post, gate, branch_scale, residual_scale, pre, w_pre, b_pre, eps, residual_dtype,
//  want_h, want_y, h, y) -> (h, y)
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Tensor& ft = cuda_tensor(a[0], "f");
    const at::Device dev = ft.device();
    const Mat f = mat(ft, "f", dev);
    if (dtype_id(f.dtype) < 0) type_error(std::string("f must be bf16, f16 or fp32, got ") + dtype_name(f.dtype));
    const int64_t T = f.rows, H = f.cols;
    at::ScalarType rdt = f.dtype;
    const bool given = as_dtype(a[12], "residual_dtype", &rdt);
    Mat r;
    if (a[1] != Py_None) {
      const at::Tensor& rt = cuda_tensor(a[1], "residual");
      need_dtype(rt, "residual", f.dtype, at::kFloat);
      r = mat(rt, "residual", dev);
      need_shape(r, "residual", T, H);
      if (given && rdt != r.dtype)
        value_error(std::string("residual_dtype ") + dtype_name(rdt) + " differs from the residual's " +
                    dtype_name(r.dtype));
      rdt = r.dtype;
    } else if (rdt != f.dtype && rdt != at::kFloat) {
      type_error(std::string("residual_dtype must be ") + dtype_name(f.dtype) + " or Float, got " + dtype_name(rdt));
    }
    at::ScalarType pdt = at::kFloat;
    const void* par[4];
    static const char* const names[4] = {"w_post", "b_post", "w_pre", "b_pre"};
    static const int at_[4] = {3, 4, 9, 10};
    bool any = false;
    for (int i = 0; i < 4; ++i) {
      at::ScalarType dt = pdt;
      par[i] = vec(a[at_[i]], names[i], dev, H, f.dtype, at::kFloat, &dt);
      if (a[at_[i]] == Py_None) continue;
      if (any && dt != pdt) type_error("w_post, b_post, w_pre and b_pre must have one dtype");
      pdt = dt;
      any = true;
    }
    Mat g;
    g.rows = g.cols = 1;
    if (a[5] != Py_None) {
      const at::Tensor& gt = cuda_tensor(a[5], "gate");
      need_dtype(gt, "gate", f.dtype, at::kFloat);
      g = mat(gt, "gate", dev);
    }
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made[2];
    Mat out[2];
    PyObject* res[2] = {Py_None, Py_None};
    static const char* const out_names[2] = {"h", "y"};
    for (int i = 0; i < 2; ++i) {
      if (!as_bool(a[13 + i])) continue;
      const at::ScalarType dt = i ? f.dtype : rdt;
      if (a[15 + i] == Py_None) {
        made[i] = empty(T, H, dt, dev);
        out[i].p = made[i].data_ptr();
        out[i].ld = H > 1 ? H : 1;
      } else {
        const at::Tensor& t = cuda_tensor(a[15 + i], out_names[i]);
        need_dtype(t, out_names[i], dt, dt);
        out[i] = mat(t, out_names[i], dev);
        need_shape(out[i], out_names[i], T, H);
        res[i] = a[15 + i];
      }
    }
    check(block_norm(f.p, f.ld, dtype_id(f.dtype), r.p, r.ld, dtype_id(rdt), as_i32(a[2]), par[0], par[1], g.p, g.ld,
                     g.rows, g.cols, dtype_id(g.dtype), as_float(a[6]), as_float(a[7]), as_i32(a[8]), par[2], par[3],
                     dtype_id(pdt), as_float(a[11]), T, H, const_cast<void*>(out[0].p), out[0].ld,
                     const_cast<void*>(out[1].p), out[1].ld, c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    PyObject* tuple = PyTuple_New(2);
    if (!tuple) return nullptr;
    for (int i = 0; i < 2; ++i) {
      PyObject* o = made[i].defined() ? THPVariable_Wrap(std::move(made[i])) : Py_NewRef(res[i]);
      if (!o) {
        Py_DECREF(tuple);
        return nullptr;
      }
      PyTuple_SET_ITEM(tuple, i, o);
    }
    return tuple;
  });
}

// (x, w, bias, act, gated, residual, out_dtype, out, ws) -> out
PyObject* py_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& xt = cuda_tensor(a[0], "x");
    const at::Device dev = xt.device();
    need_dtype(xt, "x", at::kBFloat16, at::kHalf);
    const Mat x = mat(xt, "x", dev);
    const at::Tensor& wt = cuda_tensor(a[1], "w");
    need_dtype(wt, "w", x.dtype, x.dtype);
    const Mat w = mat(wt, "w", dev);
    if (w.cols != x.cols)
      value_error("w must have " + std::to_string(x.cols) + " columns, got " + std::to_string(w.cols));
    const bool gated = as_bool(a[4]);
    if (gated && w.rows % 2)
      value_error("w must have an even number of rows when gated, got " + std::to_string(w.rows));
    const int64_t M = x.rows, N = w.rows, K = x.cols, n_out = gated ? N / 2 : N;
    at::ScalarType odt = x.dtype;
    as_dtype(a[6], "out_dtype", &odt);
    if (odt != x.dtype && odt != at::kFloat)
      type_error(std::string("out_dtype must be ") + dtype_name(x.dtype) + " or Float, got " + dtype_name(odt));
    at::ScalarType bdt = at::kFloat;
    const void* bias = vec(a[2], "bias", dev, N, x.dtype, at::kFloat, &bdt);
    Mat r, o;
    if (a[5] != Py_None) {
      const at::Tensor& rt = cuda_tensor(a[5], "residual");
      need_dtype(rt, "residual", odt, odt);
      r = mat(rt, "residual", dev);
      need_shape(r, "residual", M, n_out);
    }
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made, room;
    if (a[7] == Py_None) {
      made = empty(M, n_out, odt, dev);
      o.p = made.data_ptr();
      o.ld = n_out > 1 ? n_out : 1;
    } else {
      const at::Tensor& ot = cuda_tensor(a[7], "out");
      need_dtype(ot, "out", odt, odt);
      o = mat(ot, "out", dev);
      need_shape(o, "out", M, n_out);
    }
    void* ws = nullptr;
    int64_t ws_bytes = 0;
    if (a[8] != Py_None) {
      const at::Tensor& t = cuda_tensor(a[8], "ws");
      need_device(t, "ws", dev);
      need_dtype(t, "ws", at::kByte, at::kByte);
      if (!t.is_contiguous()) value_error("ws must be contiguous");
      ws = t.data_ptr();
      ws_bytes = t.numel();
    } else if (((reinterpret_cast<uintptr_t>(x.p) | reinterpret_cast<uintptr_t>(w.p) | static_cast<uintptr_t>(2 * x.ld) |
                 static_cast<uintptr_t>(2 * w.ld)) & 15) != 0) {  // operands without 16-byte alignment are copied there
      ws_bytes = static_cast<int64_t>(dense_linear_workspace_bytes(M, N, K));
      if (ws_bytes) {
        room = empty(1, ws_bytes, at::kByte, dev);
        ws = room.data_ptr();
      }
    }
    check(dense_linear(x.p, x.ld, w.p, w.ld, dtype_id(x.dtype), bias, dtype_id(bdt), as_i32(a[3]), gated, r.p, r.ld,
                       const_cast<void*>(o.p), o.ld, dtype_id(odt), M, N, K, ws, static_cast<size_t>(ws_bytes),
                       c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[7]);
  });
}

template <class F>
PyCFunction as_cfunction(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"init", py_init, METH_O, nullptr},
    {"route", as_cfunction(py_route), METH_FASTCALL, nullptr},
    {"norm", as_cfunction(py_norm), METH_FASTCALL, nullptr},
    {"linear", as_cfunction(py_linear), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "w4a8_torch_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w4a8_torch_ops(void) { return PyModule_Create(&module); }
