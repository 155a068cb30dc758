// Python entry of the operators around the routed experts and of the attention half: tensor checks, output tensors and the current stream in
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

#include <algorithm>
#include <array>
#include <cmath>
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

// --- the attention half ----------------------------------------------------------------------------------------

// heads [rows][heads][D] with contiguous D and any strides
struct Heads {
  const void* p = nullptr;
  int64_t rows = 0, heads = 0, D = 0, ld_t = 0, ld_h = 0;
  at::ScalarType dtype = at::kFloat;
};

// Whether two places of a tensor that is written may be one: its dimensions, by stride, each step over all that is inside.
template <size_t N>
bool overlaps(std::array<std::pair<int64_t, int64_t>, N> dims, int64_t inner) {  // (stride, size), innermost extent
  std::sort(dims.begin(), dims.end());
  int64_t reach = inner;  // places that the dimensions so far cover
  for (const auto& d : dims) {
    if (d.second <= 1) continue;
    if (d.first < reach) return true;
    reach = d.first * (d.second - 1) + reach;
  }
  return false;
}

Heads heads_of(const at::Tensor& t, const char* name, const at::Device& dev, bool written) {
  need_device(t, name, dev);
  if (t.dim() != 3) value_error(std::string(name) + " must have 3 dimensions");
  Heads h;
  h.rows = t.size(0);
  h.heads = t.size(1);
  h.D = t.size(2);
  if (h.D > 1 && t.stride(2) != 1) value_error(std::string(name) + " must have contiguous heads");
  h.ld_t = h.rows > 1 ? t.stride(0) : 0;
  h.ld_h = h.heads > 1 ? t.stride(1) : 0;
  if (written && t.numel() > 0 && overlaps<2>({{{h.ld_t, h.rows}, {h.ld_h, h.heads}}}, h.D))
    value_error(std::string(name) + " has overlapping heads");
  h.p = t.data_ptr();
  h.dtype = t.scalar_type();
  return h;
}
void need_shape(const Heads& h, const char* name, int64_t rows, int64_t heads, int64_t D) {
  if (h.rows != rows || h.heads != heads || h.D != D)
    value_error(std::string(name) + " must have shape (" + std::to_string(rows) + ", " + std::to_string(heads) + ", " +
                std::to_string(D) + "), got (" + std::to_string(h.rows) + ", " + std::to_string(h.heads) + ", " +
                std::to_string(h.D) + ")");
}

at::Tensor empty3(int64_t a, int64_t b, int64_t c, at::ScalarType dt, const at::Device& dev) {
  return at::Tensor(at::detail::empty_cuda({a, b, c}, dt, dev, std::nullopt));
}

// an optional rotation; returns whether there is one
bool rotary_of(PyObject* freqs, PyObject* positions, PyObject* interleaved, PyObject* start, PyObject* scale,
               const at::Device& dev, int64_t rows, w4a8_rotary* r) {
  *r = w4a8_rotary{};
  if (freqs == Py_None) {
    if (positions != Py_None) value_error("positions given without freqs");
    return false;
  }
  const at::Tensor& f = cuda_tensor(freqs, "freqs");
  need_device(f, "freqs", dev);
  need_dtype(f, "freqs", at::kLong, at::kLong);
  if (f.dim() != 1 || !f.is_contiguous()) value_error("freqs must be a contiguous vector");
  r->freqs = static_cast<const int64_t*>(f.data_ptr());
  r->R = 2 * f.size(0);
  r->start = as_int(start);
  r->interleaved = as_bool(interleaved);
  r->scale = as_float(scale);
  if (r->R == 0) value_error("freqs must not be empty");
  if (positions != Py_None) {
    at::ScalarType dt = at::kInt;
    r->positions = vec(positions, "positions", dev, rows, at::kInt, at::kLong, &dt);
    r->positions64 = dt == at::kLong;
  }
  return true;
}

// k_cache, v_cache [pages, page_size, heads, D] of one type, page_table [B, n], seq_lens [B], scales [heads]
w4a8_paged_cache cache_of(PyObject* k, PyObject* v, PyObject* table, PyObject* lens, PyObject* k_scale, PyObject* v_scale,
                          const at::Device& dev, at::ScalarType dtype, bool written) {
  w4a8_paged_cache c = {};
  const at::Tensor& kt = cuda_tensor(k, "k_cache");
  const at::Tensor& vt = cuda_tensor(v, "v_cache");
  const at::Tensor* both[2] = {&kt, &vt};
  static const char* const names[2] = {"k_cache", "v_cache"};
  int64_t strides[2][3];
  for (int i = 0; i < 2; ++i) {
    const at::Tensor& t = *both[i];
    need_device(t, names[i], dev);
    need_dtype(t, names[i], dtype, at::kFloat8_e4m3fn);
    if (t.dim() != 4) value_error(std::string(names[i]) + " must have 4 dimensions");
    if (i && (t.sizes() != kt.sizes() || t.scalar_type() != kt.scalar_type()))
      value_error("v_cache must have k_cache's shape and type, got " + shape_of(t) + " and " + shape_of(kt));
    if (t.size(3) > 1 && t.stride(3) != 1) value_error(std::string(names[i]) + " must have contiguous heads");
    for (int d = 0; d < 3; ++d) strides[i][d] = t.size(d) > 1 ? t.stride(d) : 0;
    if (written && t.numel() > 0 &&
        overlaps<3>({{{strides[i][0], t.size(0)}, {strides[i][1], t.size(1)}, {strides[i][2], t.size(2)}}}, t.size(3)))
      value_error(std::string(names[i]) + " has overlapping heads");
  }
  c.k = kt.data_ptr();
  c.v = vt.data_ptr();
  c.k_page = strides[0][0], c.k_slot = strides[0][1], c.k_head = strides[0][2];
  c.v_page = strides[1][0], c.v_slot = strides[1][1], c.v_head = strides[1][2];
  c.pages = kt.size(0);
  c.page_size = kt.size(1);
  c.heads = kt.size(2);
  c.D = kt.size(3);
  c.dtype = kt.scalar_type() == at::kFloat8_e4m3fn ? W4A8_DTYPE_E4M3 : dtype_id(kt.scalar_type());
  const at::Tensor& tt = cuda_tensor(table, "page_table");
  need_dtype(tt, "page_table", at::kInt, at::kInt);
  const Mat m = mat(tt, "page_table", dev);
  c.page_table = static_cast<const int32_t*>(m.p);
  c.table_ld = m.ld;
  c.table_pages = m.cols;
  c.B = m.rows;
  c.seq_lens = static_cast<const int32_t*>(vec(lens, "seq_lens", dev, c.B, at::kInt, at::kInt, nullptr));
  if (!c.seq_lens && c.B > 0) type_error("seq_lens must be a CUDA tensor");
  c.k_scale = static_cast<const float*>(vec(k_scale, "k_scale", dev, c.heads, at::kFloat, at::kFloat, nullptr));
  c.v_scale = static_cast<const float*>(vec(v_scale, "v_scale", dev, c.heads, at::kFloat, at::kFloat, nullptr));
  return c;
}

// (x, positions, freqs, interleaved, start, scale, inverse, out) -> out
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor& xt = cuda_tensor(a[0], "x");
    const at::Device dev = xt.device();
    const Heads x = heads_of(xt, "x", dev, false);
    if (dtype_id(x.dtype) < 0) type_error(std::string("x must be bf16, f16 or fp32, got ") + dtype_name(x.dtype));
    cuda_tensor(a[1], "positions");
    cuda_tensor(a[2], "freqs");
    w4a8_rotary r;
    rotary_of(a[2], a[1], a[3], a[4], a[5], dev, x.rows, &r);
    r.inverse = as_bool(a[6]);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made;
    Heads o;
    if (a[7] == Py_None) {
      made = empty3(x.rows, x.heads, x.D, x.dtype, dev);
      o = heads_of(made, "out", dev, false);
    } else {
      const at::Tensor& ot = cuda_tensor(a[7], "out");
      need_dtype(ot, "out", x.dtype, x.dtype);
      o = heads_of(ot, "out", dev, true);
      need_shape(o, "out", x.rows, x.heads, x.D);
    }
    check(rotary_embedding(x.p, x.ld_t, x.ld_h, dtype_id(x.dtype), x.rows, x.heads, x.D, &r, const_cast<void*>(o.p), o.ld_t,
                           o.ld_h, c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[7]);
  });
}

// (k, v, k_cache, v_cache, page_table, seq_lens, indptr, freqs, positions, interleaved, start, scale, k_scale, v_scale,
//  q, q_out) -> q_out
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor& kt = cuda_tensor(a[0], "k");
    const at::Device dev = kt.device();
    need_dtype(kt, "k", at::kBFloat16, at::kHalf);
    const Heads k = heads_of(kt, "k", dev, false);
    const at::Tensor& vt = cuda_tensor(a[1], "v");
    need_dtype(vt, "v", k.dtype, k.dtype);
    const Heads v = heads_of(vt, "v", dev, false);
    need_shape(v, "v", k.rows, k.heads, k.D);
    const w4a8_paged_cache c = cache_of(a[2], a[3], a[4], a[5], a[12], a[13], dev, k.dtype, true);
    if (c.heads != k.heads || c.D != k.D)
      value_error("k_cache must have heads and head size (" + std::to_string(k.heads) + ", " + std::to_string(k.D) +
                  "), got (" + std::to_string(c.heads) + ", " + std::to_string(c.D) + ")");
    const int32_t* indptr =
        static_cast<const int32_t*>(vec(a[6], "indptr", dev, c.B + 1, at::kInt, at::kInt, nullptr));
    if (!indptr && k.rows < c.B)
      value_error("k must have at least " + std::to_string(c.B) + " rows without indptr, got " + std::to_string(k.rows));
    w4a8_rotary r;
    rotary_of(a[7], a[8], a[9], a[10], a[11], dev, k.rows, &r);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made;
    Heads q, o;
    if (a[14] != Py_None) {
      const at::Tensor& qt = cuda_tensor(a[14], "q");
      need_dtype(qt, "q", k.dtype, k.dtype);
      q = heads_of(qt, "q", dev, false);
      need_shape(q, "q", k.rows, q.heads, k.D);
      if (a[15] == Py_None) {
        made = empty3(q.rows, q.heads, q.D, q.dtype, dev);
        o = heads_of(made, "q_out", dev, false);
      } else {
        const at::Tensor& ot = cuda_tensor(a[15], "q_out");
        need_dtype(ot, "q_out", k.dtype, k.dtype);
        o = heads_of(ot, "q_out", dev, true);
        need_shape(o, "q_out", q.rows, q.heads, q.D);
      }
    } else if (a[15] != Py_None) {
      value_error("q_out given without q");
    }
    const auto append = made.defined() ? paged_kv_append_whole : paged_kv_append;
    check(append(k.p, k.ld_t, k.ld_h, v.p, v.ld_t, v.ld_h, dtype_id(k.dtype), k.rows, indptr, &c, &r, q.p, q.ld_t, q.ld_h,
                 q.heads, const_cast<void*>(o.p), o.ld_t, o.ld_h, c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[15]);
  });
}

// (q, k_cache, v_cache, page_table, seq_lens, scale, window, k_scale, v_scale, return_lse, out, ws) -> out or (out, lse)
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor& qt = cuda_tensor(a[0], "q");
    const at::Device dev = qt.device();
    need_dtype(qt, "q", at::kBFloat16, at::kHalf);
    const Heads q = heads_of(qt, "q", dev, false);
    const w4a8_paged_cache c = cache_of(a[1], a[2], a[3], a[4], a[7], a[8], dev, q.dtype, false);
    if (c.B != q.rows)
      value_error("page_table must have " + std::to_string(q.rows) + " rows, got " + std::to_string(c.B));
    if (c.D != q.D)
      value_error("q must have heads of " + std::to_string(c.D) + " elements, got " + std::to_string(q.D));
    const float scale = a[5] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(q.D))) : as_float(a[5]);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made, lse, room;
    Heads o;
    if (a[10] == Py_None) {
      made = empty3(q.rows, q.heads, q.D, q.dtype, dev);
      o = heads_of(made, "out", dev, false);
    } else {
      const at::Tensor& ot = cuda_tensor(a[10], "out");
      need_dtype(ot, "out", q.dtype, q.dtype);
      o = heads_of(ot, "out", dev, true);
      need_shape(o, "out", q.rows, q.heads, q.D);
    }
    if (as_bool(a[9])) lse = empty(q.rows, q.heads, at::kFloat, dev);
    void* ws = nullptr;
    int64_t ws_bytes = 0;
    if (a[11] != Py_None) {
      const at::Tensor& t = cuda_tensor(a[11], "ws");
      need_device(t, "ws", dev);
      need_dtype(t, "ws", at::kByte, at::kByte);
      if (!t.is_contiguous()) value_error("ws must be contiguous");
      ws = t.data_ptr();
      ws_bytes = t.numel();
    } else {
      const int64_t window = as_int(a[6]), reach = c.table_pages * c.page_size;
      ws_bytes = static_cast<int64_t>(paged_attention_workspace_bytes(c.B, q.heads, c.heads, c.D, c.dtype,
                                                                      window > 0 && window < reach ? window : reach));
      if (ws_bytes) {
        room = empty(1, ws_bytes, at::kByte, dev);
        ws = room.data_ptr();
      }
    }
    check(paged_attention_decode(q.p, q.ld_t, q.ld_h, dtype_id(q.dtype), q.heads, &c, scale, as_int(a[6]),
                                 const_cast<void*>(o.p), o.ld_t, o.ld_h,
                                 lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, ws,
                                 static_cast<size_t>(ws_bytes), c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    PyObject* po = made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[10]);
    if (!po || !lse.defined()) return po;
    PyObject* pl = THPVariable_Wrap(std::move(lse));
    PyObject* r = pl ? PyTuple_Pack(2, po, pl) : nullptr;
    Py_DECREF(po);
    Py_XDECREF(pl);
    return r;
  });
}

// a contiguous matrix of E4M3 codes, as bytes or as float8_e4m3fn
Mat codes(PyObject* o, const char* name, const at::Device& dev) {
  const at::Tensor& t = cuda_tensor(o, name);
  need_dtype(t, name, at::kByte, at::kFloat8_e4m3fn);
  const Mat m = mat(t, name, dev);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return m;
}

// (A, a_scales, B, b_scales, out_dtype, out) -> out
PyObject* py_fp8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Device dev = cuda_tensor(a[0], "A").device();
    const Mat A = codes(a[0], "A", dev), B = codes(a[2], "B", dev);
    if (B.cols != A.cols)
      value_error("B must have " + std::to_string(A.cols) + " columns, got " + std::to_string(B.cols));
    const int64_t M = A.rows, N = B.rows, K = A.cols, G = K / 128;
    const at::Tensor& at_ = cuda_tensor(a[1], "a_scales");
    need_dtype(at_, "a_scales", at::kFloat, at::kFloat);
    const Mat as = mat(at_, "a_scales", dev);
    if (as.rows != G || as.cols < M)
      value_error("a_scales must have shape (" + std::to_string(G) + ", at least " + std::to_string(M) + "), got " +
                  shape_of(at_));
    const at::Tensor& bt = cuda_tensor(a[3], "b_scales");
    need_dtype(bt, "b_scales", at::kFloat, at::kFloat);
    const Mat bs = mat(bt, "b_scales", dev);
    need_shape(bs, "b_scales", (N + 127) / 128, G);
    if (!bt.is_contiguous()) value_error("b_scales must be contiguous");
    at::ScalarType odt = at::kBFloat16;
    as_dtype(a[4], "out_dtype", &odt);
    if (dtype_id(odt) < 0) type_error(std::string("out_dtype must be bf16, f16 or fp32, got ") + dtype_name(odt));
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made;
    Mat o;
    if (a[5] == Py_None) {
      made = empty(M, N, odt, dev);
      o.p = made.data_ptr();
      o.ld = N > 1 ? N : 1;
    } else {
      const at::Tensor& ot = cuda_tensor(a[5], "out");
      need_dtype(ot, "out", odt, odt);
      o = mat(ot, "out", dev);
      need_shape(o, "out", M, N);
    }
    check(fp8_block_linear(static_cast<const uint8_t*>(A.p), static_cast<const float*>(as.p), as.ld,
                           static_cast<const uint8_t*>(B.p), static_cast<const float*>(bs.p), M, N, K,
                           const_cast<void*>(o.p), o.ld, dtype_id(odt),
                           c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[5]);
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
    {"rotary", as_cfunction(py_rotary), METH_FASTCALL, nullptr},
    {"append", as_cfunction(py_append), METH_FASTCALL, nullptr},
    {"attend", as_cfunction(py_attend), METH_FASTCALL, nullptr},
    {"fp8_linear", as_cfunction(py_fp8_linear), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "w4a8_torch_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w4a8_torch_ops(void) { return PyModule_Create(&module); }
