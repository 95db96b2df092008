// Python binding of the 8-bit activation calls (awq_a8.h), the mixture of experts (awq_moe.h) and the low-rank adapters
// (awq_lora.h): argument marshalling only.  These calls run once per layer and token, where the checks and the output's
// allocation, made in Python, would take longer than the kernel; the rest of the library is bound with ctypes.  The
// library's functions are handed in as addresses (bind), so that this module does not load it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <exception>
#include <string>

#include "awq_a8.h"
#include "awq_lora.h"
#include "awq_moe.h"

namespace {

struct Lib {  // in the order of bind's addresses
  decltype(&awq_rmsnorm) rmsnorm;
  decltype(&awq_act_mul) act_mul;
  decltype(&awq_w4a8) w4a8;
  decltype(&awq_w4a8_weight_bytes) weight_bytes;
  decltype(&awq_w4a8_workspace_bytes) workspace_bytes;
  decltype(&awq_moe_route) moe_route;
  decltype(&awq_moe) moe;
  decltype(&awq_moe_layer) moe_layer;
  decltype(&awq_moe_workspace_bytes) moe_workspace_bytes;
  decltype(&awq_lora) lora;
  decltype(&awq_lora_workspace_bytes) lora_workspace_bytes;
} lib;
PyObject* act8_type = nullptr;     // awq.Act8, a tuple of two
PyObject* routing_type = nullptr;  // awq.Routing, a tuple of two
PyObject* error_type = nullptr;  // awq.AwqError(status, what)

struct Raise {  // a Python exception to set
  PyObject* type;
  std::string text;
};
[[noreturn]] void value_error(std::string text) { throw Raise{PyExc_ValueError, std::move(text)}; }
[[noreturn]] void type_error(std::string text) { throw Raise{PyExc_TypeError, std::move(text)}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return AWQ_DTYPE_F32;
    case at::kBFloat16: return AWQ_DTYPE_BF16;
    case at::kChar: return AWQ_DTYPE_I8;
    case at::kFloat8_e4m3fn: return AWQ_DTYPE_E4M3;
    default: return -1;
  }
}
bool is_codes(int code) { return code == AWQ_DTYPE_I8 || code == AWQ_DTYPE_E4M3; }
int float_code(const at::Tensor& t, const char* name) {
  const int c = type_code(t.scalar_type());
  if (c < 0 || is_codes(c)) type_error(std::string(name) + " must be float32 or bfloat16");
  return c;
}
int codes_code(const at::Tensor& t, const char* name) {
  const int c = type_code(t.scalar_type());
  if (!is_codes(c)) type_error(std::string(name) + " must be int8 or float8_e4m3fn");
  return c;
}

// [M, K] on dev with unit stride along K: its row stride (that of a single row says nothing)
int64_t row_stride(const at::Tensor& t, const char* name, c10::Device dev, int64_t M, int64_t K) {
  if (t.dim() != 2 || t.size(0) != M || t.size(1) != K || t.device() != dev)
    value_error(std::string(name) + " must be a [" + std::to_string(M) + ", " + std::to_string(K) + "] tensor on " +
                dev.str());
  if (K > 1 && t.stride(1) != 1) value_error(std::string(name) + " must have unit stride along its last axis");
  return M > 1 ? t.stride(0) : K;
}
const void* vector(const at::Tensor& t, const char* name, c10::Device dev, int64_t n) {
  if (t.dim() != 1 || t.size(0) != n || t.device() != dev || (n > 1 && t.stride(0) != 1))
    value_error(std::string(name) + " must be a contiguous vector of length " + std::to_string(n) + " on " + dev.str());
  return t.const_data_ptr();
}
void first(const at::Tensor& t, const char* name) {
  if (t.dim() != 2 || !t.is_cuda()) value_error(std::string(name) + " must be a 2-D device tensor");
}
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType t, c10::Device dev) {
  return at::empty(sizes, at::TensorOptions().dtype(t).device(dev));
}
PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw Raise{nullptr, ""};
  return o;
}
struct Ref {  // an owned reference
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {
    if (o == nullptr) throw Raise{nullptr, ""};
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* release() {
    PyObject* o = p;
    p = nullptr;
    return o;
  }
};
PyObject* pair(PyTypeObject* type, const Ref& a, const Ref& b) {
  Ref two(PyTuple_Pack(2, a.p, b.p));
  if (type == &PyTuple_Type) return two.release();
  Ref args(PyTuple_Pack(1, two.p));
  return PyTuple_Type.tp_new(type, args.p, nullptr);
}

// A row operator's output: given (a tensor, or an Act8), or made here of the dtype asked for.
struct RowOut {
  at::Tensor y, scale;
  PyObject* given = nullptr;
  int code = 0;
  int64_t ld = 0;
  float* scale_ptr = nullptr;

  RowOut(PyObject* out, PyObject* dtype, c10::Device dev, int64_t M, int64_t K) {
    at::ScalarType want = at::kBFloat16;
    const bool asked = dtype != Py_None;
    if (asked) {
      if (!THPDtype_Check(dtype)) type_error("dtype must be a torch.dtype");
      want = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    }
    if (out == Py_None) {
      code = type_code(want);
      if (code < 0) type_error("dtype must be float32, bfloat16, int8 or float8_e4m3fn");
      y = empty({M, K}, want, dev);
      ld = K;
      if (is_codes(code)) scale = empty({M}, at::kFloat, dev);
    } else {
      given = out;
      if (PyTuple_Check(out)) {
        if (PyTuple_GET_SIZE(out) != 2) type_error("out must be a tensor or an Act8");
        y = tensor(PyTuple_GET_ITEM(out, 0), "out");
        scale = tensor(PyTuple_GET_ITEM(out, 1), "out's scale");
        code = codes_code(y, "out");
        if (scale.scalar_type() != at::kFloat) type_error("out's scale must be float32");
        vector(scale, "out's scale", dev, M);
      } else {
        y = tensor(out, "out");
        code = float_code(y, "out");
      }
      if (asked && want != y.scalar_type()) value_error("dtype and out disagree");
      ld = row_stride(y, "out", dev, M, K);
    }
    if (is_codes(code)) scale_ptr = static_cast<float*>(scale.mutable_data_ptr());
  }
  PyObject* result() const {
    if (given != nullptr) return Py_NewRef(given);
    if (!is_codes(code)) return wrap(y);
    return pair(reinterpret_cast<PyTypeObject*>(act8_type), Ref(wrap(y)), Ref(wrap(scale)));
  }
};

awq_stream_t stream_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Raise{nullptr, ""};
  return static_cast<awq_stream_t>(p);
}
void check(int status, const char* name) {
  if (status == AWQ_OK) return;
  if (PyObject* e = PyObject_CallFunction(error_type, "is", status, name)) {
    PyErr_SetObject(error_type, e);
    Py_DECREF(e);
  }
  throw Raise{nullptr, ""};
}

// Runs f with n arguments; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (act8_type == nullptr) throw Raise{PyExc_RuntimeError, "the library is not bound"};
    if (got != want) type_error(std::string(name) + " takes " + std::to_string(want) + " arguments");
    return f();
  } catch (const Raise& r) {
    if (r.type != nullptr) PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// rmsnorm(X, gamma, residual, eps, dtype, out, residual_out, stream)
PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rmsnorm", n, 8, [&]() -> PyObject* {
    const at::Tensor& X = tensor(a[0], "X");
    const at::Tensor& gamma = tensor(a[1], "gamma");
    first(X, "X");
    const c10::Device dev = X.device();
    const int64_t M = X.size(0), K = X.size(1);
    const int64_t ldx = row_stride(X, "X", dev, M, K);
    const int xc = float_code(X, "X"), gc = float_code(gamma, "gamma");
    const void* gp = vector(gamma, "gamma", dev, K);
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raise{nullptr, ""};
    const bool res = a[2] != Py_None;
    at::Tensor h;
    const void* rp = nullptr;
    void* hp = nullptr;
    int rc = 0;
    int64_t ldr = 0, ldh = 0;
    if (res) {
      const at::Tensor& R = tensor(a[2], "residual");
      rc = float_code(R, "residual");
      ldr = row_stride(R, "residual", dev, M, K);
      rp = R.const_data_ptr();
      if (a[6] == Py_None) {
        h = empty({M, K}, R.scalar_type(), dev);
        ldh = K;
      } else {
        h = tensor(a[6], "residual_out");
        ldh = row_stride(h, "residual_out", dev, M, K);
        if (h.scalar_type() != R.scalar_type()) value_error("residual_out must have residual's dtype");
      }
      hp = h.mutable_data_ptr();
    } else if (a[6] != Py_None) {
      value_error("residual_out needs a residual");
    }
    RowOut out(a[5], a[4], dev, M, K);
    check(lib.rmsnorm(X.const_data_ptr(), xc, M, K, ldx, rp, rc, ldr, hp, ldh, gp, gc, (float)eps,
                      out.y.mutable_data_ptr(), out.code, out.ld, out.scale_ptr, stream_of(a[7])),
          "awq_rmsnorm");
    if (!res) return out.result();
    return pair(&PyTuple_Type, Ref(out.result()), Ref(a[6] != Py_None ? Py_NewRef(a[6]) : wrap(h)));
  });
}

// act_mul(G, U, s, act, dtype, out, stream)
PyObject* act_mul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("act_mul", n, 7, [&]() -> PyObject* {
    const at::Tensor& G = tensor(a[0], "G");
    first(G, "G");
    const c10::Device dev = G.device();
    const int64_t M = G.size(0), K = G.size(1);
    const int64_t ldg = row_stride(G, "G", dev, M, K);
    const int xc = float_code(G, "G");
    const void *up = nullptr, *sp = nullptr;
    int64_t ldu = 0;
    if (a[1] != Py_None) {
      const at::Tensor& U = tensor(a[1], "U");
      if (U.scalar_type() != G.scalar_type()) type_error("U must have G's dtype");
      ldu = row_stride(U, "U", dev, M, K);
      up = U.const_data_ptr();
    }
    if (a[2] != Py_None) {
      const at::Tensor& s = tensor(a[2], "s");
      if (s.scalar_type() != at::kFloat) type_error("s must be float32");
      sp = vector(s, "s", dev, K);
    }
    const long act = PyLong_AsLong(a[3]);
    if (act == -1 && PyErr_Occurred()) throw Raise{nullptr, ""};
    RowOut out(a[5], a[4], dev, M, K);
    check(lib.act_mul(G.const_data_ptr(), xc, M, K, ldg, up, ldu, static_cast<const float*>(sp), (int)act,
                      out.y.mutable_data_ptr(), out.code, out.ld, out.scale_ptr, stream_of(a[6])),
          "awq_act_mul");
    return out.result();
  });
}

// w4a8(q, scale, data, N, K, dtype, out, workspace, fp32_sums, stream)
PyObject* w4a8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("w4a8", n, 10, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "X.q");
    const at::Tensor& scale = tensor(a[1], "X.scale");
    const at::Tensor& data = tensor(a[2], "weight");
    const int64_t N = PyLong_AsLongLong(a[3]), K = PyLong_AsLongLong(a[4]);
    if ((N == -1 || K == -1) && PyErr_Occurred()) throw Raise{nullptr, ""};
    first(q, "X.q");
    const c10::Device dev = q.device();
    const int64_t M = q.size(0);
    if (q.size(1) != K) value_error("X and the weight disagree on K");
    const int64_t ldx = row_stride(q, "X.q", dev, M, K);
    const int xc = codes_code(q, "X.q");
    if (scale.scalar_type() != at::kFloat) type_error("X.scale must be float32");
    const void* sp = vector(scale, "X.scale", dev, M);
    const size_t bytes = lib.weight_bytes(N, K);
    if (bytes == 0 || data.device() != dev || data.scalar_type() != at::kByte || !data.is_contiguous() ||
        (size_t)data.numel() < bytes)
      value_error("weight must be the result of w4a8_weight on " + dev.str());
    at::Tensor Y;
    int64_t ldy = N;
    at::ScalarType want = at::kFloat;
    if (a[5] != Py_None) {
      if (!THPDtype_Check(a[5])) type_error("dtype must be a torch.dtype");
      want = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    }
    if (a[6] == Py_None) {
      if (want != at::kFloat && want != at::kBFloat16) type_error("dtype must be float32 or bfloat16");
      Y = empty({M, N}, want, dev);
    } else {
      Y = tensor(a[6], "out");
      ldy = row_stride(Y, "out", dev, M, N);
      if (a[5] != Py_None && want != Y.scalar_type()) value_error("dtype and out disagree");
    }
    int yc = float_code(Y, "out");
    if (a[8] != Py_None) {
      if (!PyBool_Check(a[8])) type_error("fp32_sums must be True, False or None");
      yc |= a[8] == Py_True ? AWQ_W4A8_SUMS_F32 : AWQ_W4A8_SUMS_MATRIX;
    }
    size_t need = lib.workspace_bytes(M, K, N);
    at::Tensor ws;
    if (need > 0) {
      if (a[7] == Py_None) {
        ws = empty({(int64_t)need}, at::kByte, dev);
      } else {
        ws = tensor(a[7], "workspace");
        if (!ws.is_contiguous() || ws.device() != dev) value_error("workspace must be contiguous and on " + dev.str());
        need = ws.nbytes();
      }
    }
    check(lib.w4a8(q.const_data_ptr(), xc, static_cast<const float*>(sp), M, K, ldx, data.const_data_ptr(), N, 128,
                   Y.mutable_data_ptr(), yc, ldy, ws.defined() ? ws.mutable_data_ptr() : nullptr, need,
                   stream_of(a[9])),
          "awq_w4a8");
    return a[6] != Py_None ? Py_NewRef(a[6]) : wrap(Y);
  });
}

// Activations in any of the four types: a tensor, or an Act8's codes with their scale.
struct Rows {
  at::Tensor x, scale;
  int code = 0;
  int64_t M = 0, K = 0, ld = 0;
  const float* scale_ptr = nullptr;

  explicit Rows(PyObject* o) {
    const bool codes = PyTuple_Check(o);
    if (codes) {
      if (PyTuple_GET_SIZE(o) != 2) type_error("X must be a tensor or an Act8");
      x = tensor(PyTuple_GET_ITEM(o, 0), "X.q");
      scale = tensor(PyTuple_GET_ITEM(o, 1), "X.scale");
    } else {
      x = tensor(o, "X");
    }
    first(x, codes ? "X.q" : "X");
    M = x.size(0), K = x.size(1);
    ld = row_stride(x, codes ? "X.q" : "X", x.device(), M, K);
    code = codes ? codes_code(x, "X.q") : float_code(x, "X");
    if (codes) {
      if (scale.scalar_type() != at::kFloat) type_error("X.scale must be float32");
      scale_ptr = static_cast<const float*>(vector(scale, "X.scale", x.device(), M));
    }
  }
};

// A contiguous tensor of the given type and sizes on dev.
const void* plain(const at::Tensor& t, const char* name, c10::Device dev, at::ScalarType type, const char* type_name,
                  at::IntArrayRef sizes) {
  if (t.scalar_type() != type) type_error(std::string(name) + " must be " + type_name);
  if (t.sizes() != sizes || t.device() != dev || !t.is_contiguous()) {
    std::string s;
    for (const int64_t n : sizes) s += (s.empty() ? "" : ", ") + std::to_string(n);
    value_error(std::string(name) + " must be a contiguous [" + s + "] tensor on " + dev.str());
  }
  return t.const_data_ptr();
}

int64_t whole(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raise{nullptr, ""};
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = whole(o);
  if (v < -(1 << 30) || v > (1 << 30)) value_error(std::string(name) + " is out of range");
  return (int)v;
}

// The workspace: given, or made here; its size.
size_t workspace(PyObject* given, size_t need, c10::Device dev, at::Tensor& ws) {
  if (given == Py_None) {
    ws = empty({(int64_t)(need > 0 ? need : 1)}, at::kByte, dev);
  } else {
    ws = tensor(given, "workspace");
    if (!ws.is_contiguous() || ws.device() != dev) value_error("workspace must be contiguous and on " + dev.str());
  }
  return ws.nbytes();
}

// moe_route(logits, k, score, renormalize, out, stream): (ids, weights)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("moe_route", n, 6, [&]() -> PyObject* {
    const at::Tensor& L = tensor(a[0], "logits");
    first(L, "logits");
    const c10::Device dev = L.device();
    const int64_t M = L.size(0), E = L.size(1);
    const int64_t ld = row_stride(L, "logits", dev, M, E);
    const int lc = float_code(L, "logits"), k = small(a[1], "k"), score = small(a[2], "score");
    const int renorm = PyObject_IsTrue(a[3]);
    if (renorm < 0) throw Raise{nullptr, ""};
    at::Tensor ids, weights;
    if (a[4] == Py_None) {
      if (k < 1 || k > E) value_error("k must be 1 to the number of experts");
      ids = empty({M, k}, at::kInt, dev);
      weights = empty({M, k}, at::kFloat, dev);
    } else {
      if (!PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 2) type_error("out must be a Routing");
      ids = tensor(PyTuple_GET_ITEM(a[4], 0), "out.ids");
      weights = tensor(PyTuple_GET_ITEM(a[4], 1), "out.weights");
      plain(ids, "out.ids", dev, at::kInt, "int32", {M, k});
      plain(weights, "out.weights", dev, at::kFloat, "float32", {M, k});
    }
    check(lib.moe_route(L.const_data_ptr(), lc, M, E, ld, k, score, renorm, static_cast<int32_t*>(ids.mutable_data_ptr()),
                        static_cast<float*>(weights.mutable_data_ptr()), stream_of(a[5])),
          "awq_moe_route");
    if (a[4] != Py_None) return Py_NewRef(a[4]);
    return pair(reinterpret_cast<PyTypeObject*>(routing_type), Ref(wrap(ids)), Ref(wrap(weights)));
  });
}

struct Experts {  // moe_weight's handle: (data, E, N, K)
  const void* data;
  int64_t E, N, K;
  Experts(PyObject* o, const char* name, c10::Device dev) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) type_error(std::string(name) + " must be the result of moe_weight");
    const at::Tensor& t = tensor(PyTuple_GET_ITEM(o, 0), name);
    E = whole(PyTuple_GET_ITEM(o, 1)), N = whole(PyTuple_GET_ITEM(o, 2)), K = whole(PyTuple_GET_ITEM(o, 3));
    const size_t bytes = E > 0 && N > 0 && N < INT32_MAX && E < INT32_MAX ? lib.weight_bytes(E * N, K) : 0;
    if (bytes == 0 || t.device() != dev || t.scalar_type() != at::kByte || !t.is_contiguous() || (size_t)t.numel() < bytes)
      value_error(std::string(name) + " must be the result of moe_weight on " + dev.str());
    data = t.const_data_ptr();
  }
};

// moe(X, routing or logits, k, score, renormalize, gate_up, down, act, dtype, out, workspace, stream)
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("moe", n, 12, [&]() -> PyObject* {
    const Rows X(a[0]);
    const c10::Device dev = X.x.device();
    const Experts gu(a[5], "gate_up", dev), down(a[6], "down", dev);
    if (gu.E != down.E || gu.K != X.K || down.N != X.K || gu.N % 2 != 0 || gu.N / 2 != down.K)
      value_error("X, gate_up and down disagree: [M, H], E experts of [2 I, H], E experts of [H, I]");
    const int64_t E = gu.E, I = down.K;
    const int act = small(a[7], "act"), score = small(a[3], "score");
    int k = 0, lc = 0;
    int64_t ldl = 0;
    const void *ids = nullptr, *weights = nullptr, *logits = nullptr;
    const bool routed = PyTuple_Check(a[1]);
    if (routed) {
      if (PyTuple_GET_SIZE(a[1]) != 2) type_error("routing must be a Routing or the router's logits");
      if (a[2] != Py_None) value_error("k goes with logits");
      const at::Tensor& ti = tensor(PyTuple_GET_ITEM(a[1], 0), "routing.ids");
      const at::Tensor& tw = tensor(PyTuple_GET_ITEM(a[1], 1), "routing.weights");
      if (ti.dim() != 2) value_error("routing.ids must be a [M, k] tensor");
      if (ti.size(1) > 1 << 30) value_error("routing.ids has too many columns");
      k = (int)ti.size(1);
      ids = plain(ti, "routing.ids", dev, at::kInt, "int32", {X.M, k});
      weights = plain(tw, "routing.weights", dev, at::kFloat, "float32", {X.M, k});
    } else {
      const at::Tensor& L = tensor(a[1], "routing");
      if (a[2] == Py_None) value_error("logits need k");
      k = small(a[2], "k");
      lc = float_code(L, "logits");
      ldl = row_stride(L, "logits", dev, X.M, E);
      logits = L.const_data_ptr();
    }
    const int renorm = PyObject_IsTrue(a[4]);
    if (renorm < 0) throw Raise{nullptr, ""};
    at::ScalarType want = at::kFloat;
    if (a[8] != Py_None) {
      if (!THPDtype_Check(a[8])) type_error("dtype must be a torch.dtype");
      want = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
    }
    at::Tensor Y;
    int64_t ldy = X.K;
    if (a[9] == Py_None) {
      if (want != at::kFloat && want != at::kBFloat16) type_error("dtype must be float32 or bfloat16");
      Y = empty({X.M, X.K}, want, dev);
    } else {
      Y = tensor(a[9], "out");
      ldy = row_stride(Y, "out", dev, X.M, X.K);
      if (a[8] != Py_None && want != Y.scalar_type()) value_error("dtype and out disagree");
    }
    const int yc = float_code(Y, "out");
    at::Tensor ws;
    const size_t bytes = workspace(a[10], lib.moe_workspace_bytes(X.M, E, k, X.K, I), dev, ws);
    const awq_stream_t st = stream_of(a[11]);
    if (routed)
      check(lib.moe(X.x.const_data_ptr(), X.code, X.scale_ptr, X.M, X.K, X.ld, static_cast<const int32_t*>(ids),
                    static_cast<const float*>(weights), k, gu.data, down.data, E, I, 128, act, Y.mutable_data_ptr(), yc, ldy,
                    ws.mutable_data_ptr(), bytes, st),
            "awq_moe");
    else
      check(lib.moe_layer(X.x.const_data_ptr(), X.code, X.scale_ptr, X.M, X.K, X.ld, logits, lc, ldl, k, score, renorm,
                          gu.data, down.data, E, I, 128, act, Y.mutable_data_ptr(), yc, ldy, ws.mutable_data_ptr(), bytes, st),
            "awq_moe_layer");
    return a[9] != Py_None ? Py_NewRef(a[9]) : wrap(Y);
  });
}

// lora(X, A, B, ids, base, scale, ranks, out, workspace, stream)
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("lora", n, 10, [&]() -> PyObject* {
    const Rows X(a[0]);
    const c10::Device dev = X.x.device();
    const at::Tensor& A = tensor(a[1], "A");
    const at::Tensor& B = tensor(a[2], "B");
    const at::Tensor& base = tensor(a[4], "base");
    if (A.dim() != 3 || B.dim() != 3) value_error("A must be [adapters, R, K] and B [adapters, N, R]");
    const int64_t count = A.size(0), R = A.size(1), N = B.size(1);
    const void* ap = plain(A, "A", dev, at::kBFloat16, "bfloat16", {count, R, X.K});
    const void* bp = plain(B, "B", dev, at::kBFloat16, "bfloat16", {count, N, R});
    const void* ip = plain(tensor(a[3], "ids"), "ids", dev, at::kInt, "int32", {X.M});
    const void *sp = nullptr, *rp = nullptr;
    if (a[5] != Py_None) sp = plain(tensor(a[5], "scale"), "scale", dev, at::kFloat, "float32", {count});
    if (a[6] != Py_None) rp = plain(tensor(a[6], "ranks"), "ranks", dev, at::kInt, "int32", {count});
    const int yc = float_code(base, "base");
    const int64_t ldb = row_stride(base, "base", dev, X.M, N);
    at::Tensor Y;
    int64_t ldy = N;
    if (a[7] == Py_None) {
      Y = empty({X.M, N}, base.scalar_type(), dev);
    } else {
      Y = tensor(a[7], "out");
      if (Y.scalar_type() != base.scalar_type()) type_error("out must have base's dtype");
      ldy = row_stride(Y, "out", dev, X.M, N);
    }
    at::Tensor ws;
    const size_t bytes = workspace(a[8], lib.lora_workspace_bytes(X.M, X.K, N, R), dev, ws);
    check(lib.lora(X.x.const_data_ptr(), X.code, X.scale_ptr, X.M, X.K, X.ld, ap, bp, count, R,
                   static_cast<const int32_t*>(rp), static_cast<const float*>(sp), static_cast<const int32_t*>(ip),
                   base.const_data_ptr(), ldb, Y.mutable_data_ptr(), yc, ldy, N, ws.mutable_data_ptr(), bytes, stream_of(a[9])),
          "awq_lora");
    return a[7] != Py_None ? Py_NewRef(a[7]) : wrap(Y);
  });
}

// bind(addresses, Act8, Routing, AwqError): the library's functions in Lib's order, and the types
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *functions, *act8, *routing, *error;
  if (!PyArg_ParseTuple(args, "O!O!O!O", &PyTuple_Type, &functions, &PyType_Type, &act8, &PyType_Type, &routing, &error))
    return nullptr;
  for (PyObject* t : {act8, routing}) {
    if (!PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(t), &PyTuple_Type)) {
      PyErr_SetString(PyExc_TypeError, "Act8 and Routing must be tuple types");
      return nullptr;
    }
  }
  constexpr Py_ssize_t kFunctions = sizeof(Lib) / sizeof(void*);
  if (PyTuple_GET_SIZE(functions) != kFunctions) {
    PyErr_SetString(PyExc_ValueError, "a wrong number of functions");
    return nullptr;
  }
  void* f[kFunctions];
  for (Py_ssize_t i = 0; i < kFunctions; ++i) {
    f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(functions, i));
    if (f[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is null");
      return nullptr;
    }
  }
  std::memcpy(&lib, f, sizeof(lib));
  Py_XSETREF(act8_type, Py_NewRef(act8));
  Py_XSETREF(routing_type, Py_NewRef(routing));
  Py_XSETREF(error_type, Py_NewRef(error));
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm)), METH_FASTCALL, nullptr},
    {"act_mul", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(act_mul)), METH_FASTCALL, nullptr},
    {"w4a8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(w4a8)), METH_FASTCALL, nullptr},
    {"moe_route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(moe_route)), METH_FASTCALL, nullptr},
    {"moe", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(moe)), METH_FASTCALL, nullptr},
    {"lora", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(lora)), METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_a8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__a8(void) { return PyModule_Create(&module); }
