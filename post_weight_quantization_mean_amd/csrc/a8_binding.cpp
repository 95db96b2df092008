// Python binding of the 8-bit activation calls (awq_a8.h): argument marshalling only.  These calls run once
// per layer and token, where the checks and the output's allocation, made in Python, would take longer than
// the kernel; the rest of the library is bound with ctypes.  The library's functions are handed in as
// addresses (bind), so that this module does not load it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <string>

#include "awq_a8.h"

namespace {

struct Lib {
  decltype(&awq_rmsnorm) rmsnorm;
  decltype(&awq_act_mul) act_mul;
  decltype(&awq_w4a8) w4a8;
  decltype(&awq_w4a8_weight_bytes) weight_bytes;
  decltype(&awq_w4a8_workspace_bytes) workspace_bytes;
} lib;
PyObject* act8_type = nullptr;  // awq.Act8, a tuple of two
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

// bind(rmsnorm, act_mul, w4a8, weight_bytes, workspace_bytes, Act8, AwqError): the library's addresses, and the types
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  PyObject *act8, *error;
  if (!PyArg_ParseTuple(args, "KKKKKO!O", &f[0], &f[1], &f[2], &f[3], &f[4], &PyType_Type, &act8, &error))
    return nullptr;
  if (!PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(act8), &PyTuple_Type)) {
    PyErr_SetString(PyExc_TypeError, "Act8 must be a tuple type");
    return nullptr;
  }
  lib.rmsnorm = reinterpret_cast<decltype(lib.rmsnorm)>(f[0]);
  lib.act_mul = reinterpret_cast<decltype(lib.act_mul)>(f[1]);
  lib.w4a8 = reinterpret_cast<decltype(lib.w4a8)>(f[2]);
  lib.weight_bytes = reinterpret_cast<decltype(lib.weight_bytes)>(f[3]);
  lib.workspace_bytes = reinterpret_cast<decltype(lib.workspace_bytes)>(f[4]);
  Py_XSETREF(act8_type, Py_NewRef(act8));
  Py_XSETREF(error_type, Py_NewRef(error));
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm)), METH_FASTCALL, nullptr},
    {"act_mul", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(act_mul)), METH_FASTCALL, nullptr},
    {"w4a8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(w4a8)), METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_a8", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__a8(void) { return PyModule_Create(&module); }
