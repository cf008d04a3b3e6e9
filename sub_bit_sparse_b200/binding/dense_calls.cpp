// Argument marshalling of the 8-bit integer and gated feed-forward calls, as a
// CPython extension over PyTorch's C++ tensors: the checks, the outputs that
// the caller does not give, the current stream, one call of the C ABI.
//
// These calls are short (5 to 7 us of device time for one token), and the same
// steps made from Python, attribute by attribute, took 6 us of host time a
// call besides the launch itself.  The extension holds no computation and does
// not link the library: the package hands it the entry points' addresses, so
// the release and the debug library are called the same way.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "../../include/stq1.h"

namespace {

decltype(&stq1_quantize_i8) f_quantize_i8;
decltype(&stq1_i8_matmul) f_i8_matmul;
decltype(&stq1_i8_ffn_workspace) f_i8_ffn_workspace;
decltype(&stq1_i8_ffn) f_i8_ffn;
decltype(&stq1_glu) f_glu;
decltype(&stq1_glu_backward_workspace) f_glu_backward_workspace;
decltype(&stq1_glu_backward) f_glu_backward;
PyObject* g_error = nullptr;               // the package's Stq1Error

// A refused argument: the Python exception to raise and its text.
struct Refusal {
  PyObject* type;
  std::string text;
};
// A C ABI error code.
struct Failure {
  const char* func;
  int code;
};

std::string sizes_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

std::string type_text(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kChar: return "torch.int8";
    case at::kByte: return "torch.uint8";
    case at::kHalf: return "torch.float16";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, at::ScalarType type, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    throw Refusal{PyExc_TypeError, std::string(name) + " must be a CUDA tensor"};
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type)
    throw Refusal{PyExc_TypeError, std::string(name) + " must be " + type_text(type) + ", got " + type_text(t.scalar_type())};
  if (!t.is_contiguous()) throw Refusal{PyExc_ValueError, std::string(name) + " must be contiguous"};
  return t;
}

const at::Tensor& matrix(PyObject* o, at::ScalarType type, const char* name) {
  const at::Tensor& t = tensor(o, type, name);
  if (t.dim() != 2)
    throw Refusal{PyExc_ValueError, std::string(name) + " must be a matrix, got " + std::to_string(t.dim()) + " dimensions"};
  return t;
}

// A tensor of that shape on device `dev`.
const at::Tensor& operand(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, int dev,
                          const char* name) {
  const at::Tensor& t = tensor(o, type, name);
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want)
    throw Refusal{PyExc_ValueError, std::string(name) + " must be " + sizes_text(want) + ", got " + sizes_text(t.sizes())};
  if (t.get_device() != dev)
    throw Refusal{PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                        ", the other operands on cuda:" + std::to_string(dev)};
  return t;
}

// A new tensor, straight from the caching allocator (0.3 us a tensor less than
// by way of the dispatcher).
at::Tensor made(std::initializer_list<int64_t> shape, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), type, like.device(), std::nullopt);
}

// An output: the caller's, checked, or a new one.
at::Tensor output(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const at::Tensor& like,
                  const char* name) {
  if (o != Py_None) return operand(o, type, shape, like.get_device(), name);
  return made(shape, type, like);
}

// The caller's workspace, or one of this call's own: calls on two streams, or
// captured in two graphs, then never share one.
at::Tensor scratch(PyObject* o, int64_t bytes, const at::Tensor& like) {
  if (o == Py_None) return made({bytes > 16 ? bytes : 16}, at::kByte, like);
  const at::Tensor& t = tensor(o, at::kByte, "ws");
  if (t.get_device() != like.get_device()) throw Refusal{PyExc_ValueError, "ws must be on the operands' device"};
  return t;
}

template <typename T>
T* at_(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

void* stream_of(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(t.get_device())).stream();
}

// Calls the library with t's device current and without the interpreter lock.
template <typename F>
void call(const char* func, const at::Tensor& t, F&& f) {
  int rc;
  {
    const c10::cuda::OptionalCUDAGuard guard(t.device());
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
  }
  if (rc != STQ1_OK) throw Failure{func, rc};
}

// Runs a call's body; what it throws becomes the Python exception.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const Failure& e) {
    PyObject* v = PyObject_CallFunction(g_error, "si", e.func, e.code);
    if (v) {
      PyErr_SetObject(g_error, v);
      Py_DECREF(v);
    }
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return t;
}
PyObject* wrapped(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// (src, out, scales) -> (codes, scales)
PyObject* quantize_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    const bool f32 = THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).scalar_type() == at::kFloat;
    const at::Tensor& src = matrix(a[0], f32 ? at::kFloat : at::kBFloat16, "src");
    const int64_t r = src.size(0), k = src.size(1);
    const at::Tensor q = output(a[1], at::kChar, {r, k}, src, "out"), s = output(a[2], at::kFloat, {r}, src, "scales");
    call("stq1_quantize_i8", src, [&] {
      return f_quantize_i8(src.data_ptr(), f32 ? STQ1_TYPE_F32 : STQ1_TYPE_BF16, r, k, at_<int8_t>(q), at_<float>(s),
                           stream_of(src));
    });
    return pair(wrapped(q), wrapped(s));
  });
}

// (x_q, x_scales, w_q, w_scales, out, bf16) -> y
PyObject* i8_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Tensor& x = matrix(a[0], at::kChar, "x_q");
    const at::Tensor& w = matrix(a[2], at::kChar, "w_q");
    const int64_t t = x.size(0), k = x.size(1), m = w.size(0);
    const int dev = x.get_device();
    const at::Tensor& sx = operand(a[1], at::kFloat, {t}, dev, "x_scales");
    operand(a[2], at::kChar, {m, k}, dev, "w_q");
    const at::Tensor& sw = operand(a[3], at::kFloat, {m}, dev, "w_scales");
    const bool bf16 = a[5] == Py_True;
    const at::Tensor y = output(a[4], bf16 ? at::kBFloat16 : at::kFloat, {t, m}, x, "out");
    call("stq1_i8_matmul", x, [&] {
      return f_i8_matmul(at_<int8_t>(x), at_<float>(sx), at_<int8_t>(w), at_<float>(sw), y.data_ptr(),
                         bf16 ? STQ1_TYPE_BF16 : STQ1_TYPE_F32, t, m, k, stream_of(x));
    });
    return wrapped(y);
  });
}

// (x, gateup_q, gateup_scales, down_q, down_scales, out, ws) -> out
PyObject* i8_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const at::Tensor& x = matrix(a[0], at::kBFloat16, "x");
    const int64_t t = x.size(0), h = x.size(1), m = matrix(a[1], at::kChar, "gateup_q").size(0);
    const int dev = x.get_device();
    const at::Tensor& gu = operand(a[1], at::kChar, {m, h}, dev, "gateup_q");
    const at::Tensor& sgu = operand(a[2], at::kFloat, {m}, dev, "gateup_scales");
    const at::Tensor& dn = operand(a[3], at::kChar, {h, m / 2}, dev, "down_q");
    const at::Tensor& sdn = operand(a[4], at::kFloat, {h}, dev, "down_scales");
    const at::Tensor out = output(a[5], at::kFloat, {t, h}, x, "out");
    const at::Tensor ws = scratch(a[6], static_cast<int64_t>(f_i8_ffn_workspace(t, m, h)), x);
    call("stq1_i8_ffn", x, [&] {
      return f_i8_ffn(at_<uint16_t>(x), at_<int8_t>(gu), at_<float>(sgu), at_<int8_t>(dn), at_<float>(sdn),
                      at_<float>(out), t, m, h, ws.data_ptr(), static_cast<size_t>(ws.numel()), stream_of(x));
    });
    return wrapped(out);
  });
}

// (x, w, save, out, y) -> act or (act, y)
PyObject* glu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    const at::Tensor& x = matrix(a[0], at::kBFloat16, "x");
    const int64_t t = x.size(0), k = x.size(1), m = matrix(a[1], at::kBFloat16, "w").size(0);
    const at::Tensor& w = operand(a[1], at::kBFloat16, {m, k}, x.get_device(), "w");
    const at::Tensor act = output(a[3], at::kBFloat16, {t, m / 2}, x, "out");
    at::Tensor y;
    if (a[2] == Py_True) y = output(a[4], at::kBFloat16, {t, m}, x, "y");
    call("stq1_glu", x, [&] {
      return f_glu(at_<uint16_t>(x), at_<uint16_t>(w), at_<uint16_t>(act), y.defined() ? at_<uint16_t>(y) : nullptr, t, m,
                   k, stream_of(x));
    });
    return y.defined() ? pair(wrapped(act), wrapped(y)) : wrapped(act);
  });
}

// (dact, y, x or None, w or None, dx, dw, need_dx, need_dw, ws) -> (dx or None, dw or None)
PyObject* glu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const at::Tensor& y = matrix(a[1], at::kBFloat16, "y");
    const int64_t t = y.size(0), m = y.size(1);
    const bool need_dx = a[6] == Py_True, need_dw = a[7] == Py_True;
    if (!need_dx && !need_dw) throw Refusal{PyExc_ValueError, "glu_backward: nothing to compute"};
    if ((need_dx && a[3] == Py_None) || (need_dw && a[2] == Py_None))
      throw Refusal{PyExc_ValueError, "dx needs w, and dw needs x"};
    const int64_t k = a[2] != Py_None ? matrix(a[2], at::kBFloat16, "x").size(1) : matrix(a[3], at::kBFloat16, "w").size(1);
    const int dev = y.get_device();
    const at::Tensor& dact = operand(a[0], at::kBFloat16, {t, m / 2}, dev, "dact");
    const uint16_t* x = a[2] == Py_None ? nullptr : at_<uint16_t>(operand(a[2], at::kBFloat16, {t, k}, dev, "x"));
    const uint16_t* w = a[3] == Py_None ? nullptr : at_<uint16_t>(operand(a[3], at::kBFloat16, {m, k}, dev, "w"));
    at::Tensor dx, dw;
    if (need_dx) dx = output(a[4], at::kBFloat16, {t, k}, y, "dx");
    if (need_dw) dw = output(a[5], at::kBFloat16, {m, k}, y, "dw");
    const at::Tensor ws = scratch(a[8], static_cast<int64_t>(f_glu_backward_workspace(t, m, k)), y);
    call("stq1_glu_backward", y, [&] {
      return f_glu_backward(at_<uint16_t>(dact), at_<uint16_t>(y), x, w, need_dx ? at_<uint16_t>(dx) : nullptr,
                            need_dw ? at_<uint16_t>(dw) : nullptr, t, m, k, ws.data_ptr(),
                            static_cast<size_t>(ws.numel()), stream_of(y));
    });
    return pair(wrapped(dx), wrapped(dw));
  });
}

// (addresses of the seven entry points, Stq1Error)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[7];
  PyObject* error;
  if (!PyArg_ParseTuple(args, "(KKKKKKK)O", p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6, &error)) return nullptr;
  f_quantize_i8 = reinterpret_cast<decltype(f_quantize_i8)>(p[0]);
  f_i8_matmul = reinterpret_cast<decltype(f_i8_matmul)>(p[1]);
  f_i8_ffn_workspace = reinterpret_cast<decltype(f_i8_ffn_workspace)>(p[2]);
  f_i8_ffn = reinterpret_cast<decltype(f_i8_ffn)>(p[3]);
  f_glu = reinterpret_cast<decltype(f_glu)>(p[4]);
  f_glu_backward_workspace = reinterpret_cast<decltype(f_glu_backward_workspace)>(p[5]);
  f_glu_backward = reinterpret_cast<decltype(f_glu_backward)>(p[6]);
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

#define STQ1_FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr}, STQ1_FAST(quantize_i8), STQ1_FAST(i8_matmul),
                         STQ1_FAST(i8_ffn),                     STQ1_FAST(glu),         STQ1_FAST(glu_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense_calls() { return PyModule_Create(&module); }
