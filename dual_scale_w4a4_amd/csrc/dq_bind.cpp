// dq_bind.cpp -- the Python binding's calls of the MLP operators (include/dq_mlp.h): argument
// checks, output tensors, the stream, and the call of the C entry point. A single token's
// operator is a few microseconds on the GPU, less than the same checks took in Python: on one
// box gemm_mx_epilogue cost the host 10 us a call there and 5 here.
//
// Every tensor lies on one device, the first argument's, which is made current for the call. The
// work goes to `stream` (a torch stream or None for the device's current one), on which the
// outputs allocated here belong too.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <array>
#include <optional>
#include <string>

#include "../../include/dq_mlp.h"

namespace {

PyObject* g_error = nullptr;       // DQError
PyObject* g_raw_stream = nullptr;  // device index -> the current stream's handle

template <class... A>
[[noreturn]] void refuse(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw python_error();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// The device of a call from its first tensor
c10::Device device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda() || t.dim() != 2) refuse("%s must be a 2-D CUDA (HIP) tensor", name);
  return t.device();
}

struct Arr {
  c10::Device dev;

  void* need(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef sizes) const {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != sizes || t.device() != dev || !t.is_contiguous()) {
      std::string shape;
      for (int64_t n : sizes) shape += (shape.empty() ? "" : ", ") + std::to_string(n);
      refuse("%s must be a contiguous %s tensor of shape (%s) on cuda:%d", name,
             c10::toString(type), shape.c_str(), (int)dev.index());
    }
    return t.data_ptr();
  }
  void* option(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef sizes) const {
    return o == Py_None ? nullptr : need(o, name, type, sizes);
  }
  const float* floats(PyObject* o, const char* name, int64_t n) const {
    return static_cast<const float*>(option(o, name, at::kFloat, {n}));
  }
};

// Device and stream of a call, while it lasts
struct Place {
  std::optional<c10::StreamGuard> on;
  std::optional<c10::DeviceGuard> at;
  hipStream_t stream;

  Place(c10::Device dev, PyObject* s) {
    if (s != Py_None) {
      auto number = [&](const char* name) {
        THPObjectPtr v(PyObject_GetAttrString(s, name));
        if (!v) throw python_error();
        const int64_t n = PyLong_AsLongLong(v.get());
        if (n == -1 && PyErr_Occurred()) throw python_error();
        return n;
      };
      if (number("device_index") != dev.index())
        refuse("stream belongs to another device than the tensors");
      on.emplace(c10::Stream::unpack3(number("stream_id"), dev.index(),
                                      static_cast<c10::DeviceType>(number("device_type"))));
    } else {
      at.emplace(dev);
    }
    THPObjectPtr index(PyLong_FromLong(dev.index()));
    THPObjectPtr v(PyObject_CallOneArg(g_raw_stream, index.get()));
    if (!v) throw python_error();
    stream = static_cast<hipStream_t>(PyLong_AsVoidPtr(v.get()));
    if (PyErr_Occurred()) throw python_error();
  }
};

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(dev));
}

void check(dq_status st, const char* what) {
  if (st == DQ_OK) return;
  THPObjectPtr e(PyObject_CallFunction(g_error, "is", (int)st, what));
  if (e) PyErr_SetObject(g_error, e.get());
  throw python_error();
}

bool is(PyObject* o, const char* s) {
  return PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, s) == 0;
}

int64_t integer(PyObject* o) {
  const int64_t n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw python_error();
  return n;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// A name's place in a list; `fmts` and `acts` are numbered as the enums
template <size_t N>
int choice(PyObject* o, const char* const (&names)[N], const char* what) {
  for (size_t k = 0; k < N; k++)
    if (is(o, names[k])) return (int)k;
  refuse("unknown %s %R", what, o);
}
constexpr const char* kFmts[] = {"int4_bf16", "mxint4", "mxfp4", "nvfp4", "mxfp8"};
constexpr const char* kActs[] = {"none", "relu", "silu", "gelu", "gelu_tanh"};

// ------------------------------------------------------------------- norm and quantizer

struct QuantShape {
  int fmt;
  int64_t group, tokens, cols;
  at::ScalarType scale_type;

  QuantShape(const at::Tensor& X, PyObject* f, PyObject* g)
      : fmt(choice(f, kFmts, "format")), group(integer(g)), tokens(X.size(0)), cols(X.size(1)) {
    if ((group != 16 && group != 32 && group != 64) || cols % group)
      refuse("group must be 16, 32 or 64 and divide the channels");
    scale_type = fmt == DQ_FMT_INT4_BF16 ? at::kShort : at::kByte;
  }
  std::array<int64_t, 2> codes() const { return {tokens, fmt == DQ_FMT_MXFP8 ? cols : cols / 2}; }
  std::array<int64_t, 2> scales() const { return {tokens, cols / group}; }
};

// act_outputs(X, fmt, group) -> (codes, scales)
PyObject* act_outputs(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const at::Tensor& X = tensor(a[0], "X");
  const c10::Device dev = device_of(X, "X");
  const QuantShape q(X, a[1], a[2]);
  THPObjectPtr codes(THPVariable_Wrap(make(q.codes(), at::kByte, dev)));
  THPObjectPtr scales(THPVariable_Wrap(make(q.scales(), q.scale_type, dev)));
  if (!codes || !scales) throw python_error();
  return PyTuple_Pack(2, codes.get(), scales.get());
  END_HANDLE_TH_ERRORS
}

// norm(X, fmt, group, codes, scales, status, weight, residual, residual_out, b, eps, g,
//      workspace, stream): asynchronous with a status tensor, else blocking
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const at::Tensor& X = tensor(a[0], "X");
  const Arr arr{device_of(X, "X")};
  const at::ScalarType xt = X.scalar_type();
  if ((xt != at::kFloat && xt != at::kBFloat16) || !X.is_contiguous())
    refuse("X must be a contiguous 2-D float32 or bfloat16 tensor");
  const QuantShape q(X, a[1], a[2]);
  const auto cs = q.codes(), ss = q.scales();
  void* codes = arr.need(a[3], "codes", at::kByte, cs);
  void* scales = arr.need(a[4], "scales", q.scale_type, ss);
  const void* weight = nullptr;
  dq_dtype wt = DQ_F32;
  if (a[6] != Py_None) {
    const at::ScalarType t = tensor(a[6], "weight").scalar_type();
    if (t != at::kFloat && t != at::kBFloat16) refuse("weight must be float32 or bfloat16");
    wt = t == at::kBFloat16 ? DQ_BF16 : DQ_F32;
    weight = arr.need(a[6], "weight", t, {q.cols});
  }
  const void* residual = arr.option(a[7], "residual", xt, X.sizes());
  void* residual_out = arr.option(a[8], "residual_out", xt, X.sizes());
  const float* b = arr.floats(a[9], "b", q.cols);
  const double eps = number(a[10]);
  const float g = (float)number(a[11]);
  const dq_dtype dt = xt == at::kBFloat16 ? DQ_BF16 : DQ_F32;
  if (a[5] != Py_None) {
    const at::Tensor& st = tensor(a[5], "status");
    if (st.scalar_type() != at::kInt || st.device() != arr.dev || st.numel() < 1)
      refuse("status must be an int32 tensor on X's device");
    const Place place(arr.dev, a[13]);
    check(dq_norm_quantize_act_async(X.data_ptr(), dt, residual, residual_out, q.tokens, q.cols,
                                     weight, wt, eps, b, (dq_format)q.fmt, (int)q.group, g,
                                     static_cast<uint8_t*>(codes), scales,
                                     static_cast<int*>(st.data_ptr()), place.stream),
          "dq_norm_quantize_act_async");
  } else {
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[12] != Py_None) {
      const at::Tensor& w = tensor(a[12], "workspace");
      if (w.device() != arr.dev) refuse("workspace must lie on X's device");
      ws = w.data_ptr();
      bytes = w.nbytes();
    }
    const Place place(arr.dev, a[13]);
    dq_status st;
    Py_BEGIN_ALLOW_THREADS  // it waits for the stream
    st = dq_norm_quantize_act(X.data_ptr(), dt, residual, residual_out, q.tokens, q.cols, weight,
                              wt, eps, b, (dq_format)q.fmt, (int)q.group, g,
                              static_cast<uint8_t*>(codes), scales, ws, bytes, place.stream);
    Py_END_ALLOW_THREADS
    check(st, "dq_norm_quantize_act");
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------------ products

// Packed weights: {"codes", "scales", "out", "K"}
struct Packed {
  int64_t out, K;
  PyObject *codes, *scales;

  Packed(PyObject* d, const char* name) {
    if (!PyDict_Check(d)) refuse("%s must be a dict from gemm_pack_weights", name);
    auto item = [&](const char* key) {
      PyObject* v = PyDict_GetItemString(d, key);
      if (!v) refuse("%s must be a dict from gemm_pack_weights", name);
      return v;
    };
    codes = item("codes");
    scales = item("scales");
    out = integer(item("out"));
    K = integer(item("K"));
    if (out < 1 || K < 512 || K % 512 || K > (1 << 22) || out > INT32_MAX)
      refuse("%s must be a dict from gemm_pack_weights", name);
  }
  // of (out rounded up to 32 rows) x K weights
  const uint8_t* code_ptr(const Arr& arr, const char* name) const {
    return static_cast<const uint8_t*>(arr.need(codes, name, at::kByte, {(out + 31) / 32 * 16 * K}));
  }
  const uint8_t* scale_ptr(const Arr& arr, const char* name) const {
    return static_cast<const uint8_t*>(arr.need(scales, name, at::kByte, {(out + 31) / 32 * K}));
  }
};

struct Acts {
  Arr arr;
  dq_format fmt;
  int64_t tokens;
  const uint8_t *codes, *scales;

  Acts(PyObject* c, PyObject* s, PyObject* f, int64_t K)
      : arr{device_of(tensor(c, "act_codes"), "act_codes")},
        fmt(is(f, "mxfp4") ? DQ_FMT_MXFP4 : DQ_FMT_MXFP8),
        tokens(THPVariable_Unpack(c).size(0)) {
    if (fmt == DQ_FMT_MXFP8 && !is(f, "mxfp8")) refuse("act_fmt is 'mxfp4' or 'mxfp8'");
    codes = static_cast<const uint8_t*>(
        arr.need(c, "act_codes", at::kByte, {tokens, fmt == DQ_FMT_MXFP8 ? K : K / 2}));
    scales = static_cast<const uint8_t*>(arr.need(s, "act_scales", at::kByte, {tokens, K / 32}));
  }
};

at::ScalarType out_type(PyObject* o) {
  if (is(o, "bf16")) return at::kBFloat16;
  if (!is(o, "f32")) refuse("out_dtype is 'bf16' or 'f32'");
  return at::kFloat;
}

// epilogue(act_codes, act_scales, packed, a, bias, activation, residual, act_fmt, out_dtype, y,
//          stream) -> y
PyObject* epilogue(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Packed w(a[2], "packed");
  const Acts x(a[0], a[1], a[7], w.K);
  const Arr& arr = x.arr;
  const at::ScalarType type = out_type(a[8]);
  const std::array<int64_t, 2> shape{x.tokens, w.out};
  const uint8_t *wc = w.code_ptr(arr, "packed codes"), *ws = w.scale_ptr(arr, "packed scales");
  const float *scale = arr.floats(a[3], "a", w.out), *bias = arr.floats(a[4], "bias", w.out);
  const int act = choice(a[5], kActs, "activation");
  const void* residual = arr.option(a[6], "residual", type, shape);
  void* y = arr.option(a[9], "y", type, shape);
  const Place place(arr.dev, a[10]);
  at::Tensor made;
  if (!y) {
    made = make(shape, type, arr.dev);
    y = made.data_ptr();
  }
  check(dq_gemm_mx_epilogue(x.codes, x.scales, x.fmt, x.tokens, w.K, wc, ws, scale, bias,
                            (dq_activation)act, residual, w.out,
                            type == at::kBFloat16 ? DQ_BF16 : DQ_F32, y, place.stream),
        "dq_gemm_mx_epilogue");
  if (made.defined()) return THPVariable_Wrap(std::move(made));
  Py_INCREF(a[9]);
  return a[9];
  END_HANDLE_TH_ERRORS
}

// The arguments that both forms of the gated product share: (act_codes, act_scales, gate, up,
// a_gate, a_up, activation, act_fmt)
struct Gated {
  Packed gate, up;
  Acts x;
  const uint8_t *gc, *gs, *uc, *us;
  const float *ag, *au;
  dq_activation act;

  explicit Gated(PyObject* const* a)
      : gate(a[2], "gate"), up(a[3], "up"), x(a[0], a[1], a[7], gate.K) {
    if (gate.out != up.out || gate.K != up.K) refuse("gate and up weights disagree on their channels");
    gc = gate.code_ptr(x.arr, "gate codes");
    gs = gate.scale_ptr(x.arr, "gate scales");
    uc = up.code_ptr(x.arr, "up codes");
    us = up.scale_ptr(x.arr, "up scales");
    ag = x.arr.floats(a[4], "a_gate", gate.out);
    au = x.arr.floats(a[5], "a_up", gate.out);
    act = (dq_activation)choice(a[6], kActs, "activation");
  }
};

// gated(.. as above .., out_dtype, y, stream) -> y
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Gated p(a);
  const Arr& arr = p.x.arr;
  const at::ScalarType type = out_type(a[8]);
  const std::array<int64_t, 2> shape{p.x.tokens, p.gate.out};
  void* y = arr.option(a[9], "y", type, shape);
  const Place place(arr.dev, a[10]);
  at::Tensor made;
  if (!y) {
    made = make(shape, type, arr.dev);
    y = made.data_ptr();
  }
  check(dq_gated_mx(p.x.codes, p.x.scales, p.x.fmt, p.x.tokens, p.gate.K, p.gc, p.gs, p.ag, p.uc,
                    p.us, p.au, p.act, p.gate.out, type == at::kBFloat16 ? DQ_BF16 : DQ_F32, y,
                    place.stream),
        "dq_gated_mx");
  if (made.defined()) return THPVariable_Wrap(std::move(made));
  Py_INCREF(a[9]);
  return a[9];
  END_HANDLE_TH_ERRORS
}

// gated_quantized(.. as above .., fmt, b, codes, scales, stream) -> (codes, scales)
PyObject* gated_quantized(PyObject*, PyObject* const* a, Py_ssize_t) {
  HANDLE_TH_ERRORS
  const Gated p(a);
  const Arr& arr = p.x.arr;
  const int64_t tokens = p.x.tokens, inner = p.gate.out;
  const int fmt = choice(a[8], kFmts, "format");
  if ((fmt != DQ_FMT_MXFP4 && fmt != DQ_FMT_MXFP8) || inner % 32)
    refuse("fmt is 'mxfp4' or 'mxfp8', and the channels a multiple of 32");
  const std::array<int64_t, 2> cs{tokens, fmt == DQ_FMT_MXFP8 ? inner : inner / 2},
      ss{tokens, inner / 32};
  const float* b = arr.floats(a[9], "b", inner);
  void *codes = arr.option(a[10], "codes", at::kByte, cs),
       *scales = arr.option(a[11], "scales", at::kByte, ss);
  const Place place(arr.dev, a[12]);
  THPObjectPtr co(a[10]), so(a[11]);
  Py_INCREF(a[10]);
  Py_INCREF(a[11]);
  auto fill = [&](void*& ptr, THPObjectPtr& o, at::IntArrayRef shape) {
    if (ptr) return;
    at::Tensor t = make(shape, at::kByte, arr.dev);
    ptr = t.data_ptr();
    o = THPVariable_Wrap(std::move(t));
    if (!o) throw python_error();
  };
  fill(codes, co, cs);
  fill(scales, so, ss);
  check(dq_gated_mx_quantized(p.x.codes, p.x.scales, p.x.fmt, tokens, p.gate.K, p.gc, p.gs, p.ag,
                              p.uc, p.us, p.au, p.act, inner, b, (dq_format)fmt,
                              static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                              place.stream),
        "dq_gated_mx_quantized");
  return PyTuple_Pack(2, co.get(), so.get());
  END_HANDLE_TH_ERRORS
}

// bind(DQError, raw_stream)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t) {
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(g_error, a[0]);
  Py_XSETREF(g_raw_stream, a[1]);
  Py_RETURN_NONE;
}

// Positional calls with a fixed number of arguments (the Python functions of the package make
// them); N is checked here, so the bodies index freely.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int N>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  return F(self, a, n);
}

#define DQ_METHOD(f, n) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(counted<f, n>)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {DQ_METHOD(bind, 2),      DQ_METHOD(act_outputs, 3),
                          DQ_METHOD(norm, 14),     DQ_METHOD(epilogue, 11),
                          DQ_METHOD(gated, 11),    DQ_METHOD(gated_quantized, 13),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&kModule); }
