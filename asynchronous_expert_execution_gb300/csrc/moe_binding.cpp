// Python binding of the stateless operators: argument checks, outputs and the call, in C++ because
// a small call is bound by its host side (a decode step's norm runs 3 us on the GPU; checked and
// marshalled in Python it took 10.6 us, here 4).  Nothing is computed here: every function ends
// in one moe_async_* call of the library that _native.py loaded (bind() gets their addresses).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <sstream>
#include <string>

#include "../../include/moe_async.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Library {
  decltype(&moe_async_sort_experts) sort_experts;
  decltype(&moe_async_sort_rows) sort_rows;
  decltype(&moe_async_merge_rows) merge_rows;
  decltype(&moe_async_merge_rows_backward) merge_rows_backward;
  decltype(&moe_async_route_backward) route_backward;
  decltype(&moe_async_add_rms_norm) add_rms_norm;
  decltype(&moe_async_add_rms_norm_backward_workspace) norm_workspace;
  decltype(&moe_async_add_rms_norm_backward) add_rms_norm_backward;
  decltype(&moe_async_linear) linear;
  decltype(&moe_async_linear_backward_workspace) linear_backward_workspace;
  decltype(&moe_async_linear_backward) linear_backward;
  decltype(&moe_async_act_mul_backward) act_mul_backward;
  decltype(&moe_async_linear_blocks) linear_blocks;
  decltype(&moe_async_quantize_blocks) quantize_blocks;
} lib = {};
PyObject* error_class = nullptr;

// A refused call (becomes MoEError(status, what)), or a Python error that is already set.
struct Refused {
  int status;
  std::string what;
};
struct PythonError {};

[[noreturn]] void bad(const std::string& what) { throw Refused{MOE_ERR_INVALID, what}; }

[[noreturn]] void bad(const std::string& what, const Tensor& t) {
  std::ostringstream s;
  s << what << "; got " << t.sizes() << " of " << t.scalar_type() << " on " << t.device() << ", strides " << t.strides();
  bad(s.str());
}

std::string shape(int64_t rows, int64_t width) { return "[" + std::to_string(rows) + ", " + std::to_string(width) + "]"; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + ": expected a tensor");
  const Tensor& t = THPVariable_Unpack(o);
  // nothing is recorded here: what autograd would follow has to be said to be left out
  if (t.requires_grad() && c10::GradMode::is_enabled())
    bad(std::string(name) + ": requires grad, which the operators do not record; detach it, or call under torch.no_grad() or in an "
                            "autograd.Function with the *_backward functions");
  return t;
}
const Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
template <typename T = void>
T* ptr(const Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
template <typename T = void>
T* ptr(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max()) bad(std::string(name) + ": out of range");
  return v;
}

int32_t count(int64_t n, const char* name) {
  if (n > std::numeric_limits<int32_t>::max()) bad(std::string(name) + ": 2^31 or more");
  return static_cast<int32_t>(n);
}

int32_t code(ScalarType t) { return t == at::kFloat ? MOE_F32 : t == at::kBFloat16 ? MOE_BF16 : MOE_E4M3; }

// Row stride of a [rows, width] matrix on device `dev`: adjacent columns, rows that do not overlap.
int64_t rows(const Tensor& t, const char* name, int dev, ScalarType dtype, int64_t n, int64_t width) {
  if (t.scalar_type() != dtype || !t.is_cuda() || t.get_device() != dev || t.dim() != 2 || t.size(0) != n || t.size(1) != width)
    bad(std::string(name) + ": expected " + shape(n, width) + " of " + c10::toString(dtype) + " on cuda:" + std::to_string(dev), t);
  if (width > 1 && t.stride(1) != 1) bad(std::string(name) + ": expected adjacent columns", t);
  if (n <= 1) return width;
  if (t.stride(0) < width) bad(std::string(name) + ": expected rows that do not overlap", t);
  return t.stride(0);
}

// The matrix that names the call's device.
struct Lead {
  int dev;
  int64_t n, width, ld;
  ScalarType dtype;
};
Lead lead(const Tensor& t, const char* name, std::initializer_list<ScalarType> dtypes) {
  bool known = false;
  for (ScalarType d : dtypes) known |= t.scalar_type() == d;
  if (!t.is_cuda() || t.dim() != 2 || !known) {
    std::string s = std::string(name) + ": expected a CUDA matrix of";
    for (ScalarType d : dtypes) s += std::string(" ") + c10::toString(d);
    bad(s, t);
  }
  const int dev = t.get_device();
  return {dev, t.size(0), t.size(1), rows(t, name, dev, t.scalar_type(), t.size(0), t.size(1)), t.scalar_type()};
}

// A contiguous tensor.
void whole(const Tensor& t, const char* name, int dev, ScalarType dtype, at::IntArrayRef sizes) {
  if (t.scalar_type() != dtype || !t.is_cuda() || t.get_device() != dev || t.sizes() != sizes || !t.is_contiguous()) {
    std::ostringstream s;
    s << name << ": expected contiguous " << sizes << " of " << dtype << " on cuda:" << dev;
    bad(s.str(), t);
  }
}

int64_t pairs(const Tensor& pos, int dev) {
  if (pos.dim() != 2) bad("pos: expected [T, K]", pos);
  whole(pos, "pos", dev, at::kInt, pos.sizes());
  return pos.size(1);
}

Tensor empty(at::IntArrayRef sizes, ScalarType dtype, int dev) {
  return at::detail::empty_cuda(sizes, dtype, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

// `out` as handed in (checked), or a new matrix; its row stride in ld.
Tensor output(PyObject* out, const char* name, int dev, ScalarType dtype, int64_t n, int64_t width, int64_t& ld) {
  if (out == Py_None) {
    ld = width;
    return empty({n, width}, dtype, dev);
  }
  const Tensor& t = tensor(out, name);
  ld = rows(t, name, dev, dtype, n, width);
  return t;
}

// An output that was handed in has been written over: autograd finds it where it was saved before.
void written(PyObject* out) {
  if (out == Py_None) return;
  const Tensor& t = THPVariable_Unpack(out);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();     // an inference tensor has no version
}

// The call's device and stream, made current while it runs: what the call allocates belongs to that
// stream, so memory that other streams gave back is not written before they are done with it.
struct On {
  int dev;
  cudaStream_t stream;
  c10::cuda::OptionalCUDAStreamGuard guard;
  c10::cuda::OptionalCUDAGuard device;
  On(int d, PyObject* s) : dev(d) {
    if (s == Py_None) {
      if (c10::cuda::current_device() != d) device.set_index(static_cast<c10::DeviceIndex>(d));
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(d)).stream();
      return;
    }
    PyObject* v = PyObject_GetAttrString(s, "cuda_stream");
    if (!v) throw PythonError{};
    stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
    Py_DECREF(v);
    if (PyErr_Occurred()) throw PythonError{};
    if (PyObject* index = PyObject_GetAttrString(s, "device_index")) {      // an object that names no device is taken at its word
      const long at = PyLong_AsLong(index);
      Py_DECREF(index);
      if (at == -1 && PyErr_Occurred()) throw PythonError{};
      if (at != d) bad("stream: on cuda:" + std::to_string(at) + ", the tensors on cuda:" + std::to_string(d));
    } else {
      PyErr_Clear();
    }
    guard.reset_stream(c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(d)));
  }
};

template <typename F>
void call(const char* what, const On& on, F f) {
  int status;
  PyThreadState* state = PyEval_SaveThread();        // a launch may wait for room in the stream
  try {
    status = f(static_cast<void*>(on.stream));
  } catch (...) {
    PyEval_RestoreThread(state);
    throw;
  }
  PyEval_RestoreThread(state);
  if (status != MOE_OK) throw Refused{status, what};
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

// ------------------------------------------------------------------ the operators
// Arguments come in the order of the functions in ops.py.

// expert, num_experts, stream
PyObject* sort_experts(PyObject* const* a) {
  const Tensor& expert = tensor(a[0], "expert");
  const Lead l = lead(expert, "expert", {at::kInt});
  const On on(l.dev, a[2]);
  if (!expert.is_contiguous()) bad("expert: expected contiguous", expert);
  const int64_t E = integer(a[1], "num_experts");
  if (E < 1) bad("num_experts: expected at least 1");
  const int32_t T = count(l.n, "tokens"), K = count(l.width, "top_k");
  Tensor offsets = empty({E + 1}, at::kInt, l.dev), pos = empty({T, K}, at::kInt, l.dev), pair = empty({l.n * l.width}, at::kInt, l.dev);
  call("sort_experts", on, [&](void* s) {
    return lib.sort_experts(ptr<int32_t>(expert), T, K, static_cast<int32_t>(E), ptr<int32_t>(offsets), ptr<int32_t>(pos),
                            ptr<int32_t>(pair), s);
  });
  return tuple({wrap(offsets), wrap(pos), wrap(pair)});
}

// x, pos, out, stream
PyObject* sort_rows(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &pos = tensor(a[1], "pos");
  const Lead l = lead(x, "x", {at::kFloat, at::kBFloat16});
  const On on(l.dev, a[3]);
  const int64_t K = pairs(pos, l.dev);
  if (pos.size(0) != l.n) bad("pos: expected a row per row of x", pos);
  int64_t ldo, R = a[2] == Py_None ? l.n * K : tensor(a[2], "out").dim() == 2 ? tensor(a[2], "out").size(0) : 0;
  const Tensor out = output(a[2], "out", l.dev, l.dtype, R, l.width, ldo);
  call("sort_rows", on, [&](void* s) {
    return lib.sort_rows(code(l.dtype), ptr(x), l.ld, ptr<int32_t>(pos), count(l.n, "tokens"), count(K, "top_k"),
                         count(l.width, "width"), ptr(out), ldo, R, s);
  });
  written(a[2]);
  return wrap(out);
}

// rows, pos, w, residual, out, stream
PyObject* merge_rows(PyObject* const* a) {
  const Tensor &r = tensor(a[0], "rows"), &pos = tensor(a[1], "pos");
  const Tensor *w = maybe(a[2], "w"), *res = maybe(a[3], "residual");
  const Lead l = lead(r, "rows", {at::kFloat, at::kBFloat16});
  const On on(l.dev, a[5]);
  const int64_t K = pairs(pos, l.dev), T = pos.size(0);
  if (w) whole(*w, "w", l.dev, at::kFloat, {T, K});
  const int64_t ldres = res ? rows(*res, "residual", l.dev, l.dtype, T, l.width) : l.width;
  int64_t ldo;
  const Tensor out = output(a[4], "out", l.dev, l.dtype, T, l.width, ldo);
  call("merge_rows", on, [&](void* s) {
    return lib.merge_rows(code(l.dtype), ptr(r), l.ld, l.n, ptr<int32_t>(pos), ptr<float>(w), count(T, "tokens"), count(K, "top_k"),
                          count(l.width, "width"), ptr(res), ldres, ptr(out), ldo, s);
  });
  written(a[4]);
  return wrap(out);
}

// grad, rows, pos, w, out, stream
PyObject* merge_rows_backward(PyObject* const* a) {
  const Tensor &grad = tensor(a[0], "grad"), &r = tensor(a[1], "rows"), &pos = tensor(a[2], "pos"), &w = tensor(a[3], "w");
  const Lead l = lead(r, "rows", {at::kFloat, at::kBFloat16});
  const On on(l.dev, a[5]);
  const int64_t K = pairs(pos, l.dev), T = pos.size(0);
  whole(w, "w", l.dev, at::kFloat, {T, K});
  const int64_t ldg = rows(grad, "grad", l.dev, l.dtype, T, l.width);
  int64_t ldo;
  const Tensor out = output(a[4], "out", l.dev, l.dtype, l.n, l.width, ldo);
  Tensor grad_w = empty({T, K}, at::kFloat, l.dev);
  call("merge_rows_backward", on, [&](void* s) {
    return lib.merge_rows_backward(code(l.dtype), ptr(grad), ldg, ptr(r), l.ld, l.n, ptr<int32_t>(pos), ptr<float>(w),
                                   count(T, "tokens"), count(K, "top_k"), count(l.width, "width"), ptr(out), ldo,
                                   ptr<float>(grad_w), s);
  });
  written(a[4]);
  return tuple({wrap(out), wrap(grad_w)});
}

// idx, w, grad_w, num_experts, stream
PyObject* route_backward(PyObject* const* a) {
  const Tensor &idx = tensor(a[0], "idx"), &w = tensor(a[1], "w"), &grad_w = tensor(a[2], "grad_w");
  const Lead l = lead(w, "w", {at::kFloat});
  const On on(l.dev, a[4]);
  whole(w, "w", l.dev, at::kFloat, {l.n, l.width});
  whole(idx, "idx", l.dev, at::kInt, {l.n, l.width});
  whole(grad_w, "grad_w", l.dev, at::kFloat, {l.n, l.width});
  const int64_t E = integer(a[3], "num_experts");
  if (E < 1) bad("num_experts: expected at least 1");
  Tensor out = empty({l.n, E}, at::kFloat, l.dev);
  call("route_backward", on, [&](void* s) {
    return lib.route_backward(ptr<int32_t>(idx), ptr<float>(w), ptr<float>(grad_w), count(l.n, "tokens"), static_cast<int32_t>(E),
                              count(l.width, "top_k"), ptr<float>(out), s);
  });
  return wrap(out);
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}

// x, residual, gain, eps, out, out_h, stream, e4m3 -> (y, scale or None, h)
PyObject* add_rms_norm(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Tensor *res = maybe(a[1], "residual"), *gain = maybe(a[2], "gain");
  const float eps = real(a[3]);
  const bool e4m3 = a[7] == Py_True;
  const Lead l = lead(x, "x", {at::kFloat, at::kBFloat16});
  const On on(l.dev, a[6]);
  const int64_t T = l.n, H = l.width;
  if (gain) whole(*gain, "gain", l.dev, at::kFloat, {H});
  int64_t ldr = H, ldh = H, ldo;
  Tensor h;
  if (res) {
    ldr = rows(*res, "residual", l.dev, l.dtype, T, H);
    h = output(a[5], "out_h", l.dev, l.dtype, T, H, ldh);
  } else if (a[5] != Py_None) {
    bad("out_h: there is no sum without a residual");
  }
  const Tensor out = output(a[4], "out", l.dev, e4m3 ? at::kFloat8_e4m3fn : l.dtype, T, H, ldo);
  Tensor scale;
  if (e4m3) scale = empty({T}, at::kFloat, l.dev);
  call("add_rms_norm", on, [&](void* s) {
    return lib.add_rms_norm(code(l.dtype), ptr(x), l.ld, ptr(res), ldr, ptr<float>(gain), eps, count(T, "rows"), count(H, "width"),
                            res ? ptr(h) : nullptr, ldh, ptr(out), ldo, e4m3 ? ptr<float>(scale) : nullptr, s);
  });
  written(a[4]);
  written(a[5]);
  return tuple({wrap(out), e4m3 ? wrap(scale) : same(Py_None), !res ? same(a[0]) : a[5] != Py_None ? same(a[5]) : wrap(h)});
}

// grad, h, gain, eps, grad_h, out, stream -> (grad_x, grad_gain or None)
PyObject* add_rms_norm_backward(PyObject* const* a) {
  const Tensor &grad = tensor(a[0], "grad"), &h = tensor(a[1], "h");
  const Tensor *gain = maybe(a[2], "gain"), *gh = maybe(a[4], "grad_h");
  const float eps = real(a[3]);
  const Lead l = lead(h, "h", {at::kFloat, at::kBFloat16});
  const On on(l.dev, a[6]);
  const int64_t T = l.n, H = l.width;
  const int64_t ldg = rows(grad, "grad", l.dev, l.dtype, T, H), ldgh = gh ? rows(*gh, "grad_h", l.dev, l.dtype, T, H) : H;
  int64_t ldo, size = 0;
  const Tensor out = output(a[5], "out", l.dev, l.dtype, T, H, ldo);
  Tensor grad_gain, ws;
  if (gain) {
    whole(*gain, "gain", l.dev, at::kFloat, {H});
    grad_gain = empty({H}, at::kFloat, l.dev);
    size = lib.norm_workspace(count(T, "rows"), count(H, "width"));
    ws = empty({size}, at::kByte, l.dev);
  }
  call("add_rms_norm_backward", on, [&](void* s) {
    return lib.add_rms_norm_backward(code(l.dtype), ptr(grad), ldg, ptr(h), l.ld, ptr<float>(gain), eps, count(T, "rows"),
                                     count(H, "width"), ptr(gh), ldgh, ptr(out), ldo, gain ? ptr<float>(grad_gain) : nullptr,
                                     gain ? ptr(ws) : nullptr, size, s);
  });
  written(a[5]);
  return tuple({wrap(out), gain ? wrap(grad_gain) : same(Py_None)});
}

// x, weight, bias, act code, mul, residual, offsets, x_scale, w_scale, out dtype or None, out, stream
PyObject* linear(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
  const Tensor *bias = maybe(a[2], "bias"), *mul = maybe(a[4], "mul"), *res = maybe(a[5], "residual"),
               *offsets = maybe(a[6], "offsets"), *sx = maybe(a[7], "x_scale"), *sw = maybe(a[8], "w_scale"),
               *given = maybe(a[10], "out");
  const Lead l = lead(x, "x", {at::kBFloat16, at::kFloat8_e4m3fn});
  const On on(l.dev, a[11]);
  const bool e4m3 = l.dtype == at::kFloat8_e4m3fn;
  const int64_t T = l.n, F = l.width;
  moe_async_linear_args p = {};
  int64_t N, per[2];
  size_t dims = 1;
  if (!offsets) {
    if (weight.dim() != 2) bad("weight: expected [N, fan_in]", weight);
    per[0] = N = weight.size(0);
    p.w_stride = rows(weight, "weight", l.dev, l.dtype, N, F);
  } else {
    if (weight.dim() != 3 || weight.size(0) < 1) bad("weight: expected [G, N, fan_in] with offsets", weight);
    per[0] = weight.size(0);
    per[1] = N = weight.size(1);
    dims = 2;
    whole(weight, "weight", l.dev, l.dtype, {per[0], N, F});
    whole(*offsets, "offsets", l.dev, at::kInt, {per[0] + 1});
    p.w_stride = F;
    p.groups = count(per[0], "groups");
  }
  const at::IntArrayRef vec(per, dims);
  ScalarType od = at::kBFloat16;
  if (a[9] != Py_None) {
    if (!THPDtype_Check(a[9])) bad("out_dtype: expected a dtype");
    od = reinterpret_cast<THPDtype*>(a[9])->scalar_type;
  } else if (given) {
    od = given->scalar_type();
  }
  if (od != at::kFloat && od != at::kBFloat16) bad("out_dtype: expected float32 or bfloat16");
  if ((sx != nullptr) != e4m3 || (sw != nullptr) != e4m3) bad("x_scale, w_scale: both with e4m3 operands, none with bf16");
  const int64_t KB = (F + 127) / 128;
  const bool blocks = e4m3 && sx->dim() == 2;        // a scale per 128 columns of a token and per 128 x 128 of a weight
  if (blocks) {
    if (sx->scalar_type() != at::kFloat || !sx->is_cuda() || sx->get_device() != l.dev || sx->size(0) != T || sx->size(1) != KB)
      bad("x_scale: expected " + shape(T, KB) + " of float on cuda:" + std::to_string(l.dev), *sx);
    const int64_t sizes[3] = {offsets ? per[0] : (N + 127) / 128, offsets ? (N + 127) / 128 : KB, KB};
    whole(*sw, "w_scale", l.dev, at::kFloat, at::IntArrayRef(sizes, offsets ? 3 : 2));
  } else if (e4m3) {
    whole(*sx, "x_scale", l.dev, at::kFloat, {T});
    whole(*sw, "w_scale", l.dev, at::kFloat, vec);
  }
  if (bias) whole(*bias, "bias", l.dev, at::kFloat, vec);
  p.mul_stride = mul ? rows(*mul, "mul", l.dev, od, T, N) : N;
  p.residual_stride = res ? rows(*res, "residual", l.dev, od, T, N) : N;
  const Tensor out = output(a[10], "out", l.dev, od, T, N, p.y_stride);
  p.dtype = code(l.dtype);
  p.out_dtype = code(od);
  p.act = static_cast<int32_t>(integer(a[3], "act"));
  p.rows = count(T, "rows");
  p.fan_in = count(F, "fan_in");
  p.fan_out = count(N, "fan_out");
  p.x_stride = l.ld;
  p.d_x = ptr(x);
  p.d_w = ptr(weight);
  p.d_bias = ptr<float>(bias);
  p.d_x_scale = ptr<float>(sx);
  p.d_w_scale = ptr<float>(sw);
  p.d_mul = ptr(mul);
  p.d_residual = ptr(res);
  p.d_offsets = ptr<int32_t>(offsets);
  p.d_y = ptr(out);
  call("linear", on, [&](void* s) { return blocks ? lib.linear_blocks(&p, sx->stride(0), sx->stride(1), s) : lib.linear(&p, s); });
  written(a[10]);
  return given ? same(a[10]) : wrap(out);
}

// float32 or bfloat16 as asked for, as the output that was handed in has, or bfloat16
ScalarType result_dtype(PyObject* asked, const Tensor* given, const char* name) {
  ScalarType d = at::kBFloat16;
  if (asked != Py_None) {
    if (!THPDtype_Check(asked)) bad(std::string(name) + ": expected a dtype");
    d = reinterpret_cast<THPDtype*>(asked)->scalar_type;
  } else if (given) {
    d = given->scalar_type();
  }
  if (d != at::kFloat && d != at::kBFloat16) bad(std::string(name) + ": expected float32 or bfloat16");
  return d;
}

// grad, x, weight, offsets, bias, residual, out dtype, weight dtype, out_x, out_weight, out_bias, accumulate, stream
// -> (grad_x, grad_weight, grad_bias), None for what was not asked for
PyObject* linear_backward(PyObject* const* a) {
  const Tensor& grad = tensor(a[0], "grad");
  const Tensor *x = maybe(a[1], "x"), *weight = maybe(a[2], "weight"), *offsets = maybe(a[3], "offsets"), *res = maybe(a[5], "residual"),
               *given_x = maybe(a[8], "out_x"), *given_w = maybe(a[9], "out_weight"), *given_b = maybe(a[10], "out_bias");
  const int bias = PyObject_IsTrue(a[4]), add = PyObject_IsTrue(a[11]);
  if (bias < 0 || add < 0) throw PythonError{};
  const Lead l = lead(grad, "grad", {at::kBFloat16});
  const On on(l.dev, a[12]);
  const int64_t T = l.n, N = l.width;
  if (!x && !weight && !bias) bad("x, weight, bias: nothing to compute");
  if ((!weight && (given_x || res)) || (!x && given_w) || (!bias && given_b))
    bad("out_x and residual need weight, out_weight needs x, out_bias needs bias=True");
  if (add && ((x && !given_w) || (bias && !given_b))) bad("accumulate: needs out_weight and out_bias, as far as they are computed");
  moe_async_linear_backward_args p = {};
  int64_t G = 0, F = 8;
  if (offsets) {
    if (offsets->dim() != 1 || offsets->size(0) < 2) bad("offsets: expected [G + 1]", *offsets);
    G = offsets->size(0) - 1;
    whole(*offsets, "offsets", l.dev, at::kInt, {G + 1});
  }
  if (x) {
    if (x->dim() != 2) bad("x: expected [T, fan_in]", *x);
    F = x->size(1);
    p.x_stride = rows(*x, "x", l.dev, at::kBFloat16, T, F);
  } else if (weight) {
    F = weight->dim() > 0 ? weight->size(-1) : 0;
  }
  p.x_dtype = p.w_dtype = MOE_BF16;
  Tensor out_x, out_w, out_b;
  if (weight) {
    if (offsets) {
      whole(*weight, "weight", l.dev, at::kBFloat16, {G, N, F});
      p.w_stride = F;
    } else {
      p.w_stride = rows(*weight, "weight", l.dev, at::kBFloat16, N, F);
    }
    const ScalarType d = result_dtype(a[6], given_x, "out_dtype");
    p.x_dtype = code(d);
    p.residual_stride = res ? rows(*res, "residual", l.dev, d, T, F) : F;
    out_x = output(a[8], "out_x", l.dev, d, T, F, p.grad_x_stride);
  }
  if (x) {
    const ScalarType d = result_dtype(a[7], given_w, "weight_dtype");
    p.w_dtype = code(d);
    if (!offsets) {
      out_w = output(a[9], "out_weight", l.dev, d, N, F, p.grad_w_stride);
    } else {
      if (given_w) whole(*given_w, "out_weight", l.dev, d, {G, N, F});
      out_w = given_w ? *given_w : empty({G, N, F}, d, l.dev);
      p.grad_w_stride = F;
    }
  }
  if (bias) {
    const int64_t per[2] = {offsets ? G : N, N};
    const at::IntArrayRef vec(per, offsets ? 2 : 1);
    if (given_b) whole(*given_b, "out_bias", l.dev, at::kFloat, vec);
    out_b = given_b ? *given_b : empty(vec, at::kFloat, l.dev);
  }
  p.rows = count(T, "rows");
  p.fan_in = count(F, "fan_in");
  p.fan_out = count(N, "fan_out");
  p.groups = count(G, "groups");
  p.accumulate = add;
  p.grad_stride = l.ld;
  p.d_grad = ptr(grad);
  p.d_x = ptr(x);
  p.d_w = ptr(weight);
  p.d_residual = ptr(res);
  p.d_offsets = ptr<int32_t>(offsets);
  p.d_grad_x = weight ? ptr(out_x) : nullptr;
  p.d_grad_w = x ? ptr(out_w) : nullptr;
  p.d_grad_bias = bias ? ptr<float>(out_b) : nullptr;
  Tensor ws;
  p.workspace_bytes = lib.linear_backward_workspace(&p);
  if (p.workspace_bytes > 0) {
    ws = empty({p.workspace_bytes}, at::kByte, l.dev);
    p.d_workspace = ptr(ws);
  }
  call("linear_backward", on, [&](void* s) { return lib.linear_backward(&p, s); });
  for (int i = 8; i < 11; ++i) written(a[i]);
  const auto result = [&](PyObject* given, const Tensor& t, bool some) { return !some ? same(Py_None) : given != Py_None ? same(given) : wrap(t); };
  return tuple({result(a[8], out_x, weight != nullptr), result(a[9], out_w, x != nullptr), result(a[10], out_b, bias != 0)});
}

// grad, z, mul, act code, out_z, out_mul, stream -> (grad_z, grad_mul or None)
PyObject* act_mul_backward(PyObject* const* a) {
  const Tensor &grad = tensor(a[0], "grad"), &z = tensor(a[1], "z");
  const Tensor* mul = maybe(a[2], "mul");
  const Lead l = lead(z, "z", {at::kFloat, at::kBFloat16});
  const On on(l.dev, a[6]);
  const int64_t T = l.n, H = l.width;
  const int32_t act = static_cast<int32_t>(integer(a[3], "act"));
  const int64_t ldg = rows(grad, "grad", l.dev, l.dtype, T, H), ldm = mul ? rows(*mul, "mul", l.dev, l.dtype, T, H) : H;
  if (!mul && a[5] != Py_None) bad("out_mul: there is no gradient of mul without mul");
  int64_t ldz, ldgm = H;
  const Tensor out_z = output(a[4], "out_z", l.dev, l.dtype, T, H, ldz);
  Tensor out_mul;
  if (mul) out_mul = output(a[5], "out_mul", l.dev, l.dtype, T, H, ldgm);
  call("act_mul_backward", on, [&](void* s) {
    return lib.act_mul_backward(code(l.dtype), act, ptr(grad), ldg, ptr(z), l.ld, ptr(mul), ldm, count(T, "rows"), count(H, "width"), ptr(out_z), ldz,
                                mul ? ptr(out_mul) : nullptr, ldgm, s);
  });
  written(a[4]);
  written(a[5]);
  return tuple({a[4] != Py_None ? same(a[4]) : wrap(out_z), !mul ? same(Py_None) : a[5] != Py_None ? same(a[5]) : wrap(out_mul)});
}

// x, out, stream -> (q, scale): a scale per 128 columns of a row
PyObject* quantize_blocks(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const Lead l = lead(x, "x", {at::kFloat, at::kBFloat16});
  const On on(l.dev, a[2]);
  const int64_t T = l.n, F = l.width, KB = (F + 127) / 128;
  int64_t ldo;
  const Tensor q = output(a[1], "out", l.dev, at::kFloat8_e4m3fn, T, F, ldo);
  const Tensor scale = empty({KB, T}, at::kFloat, l.dev);
  const int64_t sizes[2] = {T, KB}, strides[2] = {1, T};                 // tokens adjacent: the product reads a block's together
  scale.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(sizes, 2), at::IntArrayRef(strides, 2));
  call("quantize_blocks", on, [&](void* s) {
    return lib.quantize_blocks(code(l.dtype), ptr(x), l.ld, 1, count(T, "rows"), count(F, "width"), 1, ptr(q), ldo, ptr<float>(scale), 1, T, s);
  });
  written(a[1]);
  return tuple({a[1] != Py_None ? same(a[1]) : wrap(q), wrap(scale)});
}

// w, out, stream -> (q, scale): a scale per 128 x 128 of a matrix, or of each of several
PyObject* quantize_weight_blocks(PyObject* const* a) {
  const Tensor& w = tensor(a[0], "w");
  if (w.dim() != 2 && w.dim() != 3) bad("w: expected [N, F] or [G, N, F]", w);
  if ((w.scalar_type() != at::kFloat && w.scalar_type() != at::kBFloat16) || !w.is_cuda()) bad("w: expected CUDA matrices of Float BFloat16", w);
  const int dev = w.get_device();
  const On on(dev, a[2]);
  const bool many = w.dim() == 3;
  const int64_t G = many ? w.size(0) : 1, N = w.size(-2), F = w.size(-1), NB = (N + 127) / 128, KB = (F + 127) / 128;
  int64_t ldw = F, ldo = F;
  if (many)
    whole(w, "w", dev, w.scalar_type(), {G, N, F});
  else
    ldw = rows(w, "w", dev, w.scalar_type(), N, F);
  Tensor q;
  if (!many) {
    q = output(a[1], "out", dev, at::kFloat8_e4m3fn, N, F, ldo);
  } else if (a[1] == Py_None) {
    q = empty({G, N, F}, at::kFloat8_e4m3fn, dev);
  } else {
    q = tensor(a[1], "out");
    whole(q, "out", dev, at::kFloat8_e4m3fn, {G, N, F});
  }
  const int64_t sizes[3] = {many ? G : NB, many ? NB : KB, KB};
  const Tensor scale = empty(at::IntArrayRef(sizes, many ? 3 : 2), at::kFloat, dev);
  if (G > 0 && N > 0)
    call("quantize_weight_blocks", on, [&](void* s) {
      return lib.quantize_blocks(code(w.scalar_type()), ptr(w), ldw, count(G, "groups"), count(N, "rows"), count(F, "width"), 128, ptr(q), ldo, ptr<float>(scale),
                                 KB, 1, s);
    });
  written(a[1]);
  return tuple({a[1] != Py_None ? same(a[1]) : wrap(q), wrap(scale)});
}

// ------------------------------------------------------------------ module

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N || !error_class) {
    PyErr_SetString(PyExc_TypeError, "call the functions of ops.py");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(error_class, "is", r.status, r.what.c_str());
    if (e) {
      PyErr_SetObject(error_class, e);
      Py_DECREF(e);
    }
  } catch (const PythonError&) {
  } catch (const std::exception& e) {                // an allocation that failed, say
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(MoEError, address of moe_async_sort_experts, ...): in the order of Library
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 1 + static_cast<Py_ssize_t>(sizeof(lib) / sizeof(void*))) {
    PyErr_SetString(PyExc_TypeError, "bind: the error class and one address per operator");
    return nullptr;
  }
  void** slot = reinterpret_cast<void**>(&lib);
  for (Py_ssize_t i = 1; i < n; ++i) {
    slot[i - 1] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(args[0]);
  Py_XDECREF(error_class);
  error_class = args[0];
  Py_RETURN_NONE;
}

#define OP(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
                         OP(sort_experts, 3),
                         OP(sort_rows, 4),
                         OP(merge_rows, 6),
                         OP(merge_rows_backward, 6),
                         OP(route_backward, 5),
                         OP(add_rms_norm, 8),
                         OP(add_rms_norm_backward, 7),
                         OP(linear, 12),
                         OP(linear_backward, 13),
                         OP(act_mul_backward, 7),
                         OP(quantize_blocks, 3),
                         OP(quantize_weight_blocks, 3),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", MOE_BINDING_TAG) < 0) Py_CLEAR(m);
  return m;
}
