// The Python binding of the entries that run between a block's linears, as a
// CPython extension over PyTorch's tensors: it checks and marshals what
// __init__.py's ctypes binding does for the other entries, in a third of the
// time (a call of qk_norm_rope took 15 us of interpreter and ctypes around a
// kernel of 4).  It holds no state but the library's entry points, handed over by
// bind(), and does no arithmetic.
//
// Every function takes its arguments by position, None for an absent one, and
// raises TypeError or ValueError for tensors the library cannot take and
// W4A4Error for a status it returns.  Kernels go to the current stream of the
// tensors' own device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <optional>
#include <stdexcept>
#include <string>

#include "w4a4.h"

namespace {

decltype(&w4a4_linear_w4a16) linear_fn = nullptr;
decltype(&w4a4_qk_norm_rope) rope_fn = nullptr;
decltype(&w4a4_attention) attention_fn = nullptr;
decltype(&w4a4_attention_workspace_bytes) attention_bytes_fn = nullptr;
PyObject* error_type = nullptr;      // W4A4Error(status, what)

// A Python exception is set: leave through the entry point.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
  return t;
}

// W4A4_BF16 or W4A4_FP16.
int type_code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return W4A4_BF16;
  if (t.scalar_type() == at::kHalf) return W4A4_FP16;
  raise(PyExc_TypeError, std::string(name) + " must be torch.bfloat16 or torch.float16, got " + toString(t.scalar_type()));
}

void need(const at::Tensor& t, at::ScalarType type, const at::Device& device, const char* name) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor of " + toString(type) + ", got " + toString(t.scalar_type()));
  if (t.device() != device)
    raise(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
}

// A contiguous operand of the given type and shape; its address (null for None).
void* operand(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const at::Device& device, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  need(t, type, device, name);
  if (t.sizes() != shape || !t.is_contiguous())
    raise(PyExc_ValueError, std::string(name) + " must be contiguous with shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  return t.data_ptr();
}

// A [tokens, heads, D] tensor with contiguous D; a dimension of one or no
// element has no stride of its own.
struct Heads {
  void* at = nullptr;
  int64_t token = 0, head = 0;
  Heads() = default;
  Heads(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const at::Device& device, const char* name) {
    need(t, type, device, name);
    if (t.sizes() != shape)
      raise(PyExc_ValueError, std::string(name) + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (t.numel() != 0 && shape[2] > 1 && t.stride(2) != 1)
      raise(PyExc_ValueError, std::string(name) + " must have a contiguous last dimension");
    at = t.data_ptr();
    head = shape[1] > 1 && t.numel() != 0 ? t.stride(1) : shape[2];
    token = shape[0] > 1 && t.numel() != 0 ? t.stride(0) : shape[1] * shape[2];
  }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& device) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

// The tensors' device made current for the launch, and its current stream.
struct Launch {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit Launch(const at::Device& device) {
    if (device.index() != c10::cuda::current_device()) guard.set_device(device);
    stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  }
};

void check(int status, const char* what) {
  if (status == W4A4_OK) return;
  PyObject* e = PyObject_CallFunction(error_type, "is", status, what);
  if (e != nullptr) {
    PyErr_SetObject(error_type, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

void count(Py_ssize_t n, Py_ssize_t want, const char* what) {
  if (n != want) raise(PyExc_TypeError, std::string(what) + " takes " + std::to_string(want) + " arguments");
}

// linear_w4a16(x, Wq, scale, offset, bias, out)
PyObject* linear_w4a16(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count(n, 6, "linear_w4a16");
    const at::Tensor& x = tensor(a[0], "x");
    const int code = type_code(x, "x");
    const at::ScalarType type = x.scalar_type();
    const at::Device device = x.device();
    if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
      raise(PyExc_ValueError, "x must be a 2-D tensor with a contiguous inner dimension");
    const int64_t M = x.size(0), K = x.size(1);
    const at::Tensor& Wq = tensor(a[1], "Wq");
    if (Wq.dim() != 2) raise(PyExc_ValueError, "Wq must be a contiguous [N, K/2] int8 tensor on x's device");
    const int64_t N = Wq.size(0);
    void* w = operand(a[1], at::kChar, {N, K / 2}, device, "Wq");
    const at::Tensor& scale = tensor(a[2], "scale");
    if (scale.dim() != 2 || scale.size(1) < 1 || K % scale.size(1) != 0)
      raise(PyExc_ValueError, "scale must be a [N, K/group] tensor");
    const int64_t groups = scale.size(1);
    void* s = operand(a[2], type, {N, groups}, device, "scale");
    void* o = operand(a[3], type, {N, groups}, device, "offset");
    void* b = operand(a[4], type, {N}, device, "bias");
    at::Tensor y;
    if (a[5] == Py_None) {
      y = empty({M, N}, type, device);
    } else {
      y = tensor(a[5], "out");
      need(y, type, device, "out");
      if (y.dim() != 2 || y.size(0) != M || y.size(1) != N || (N > 1 && y.stride(1) != 1))
        raise(PyExc_ValueError, "out must be a [" + std::to_string(M) + ", " + std::to_string(N) +
                                    "] tensor with a contiguous inner dimension");
    }
    const Launch launch(device);
    check(linear_fn(x.data_ptr(), M > 1 ? x.stride(0) : K, static_cast<const int8_t*>(w), s, o,
                    static_cast<int>(K / groups), b, y.data_ptr(), M > 1 ? y.stride(0) : N, M, N, K, code,
                    launch.stream),
          "w4a4_linear_w4a16");
    return THPVariable_Wrap(std::move(y));
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// qk_norm_rope(q, k, q_weight, k_weight, positions, freq, axis, interleaved, eps, q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count(n, 11, "qk_norm_rope");
    const at::Tensor& q = tensor(a[0], "q");
    const int code = type_code(q, "q");
    const at::ScalarType type = q.scalar_type();
    const at::Device device = q.device();
    if (q.dim() != 3) raise(PyExc_ValueError, "q must be [T, Hq, D]");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    const Heads qi(q, q.sizes(), type, device, "q");
    at::Tensor q_out = a[9] == Py_None ? empty({T, Hq, D}, type, device) : tensor(a[9], "q_out");
    const Heads qo(q_out, q.sizes(), type, device, "q_out");
    int64_t Hk = 0;
    Heads ki, ko;
    at::Tensor k_out;
    if (a[1] != Py_None) {
      const at::Tensor& k = tensor(a[1], "k");
      if (k.dim() != 3 || k.size(0) != T || k.size(2) != D)
        raise(PyExc_ValueError, "k must be [" + std::to_string(T) + ", Hk, " + std::to_string(D) + "], got " + shape_text(k.sizes()));
      Hk = k.size(1);
      ki = Heads(k, k.sizes(), type, device, "k");
      k_out = a[10] == Py_None ? empty({T, Hk, D}, type, device) : tensor(a[10], "k_out");
      ko = Heads(k_out, k.sizes(), type, device, "k_out");
    } else if (a[3] != Py_None || a[10] != Py_None) {
      raise(PyExc_ValueError, "k_weight and k_out need k");
    }
    void* qw = operand(a[2], type, {D}, device, "q_weight");
    void* kw = operand(a[3], type, {D}, device, "k_weight");
    void *positions = nullptr, *freq = nullptr, *axis = nullptr;
    int bits = 0;
    int64_t row = 0, axes = 0, half = 0;
    if (a[4] != Py_None) {
      const at::Tensor& p = tensor(a[4], "positions");
      bits = p.scalar_type() == at::kInt ? 32 : p.scalar_type() == at::kLong ? 64 : 0;
      if (bits == 0)
        raise(PyExc_TypeError, std::string("positions must be torch.int32 or torch.int64, got ") + toString(p.scalar_type()));
      need(p, p.scalar_type(), device, "positions");
      if ((p.dim() != 1 && p.dim() != 2) || p.size(0) != T)
        raise(PyExc_ValueError, "positions must be [" + std::to_string(T) + ", axes] or [" + std::to_string(T) + "], got " + shape_text(p.sizes()));
      axes = p.dim() == 2 ? p.size(1) : 1;
      if (axes > 1 && p.stride(1) != 1) raise(PyExc_ValueError, "positions must have a contiguous inner dimension");
      if (axes > 0x7FFFFFFF) raise(PyExc_ValueError, "positions has too many axes");
      row = T > 1 ? p.stride(0) : axes;
      positions = p.data_ptr();
      if (a[5] == Py_None || a[6] == Py_None) raise(PyExc_ValueError, "positions need freq and axis (rotary_frequencies)");
      half = tensor(a[5], "freq").numel();
      freq = operand(a[5], at::kDouble, {half}, device, "freq");
      axis = operand(a[6], at::kInt, {half}, device, "axis");
    }
    const bool interleaved = truth(a[7]);
    const float eps = static_cast<float>(number(a[8]));
    const Launch launch(device);
    check(rope_fn(qi.at, qi.token, qi.head, Hq, ki.at, ki.token, ki.head, Hk, qw, kw, eps, positions, bits, row,
                  static_cast<int>(axes), static_cast<const double*>(freq), static_cast<const int32_t*>(axis), 2 * half,
                  interleaved ? 1 : 0, qo.at, qo.token, qo.head, ko.at, ko.token, ko.head, T, D, code, launch.stream),
          "w4a4_qk_norm_rope");
    PyObject* first = THPVariable_Wrap(std::move(q_out));
    if (first == nullptr) return nullptr;
    PyObject* second = k_out.defined() ? THPVariable_Wrap(std::move(k_out)) : Py_NewRef(Py_None);
    if (second == nullptr) {
      Py_DECREF(first);
      return nullptr;
    }
    PyObject* both = PyTuple_New(2);
    if (both == nullptr) {
      Py_DECREF(first);
      Py_DECREF(second);
      return nullptr;
    }
    PyTuple_SET_ITEM(both, 0, first);
    PyTuple_SET_ITEM(both, 1, second);
    return both;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// attention(q, k, v, cu_seqlens_q, cu_seqlens_k, causal, scale, out, return_lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count(n, 9, "attention");
    const at::Tensor& q = tensor(a[0], "q");
    const int code = type_code(q, "q");
    const at::ScalarType type = q.scalar_type();
    const at::Device device = q.device();
    const at::Tensor& k = tensor(a[1], "k");
    const at::Tensor& v = tensor(a[2], "v");
    if (q.dim() != 3 || k.dim() != 3) raise(PyExc_ValueError, "q must be [Tq, Hq, D] and k, v [Tk, Hk, D]");
    const int64_t Tq = q.size(0), Hq = q.size(1), D = q.size(2), Tk = k.size(0), Hk = k.size(1);
    if (k.size(2) != D) raise(PyExc_ValueError, "q and k must have the same last dimension");
    const Heads qi(q, q.sizes(), type, device, "q"), ki(k, k.sizes(), type, device, "k"), vi(v, k.sizes(), type, device, "v");
    at::Tensor out = a[7] == Py_None ? empty({Tq, Hq, D}, type, device) : tensor(a[7], "out");
    const Heads oi(out, q.sizes(), type, device, "out");
    int64_t B = 1;
    void *cq = nullptr, *ck = nullptr;
    if (a[3] != Py_None || a[4] != Py_None) {
      if (a[3] == Py_None || a[4] == Py_None) raise(PyExc_ValueError, "cu_seqlens_q and cu_seqlens_k go together");
      B = tensor(a[3], "cu_seqlens_q").numel() - 1;
      if (B < 1) raise(PyExc_ValueError, "cu_seqlens_q must hold at least two numbers");
      cq = operand(a[3], at::kInt, {B + 1}, device, "cu_seqlens_q");
      ck = operand(a[4], at::kInt, {B + 1}, device, "cu_seqlens_k");
    }
    const float scale = static_cast<float>(a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : number(a[6]));
    const bool causal = truth(a[5]);
    at::Tensor lse;
    if (truth(a[8])) lse = empty({Tq, Hq}, at::kFloat, device);
    // the workspace is this call's own and lives in PyTorch's allocator (or a
    // graph's pool) until the stream is past it, so overlapping calls and
    // captured graphs never share one
    const size_t bytes = attention_bytes_fn(Tq, Tk, B, Hq, Hk, D);
    at::Tensor ws;
    if (bytes != 0) ws = empty({static_cast<int64_t>(bytes)}, at::kByte, device);
    const Launch launch(device);
    check(attention_fn(qi.at, qi.token, qi.head, ki.at, ki.token, ki.head, vi.at, vi.token, vi.head, oi.at, oi.token,
                       oi.head, lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                       static_cast<const int32_t*>(cq), static_cast<const int32_t*>(ck), B, Tq, Tk, Hq, Hk, D,
                       causal ? 1 : 0, scale, code, bytes != 0 ? ws.data_ptr() : nullptr, bytes, launch.stream),
          "w4a4_attention");
    PyObject* first = THPVariable_Wrap(std::move(out));
    if (first == nullptr || !lse.defined()) return first;
    PyObject* second = THPVariable_Wrap(std::move(lse));
    PyObject* both = second != nullptr ? PyTuple_New(2) : nullptr;
    if (both == nullptr) {
      Py_DECREF(first);
      Py_XDECREF(second);
      return nullptr;
    }
    PyTuple_SET_ITEM(both, 0, first);
    PyTuple_SET_ITEM(both, 1, second);
    return both;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(error_type, linear_w4a16, qk_norm_rope, attention, attention_workspace_bytes): the
// library's entry points as addresses.
PyObject* bind(PyObject*, PyObject* args) {
  PyObject* type = nullptr;
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "OKKKK", &type, &f[0], &f[1], &f[2], &f[3])) return nullptr;
  Py_INCREF(type);
  Py_XSETREF(error_type, type);
  linear_fn = reinterpret_cast<decltype(linear_fn)>(f[0]);
  rope_fn = reinterpret_cast<decltype(rope_fn)>(f[1]);
  attention_fn = reinterpret_cast<decltype(attention_fn)>(f[2]);
  attention_bytes_fn = reinterpret_cast<decltype(attention_bytes_fn)>(f[3]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"linear_w4a16", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_w4a16)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk_norm_rope)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

// The documentation names what the extension was compiled for (BUILT_FOR comes
// from build.py, which looks for it in the file before it loads or keeps it).
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", BUILT_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
