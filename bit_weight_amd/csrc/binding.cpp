// Argument marshalling of the feed-forward and attention operators: checks torch tensors,
// allocates outputs and scratch memory and calls the library's C ABI on the
// current stream of the tokens' device.  It holds no arithmetic.  (A CPython
// module and not ctypes because a decode step's kernel takes 5 to 10 us: the
// same checks and calls written in Python take 11 us a call on the host.)
//
// setup() gives it the library's entry points as addresses, the zeroed split-K
// workspaces by (device index, stream), a callable (device index, bytes) ->
// workspace for when there is none that serves, the activations' codes by
// name, and a callable (status, name) that raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstring>
#include <memory>
#include <string>

#include "../../include/sherry.h"

namespace {

PyObject* g_workspaces = nullptr;     // dict
PyObject* g_workspace = nullptr;
PyObject* g_activations = nullptr;    // dict
PyObject* g_error = nullptr;

decltype(&sherry_packed_bytes) f_packed_bytes;
decltype(&sherry_gemm_fused) f_gemm_fused;
decltype(&sherry_gemm_fused_workspace_bytes) f_gemm_fused_workspace_bytes;
decltype(&sherry_gemm_fused_backward) f_gemm_fused_backward;
decltype(&sherry_gemm_fused_backward_scratch_bytes) f_gemm_fused_backward_scratch_bytes;
decltype(&sherry_glu) f_glu;
decltype(&sherry_glu_workspace_bytes) f_glu_workspace_bytes;
decltype(&sherry_glu_backward) f_glu_backward;
decltype(&sherry_glu_backward_scratch_bytes) f_glu_backward_scratch_bytes;
decltype(&sherry_layernorm) f_layernorm;
decltype(&sherry_layernorm_quantize) f_layernorm_quantize;
decltype(&sherry_layernorm_backward) f_layernorm_backward;
decltype(&sherry_layernorm_backward_scratch_bytes) f_layernorm_backward_scratch_bytes;
decltype(&sherry_qk_norm_rope) f_qk_norm_rope;
decltype(&sherry_qk_norm_rope_backward) f_qk_norm_rope_backward;
decltype(&sherry_qk_norm_rope_backward_scratch_bytes) f_qk_norm_rope_backward_scratch_bytes;
decltype(&sherry_cache_write) f_cache_write;
decltype(&sherry_cache_read) f_cache_read;
decltype(&sherry_cache_attention) f_cache_attention;
decltype(&sherry_cache_attention_workspace_bytes) f_cache_attention_workspace_bytes;
decltype(&sherry_cache_attention_scratch_bytes) f_cache_attention_scratch_bytes;

struct Entry {
  const char* name;
  void* at;
};
const Entry kEntries[] = {
    {"sherry_packed_bytes", &f_packed_bytes},
    {"sherry_gemm_fused", &f_gemm_fused},
    {"sherry_gemm_fused_workspace_bytes", &f_gemm_fused_workspace_bytes},
    {"sherry_gemm_fused_backward", &f_gemm_fused_backward},
    {"sherry_gemm_fused_backward_scratch_bytes", &f_gemm_fused_backward_scratch_bytes},
    {"sherry_glu", &f_glu},
    {"sherry_glu_workspace_bytes", &f_glu_workspace_bytes},
    {"sherry_glu_backward", &f_glu_backward},
    {"sherry_glu_backward_scratch_bytes", &f_glu_backward_scratch_bytes},
    {"sherry_layernorm", &f_layernorm},
    {"sherry_layernorm_quantize", &f_layernorm_quantize},
    {"sherry_layernorm_backward", &f_layernorm_backward},
    {"sherry_layernorm_backward_scratch_bytes", &f_layernorm_backward_scratch_bytes},
    {"sherry_qk_norm_rope", &f_qk_norm_rope},
    {"sherry_qk_norm_rope_backward", &f_qk_norm_rope_backward},
    {"sherry_qk_norm_rope_backward_scratch_bytes", &f_qk_norm_rope_backward_scratch_bytes},
    {"sherry_cache_write", &f_cache_write},
    {"sherry_cache_read", &f_cache_read},
    {"sherry_cache_attention", &f_cache_attention},
    {"sherry_cache_attention_workspace_bytes", &f_cache_attention_workspace_bytes},
    {"sherry_cache_attention_scratch_bytes", &f_cache_attention_scratch_bytes},
};

// A Python error is set; unwinds to the method's entry.
struct Raised {};

[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised{};
}

const char* type_name(at::ScalarType t) { return c10::toString(t); }

const at::Tensor& tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// A contiguous tensor of type t on a GPU; index >= 0: on that one.
void check_tensor(const at::Tensor& t, const char* name, at::ScalarType type, int index) {
  if (t.layout() != at::kStrided) fail(PyExc_RuntimeError, "%s must be a dense tensor", name);
  if (!t.is_cuda()) fail(PyExc_RuntimeError, "%s must be on a GPU device, got %s", name, t.device().str().c_str());
  if (t.scalar_type() != type)
    fail(PyExc_RuntimeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
  if (!t.is_contiguous()) fail(PyExc_RuntimeError, "%s must be contiguous", name);
  if (index >= 0 && t.get_device() != index)
    fail(PyExc_RuntimeError, "%s must be on cuda:%d, got %s", name, index, t.device().str().c_str());
}

// Pointer of an operand of n values (None: nullptr where it may be missing).
void* vector_of(PyObject* o, const char* name, at::ScalarType type, int index, int64_t n, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = tensor_of(o, name);
  check_tensor(t, name, type, index);
  if (t.numel() != n)
    fail(PyExc_RuntimeError, "%s must hold %lld values, got %lld", name, (long long)n, (long long)t.numel());
  return t.data_ptr();
}

void* matrix_of(const at::Tensor& t, const char* name, at::ScalarType type, int index, int64_t M, int64_t N) {
  check_tensor(t, name, type, index);
  if (t.dim() != 2 || t.size(0) != M || t.size(1) != N)
    fail(PyExc_RuntimeError, "%s must be [%lld,%lld]", name, (long long)M, (long long)N);
  return t.data_ptr();
}

void* matrix_of(PyObject* o, const char* name, at::ScalarType type, int index, int64_t M, int64_t N,
                bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  return matrix_of(tensor_of(o, name), name, type, index, M, N);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

int dtype_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return SHERRY_F32;
    case at::kHalf: return SHERRY_F16;
    case at::kBFloat16: return SHERRY_BF16;
    default: fail(PyExc_RuntimeError, "type must be float32, float16 or bfloat16, got %s", type_name(t));
  }
}

at::ScalarType scalar_of(PyObject* dtype) {
  if (!THPDtype_Check(dtype)) fail(PyExc_TypeError, "dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(dtype)->scalar_type;
}

int activation_of(PyObject* name) {
  PyObject* code = PyDict_GetItemWithError(g_activations, name);
  if (!code) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "act must be one of %R, got %R", g_activations, name);
    throw Raised{};
  }
  return (int)integer(code);
}

// The tokens x [M,K] (int8) and what follows from them.
struct Tokens {
  int64_t M, N, K;
  int index;
  at::Device device;
  const int8_t* x;
  const float* s_x;
  Tokens(PyObject* px, PyObject* ps, PyObject* pn, PyObject* pk) : device(at::kCPU) {
    const at::Tensor& t = tensor_of(px, "x");
    N = integer(pn);
    K = integer(pk);
    check_tensor(t, "x", at::kChar, -1);
    if (t.dim() != 2 || t.size(1) != K) fail(PyExc_RuntimeError, "x must be [M,%lld]", (long long)K);
    M = t.size(0);
    index = (int)t.get_device();
    device = t.device();
    x = static_cast<const int8_t*>(t.data_ptr());
    s_x = static_cast<const float*>(vector_of(ps, "s_x", at::kFloat, index, M));
  }
};

struct Weights {
  const void* packed;
  const float* alpha;
  Weights(PyObject* pp, PyObject* pa, const char* packed_name, const char* alpha_name, const Tokens& t) {
    const size_t bytes = f_packed_bytes(t.N, t.K);
    if (bytes == 0) {
      Py_XDECREF(PyObject_CallFunction(g_error, "is", SHERRY_ERR_SHAPE, "weights [N,K]"));
      throw Raised{};
    }
    packed = vector_of(pp, packed_name, at::kByte, t.index, (int64_t)bytes);
    alpha = static_cast<const float*>(vector_of(pa, alpha_name, at::kFloat, t.index, t.N));
  }
};

// (the allocation itself: at::empty's dispatch takes 0.3 us more, and a small
// operator's host time is about its kernel's)
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, at::Device device) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, device, std::nullopt));
}

// The output: the caller's, or a new one.
at::Tensor output_of(PyObject* o, int64_t M, int64_t N, at::ScalarType type, int index, at::Device device) {
  if (o == Py_None) return empty({M, N}, type, device);
  const at::Tensor& t = tensor_of(o, "out");
  matrix_of(t, "out", type, index, M, N);
  return t;
}

// Runs `call(stream)` with the device current and reports its status.
template <typename F>
void launch(const char* name, int index, F call) {
  const c10::OptionalDeviceGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)index));
  const int status = call(static_cast<void*>(c10::hip::getCurrentHIPStream((c10::DeviceIndex)index).stream()));
  if (status != SHERRY_OK) {
    Py_XDECREF(PyObject_CallFunction(g_error, "is", status, name));
    throw Raised{};
  }
}

// The zeroed workspace: the caller's tensor, none needed, or the module's.
struct Workspace {
  void* at = nullptr;
  size_t bytes = 0;
  at::Tensor keep;
  template <typename Operand>
  Workspace(PyObject* o, size_t need, const Operand& t) {
    if (o != Py_None) {
      keep = tensor_of(o, "workspace");
      check_tensor(keep, "workspace", at::kByte, t.index);
    } else if (need > 0) {
      const c10::OptionalDeviceGuard guard(t.device);
      if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) {
        const auto stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)t.index).stream();
        PyObject* key = Py_BuildValue("(iK)", t.index, (unsigned long long)reinterpret_cast<uintptr_t>(stream));
        if (!key) throw Raised{};
        PyObject* w = PyDict_GetItemWithError(g_workspaces, key);
        Py_DECREF(key);
        if (!w && PyErr_Occurred()) throw Raised{};
        if (w) keep = tensor_of(w, "workspace");
      }
      if (!keep.defined() || (size_t)keep.numel() < need) {
        PyObject* w = PyObject_CallFunction(g_workspace, "in", t.index, (Py_ssize_t)need);
        if (!w) throw Raised{};
        keep = tensor_of(w, "workspace");
        Py_DECREF(w);
      }
    } else {
      return;
    }
    at = keep.data_ptr();
    bytes = (size_t)keep.numel();
  }
};

// Forward mode: the operators have no such derivatives.  A tensor that carries a tangent
// is refused, as torch's functions without one do, unless forward mode is off (as in the
// forward of a torch.autograd.Function with a jvp of its own); it does not go by the grad
// mode.
void refuse_tangent(const char* name, const at::Tensor& t) {
  if (t._fw_grad(/*level=*/0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
    fail(PyExc_NotImplementedError, "bit_weight_amd.%s has no forward-mode derivative, but a tensor carries a tangent", name);
}

// Autograd: the operators have backward passes of their own and no grad_fn.
// Where one of the tensors requires a gradient the outputs are made to say
// so, and a backward pass through them fails by the operator's name instead
// of leaving that gradient out.  A caller's output cannot carry this: refused,
// as torch's functions do.
class Gradients {
 public:
  Gradients(const char* name, std::initializer_list<PyObject*> inputs, PyObject* out = Py_None) : name_(name) {
    for (PyObject* o : inputs)
      if (o != Py_None) refuse_tangent(name, THPVariable_Unpack(o));
    if (out != Py_None) refuse_tangent(name, THPVariable_Unpack(out));
    if (!c10::GradMode::is_enabled()) return;
    for (PyObject* o : inputs)
      if (o != Py_None && THPVariable_Unpack(o).requires_grad())
        edges_.push_back(torch::autograd::impl::gradient_edge(THPVariable_Unpack(o)));
    if (out != Py_None && (!edges_.empty() || THPVariable_Unpack(out).requires_grad()))
      fail(PyExc_RuntimeError, "%s with out= cannot carry gradients, but a tensor requires one: call it in torch.no_grad()",
           name);
  }
  void mark(std::initializer_list<at::Tensor> outputs) {
    if (edges_.empty()) return;
    const std::shared_ptr<torch::autograd::Node> node(
        new torch::autograd::NotImplemented(
            std::string("bit_weight_amd.") + name_ + " (put it and its backward pass into a torch.autograd.Function)",
            std::move(edges_)),
        torch::autograd::deleteNode);
    for (const at::Tensor& t : outputs)
      if (t.defined() && at::isFloatingType(t.scalar_type())) torch::autograd::set_history(t, node);
  }

 private:
  const char* name_;
  torch::autograd::edge_list edges_;
};

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// Every method: a fixed count of arguments, C++ errors (an allocation's) turned
// into torch's Python ones.
template <int kCount, PyObject* (*kBody)(PyObject* const*)>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kCount) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kCount, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return kBody(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// x, s_x, packed, alpha, N, K, bias, act, residual, dtype, out, workspace
PyObject* gemm_fused(PyObject* const* a) {
  const Tokens t(a[0], a[1], a[4], a[5]);
  const Weights w(a[2], a[3], "packed", "alpha", t);
  const int act = activation_of(a[7]);
  const at::ScalarType type = scalar_of(a[9]);
  const int dtype = dtype_of(type);
  const auto* bias = static_cast<const float*>(vector_of(a[6], "bias", at::kFloat, t.index, t.N, true));
  const void* residual = matrix_of(a[8], "residual", type, t.index, t.M, t.N, true);
  const at::Tensor y = output_of(a[10], t.M, t.N, type, t.index, t.device);
  const Workspace ws(a[11], f_gemm_fused_workspace_bytes(t.M, t.N, t.K), t);
  Gradients gradients("gemm_fused", {a[1], a[3], a[6], a[8]}, a[10]);
  launch("sherry_gemm_fused", t.index, [&](void* stream) {
    return f_gemm_fused(t.x, t.s_x, w.packed, w.alpha, bias, act, residual, y.data_ptr(), dtype, t.M, t.N, t.K,
                        ws.at, ws.bytes, stream);
  });
  gradients.mark({y});
  return wrap(y);
}

// dy, x, s_x, packed, alpha, N, K, bias, act
PyObject* gemm_fused_backward(PyObject* const* a) {
  const Tokens t(a[1], a[2], a[5], a[6]);
  const Weights w(a[3], a[4], "packed", "alpha", t);
  const int act = activation_of(a[8]);
  const auto* bias = static_cast<const float*>(vector_of(a[7], "bias", at::kFloat, t.index, t.N, true));
  const at::Tensor& dy = tensor_of(a[0], "dy");
  const int dtype = dtype_of(dy.scalar_type());
  const void* pdy = matrix_of(dy, "dy", dy.scalar_type(), t.index, t.M, t.N);
  const size_t bytes = f_gemm_fused_backward_scratch_bytes(t.M, t.N, t.K, dtype);
  const at::Tensor dx = empty({t.M, t.K}, dy.scalar_type(), t.device), da = empty({t.N}, at::kFloat, t.device),
                   db = empty({t.N}, at::kFloat, t.device), scratch = empty({(int64_t)bytes}, at::kByte, t.device);
  Gradients gradients("gemm_fused_backward", {a[0], a[2], a[4], a[7]});
  launch("sherry_gemm_fused_backward", t.index, [&](void* stream) {
    return f_gemm_fused_backward(pdy, t.x, t.s_x, w.packed, w.alpha, bias, act, dx.data_ptr(),
                                 da.data_ptr<float>(), db.data_ptr<float>(), dtype, t.M, t.N, t.K,
                                 scratch.data_ptr(), bytes, stream);
  });
  gradients.mark({dx, da, db});
  return wrap_all({dx, da, db});
}

// x, s_x, packed_gate, alpha_gate, packed_up, alpha_up, N, K, act, dtype, out, workspace
PyObject* glu(PyObject* const* a) {
  const Tokens t(a[0], a[1], a[6], a[7]);
  const Weights g(a[2], a[3], "packed_gate", "alpha_gate", t), u(a[4], a[5], "packed_up", "alpha_up", t);
  const int act = activation_of(a[8]);
  const at::ScalarType type = scalar_of(a[9]);
  const int dtype = dtype_of(type);
  const at::Tensor h = output_of(a[10], t.M, t.N, type, t.index, t.device);
  const Workspace ws(a[11], f_glu_workspace_bytes(t.M, t.N, t.K), t);
  Gradients gradients("glu", {a[1], a[3], a[5]}, a[10]);
  launch("sherry_glu", t.index, [&](void* stream) {
    return f_glu(t.x, t.s_x, g.packed, g.alpha, u.packed, u.alpha, act, h.data_ptr(), dtype, t.M, t.N, t.K, ws.at,
                 ws.bytes, stream);
  });
  gradients.mark({h});
  return wrap(h);
}

// dh, x, s_x, packed_gate, alpha_gate, packed_up, alpha_up, N, K, act
PyObject* glu_backward(PyObject* const* a) {
  const Tokens t(a[1], a[2], a[7], a[8]);
  const Weights g(a[3], a[4], "packed_gate", "alpha_gate", t), u(a[5], a[6], "packed_up", "alpha_up", t);
  const int act = activation_of(a[9]);
  const at::Tensor& dh = tensor_of(a[0], "dh");
  const int dtype = dtype_of(dh.scalar_type());
  const void* pdh = matrix_of(dh, "dh", dh.scalar_type(), t.index, t.M, t.N);
  const size_t bytes = f_glu_backward_scratch_bytes(t.M, t.N, t.K, dtype);
  const at::Tensor dx = empty({t.M, t.K}, dh.scalar_type(), t.device), dg = empty({t.N}, at::kFloat, t.device),
                   du = empty({t.N}, at::kFloat, t.device), scratch = empty({(int64_t)bytes}, at::kByte, t.device);
  Gradients gradients("glu_backward", {a[0], a[2], a[4], a[6]});
  launch("sherry_glu_backward", t.index, [&](void* stream) {
    return f_glu_backward(pdh, t.x, t.s_x, g.packed, g.alpha, u.packed, u.alpha, act, dx.data_ptr(),
                          dg.data_ptr<float>(), du.data_ptr<float>(), dtype, t.M, t.N, t.K, scratch.data_ptr(),
                          bytes, stream);
  });
  gradients.mark({dx, dg, du});
  return wrap_all({dx, dg, du});
}

// The tokens x [M,K] of a norm (float32, float16 or bfloat16).
struct Features {
  int64_t M, K;
  int index, dtype;
  at::ScalarType type;
  at::Device device;
  const void* x;
  explicit Features(PyObject* px) : device(at::kCPU) {
    const at::Tensor& t = tensor_of(px, "x");
    type = t.scalar_type();
    dtype = dtype_of(type);
    check_tensor(t, "x", type, -1);
    if (t.dim() != 2) fail(PyExc_RuntimeError, "x must be 2-D [M,K]");
    M = t.size(0);
    K = t.size(1);
    index = (int)t.get_device();
    device = t.device();
    x = t.data_ptr();
  }
};

struct Stats {
  at::Tensor mean, rstd;
  float* pm = nullptr;
  float* pr = nullptr;
  Stats(PyObject* wanted, const Features& f) {
    const int truth = PyObject_IsTrue(wanted);
    if (truth < 0) throw Raised{};
    if (!truth) return;
    mean = empty({f.M}, at::kFloat, f.device);
    rstd = empty({f.M}, at::kFloat, f.device);
    pm = mean.data_ptr<float>();
    pr = rstd.data_ptr<float>();
  }
};

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

// x, weight, bias, eps, stats, out
PyObject* layernorm(PyObject* const* a) {
  const Features f(a[0]);
  const auto* w = static_cast<const float*>(vector_of(a[1], "weight", at::kFloat, f.index, f.K, true));
  const auto* b = static_cast<const float*>(vector_of(a[2], "bias", at::kFloat, f.index, f.K, true));
  const float eps = number(a[3]);
  const at::Tensor y = output_of(a[5], f.M, f.K, f.type, f.index, f.device);
  const Stats s(a[4], f);
  Gradients gradients("layernorm", {a[0], a[1], a[2]}, a[5]);
  launch("sherry_layernorm", f.index, [&](void* stream) {
    return f_layernorm(f.x, w, b, eps, y.data_ptr(), s.pm, s.pr, f.dtype, f.M, f.K, stream);
  });
  gradients.mark({y, s.mean, s.rstd});
  return s.pm ? wrap_all({y, s.mean, s.rstd}) : wrap(y);
}

// x, weight, bias, eps, stats
PyObject* layernorm_quantize(PyObject* const* a) {
  const Features f(a[0]);
  const auto* w = static_cast<const float*>(vector_of(a[1], "weight", at::kFloat, f.index, f.K, true));
  const auto* b = static_cast<const float*>(vector_of(a[2], "bias", at::kFloat, f.index, f.K, true));
  const float eps = number(a[3]);
  const at::Tensor q = empty({f.M, f.K}, at::kChar, f.device), s_x = empty({f.M}, at::kFloat, f.device);
  const Stats s(a[4], f);
  Gradients gradients("layernorm_quantize", {a[0], a[1], a[2]});
  launch("sherry_layernorm_quantize", f.index, [&](void* stream) {
    return f_layernorm_quantize(f.x, w, b, eps, static_cast<int8_t*>(q.data_ptr()), s_x.data_ptr<float>(), s.pm,
                                s.pr, f.dtype, f.M, f.K, stream);
  });
  gradients.mark({s_x, s.mean, s.rstd});
  return s.pm ? wrap_all({q, s_x, s.mean, s.rstd}) : wrap_all({q, s_x});
}

// dy, x, mean, rstd, weight, out
PyObject* layernorm_backward(PyObject* const* a) {
  const Features f(a[1]);
  const void* dy = matrix_of(a[0], "dy", f.type, f.index, f.M, f.K);
  const auto* mean = static_cast<const float*>(vector_of(a[2], "mean", at::kFloat, f.index, f.M));
  const auto* rstd = static_cast<const float*>(vector_of(a[3], "rstd", at::kFloat, f.index, f.M));
  const auto* w = static_cast<const float*>(vector_of(a[4], "weight", at::kFloat, f.index, f.K, true));
  const at::Tensor dx = output_of(a[5], f.M, f.K, f.type, f.index, f.device);
  const size_t bytes = f_layernorm_backward_scratch_bytes(f.M, f.K);
  const at::Tensor dw = empty({f.K}, at::kFloat, f.device), db = empty({f.K}, at::kFloat, f.device),
                   scratch = empty({(int64_t)bytes}, at::kByte, f.device);
  Gradients gradients("layernorm_backward", {a[0], a[1], a[2], a[3], a[4]}, a[5]);
  launch("sherry_layernorm_backward", f.index, [&](void* stream) {
    return f_layernorm_backward(dy, f.x, mean, rstd, w, dx.data_ptr(), dw.data_ptr<float>(), db.data_ptr<float>(),
                                f.dtype, f.M, f.K, scratch.data_ptr(), bytes, stream);
  });
  gradients.mark({dx, dw, db});
  return wrap_all({dx, dw, db});
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

// A matrix whose rows may lie further apart than they are long (a slice of a
// stacked product): its rows' distance.
void check_rows(const at::Tensor& t, const char* name, at::ScalarType type, int index) {
  if (t.layout() != at::kStrided) fail(PyExc_RuntimeError, "%s must be a dense tensor", name);
  if (!t.is_cuda()) fail(PyExc_RuntimeError, "%s must be on a GPU device, got %s", name, t.device().str().c_str());
  if (t.scalar_type() != type)
    fail(PyExc_RuntimeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
  if (index >= 0 && t.get_device() != index)
    fail(PyExc_RuntimeError, "%s must be on cuda:%d, got %s", name, index, t.device().str().c_str());
}

int64_t stride_of(const at::Tensor& t, int64_t width) { return t.size(0) > 1 ? t.stride(0) : (width + 7) / 8 * 8; }

// [T, heads, dim], a row's heads one after another.
int64_t heads_of(const at::Tensor& t, const char* name, at::ScalarType type, int index, int64_t T, int64_t heads,
                 int64_t dim) {
  check_rows(t, name, type, index);
  if (t.dim() != 3 || t.size(0) != T || t.size(1) != heads || t.size(2) != dim)
    fail(PyExc_RuntimeError, "%s must be [%lld,%lld,%lld]", name, (long long)T, (long long)heads, (long long)dim);
  if ((dim > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != dim))
    fail(PyExc_RuntimeError, "%s must have its rows' %lld values one after another", name, (long long)(heads * dim));
  return stride_of(t, heads * dim);
}

// What qk_norm_rope and its backward share: x [T, width], positions, freqs, weights.
struct Stacked {
  int64_t T, width, stride;
  int index, dtype;
  at::ScalarType type;
  at::Device device;
  const void* x;
  const int32_t* positions;
  const double* freqs;
  int64_t rotary;
  float eps;
  bool norm;
  const float *wq, *wk;
  Stacked(PyObject* px, PyObject* pp, PyObject* pf, PyObject* pwq, PyObject* pwk, PyObject* pe, PyObject* pn,
          int64_t dim)
      : device(at::kCPU) {
    const at::Tensor& t = tensor_of(px, "x");
    type = t.scalar_type();
    dtype = dtype_of(type);
    check_rows(t, "x", type, -1);
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1)) fail(PyExc_RuntimeError, "x must be 2-D with contiguous rows");
    T = t.size(0);
    width = t.size(1);
    stride = stride_of(t, width);
    index = (int)t.get_device();
    device = t.device();
    x = t.data_ptr();
    positions = static_cast<const int32_t*>(vector_of(pp, "positions", at::kInt, index, T));
    const at::Tensor& f = tensor_of(pf, "freqs");
    check_tensor(f, "freqs", at::kDouble, index);
    rotary = 2 * f.numel();
    freqs = rotary ? f.data_ptr<double>() : nullptr;
    norm = truth(pn);
    eps = number(pe);
    wq = static_cast<const float*>(vector_of(pwq, "q_weight", at::kFloat, index, dim, true));
    wk = static_cast<const float*>(vector_of(pwk, "k_weight", at::kFloat, index, dim, true));
    if (!norm && (wq || wk)) fail(PyExc_ValueError, "norm=False takes no weights");
  }
};

// x, positions, freqs, q_heads, k_heads, dim, q_weight, k_weight, eps, norm, interleaved
PyObject* qk_norm_rope(PyObject* const* a) {
  const int64_t hq = integer(a[3]), hk = integer(a[4]), dim = integer(a[5]);
  const Stacked s(a[0], a[1], a[2], a[6], a[7], a[8], a[9], dim);
  if (hq < 1 || hk < 1 || dim < 1 || hq > 1024 || hk > 1024 || dim > 256 || s.width < (hq + hk) * dim)
    fail(PyExc_RuntimeError, "x must hold (q_heads + k_heads) * dim values a row, at most 1024 heads of 256");
  const bool interleaved = truth(a[10]);
  const at::Tensor q = empty({s.T, hq, dim}, s.type, s.device), k = empty({s.T, hk, dim}, s.type, s.device);
  Gradients gradients("qk_norm_rope", {a[0], a[2], a[6], a[7]});
  launch("sherry_qk_norm_rope", s.index, [&](void* stream) {
    return f_qk_norm_rope(s.x, s.stride, s.wq, s.wk, s.eps, s.norm, s.freqs, s.rotary, interleaved, s.positions,
                          q.data_ptr(), k.data_ptr(), s.dtype, s.T, hq, hk, dim, stream);
  });
  gradients.mark({q, k});
  return wrap_all({q, k});
}

// dq, dk, x, positions, freqs, q_weight, k_weight, eps, norm, interleaved, out
PyObject* qk_norm_rope_backward(PyObject* const* a) {
  const at::Tensor &dq = tensor_of(a[0], "dq"), &dk = tensor_of(a[1], "dk");
  if (dq.dim() != 3 || dk.dim() != 3 || dq.size(2) != dk.size(2))
    fail(PyExc_RuntimeError, "dq and dk must be [T,heads,dim]");
  const int64_t hq = dq.size(1), hk = dk.size(1), dim = dq.size(2), width = (hq + hk) * dim;
  const Stacked s(a[2], a[3], a[4], a[5], a[6], a[7], a[8], dim);
  if (s.width < width) fail(PyExc_RuntimeError, "x must hold dq's and dk's heads, %lld values a row", (long long)width);
  check_tensor(dq, "dq", s.type, s.index);
  check_tensor(dk, "dk", s.type, s.index);
  if (dq.size(0) != s.T || dk.size(0) != s.T) fail(PyExc_RuntimeError, "dq and dk must have x's %lld rows", (long long)s.T);
  const bool interleaved = truth(a[9]);
  at::Tensor dx;
  int64_t stride = width;
  if (a[10] == Py_None) {
    dx = empty({s.T, width}, s.type, s.device);
  } else {
    dx = tensor_of(a[10], "out");
    check_rows(dx, "out", s.type, s.index);
    if (dx.dim() != 2 || dx.size(0) != s.T || dx.size(1) < width || (dx.size(1) > 1 && dx.stride(1) != 1))
      fail(PyExc_RuntimeError, "out must be [%lld,at least %lld] with contiguous rows", (long long)s.T, (long long)width);
    stride = stride_of(dx, dx.size(1));
  }
  at::Tensor dwq, dwk, scratch;
  size_t bytes = 0;
  if (s.norm) {
    bytes = f_qk_norm_rope_backward_scratch_bytes(s.T, hq, hk, dim);
    dwq = empty({dim}, at::kFloat, s.device);
    dwk = empty({dim}, at::kFloat, s.device);
    scratch = empty({(int64_t)bytes}, at::kByte, s.device);
  }
  Gradients gradients("qk_norm_rope_backward", {a[0], a[1], a[2], a[4], a[5], a[6]}, a[10]);
  launch("sherry_qk_norm_rope_backward", s.index, [&](void* stream) {
    return f_qk_norm_rope_backward(dq.data_ptr(), dk.data_ptr(), s.x, s.stride, s.wq, s.wk, s.eps, s.norm, s.freqs,
                                   s.rotary, interleaved, s.positions, dx.data_ptr(), stride,
                                   s.norm ? dwq.data_ptr<float>() : nullptr, s.norm ? dwk.data_ptr<float>() : nullptr,
                                   s.dtype, s.T, hq, hk, dim, s.norm ? scratch.data_ptr() : nullptr, bytes, stream);
  });
  gradients.mark({dx, dwq, dwk});
  return wrap_all({dx, dwq, dwk});      // (an undefined tensor becomes None)
}

// The cache's tensors and the sequences of a call.
struct Cache {
  sherry_kv_cache c;
  int index;
  at::Device device;
  int64_t S, table_width;
  const int32_t *table, *starts, *lens;
  // k, v, k_scale, v_scale and table, starts, lens
  Cache(PyObject* const* a, PyObject* const* b) : device(at::kCPU) {
    const at::Tensor& k = tensor_of(a[0], "cache.k");
    check_tensor(k, "cache.k", at::kChar, -1);
    if (k.dim() != 6 || k.size(4) != 16 || k.size(5) != 16)
      fail(PyExc_RuntimeError, "cache.k must be [pages,heads,page_size/16,dim/16,16,16]");
    index = (int)k.get_device();
    device = k.device();
    const at::Tensor& v = tensor_of(a[1], "cache.v");
    check_tensor(v, "cache.v", at::kChar, index);
    if (v.sizes() != k.sizes()) fail(PyExc_RuntimeError, "cache.v must have cache.k's shape");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.pages = k.size(0);
    c.heads = k.size(1);
    c.page_size = 16 * k.size(2);
    c.dim = 16 * k.size(3);
    float* scales[2];
    const char* names[2] = {"cache.k_scale", "cache.v_scale"};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor& s = tensor_of(a[2 + i], names[i]);
      check_tensor(s, names[i], at::kFloat, index);
      if (s.dim() != 3 || s.size(0) != k.size(0) || s.size(1) != k.size(1) || s.size(2) != k.size(2))
        fail(PyExc_RuntimeError, "%s must be [pages,heads,page_size/16]", names[i]);
      scales[i] = s.data_ptr<float>();
    }
    c.k_scale = scales[0];
    c.v_scale = scales[1];
    const at::Tensor& t = tensor_of(b[0], "table");
    check_tensor(t, "table", at::kInt, index);
    if (t.dim() != 2) fail(PyExc_RuntimeError, "table must be 2-D [sequences,pages of one]");
    S = t.size(0);
    table_width = t.size(1);
    table = t.data_ptr<int32_t>();
    starts = static_cast<const int32_t*>(vector_of(b[1], "starts", at::kInt, index, S + 1));
    lens = static_cast<const int32_t*>(vector_of(b[2], "lens", at::kInt, index, S));
  }
};

// k, v, k_scale, v_scale of the cache; k, v, table, starts, lens
PyObject* cache_write(PyObject* const* a) {
  const Cache c(a, a + 6);
  const at::Tensor &k = tensor_of(a[4], "k"), &v = tensor_of(a[5], "v");
  const int dtype = dtype_of(k.scalar_type());
  if (k.dim() != 3) fail(PyExc_RuntimeError, "k must be [T,heads,dim]");
  const int64_t T = k.size(0);
  const int64_t ks = heads_of(k, "k", k.scalar_type(), c.index, T, c.c.heads, c.c.dim);
  const int64_t vs = heads_of(v, "v", k.scalar_type(), c.index, T, c.c.heads, c.c.dim);
  bool graded = k.requires_grad() || v.requires_grad();
  for (int i : {2, 3}) graded |= tensor_of(a[i], "cache").requires_grad();
  for (int i : {2, 3, 4, 5}) refuse_tangent("cache_write", tensor_of(a[i], "cache"));
  if (c10::GradMode::is_enabled() && graded)
    fail(PyExc_RuntimeError, "cache_write cannot carry gradients, but a tensor requires one: call it in torch.no_grad()");
  launch("sherry_cache_write", c.index, [&](void* stream) {
    return f_cache_write(&c.c, k.data_ptr(), ks, v.data_ptr(), vs, dtype, c.table, c.table_width, c.starts, c.lens,
                         c.S, T, stream);
  });
  Py_RETURN_NONE;
}

// k, v, k_scale, v_scale of the cache; table, starts, lens, tokens, dtype
PyObject* cache_read(PyObject* const* a) {
  const Cache c(a, a + 4);
  const int64_t T = integer(a[7]);
  const at::ScalarType type = scalar_of(a[8]);
  const int dtype = dtype_of(type);
  if (T < 1 || T > (1 << 20)) fail(PyExc_RuntimeError, "tokens must be from 1 to 2^20, got %lld", (long long)T);
  const at::Tensor k = empty({T, c.c.heads, c.c.dim}, type, c.device), v = empty({T, c.c.heads, c.c.dim}, type, c.device);
  Gradients gradients("cache_read", {a[2], a[3]});
  launch("sherry_cache_read", c.index, [&](void* stream) {
    return f_cache_read(&c.c, k.data_ptr(), v.data_ptr(), dtype, c.table, c.table_width, c.starts, c.lens, c.S, T,
                        stream);
  });
  gradients.mark({k, v});
  return wrap_all({k, v});
}

// q; k, v, k_scale, v_scale of the cache; table, starts, lens, scale, window, sinks, out, lse
PyObject* cache_attention(PyObject* const* a) {
  const Cache c(a + 1, a + 5);
  const at::Tensor& q = tensor_of(a[0], "q");
  const at::ScalarType type = q.scalar_type();
  const int dtype = dtype_of(type);
  if (q.dim() != 3) fail(PyExc_RuntimeError, "q must be [T,q_heads,dim]");
  const int64_t T = q.size(0), heads = q.size(1);
  const int64_t stride = heads_of(q, "q", type, c.index, T, heads, c.c.dim);
  const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)c.c.dim)) : number(a[8]);
  const int64_t window = a[9] == Py_None ? 0 : integer(a[9]), sinks = integer(a[10]);
  if (a[9] != Py_None && window < 1) fail(PyExc_ValueError, "window must be at least 1, or None");
  at::Tensor y;
  if (a[11] == Py_None) {
    y = empty({T, heads, c.c.dim}, type, c.device);
  } else {
    y = tensor_of(a[11], "out");
    check_tensor(y, "out", type, c.index);
    if (y.sizes() != q.sizes()) fail(PyExc_RuntimeError, "out must have q's shape");
  }
  at::Tensor lse;
  if (truth(a[12])) lse = empty({T, heads}, at::kFloat, c.device);
  const size_t bytes = f_cache_attention_scratch_bytes(T, c.S, heads, c.c.heads, c.c.dim);
  const at::Tensor scratch = empty({(int64_t)bytes}, at::kByte, c.device);
  const Workspace ws(Py_None, f_cache_attention_workspace_bytes(), c);
  Gradients gradients("cache_attention", {a[0], a[3], a[4]}, a[11]);
  launch("sherry_cache_attention", c.index, [&](void* stream) {
    return f_cache_attention(q.data_ptr(), stride, heads, &c.c, c.table, c.table_width, c.starts, c.lens, c.S, T,
                             scale, window, sinks, y.data_ptr(), lse.defined() ? lse.data_ptr<float>() : nullptr,
                             dtype, ws.at, ws.bytes, scratch.data_ptr(), bytes, stream);
  });
  gradients.mark({y, lse});
  return lse.defined() ? wrap_all({y, lse}) : wrap(y);
}

// functions (dict of name -> address), workspaces, workspace, activations, error
PyObject* setup(PyObject* const* a) {
  if (!PyDict_Check(a[0]) || !PyDict_Check(a[1]) || !PyDict_Check(a[3])) fail(PyExc_TypeError, "expected a dict");
  for (const Entry& e : kEntries) {
    PyObject* v = PyDict_GetItemString(a[0], e.name);
    if (!v) fail(PyExc_KeyError, "%s", e.name);
    void* p = PyLong_AsVoidPtr(v);
    if (!p) {
      if (PyErr_Occurred()) throw Raised{};
      fail(PyExc_ValueError, "%s has no address", e.name);
    }
    std::memcpy(e.at, &p, sizeof p);
  }
  PyObject** const to[] = {&g_workspaces, &g_workspace, &g_activations, &g_error};
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(a[1 + i]);
    Py_XSETREF(*to[i], a[1 + i]);
  }
  Py_RETURN_NONE;
}

#define SHERRY_METHOD(name, count) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&method<count, name>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    SHERRY_METHOD(setup, 5),           SHERRY_METHOD(gemm_fused, 12),        SHERRY_METHOD(gemm_fused_backward, 9),
    SHERRY_METHOD(glu, 12),            SHERRY_METHOD(glu_backward, 10),      SHERRY_METHOD(layernorm, 6),
    SHERRY_METHOD(layernorm_quantize, 5), SHERRY_METHOD(layernorm_backward, 6),
    SHERRY_METHOD(qk_norm_rope, 11),   SHERRY_METHOD(qk_norm_rope_backward, 11), SHERRY_METHOD(cache_write, 9),
    SHERRY_METHOD(cache_read, 9),      SHERRY_METHOD(cache_attention, 13),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
