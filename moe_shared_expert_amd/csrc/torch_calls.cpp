// Python entry points of the calls whose GPU work takes only a few microseconds: checks of
// the tensors, outputs and workspace from torch's allocator, the current stream, and one call
// of the C ABI.  No computation happens here.
//
// A module of the CPython C API on torch's C++ tensors: taking the same steps in Python costs
// more than the kernels (one routing call 8.7 us of host time through ctypes).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "smlp.h"

namespace {

PyObject* g_check = nullptr;  // binding._check: raises for a status other than SMLP_OK

// Raised as ValueError.
struct Refused {
  std::string what;
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// Type, shape, place and (dense) layout; returns the address.
void* want(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (t.scalar_type() != type || t.sizes() != shape)
    throw Refused{std::string(name) + " must be " + c10::toString(type) + " " + shape_text(shape) + ", not " +
                  c10::toString(t.scalar_type()) + " " + shape_text(t.sizes())};
  if (!t.is_cuda() || !t.is_contiguous()) throw Refused{std::string(name) + " must be a contiguous GPU tensor"};
  if (t.get_device() != dev) throw Refused{std::string(name) + " is on another GPU"};
  return t.data_ptr();
}

int64_t blocks128(int64_t n) { return (n + 127) / 128; }

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// A C int: the library's options are narrower than Python's integers.
int small_integer(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != (int)v) throw Refused{std::string(name) + " = " + std::to_string(v) + " is out of range"};
  return (int)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// Makes GPU `dev` the current one for a call.  Usually it is, and asking takes 0.1 us of a 5 us
// call, so a process that sees one GPU does not ask.
struct OnGpu {
  c10::OptionalDeviceGuard guard;
  explicit OnGpu(int dev) {
    static const bool several = c10::hip::device_count() > 1;
    if (several && c10::hip::current_device() != dev) guard.reset_device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  }
};

// Work and allocations go to the current stream of the tensors' GPU (the binding makes a caller's
// stream current), with that GPU as the current one: launches on a default stream go there.
hipStream_t queue(int dev) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

void checked(int rc) {
  if (rc == SMLP_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", rc);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the library refused the call");
  throw python_error();
}

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (python_error& e) {
    e.restore();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool counted(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments instead of %zd", n, want);
  return false;
}

// route(logits, topk, score, bias, groups, top_groups, group_top, renormalize, scale)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& logits = tensor(a[0], "logits");
    if (logits.dim() != 2 || !logits.is_cuda() || (logits.size(1) > 1 && logits.stride(1) != 1))
      throw Refused{"logits must be a GPU matrix with unit column stride"};
    const auto type = logits.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) throw Refused{"logits must be bfloat16 or float32"};
    const int64_t T = logits.size(0), E = logits.size(1), topk = integer(a[1]);
    if (topk < 1 || topk > SMLP_MAX_TOPK) throw Refused{"topk = " + std::to_string(topk) + " is out of range"};
    const int dev = logits.get_device();
    const OnGpu current(dev);
    const float* bias = nullptr;
    if (a[3] != Py_None) bias = static_cast<const float*>(want(tensor(a[3], "bias"), "bias", at::kFloat, {E}, dev));
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    const smlp_route r{small_integer(a[2], "score"), small_integer(a[4], "groups"), small_integer(a[5], "top_groups"),
                       small_integer(a[6], "group_top"), (int)topk, truth(a[7]), (float)scale};
    at::Tensor ids = fresh({T, topk}, at::kInt, logits), weights = fresh({T, topk}, at::kFloat, logits);
    checked(shared_mlp_route(logits.data_ptr(), type == at::kFloat ? SMLP_FP32 : SMLP_BF16, T, E,
                             T > 1 ? logits.stride(0) : E, bias, &r, static_cast<int32_t*>(ids.data_ptr()),
                             static_cast<float*>(weights.data_ptr()), queue(dev)));
    PyObject* i = THPVariable_Wrap(std::move(ids));
    PyObject* w = THPVariable_Wrap(std::move(weights));
    PyObject* both = i && w ? PyTuple_Pack(2, i, w) : nullptr;
    Py_XDECREF(i);
    Py_XDECREF(w);
    return both;
  });
}

// A caller's workspace, or one of `need` bytes from torch (kept alive by `own`).
void* scratch(PyObject* given, size_t need, const at::Tensor& like, at::Tensor& own, size_t& bytes) {
  if (given != Py_None) {
    const at::Tensor& t = tensor(given, "workspace");
    if (!t.is_cuda() || !t.is_contiguous() || t.get_device() != like.get_device())
      throw Refused{"workspace must be a contiguous tensor on the same GPU"};
    bytes = t.nbytes();
    return t.data_ptr();
  }
  bytes = need;
  if (!need) return nullptr;
  own = fresh({(int64_t)need}, at::kByte, like);
  return own.data_ptr();
}

// linear_fp8(x, w, w_scales, x_scales, out_fp32, workspace)
PyObject* linear_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
    if (x.dim() != 2 || w.dim() != 2) throw Refused{"x and w must be matrices"};
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0), KB = blocks128(K);
    const int dev = x.is_cuda() ? x.get_device() : -1;
    const bool given = a[3] != Py_None;
    const bool f32 = truth(a[4]);
    const void* xp = want(x, "x", given ? at::kFloat8_e4m3fn : at::kBFloat16, {M, K}, dev);
    const OnGpu current(dev);
    const void* wp = want(w, "w", at::kFloat8_e4m3fn, {N, K}, dev);
    const float* wsp = static_cast<const float*>(want(tensor(a[2], "w_scales"), "w_scales", at::kFloat, {blocks128(N), KB}, dev));
    const float* xsp = given ? static_cast<const float*>(want(tensor(a[3], "x_scales"), "x_scales", at::kFloat, {M, KB}, dev)) : nullptr;
    size_t need = 0, bytes = 0;
    checked(shared_mlp_linear_fp8_workspace_bytes(M, K, N, given, &need));
    at::Tensor own;
    void* ws = scratch(a[5], need, x, own, bytes);
    at::Tensor y = fresh({M, N}, f32 ? at::kFloat : at::kBFloat16, x);
    checked(shared_mlp_linear_fp8(xp, xsp, wp, wsp, y.data_ptr(), M, K, N, N, f32, ws, bytes, queue(dev)));
    return THPVariable_Wrap(std::move(y));
  });
}

// experts_fp8(x, ids, weights, w_gate_up, s_gate_up, w_down, s_down, first_expert, partial_fp32, workspace)
PyObject* experts_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!counted(n, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &ids = tensor(a[1], "ids"), &wd = tensor(a[5], "w_down");
    if (x.dim() != 2 || ids.dim() != 2 || wd.dim() != 3) throw Refused{"x and ids must be matrices, w_down [E, H, I]"};
    const int64_t T = x.size(0), H = x.size(1), E = wd.size(0), I = wd.size(2), topk = ids.size(1);
    const int64_t HB = blocks128(H), IB = blocks128(I);
    const int dev = x.is_cuda() ? x.get_device() : -1;
    const bool f32 = truth(a[8]);
    const void* xp = want(x, "x", at::kBFloat16, {T, H}, dev);
    const OnGpu current(dev);
    const void* ip = want(ids, "ids", at::kInt, {T, topk}, dev);
    const void* rp = want(tensor(a[2], "weights"), "weights", at::kFloat, {T, topk}, dev);
    const void* gp = want(tensor(a[3], "w_gate_up"), "w_gate_up", at::kFloat8_e4m3fn, {E, 2 * I, H}, dev);
    const void* gs = want(tensor(a[4], "s_gate_up"), "s_gate_up", at::kFloat, {E, 2 * IB, HB}, dev);
    const void* dp = want(wd, "w_down", at::kFloat8_e4m3fn, {E, H, I}, dev);
    const void* ds = want(tensor(a[6], "s_down"), "s_down", at::kFloat, {E, HB, IB}, dev);
    size_t need = 0, bytes = 0;
    checked(shared_mlp_experts_fp8_workspace_bytes(T, H, I, E, topk, f32, &need));
    at::Tensor own;
    void* ws = scratch(a[9], need, x, own, bytes);
    at::Tensor out = fresh({T, H}, f32 ? at::kFloat : at::kBFloat16, x);
    checked(shared_mlp_experts_fp8(xp, static_cast<const int32_t*>(ip), static_cast<const float*>(rp), gp,
                                   static_cast<const float*>(gs), dp, static_cast<const float*>(ds), out.data_ptr(), T,
                                   H, I, E, topk, integer(a[7]), f32, ws, bytes, queue(dev)));
    return THPVariable_Wrap(std::move(out));
  });
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_XDECREF(g_check);
  Py_INCREF(f);
  g_check = f;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route)), METH_FASTCALL, nullptr},
    {"linear_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_fp8)), METH_FASTCALL, nullptr},
    {"experts_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(experts_fp8)), METH_FASTCALL, nullptr},
    {"set_check", set_check, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__calls() { return PyModule_Create(&module); }
