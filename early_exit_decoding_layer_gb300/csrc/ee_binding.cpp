// Python binding of the paged-cache operators (the _binding module): the checks of their
// tensors, the results' allocation and the call of libee.so.
//
// A decode step calls these once per layer.  Through ctypes a call cost 8 to 16 us of
// host time, three quarters of it in looking the tensors over from Python; here it is
// 2.4 to 5.5 us, of which the launch is 2 to 4.
//
// Refusals raise the package's EEError with EE_ERR_INVALID_ARG before any launch.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <sstream>
#include <string>

#include "../../include/ee.h"

namespace {

struct Refused {
  std::string why;
};
struct PythonError {};  // a Python error is set

// Element types by kind: fp16 (or its bits in 16-bit integers), fp32, int32.
enum Kind { kHalf, kF32, kI32 };

bool is_kind(const at::Tensor& t, Kind k) {
  const auto s = t.scalar_type();
  if (k == kF32) return s == c10::ScalarType::Float;
  if (k == kI32) return s == c10::ScalarType::Int;
  return s == c10::ScalarType::Half || s == c10::ScalarType::Short || s == c10::ScalarType::UInt16;
}

[[noreturn]] void refuse(const char* name, const at::Tensor& t, Kind k, c10::IntArrayRef shape, int dev, const char* how) {
  static const char* const kinds[] = {"fp16", "fp32", "int32"};
  std::ostringstream s;
  s << name << " has to be a " << how << " " << kinds[k] << " tensor of shape " << shape << " on cuda:" << dev << ", not "
    << t.scalar_type() << " " << t.sizes() << ", strides " << t.strides() << " on " << t.device();
  throw Refused{s.str()};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " has to be a tensor"};
  return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) throw Refused{std::string(name) + " has to be a tensor on a CUDA device"};
  return t.get_device();
}

int64_t size(const at::Tensor& t, int dim, int dims, const char* name) {
  if (t.dim() != dims) throw Refused{std::string(name) + " has to have " + std::to_string(dims) + " dimensions"};
  return t.size(dim);
}

void* address(const at::Tensor& t, const char* name, int dev, Kind k, c10::IntArrayRef shape) {
  if (!t.is_cuda() || t.get_device() != dev || !is_kind(t, k) || t.sizes() != shape || !t.is_contiguous())
    refuse(name, t, k, shape, dev, "contiguous");
  return t.data_ptr();
}

// Rows that may lie apart, their values side by side.
void* rows(const at::Tensor& t, const char* name, int dev, int64_t n, int64_t width, int64_t* stride) {
  *stride = width;
  const bool same = t.is_cuda() && t.get_device() == dev && is_kind(t, kHalf) && t.sizes() == c10::IntArrayRef({n, width});
  if (same && !t.is_contiguous()) *stride = n > 1 ? t.stride(0) : width;
  if (!same || (width > 1 && t.stride(1) != 1) || *stride < width) refuse(name, t, kHalf, {n, width}, dev, "row-wise contiguous");
  return t.data_ptr();
}

int32_t integer(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw PythonError{};
    PyErr_Clear();
    throw Refused{std::string(name) + " is out of range"};
  }
  if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(name) + " is out of range"};
  return (int32_t)v;
}

int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) throw Refused{std::string(name) + " is too large"};
  return (int32_t)n;
}

int32_t* error_word(PyObject* o, int dev) {
  return o == Py_None ? nullptr : (int32_t*)address(tensor(o, "err"), "err", dev, kI32, {1});
}

at::Tensor empty(c10::IntArrayRef shape, c10::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev)));
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// EEError(status, "what: why")
void raise(ee_status status, const char* what, const std::string& why) {
  PyObject* pkg = PyImport_ImportModule("early_exit_decoding_layer_gb300");
  PyObject* cls = pkg ? PyObject_GetAttrString(pkg, "EEError") : nullptr;
  PyObject* e = cls ? PyObject_CallFunction(cls, "is", (int)status, (why.empty() ? what : (what + (": " + why))).c_str()) : nullptr;
  if (e) PyErr_SetObject(cls, e);
  Py_XDECREF(e);
  Py_XDECREF(cls);
  Py_XDECREF(pkg);
}

// Runs f, which returns a new reference or throws.
template <typename F>
PyObject* guarded(const char* what, F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused& r) {
    raise(EE_ERR_INVALID_ARG, what, r.why);
  } catch (const PythonError&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

void check(const char* what, ee_status s) {
  if (s == EE_OK) return;
  raise(s, what, "");
  throw PythonError{};
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = x ? THPVariable_Wrap(b) : nullptr;
  PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw Refused{"takes " + std::to_string(want) + " arguments"};
}

// (q, kcache, vcache, block_table, cu_q, ctx, n_heads, n_kv_heads, head_dim, max_ctx, out, err)
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  static const char* const what = "ee_op_prompt_attention";
  return guarded(what, [&]() -> PyObject* {
    count(n, 12);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "kcache"), &v = tensor(a[2], "vcache"),
                     &table = tensor(a[3], "block_table"), &cu = tensor(a[4], "cu_q"), &ctx = tensor(a[5], "ctx");
    const int dev = device_of(q, "q");
    const int64_t hq = integer(a[6], "n_heads"), hkv = integer(a[7], "n_kv_heads"), hd = integer(a[8], "head_dim");
    const int32_t max_ctx = integer(a[9], "max_ctx");
    const int64_t T = size(q, 0, 2, "q"), S = size(ctx, 0, 1, "ctx"), W = size(table, 1, 2, "block_table"),
                  nb = size(k, 0, 4, "kcache"), width = hq * hd;
    int64_t qs, os;
    const void* qp = rows(q, "q", dev, T, width, &qs);
    const void* kp = address(k, "kcache", dev, kHalf, {nb, hkv, 16, hd});
    const void* vp = address(v, "vcache", dev, kHalf, {nb, hkv, 16, hd});
    const void* tp = address(table, "block_table", dev, kI32, {S, W});
    const void* cp = address(cu, "cu_q", dev, kI32, {S + 1});
    const void* xp = address(ctx, "ctx", dev, kI32, {S});
    int32_t* ep = error_word(a[11], dev);
    const at::Tensor o = a[10] == Py_None ? empty({T, width}, c10::ScalarType::Half, dev) : tensor(a[10], "out");
    void* op = rows(o, "out", dev, T, width, &os);
    const at::Tensor lse = empty({hq, T}, c10::ScalarType::Float, dev);
    const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
    check(what, ee_op_prompt_attention(size32(S, "ctx"), size32(T, "q"), (int32_t)hq, (int32_t)hkv, (int32_t)hd, max_ctx,
                                       (const uint16_t*)qp, qs, (const uint16_t*)kp, (const uint16_t*)vp, size32(nb, "kcache"),
                                       (const int32_t*)tp, size32(W, "block_table"), (const int32_t*)cp, (const int32_t*)xp,
                                       (uint16_t*)op, os, (float*)lse.data_ptr(), ep, stream_of(dev)));
    return pair(o, lse);
  });
}

// (q, kcache, block_table, cu_q, ctx, lse, weights, n_heads, n_kv_heads, head_dim, max_ctx, err)
PyObject* prompt_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  static const char* const what = "ee_op_prompt_weights";
  return guarded(what, [&]() -> PyObject* {
    count(n, 12);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "kcache"), &table = tensor(a[2], "block_table"),
                     &cu = tensor(a[3], "cu_q"), &ctx = tensor(a[4], "ctx"), &lse = tensor(a[5], "lse"),
                     &w = tensor(a[6], "weights");
    const int dev = device_of(q, "q");
    const int64_t hq = integer(a[7], "n_heads"), hkv = integer(a[8], "n_kv_heads"), hd = integer(a[9], "head_dim");
    const int32_t max_ctx = integer(a[10], "max_ctx");
    const int64_t T = size(q, 0, 2, "q"), S = size(ctx, 0, 1, "ctx"), W = size(table, 1, 2, "block_table"),
                  nb = size(k, 0, 4, "kcache");
    int64_t qs;
    const void* qp = rows(q, "q", dev, T, hq * hd, &qs);
    const void* kp = address(k, "kcache", dev, kHalf, {nb, hkv, 16, hd});
    const void* tp = address(table, "block_table", dev, kI32, {S, W});
    const void* cp = address(cu, "cu_q", dev, kI32, {S + 1});
    const void* xp = address(ctx, "ctx", dev, kI32, {S});
    const void* lp = address(lse, "lse", dev, kF32, {hq, T});
    void* wp = address(w, "weights", dev, kF32, {nb, hkv, 16});
    int32_t* ep = error_word(a[11], dev);
    const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
    check(what, ee_op_prompt_weights(size32(S, "ctx"), size32(T, "q"), (int32_t)hq, (int32_t)hkv, (int32_t)hd, max_ctx,
                                     (const uint16_t*)qp, qs, (const uint16_t*)kp, size32(nb, "kcache"), (const int32_t*)tp,
                                     size32(W, "block_table"), (const int32_t*)cp, (const int32_t*)xp, (const float*)lp,
                                     (float*)wp, ep, stream_of(dev)));
    Py_INCREF(a[6]);
    return a[6];
  });
}

// (q, kcache, vcache, block_table, pos, weights, n_heads, n_kv_heads, head_dim, max_ctx, out, err)
PyObject* attention_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  static const char* const what = "ee_op_attention_weights";
  return guarded(what, [&]() -> PyObject* {
    count(n, 12);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "kcache"), &v = tensor(a[2], "vcache"),
                     &table = tensor(a[3], "block_table"), &pos = tensor(a[4], "pos"), &w = tensor(a[5], "weights");
    const int dev = device_of(q, "q");
    const int64_t hq = integer(a[6], "n_heads"), hkv = integer(a[7], "n_kv_heads"), hd = integer(a[8], "head_dim");
    const int32_t max_ctx = integer(a[9], "max_ctx");
    const int64_t B = size(pos, 0, 1, "pos"), W = size(table, 1, 2, "block_table"), nb = size(k, 0, 4, "kcache"), width = hq * hd;
    const void* qp = address(q, "q", dev, kF32, {B, width});
    const void* kp = address(k, "kcache", dev, kHalf, {nb, hkv, 16, hd});
    const void* vp = address(v, "vcache", dev, kHalf, {nb, hkv, 16, hd});
    const void* tp = address(table, "block_table", dev, kI32, {B, W});
    const void* pp = address(pos, "pos", dev, kI32, {B});
    void* wp = address(w, "weights", dev, kF32, {nb, hkv, 16});
    int32_t* ep = error_word(a[11], dev);
    const at::Tensor o = a[10] == Py_None ? empty({B, width}, c10::ScalarType::Float, dev) : tensor(a[10], "out");
    void* op = address(o, "out", dev, kF32, {B, width});
    const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
    check(what, ee_op_attention_weights(size32(B, "pos"), (int32_t)hq, (int32_t)hkv, (int32_t)hd, max_ctx, (const float*)qp,
                                        (const uint16_t*)kp, (const uint16_t*)vp, size32(nb, "kcache"), (const int32_t*)tp,
                                        size32(W, "block_table"), (const int32_t*)pp, (float*)op, (float*)wp, ep,
                                        stream_of(dev)));
    return THPVariable_Wrap(o);
  });
}

// (kcache, vcache, weights, block_table, ctx, keep, recent, max_ctx, dst_table, err)
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  static const char* const what = "ee_op_evict";
  return guarded(what, [&]() -> PyObject* {
    count(n, 10);
    const at::Tensor &k = tensor(a[0], "kcache"), &v = tensor(a[1], "vcache"), &w = tensor(a[2], "weights"),
                     &table = tensor(a[3], "block_table"), &ctx = tensor(a[4], "ctx");
    const int dev = device_of(k, "kcache");
    const int32_t keep = integer(a[5], "keep"), recent = integer(a[6], "recent"), max_ctx = integer(a[7], "max_ctx");
    const int64_t nb = size(k, 0, 4, "kcache"), hkv = k.size(1), hd = k.size(3), B = size(ctx, 0, 1, "ctx"),
                  W = size(table, 1, 2, "block_table");
    void* kp = address(k, "kcache", dev, kHalf, {nb, hkv, 16, hd});
    void* vp = address(v, "vcache", dev, kHalf, {nb, hkv, 16, hd});
    void* wp = address(w, "weights", dev, kF32, {nb, hkv, 16});
    const void* tp = address(table, "block_table", dev, kI32, {B, W});
    const void* xp = address(ctx, "ctx", dev, kI32, {B});
    const void* dp = nullptr;
    int64_t D = 0;
    if (a[8] != Py_None) {
      const at::Tensor& dst = tensor(a[8], "dst_table");
      D = size(dst, 1, 2, "dst_table");
      dp = address(dst, "dst_table", dev, kI32, {B, D});
    }
    if (keep < 1 || keep > 16384 || (a[8] != Py_None && D * 16 < std::min(keep, max_ctx)))
      throw Refused{"keep has to be in [1, 16384] and to fit dst_table"};
    int32_t* ep = error_word(a[9], dev);
    const at::Tensor kept = empty({B, hkv, keep}, c10::ScalarType::Int, dev), len = empty({B}, c10::ScalarType::Int, dev);
    const c10::cuda::CUDAGuard on((c10::DeviceIndex)dev);
    check(what, ee_op_evict(size32(B, "ctx"), size32(hkv, "kcache"), size32(hd, "kcache"), max_ctx, keep, recent, (uint16_t*)kp,
                            (uint16_t*)vp, (float*)wp, size32(nb, "kcache"), (const int32_t*)tp, size32(W, "block_table"),
                            (const int32_t*)dp, size32(D, "dst_table"), (const int32_t*)xp, (int32_t*)len.data_ptr(),
                            (int32_t*)kept.data_ptr(), ep, stream_of(dev)));
    return pair(kept, len);
  });
}

PyMethodDef methods[] = {
    {"prompt_attention", (PyCFunction)(void (*)(void))prompt_attention, METH_FASTCALL, nullptr},
    {"prompt_weights", (PyCFunction)(void (*)(void))prompt_weights, METH_FASTCALL, nullptr},
    {"attention_weights", (PyCFunction)(void (*)(void))attention_weights, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void (*)(void))evict, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // inlined accessors of tensors fit the PyTorch that they were compiled against alone
  if (m && PyModule_AddStringConstant(m, "torch_version", EE_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
