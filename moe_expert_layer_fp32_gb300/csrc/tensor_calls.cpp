// The tensor calls' fast path: selection, its gradient, quantisation and the 4-bit product from
// torch tensors, for small batches, where the host's part of a call is longer than the kernel's
// (GB300's host, route_select of one token: 13 us through the interpreter and ctypes, of which
// the launch is 4).
//
// Each function takes the arguments of its Python namesake in order and either makes the whole
// call - checks, output allocation, the C ABI function - and returns its result, or returns
// None without having done anything where an argument is not of the plain kind; the Python
// path then says what is wrong with it, or handles it.  A status other than MOE_OK comes back
// as an int.  The library's functions are looked up in the library that the package loaded.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

struct Library {
  decltype(&moe_select_workspace_bytes) select_workspace_bytes = nullptr;
  decltype(&moe_route_select) route_select = nullptr;
  decltype(&moe_route_select_bwd) route_select_bwd = nullptr;
  decltype(&moe_mx4_quantize) mx4_quantize = nullptr;
  decltype(&moe_mx4_packed_bytes) mx4_packed_bytes = nullptr;
  decltype(&moe_mx4_expert_product) mx4_expert_product = nullptr;
} lib;

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MOE_DTYPE_F32;
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_F16;
    default: return -1;
  }
}

// A dense CUDA tensor of this type on this device with these sizes (-1: any).
bool plain(const at::Tensor& t, at::ScalarType type, int device, std::initializer_list<int64_t> sizes) {
  if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type || !t.is_contiguous() ||
      t.dim() != (int64_t)sizes.size())
    return false;
  int64_t i = 0;
  for (int64_t s : sizes) {
    if (s >= 0 && t.size(i) != s) return false;
    ++i;
  }
  return true;
}

// A dense 2D CUDA tensor of a supported type on the current device.
bool matrix(PyObject* o, at::Tensor& t, int& dtype, int& device) {
  if (!THPVariable_Check(o)) return false;
  t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.dim() != 2 || !t.is_contiguous()) return false;
  dtype = dtype_of(t);
  device = (int)t.get_device();
  return dtype >= 0 && device == (int)c10::cuda::current_device() && t.size(0) <= INT32_MAX &&
         t.size(1) <= INT32_MAX;
}

// None or a tensor
bool maybe(PyObject* o, at::Tensor& t) {
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  t = THPVariable_Unpack(o);
  return true;
}

void* current_stream(int device) {
  return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
}

// A moe_select_opts structure (through the buffer protocol)
bool opts_of(PyObject* o, moe_select_opts& out) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    return false;
  }
  const bool ok = b.len == (Py_ssize_t)sizeof(out);
  if (ok) memcpy(&out, b.buf, sizeof(out));
  PyBuffer_Release(&b);
  return ok;
}

bool int_of(PyObject* o, int64_t& v) {
  if (!PyLong_Check(o)) return false;
  int overflow = 0;
  v = PyLong_AsLongLongAndOverflow(o, &overflow);
  return overflow == 0 && v >= 0 && v <= INT32_MAX;
}

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, int device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// (logits, k, opts, bias, want_prob_sum)
PyObject* route_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Tensor l, bias;
  int dt, dev;
  int64_t k;
  moe_select_opts o;
  if (n != 5 || !matrix(a[0], l, dt, dev) || !int_of(a[1], k) || !opts_of(a[2], o) ||
      !maybe(a[3], bias))
    Py_RETURN_NONE;
  const int64_t T = l.size(0), E = l.size(1);
  // (a k outside the limits: the Python path refuses it before it allocates)
  if (k < 1 || k > 16 || k > E || (bias.defined() && !plain(bias, at::kFloat, dev, {E})))
    Py_RETURN_NONE;
  at::Tensor idx = make({T, k}, at::kInt, dev), w = make({T, k}, at::kFloat, dev), prob, ws;
  size_t bytes = 0;
  if (a[4] == Py_True) {
    bytes = lib.select_workspace_bytes((int32_t)T, (int32_t)E);
    prob = make({E}, at::kFloat, dev);
    ws = make({(int64_t)bytes}, at::kByte, dev);
  }
  const int r = lib.route_select(l.data_ptr(), dt, E, (const float*)ptr(bias), &o, (int32_t)T,
                                 (int32_t)E, (int32_t)k, (int32_t*)idx.data_ptr(),
                                 (float*)w.data_ptr(), (float*)ptr(prob), ptr(ws), bytes,
                                 current_stream(dev));
  if (r != MOE_OK) return PyLong_FromLong(r);
  return prob.defined() ? pack({idx, w, prob}) : pack({idx, w});
  END_HANDLE_TH_ERRORS
}

// (logits, topk_idx, d_topk_w, opts, bias, d_prob_sum, want_d_bias)
PyObject* route_select_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Tensor l, idx, dw, bias, dp;
  int dt, dev;
  moe_select_opts o;
  if (n != 7 || !matrix(a[0], l, dt, dev) || a[1] == Py_None || !maybe(a[1], idx) ||
      a[2] == Py_None || !maybe(a[2], dw) || !opts_of(a[3], o) || !maybe(a[4], bias) ||
      !maybe(a[5], dp))
    Py_RETURN_NONE;
  const int64_t T = l.size(0), E = l.size(1);
  if (!plain(idx, at::kInt, dev, {T, -1})) Py_RETURN_NONE;
  const int64_t k = idx.size(1);
  if (!plain(dw, at::kFloat, dev, {T, k}) || (bias.defined() && !plain(bias, at::kFloat, dev, {E})) ||
      (dp.defined() && !plain(dp, at::kFloat, dev, {E})))
    Py_RETURN_NONE;
  at::Tensor d = make({T, E}, l.scalar_type(), dev), db, ws;
  size_t bytes = 0;
  if (a[6] == Py_True) {
    bytes = lib.select_workspace_bytes((int32_t)T, (int32_t)E);
    db = make({E}, at::kFloat, dev);
    ws = make({(int64_t)bytes}, at::kByte, dev);
  }
  const int r = lib.route_select_bwd(
      l.data_ptr(), dt, E, (const float*)ptr(bias), &o, (int32_t)T, (int32_t)E, (int32_t)k,
      (const int32_t*)idx.data_ptr(), (const float*)dw.data_ptr(), (const float*)ptr(dp),
      d.data_ptr(), E, (float*)ptr(db), ptr(ws), bytes, current_stream(dev));
  if (r != MOE_OK) return PyLong_FromLong(r);
  return db.defined() ? pack({d, db}) : THPVariable_Wrap(d);
  END_HANDLE_TH_ERRORS
}

// (x, want_values)
PyObject* mx4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Tensor x;
  int dt, dev;
  if (n != 2 || !matrix(a[0], x, dt, dev)) Py_RETURN_NONE;
  const int64_t R = x.size(0), K = x.size(1);
  at::Tensor codes = make({R, K / 2}, at::kByte, dev), scales = make({R, K / 32}, at::kByte, dev), values;
  if (a[1] == Py_True) values = make({R, K}, at::kBFloat16, dev);
  const int r = lib.mx4_quantize(x.data_ptr(), dt, K, R, (int32_t)K, codes.data_ptr(),
                                 scales.data_ptr(), ptr(values), current_stream(dev));
  if (r != MOE_OK) return PyLong_FromLong(r);
  return values.defined() ? pack({codes, scales, values}) : pack({codes, scales});
  END_HANDLE_TH_ERRORS
}

// (x, offsets, packed, N, workspace, bf16)
PyObject* mx4_expert_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Tensor x, off, packed, ws;
  int dt, dev;
  int64_t N;
  if (n != 6 || !matrix(a[0], x, dt, dev) || a[1] == Py_None || !maybe(a[1], off) ||
      a[2] == Py_None || !maybe(a[2], packed) || !int_of(a[3], N) || a[4] == Py_None ||
      !maybe(a[4], ws))
    Py_RETURN_NONE;
  if (!plain(off, at::kInt, dev, {-1}) || off.size(0) < 2 || !plain(packed, at::kByte, dev, {-1}) ||
      !plain(ws, at::kByte, dev, {-1}))
    Py_RETURN_NONE;
  const int64_t R = x.size(0), K = x.size(1), E = off.size(0) - 1;
  if (E > INT32_MAX || (size_t)packed.size(0) != lib.mx4_packed_bytes((int32_t)E, (int32_t)K, (int32_t)N))
    Py_RETURN_NONE;
  const bool bf16 = a[5] == Py_True;
  at::Tensor y = make({R, N}, bf16 ? at::kBFloat16 : at::kFloat, dev);
  const int r = lib.mx4_expert_product(x.data_ptr(), dt, (const int32_t*)off.data_ptr(),
                                       packed.data_ptr(), (int32_t)R, (int32_t)K, (int32_t)N,
                                       (int32_t)E, y.data_ptr(), bf16 ? MOE_DTYPE_BF16 : MOE_DTYPE_F32,
                                       ws.data_ptr(), (size_t)ws.size(0), current_stream(dev));
  if (r != MOE_OK) return PyLong_FromLong(r);
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// (path of the library): the package has it loaded
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (p == nullptr) return nullptr;
  void* h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  bool ok = h != nullptr;
  auto get = [&](auto& f, const char* name) {
    f = ok ? reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name)) : nullptr;
    ok = ok && f != nullptr;
  };
  get(lib.select_workspace_bytes, "moe_select_workspace_bytes");
  get(lib.route_select, "moe_route_select");
  get(lib.route_select_bwd, "moe_route_select_bwd");
  get(lib.mx4_quantize, "moe_mx4_quantize");
  get(lib.mx4_packed_bytes, "moe_mx4_packed_bytes");
  get(lib.mx4_expert_product, "moe_mx4_expert_product");
  if (!ok) {
    PyErr_Format(PyExc_ImportError, "%s: %s", p, dlerror());
    return nullptr;
  }
  Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(route_select),
                         FAST(route_select_backward),
                         FAST(mx4_quantize),
                         FAST(mx4_expert_product),
                         {"bind", bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods};

}  // namespace

// torch_version: the torch whose headers this was built with; the package uses it with no other
PyMODINIT_FUNC PyInit__tensor_calls() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", MOE_BUILT_WITH_TORCH) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
