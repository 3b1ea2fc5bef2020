// k3attn_binding.cpp -- native side of attn.py: checks an operator's tensors (type, shape,
// device, strides) and calls the C ABI on their pointers.  A decode step's kernels take a few
// microseconds; the same checks in Python took as long as they (append: 9.4 us of host time).
//
// Every function takes the address of the k3attn_dims (and of the k3attn_cache, with its device,
// heads and head dim for comparison), the tensors, which all have to be on one device, and a
// stream handle or None for the current stream of that device.  The call is made with that device
// current.  It returns the k3moe_status, or raises ValueError for a tensor that does not fit.  No
// C++ exception leaves it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "../../../include/k3attn.h"

namespace {

// the C ABI's functions in libk3moe.so, set by bind()
decltype(&k3attn_qk_norm_rope) f_norm_rope;
decltype(&k3attn_kv_write) f_write;
decltype(&k3attn_kv_append) f_append;
decltype(&k3attn_kv_read) f_read;
decltype(&k3attn_decode) f_decode;

struct Refused {};  // a Python error is set

std::string list_of(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

// The device of a call's tensors: that of the first one.
struct Device {
  int index = -1;
  bool takes(const at::Tensor& t) {
    const int i = (int)t.get_device();
    if (index < 0) index = i;
    return i == index;
  }
  std::string where() const { return index < 0 ? "" : ", on cuda:" + std::to_string(index) + ","; }
};

[[noreturn]] void refuse(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, const char* how,
                         const Device& dev) {
  std::string got;
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    got = list_of(t.sizes()) + " (strides " + list_of(t.strides()) + ") of " + c10::toString(t.scalar_type()) + " on " +
          t.device().str();
  } else {
    got = Py_TYPE(o)->tp_name;
  }
  PyErr_Format(PyExc_ValueError, "%s: a CUDA tensor %s of %s%s%s is needed, got %s", name, list_of(shape).c_str(),
               c10::toString(type), how, dev.where().c_str(), got.c_str());
  throw Refused{};
}

// a contiguous tensor's pointer
template <typename T>
T* dense(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, Device& dev) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == type && t.is_cuda() && t.sizes().equals(shape) && t.is_contiguous() && dev.takes(t))
      return static_cast<T*>(t.data_ptr());
  }
  refuse(o, name, type, shape, ", contiguous", dev);
}

struct Rows {
  const uint16_t* p;
  int64_t stride;
};
// a [T, heads, D] bf16 tensor whose tokens' rows are dense: its pointer and token stride
Rows rows(PyObject* o, const char* name, int64_t T, int64_t heads, int64_t D, Device& dev) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == at::kBFloat16 && t.is_cuda() && t.sizes().equals({T, heads, D}) && t.stride(2) == 1 &&
        (t.stride(1) == D || heads == 1) && dev.takes(t))
      return {static_cast<const uint16_t*>(t.data_ptr()), T > 1 ? t.stride(0) : heads * D};
  }
  refuse(o, name, at::kBFloat16, {T, heads, D}, ", the heads of a token dense", dev);
}

// the first size of a tensor (the tokens of a call)
int32_t first_size(PyObject* o, const char* name) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() > 0 && t.size(0) <= INT32_MAX) return (int32_t)t.size(0);
  }
  PyErr_Format(PyExc_ValueError, "%s: a tensor of at most 2^31 - 1 tokens is needed", name);
  throw Refused{};
}

struct Work {
  void* p;
  size_t bytes;
};
Work workspace(PyObject* o, Device& dev) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == at::kByte && t.is_cuda() && t.is_contiguous() && dev.takes(t))
      return {t.data_ptr(), (size_t)t.numel()};
  }
  PyErr_Format(PyExc_ValueError, "ws: a contiguous uint8 CUDA tensor%s is needed", dev.where().c_str());
  throw Refused{};
}

// The tensors' device made current (where it is not: looking costs less than a guard's two changes),
// and the call's stream there.
struct Stream {
  c10::cuda::OptionalCUDAGuard guard;
  void* handle;
  Stream(PyObject* stream, const Device& dev) {
    if (c10::cuda::current_device() != dev.index) guard.set_index((c10::DeviceIndex)dev.index);
    if (stream == Py_None) {
      handle = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
    } else {
      handle = PyLong_AsVoidPtr(stream);
      if (!handle && PyErr_Occurred()) throw Refused{};
    }
  }
};

template <typename T>
const T* struct_at(PyObject* address) {
  const T* p = static_cast<const T*>(PyLong_AsVoidPtr(address));
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null struct");
    throw Refused{};
  }
  return p;
}

// the cache at `address` on the call's device, whose rows are `heads` x `D` (one number: device *
// 2^32 + heads * 65536 + D)
const k3attn_cache* cache_at(PyObject* address, PyObject* what, const k3attn_dims& d, const Device& dev) {
  const long s = PyLong_AsLong(what), shape = s & 0xFFFFFFFFl;
  if (PyErr_Occurred()) throw Refused{};
  if (shape != (long)d.n_kv_heads * 65536 + d.head_dim) {
    PyErr_Format(PyExc_ValueError, "the cache's (Hkv, D) are (%ld, %ld), the dims' (%d, %d)", shape / 65536,
                 shape % 65536, (int)d.n_kv_heads, (int)d.head_dim);
    throw Refused{};
  }
  if (s >> 32 != dev.index) {
    PyErr_Format(PyExc_ValueError, "the cache is on cuda:%ld, the tensors are on cuda:%d", s >> 32, dev.index);
    throw Refused{};
  }
  return struct_at<k3attn_cache>(address);
}

// what the norms and the rotation read beside the rows
struct Norm {
  const int32_t* positions;
  const double* inv_freq;
  const float *q_w, *k_w;
};
Norm norm(const k3attn_dims& d, int64_t T, PyObject* positions, PyObject* inv_freq, PyObject* q_w, PyObject* k_w,
          Device& dev) {
  Norm n;
  n.positions = dense<int32_t>(positions, "positions", at::kInt, {T}, dev);
  n.inv_freq = d.rot_dim ? dense<double>(inv_freq, "inv_freq", at::kDouble, {d.rot_dim / 2}, dev) : nullptr;
  n.q_w = dense<float>(q_w, "q_w", at::kFloat, {d.head_dim}, dev);
  n.k_w = dense<float>(k_w, "k_w", at::kFloat, {d.head_dim}, dev);
  return n;
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return PyLong_FromLong((long)f());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// dims, q, k, positions, inv_freq, q_w, k_w, q_out, k_out, stream
PyObject* py_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const k3attn_dims& d = *struct_at<k3attn_dims>(a[0]);
    Device dev;
    const int32_t T = first_size(a[1], "q");
    const Rows q = rows(a[1], "q", T, d.n_heads, d.head_dim, dev),
               k = rows(a[2], "k", T, d.n_kv_heads, d.head_dim, dev);
    const Norm m = norm(d, T, a[3], a[4], a[5], a[6], dev);
    uint16_t* q_out = dense<uint16_t>(a[7], "q_out", at::kBFloat16, {T, d.n_heads, d.head_dim}, dev);
    uint16_t* k_out = dense<uint16_t>(a[8], "k_out", at::kBFloat16, {T, d.n_kv_heads, d.head_dim}, dev);
    return f_norm_rope(&d, T, q.p, q.stride, k.p, k.stride, m.positions, m.inv_freq, m.q_w, m.k_w, q_out, k_out,
                       Stream(a[9], dev).handle);
  });
}

// dims, k, v, slots, cache, cache shape, ws, stream
PyObject* py_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const k3attn_dims& d = *struct_at<k3attn_dims>(a[0]);
    Device dev;
    const int32_t T = first_size(a[1], "k");
    const Rows k = rows(a[1], "k", T, d.n_kv_heads, d.head_dim, dev),
               v = rows(a[2], "v", T, d.n_kv_heads, d.head_dim, dev);
    const int32_t* slots = dense<int32_t>(a[3], "slots", at::kInt, {T}, dev);
    const k3attn_cache* c = cache_at(a[4], a[5], d, dev);
    const Work w = workspace(a[6], dev);
    return f_write(&d, T, k.p, k.stride, v.p, v.stride, slots, c, w.p, w.bytes, Stream(a[7], dev).handle);
  });
}

// dims, q, k, v, positions, slots, inv_freq, q_w, k_w, cache, cache shape, q_out, k_out, ws, stream
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const k3attn_dims& d = *struct_at<k3attn_dims>(a[0]);
    Device dev;
    const int32_t T = first_size(a[1], "q");
    const Rows q = rows(a[1], "q", T, d.n_heads, d.head_dim, dev),
               k = rows(a[2], "k", T, d.n_kv_heads, d.head_dim, dev),
               v = rows(a[3], "v", T, d.n_kv_heads, d.head_dim, dev);
    const Norm m = norm(d, T, a[4], a[6], a[7], a[8], dev);
    const int32_t* slots = dense<int32_t>(a[5], "slots", at::kInt, {T}, dev);
    const k3attn_cache* c = cache_at(a[9], a[10], d, dev);
    uint16_t* q_out = dense<uint16_t>(a[11], "q_out", at::kBFloat16, {T, d.n_heads, d.head_dim}, dev);
    uint16_t* k_out = a[12] == Py_None
                          ? nullptr
                          : dense<uint16_t>(a[12], "k_out", at::kBFloat16, {T, d.n_kv_heads, d.head_dim}, dev);
    const Work w = workspace(a[13], dev);
    return f_append(&d, T, q.p, q.stride, k.p, k.stride, v.p, v.stride, m.positions, slots, m.inv_freq, m.q_w, m.k_w, c,
                    q_out, k_out, w.p, w.bytes, Stream(a[14], dev).handle);
  });
}

// dims, slots, cache, cache shape, k_out, v_out, ws, stream
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const k3attn_dims& d = *struct_at<k3attn_dims>(a[0]);
    Device dev;
    const int32_t T = first_size(a[1], "slots");
    const int32_t* slots = dense<int32_t>(a[1], "slots", at::kInt, {T}, dev);
    const k3attn_cache* c = cache_at(a[2], a[3], d, dev);
    uint16_t* k_out = dense<uint16_t>(a[4], "k_out", at::kBFloat16, {T, d.n_kv_heads, d.head_dim}, dev);
    uint16_t* v_out = dense<uint16_t>(a[5], "v_out", at::kBFloat16, {T, d.n_kv_heads, d.head_dim}, dev);
    const Work w = workspace(a[6], dev);
    return f_read(&d, T, slots, c, k_out, v_out, w.p, w.bytes, Stream(a[7], dev).handle);
  });
}

// dims, q, cache, cache shape, page_table, lens, out, lse, ws, stream
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const k3attn_dims& d = *struct_at<k3attn_dims>(a[0]);
    Device dev;
    const int32_t B = first_size(a[1], "q");
    const Rows q = rows(a[1], "q", B, d.n_heads, d.head_dim, dev);
    const k3attn_cache* c = cache_at(a[2], a[3], d, dev);
    int64_t width = -1;
    if (THPVariable_Check(a[4]) && THPVariable_Unpack(a[4]).dim() == 2) width = THPVariable_Unpack(a[4]).size(1);
    const int32_t* table = dense<int32_t>(a[4], "page_table", at::kInt, {B, width}, dev);
    const int32_t* lens = dense<int32_t>(a[5], "lens", at::kInt, {B}, dev);
    uint16_t* out = dense<uint16_t>(a[6], "out", at::kBFloat16, {B, d.n_heads, d.head_dim}, dev);
    float* lse = a[7] == Py_None ? nullptr : dense<float>(a[7], "lse", at::kFloat, {B, d.n_heads}, dev);
    const Work w = workspace(a[8], dev);
    if (width > INT32_MAX) return K3MOE_ERR_SHAPE;
    return f_decode(&d, B, q.p, q.stride, c, table, (int32_t)width, lens, out, lse, w.p, w.bytes,
                    Stream(a[9], dev).handle);
  });
}

// the addresses of k3attn_qk_norm_rope, _kv_write, _kv_append, _kv_read, _decode
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&] {
    void* f[5];
    for (int i = 0; i < 5; ++i) f[i] = const_cast<void*>(struct_at<void>(a[i]));
    f_norm_rope = reinterpret_cast<decltype(f_norm_rope)>(f[0]);
    f_write = reinterpret_cast<decltype(f_write)>(f[1]);
    f_append = reinterpret_cast<decltype(f_append)>(f[2]);
    f_read = reinterpret_cast<decltype(f_read)>(f[3]);
    f_decode = reinterpret_cast<decltype(f_decode)>(f[4]);
    return 0;
  });
}

#define K3_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", K3_FAST(py_bind), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", K3_FAST(py_norm_rope), METH_FASTCALL, nullptr},
                         {"kv_write", K3_FAST(py_write), METH_FASTCALL, nullptr},
                         {"kv_append", K3_FAST(py_append), METH_FASTCALL, nullptr},
                         {"kv_read", K3_FAST(py_read), METH_FASTCALL, nullptr},
                         {"decode", K3_FAST(py_decode), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "k3attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_k3attn_binding() { return PyModule_Create(&module); }
