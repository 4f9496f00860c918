// torch_args.cpp -- marshalling of torch tensors for the calls whose kernels
// take a few microseconds: checking eight to fourteen tensors in Python costs
// more than the kernel behind them (GB300's host cores: 9 to 15 us a call from
// Python, 3 to 4.5 us from here).
//
// Each function checks dtype, shape, layout and device of its arguments and
// calls the C ABI (include/w4a16.h) on the current stream.  It returns the
// result; or an int, the library's error code; or None for anything that is
// not the plain case (a wrong tensor, no workspace, another device than the
// current one), which the binding's checked path then handles or refuses.
// No part of an operation is computed here.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <initializer_list>

#include "w4a16.h"

namespace {

// The library's entries, given by address (the library is loaded by the binding).
decltype(&::kv_append_rope_int4) f_append = nullptr;
decltype(&::kv_read_int4) f_read = nullptr;
decltype(&::paged_gqa_decode_int4) f_decode = nullptr;
decltype(&::paged_gqa_decode_rope_append_int4) f_step = nullptr;
decltype(&::paged_gqa_decode_window) f_win16 = nullptr;
decltype(&::paged_gqa_decode_window_fp8) f_win8 = nullptr;
decltype(&::paged_gqa_decode_window_int4) f_win4 = nullptr;

constexpr int64_t D = 128;

struct NotPlain {};  // the checked path takes the call

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw NotPlain();
  return THPVariable_Unpack(o);
}

// the tensor's address, after the checks; `shape` entries < 0 match anything
void* checked(const at::Tensor& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() ||
      t.dim() != (int64_t)shape.size())
    throw NotPlain();
  int64_t i = 0;
  for (int64_t n : shape) {
    if (n >= 0 && t.size(i) != n) throw NotPlain();
    ++i;
  }
  return t.data_ptr();
}
void* checked(PyObject* o, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return checked(tensor(o), type, dev, shape);
}
int32_t* err_flag(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() || t.numel() < 1)
    throw NotPlain();
  return static_cast<int32_t*>(t.data_ptr());
}

int64_t whole(PyObject* o) {
  if (!PyLong_Check(o)) throw NotPlain();
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotPlain();
  }
  return v;
}
int small(PyObject* o) {
  const int64_t v = whole(o);
  if (v < INT32_MIN || v > INT32_MAX) throw NotPlain();
  return (int)v;
}
int narrow(int64_t v) {
  if (v > INT32_MAX) throw NotPlain();
  return (int)v;
}
float real(PyObject* o) {
  if (!PyFloat_Check(o)) throw NotPlain();
  return (float)PyFloat_AS_DOUBLE(o);
}

struct Paging {
  void *k, *v;
  const int32_t *bt, *lens;
  int pages, Hkv, B, blocks, dev;
};
enum Kind { FP16, FP8, INT4 };
Paging paging(PyObject* ko, PyObject* vo, PyObject* bto, PyObject* lo, Kind kind) {
  const at::Tensor& k = tensor(ko);
  if (!k.is_cuda() || k.dim() != (kind == INT4 ? 3 : 4)) throw NotPlain();
  Paging p;
  p.dev = k.get_device();
  if (p.dev != c10::cuda::current_device()) throw NotPlain();
  p.pages = narrow(k.size(0));
  p.Hkv = narrow(k.size(1));
  const at::ScalarType type = kind == FP16 ? at::kHalf : at::kByte;
  if (kind == INT4) {
    p.k = checked(k, type, p.dev, {-1, -1, W4A16_KV4_SLICE});
    p.v = checked(vo, type, p.dev, {p.pages, p.Hkv, W4A16_KV4_SLICE});
  } else {
    p.k = checked(k, type, p.dev, {-1, -1, 16, D});
    p.v = checked(vo, type, p.dev, {p.pages, p.Hkv, 16, D});
  }
  const at::Tensor& bt = tensor(bto);
  p.bt = static_cast<const int32_t*>(checked(bt, at::kInt, p.dev, {-1, -1}));
  p.B = narrow(bt.size(0));
  p.blocks = narrow(bt.size(1));
  p.lens = static_cast<const int32_t*>(checked(lo, at::kInt, p.dev, {p.B}));
  return p;
}

w4a16_stream_t stream_of(int dev) {
  return reinterpret_cast<w4a16_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}
at::Tensor fresh(const at::Tensor& like, c10::IntArrayRef shape) {
  return at::empty(shape, like.options().dtype(at::kHalf).requires_grad(false));
}
uint16_t* half(void* p) { return static_cast<uint16_t*>(p); }
uint8_t* byte(void* p) { return static_cast<uint8_t*>(p); }

// runs `call` without the interpreter lock: a full launch queue makes it wait
template <class F>
int unlocked(F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  return rc;
}

template <class F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const NotPlain&) {
    Py_RETURN_NONE;
  } catch (const std::exception& e) {  // (an allocation that failed, for instance)
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
    return nullptr;
  }
}

PyObject* result(int rc, const at::Tensor& t) { return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(t); }
PyObject* result(int rc, PyObject* o) {
  if (rc) return PyLong_FromLong(rc);
  Py_INCREF(o);
  return o;
}

// (q, k, v, k_pool, v_pool, block_table, context_lens, theta, q_out or None, err_flag or None)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10) throw NotPlain();
    const Paging p = paging(a[3], a[4], a[5], a[6], INT4);
    const at::Tensor& q = tensor(a[0]);
    void* qp = checked(q, at::kHalf, p.dev, {p.B, -1, D});
    const int64_t Hq = q.size(1);
    void* kp = checked(a[1], at::kHalf, p.dev, {p.B, p.Hkv, D});
    void* vp = checked(a[2], at::kHalf, p.dev, {p.B, p.Hkv, D});
    void* qo = a[8] == Py_None ? nullptr : checked(a[8], at::kHalf, p.dev, {p.B, Hq, D});
    const float theta = real(a[7]);
    int32_t* err = err_flag(a[9], p.dev);
    const w4a16_stream_t s = stream_of(p.dev);
    const int rc = unlocked([&] {
      return f_append(half(qp), half(kp), half(vp), 0, half(qo), byte(p.k), byte(p.v), p.pages, p.bt, p.blocks, p.lens,
                      p.B, (int)Hq, p.Hkv, (int)D, theta, err, s);
    });
    return result(rc, a[8] == Py_None ? a[0] : a[8]);
  });
}

// (k_pool, v_pool, block_table, context_lens, T, starts or None, k_out or None, v_out or None, err_flag or None)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) throw NotPlain();
    const Paging p = paging(a[0], a[1], a[2], a[3], INT4);
    const int T = small(a[4]);
    if (T < 1) throw NotPlain();
    const int32_t* starts = a[5] == Py_None ? nullptr : static_cast<const int32_t*>(checked(a[5], at::kInt, p.dev, {p.B}));
    const bool make = a[6] == Py_None && a[7] == Py_None;
    at::Tensor ko, vo;
    if (make) {
      ko = fresh(tensor(a[0]), {p.B, T, p.Hkv, D});
      vo = fresh(tensor(a[0]), {p.B, T, p.Hkv, D});
    } else {
      checked(ko = tensor(a[6]), at::kHalf, p.dev, {p.B, T, p.Hkv, D});
      checked(vo = tensor(a[7]), at::kHalf, p.dev, {p.B, T, p.Hkv, D});
    }
    int32_t* err = err_flag(a[8], p.dev);
    const w4a16_stream_t s = stream_of(p.dev);
    const int rc = unlocked([&] {
      return f_read(byte(p.k), byte(p.v), p.pages, p.bt, p.blocks, starts, p.lens, T, p.B, p.Hkv, (int)D,
                    half(ko.data_ptr()), half(vo.data_ptr()), make, err, s);
    });
    if (rc) return PyLong_FromLong(rc);
    PyObject* k = make ? THPVariable_Wrap(ko) : (Py_INCREF(a[6]), a[6]);
    PyObject* v = make ? THPVariable_Wrap(vo) : (Py_INCREF(a[7]), a[7]);
    PyObject* t = k && v ? PyTuple_Pack(2, k, v) : nullptr;
    Py_XDECREF(k);
    Py_XDECREF(v);
    return t;
  });
}

// (q, k_pool, v_pool, block_table, context_lens, max_context, sm_scale, workspace, out or None, err_flag or None,
//  qkv_theta or None, n_q_heads or None)
PyObject* decode_int4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 12) throw NotPlain();
    const Paging p = paging(a[1], a[2], a[3], a[4], INT4);
    const at::Tensor& q = tensor(a[0]);
    const bool fuse = a[10] != Py_None;
    int64_t Hq;
    void* qp;
    if (fuse) {
      Hq = small(a[11]);
      qp = checked(q, at::kHalf, p.dev, {p.B, -1});
      if (Hq < 1 || q.size(1) < (Hq + 2 * (int64_t)p.Hkv) * D) throw NotPlain();
    } else {
      if (a[11] != Py_None) throw NotPlain();
      qp = checked(q, at::kHalf, p.dev, {p.B, -1, D});
      Hq = q.size(1);
    }
    const int mc = small(a[5]), heads = narrow(Hq), pitch = fuse ? narrow(q.size(1)) : 0;
    const float scale = real(a[6]), theta = fuse ? real(a[10]) : 0.f;
    const at::Tensor& ws = tensor(a[7]);
    void* wp = checked(ws, at::kByte, p.dev, {-1});
    const at::Tensor out = a[8] == Py_None ? fresh(q, {p.B, Hq, D}) : tensor(a[8]);
    void* op = checked(out, at::kHalf, p.dev, {p.B, Hq, D});
    int32_t* err = err_flag(a[9], p.dev);
    const size_t wb = (size_t)ws.numel();
    const w4a16_stream_t s = stream_of(p.dev);
    const int rc = unlocked([&] {
      return fuse ? f_step(half(qp), pitch, byte(p.k), byte(p.v), p.pages, p.bt, p.blocks, p.lens, mc, p.B, heads, p.Hkv,
                           (int)D, theta, scale, wp, wb, half(op), err, s)
                  : f_decode(half(qp), 0, byte(p.k), byte(p.v), p.pages, p.bt, p.blocks, p.lens, mc, p.B, heads, p.Hkv,
                             (int)D, scale, wp, wb, half(op), err, s);
    });
    return a[8] == Py_None ? result(rc, out) : result(rc, a[8]);
  });
}

// (q, k_pool, v_pool, k_scale or None, v_scale or None, block_table, context_lens, max_context, window, sinks,
//  sm_scale, workspace, out or None, err_flag or None)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 14) throw NotPlain();
    const bool scaled = a[3] != Py_None;
    if (scaled != (a[4] != Py_None)) throw NotPlain();
    const Kind kind = scaled ? FP8 : tensor(a[1]).scalar_type() == at::kByte ? INT4 : FP16;
    const Paging p = paging(a[1], a[2], a[5], a[6], kind);
    const float *ks = nullptr, *vs = nullptr;
    if (scaled) {
      ks = static_cast<const float*>(checked(a[3], at::kFloat, p.dev, {p.pages, p.Hkv, 16}));
      vs = static_cast<const float*>(checked(a[4], at::kFloat, p.dev, {p.pages, p.Hkv, 16}));
    }
    const at::Tensor& q = tensor(a[0]);
    void* qp = checked(q, at::kHalf, p.dev, {p.B, -1, D});
    const int Hq = narrow(q.size(1)), mc = small(a[7]);
    const int64_t win = whole(a[8]), sk = whole(a[9]);
    if (win < 0 || sk < 0) throw NotPlain();
    const int window = (int)std::min<int64_t>(win, mc), sinks = (int)std::min<int64_t>(sk, mc);
    const float scale = real(a[10]);
    const at::Tensor& ws = tensor(a[11]);
    void* wp = checked(ws, at::kByte, p.dev, {-1});
    const at::Tensor out = a[12] == Py_None ? fresh(q, {p.B, Hq, D}) : tensor(a[12]);
    void* op = checked(out, at::kHalf, p.dev, {p.B, Hq, D});
    int32_t* err = err_flag(a[13], p.dev);
    const size_t wb = (size_t)ws.numel();
    const w4a16_stream_t s = stream_of(p.dev);
    const int rc = unlocked([&] {
      if (kind == FP16)
        return f_win16(half(qp), 0, half(p.k), half(p.v), p.pages, p.bt, p.blocks, p.lens, mc, window, sinks, p.B, Hq,
                       p.Hkv, (int)D, scale, wp, wb, half(op), err, s);
      if (kind == FP8)
        return f_win8(half(qp), 0, byte(p.k), byte(p.v), ks, vs, p.pages, p.bt, p.blocks, p.lens, mc, window, sinks, p.B,
                      Hq, p.Hkv, (int)D, scale, wp, wb, half(op), err, s);
      return f_win4(half(qp), 0, byte(p.k), byte(p.v), p.pages, p.bt, p.blocks, p.lens, mc, window, sinks, p.B, Hq,
                    p.Hkv, (int)D, scale, wp, wb, half(op), err, s);
    });
    return a[12] == Py_None ? result(rc, out) : result(rc, a[12]);
  });
}

// (addresses of the seven entries, in the order of the declarations above)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[7];
  if (n != 7) {
    PyErr_SetString(PyExc_ValueError, "bind: seven addresses expected");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
  }
  f_append = reinterpret_cast<decltype(f_append)>(p[0]);
  f_read = reinterpret_cast<decltype(f_read)>(p[1]);
  f_decode = reinterpret_cast<decltype(f_decode)>(p[2]);
  f_step = reinterpret_cast<decltype(f_step)>(p[3]);
  f_win16 = reinterpret_cast<decltype(f_win16)>(p[4]);
  f_win8 = reinterpret_cast<decltype(f_win8)>(p[5]);
  f_win4 = reinterpret_cast<decltype(f_win4)>(p[6]);
  Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(append), ENTRY(read), ENTRY(decode_int4), ENTRY(decode_window), ENTRY(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w4a16_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w4a16_torch(void) { return PyModule_Create(&module); }
