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

#include <ATen/Context.h>
#include <ATen/core/TensorBody.h>
#include <ATen/EmptyTensor.h>
#include <ATen/PythonTorchFunctionTLS.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDACachingAllocator.h>
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
decltype(&::mxfp4_quantize) f_mxq = nullptr;
decltype(&::mxfp4_dequantize) f_mxd = nullptr;
decltype(&::w4a16_gemm_mxfp4) f_mx16 = nullptr;
decltype(&::w4a16_gemm_silu_mul_mxfp4) f_mxsilu = nullptr;
decltype(&::w4a4_gemm_mxfp4) f_mx4 = nullptr;

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

// An MXFP4 matrix: codes [rows][K/8] (int32), scale tiles [rows/128 rounded up][K/128][512].
struct Mx {
  const uint32_t* codes;
  const uint8_t* scales;
  int rows, K, dev;
};
int64_t tiles(int64_t rows) { return (rows + 127) / 128; }
Mx mx(PyObject* co, PyObject* so, int64_t K = -1) {
  const at::Tensor& c = tensor(co);
  if (!c.is_cuda() || c.dim() != 2) throw NotPlain();
  Mx m;
  m.dev = c.get_device();
  if (m.dev != c10::cuda::current_device()) throw NotPlain();
  const int64_t rows = c.size(0), k = c.size(1) * 8;
  if (rows < 1 || k < 128 || k % 128 != 0 || (K >= 0 && k != K)) throw NotPlain();
  m.rows = narrow(rows);
  m.K = narrow(k);
  m.codes = static_cast<const uint32_t*>(checked(c, at::kInt, m.dev, {rows, k / 8}));
  m.scales = static_cast<const uint8_t*>(checked(so, at::kByte, m.dev, {tiles(rows), k / 128, 512}));
  return m;
}
// activations fp16 [M][K]
struct Rows {
  uint16_t* x;
  int M, K, dev;
};
Rows rows_of(PyObject* o) {
  const at::Tensor& t = tensor(o);
  if (!t.is_cuda() || t.dim() != 2) throw NotPlain();
  Rows r;
  r.dev = t.get_device();
  if (r.dev != c10::cuda::current_device()) throw NotPlain();
  if (t.size(0) < 1 || t.size(1) < 128 || t.size(1) % 128 != 0) throw NotPlain();
  r.M = narrow(t.size(0));
  r.K = narrow(t.size(1));
  r.x = half(checked(t, at::kHalf, r.dev, {r.M, r.K}));
  return r;
}
// a new tensor on the current device, straight from torch's caching allocator (the
// dispatcher's share of at::empty is 0.8 us); where a mode wants to see it made, or new
// memory is to be filled, the checked path makes it
at::Tensor made(at::ScalarType type, c10::IntArrayRef shape) {
  if (c10::impl::TorchDispatchModeTLS::any_modes_set() || at::impl::torch_function_mode_enabled() ||
      (at::globalContext().deterministicAlgorithms() && at::globalContext().deterministicFillUninitializedMemory()))
    throw NotPlain();
  return at::Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                              c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
}
uint16_t* optional_half(PyObject* o, int dev, std::initializer_list<int64_t> shape) {
  return o == Py_None ? nullptr : half(checked(o, at::kHalf, dev, shape));
}
// what the products share: output (given or made), workspace, error word
struct Product {
  at::Tensor out;
  uint16_t* y;
  void* ws;
  size_t wb;
  int32_t* err;
  w4a16_stream_t s;
};
Product product(int M, int N, int dev, PyObject* out, PyObject* ws, PyObject* err) {
  Product p;
  const at::Tensor& w = tensor(ws);
  p.ws = checked(w, at::kByte, dev, {-1});
  p.wb = (size_t)w.numel();
  p.err = err_flag(err, dev);
  p.out = out == Py_None ? made(at::kHalf, {M, N}) : tensor(out);
  p.y = half(checked(p.out, at::kHalf, dev, {M, N}));
  p.s = stream_of(dev);
  return p;
}
PyObject* finished(int rc, const Product& p, PyObject* out) { return out == Py_None ? result(rc, p.out) : result(rc, out); }

// (x, codes or None, scales or None)
PyObject* mx_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 3) throw NotPlain();
    const Rows r = rows_of(a[0]);
    const at::Tensor c = a[1] == Py_None ? made(at::kInt, {r.M, r.K / 8}) : tensor(a[1]);
    const at::Tensor t = a[2] == Py_None ? made(at::kByte, {tiles(r.M), r.K / 128, 512}) : tensor(a[2]);
    void* cp = checked(c, at::kInt, r.dev, {r.M, r.K / 8});
    void* sp = checked(t, at::kByte, r.dev, {tiles(r.M), r.K / 128, 512});
    const w4a16_stream_t s = stream_of(r.dev);
    const int rc = unlocked([&] { return f_mxq(r.x, r.M, r.K, static_cast<uint32_t*>(cp), byte(sp), s); });
    if (rc) return PyLong_FromLong(rc);
    PyObject* co = a[1] == Py_None ? THPVariable_Wrap(c) : (Py_INCREF(a[1]), a[1]);
    PyObject* so = a[2] == Py_None ? THPVariable_Wrap(t) : (Py_INCREF(a[2]), a[2]);
    PyObject* pair = co && so ? PyTuple_Pack(2, co, so) : nullptr;
    Py_XDECREF(co);
    Py_XDECREF(so);
    return pair;
  });
}

// (codes, scales, out or None)
PyObject* mx_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 3) throw NotPlain();
    const Mx m = mx(a[0], a[1]);
    const at::Tensor out = a[2] == Py_None ? made(at::kHalf, {m.rows, m.K}) : tensor(a[2]);
    void* op = checked(out, at::kHalf, m.dev, {m.rows, m.K});
    const w4a16_stream_t s = stream_of(m.dev);
    const int rc = unlocked([&] { return f_mxd(m.codes, m.scales, m.rows, m.K, half(op), s); });
    return a[2] == Py_None ? result(rc, out) : result(rc, a[2]);
  });
}

// (x, codes, scales, bias or None, residual or None, out or None, workspace, err_flag or None)
PyObject* mx_gemm16(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) throw NotPlain();
    const Rows r = rows_of(a[0]);
    const Mx w = mx(a[1], a[2], r.K);
    const uint16_t *bias = optional_half(a[3], r.dev, {w.rows}), *res = optional_half(a[4], r.dev, {r.M, w.rows});
    const Product p = product(r.M, w.rows, r.dev, a[5], a[6], a[7]);
    const int rc = unlocked([&] {
      return f_mx16(r.x, r.M, r.K, w.codes, w.scales, w.rows, bias, res, p.y, p.ws, p.wb, p.err, p.s);
    });
    return finished(rc, p, a[5]);
  });
}

// (x, codes_gate, scales_gate, codes_up, scales_up, out or None, workspace, err_flag or None)
PyObject* mx_silu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) throw NotPlain();
    const Rows r = rows_of(a[0]);
    const Mx g = mx(a[1], a[2], r.K), u = mx(a[3], a[4], r.K);
    if (g.rows != u.rows) throw NotPlain();
    const Product p = product(r.M, g.rows, r.dev, a[5], a[6], a[7]);
    const int rc = unlocked([&] {
      return f_mxsilu(r.x, r.M, r.K, g.codes, g.scales, u.codes, u.scales, g.rows, p.y, p.ws, p.wb, p.err, p.s);
    });
    return finished(rc, p, a[5]);
  });
}

// (x_codes, x_scales, codes, scales, bias or None, residual or None, out or None, workspace, err_flag or None)
PyObject* mx_gemm4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) throw NotPlain();
    const Mx x = mx(a[0], a[1]), w = mx(a[2], a[3], x.K);
    if (w.dev != x.dev) throw NotPlain();
    const uint16_t *bias = optional_half(a[4], x.dev, {w.rows}), *res = optional_half(a[5], x.dev, {x.rows, w.rows});
    const Product p = product(x.rows, w.rows, x.dev, a[6], a[7], a[8]);
    const int rc = unlocked([&] {
      return f_mx4(x.codes, x.scales, x.rows, x.K, w.codes, w.scales, w.rows, bias, res, p.y, p.ws, p.wb, p.err, p.s);
    });
    return finished(rc, p, a[6]);
  });
}

// (addresses of the entries, in the order of the declarations above)
constexpr int ENTRIES = 12;
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[ENTRIES];
  if (n != ENTRIES) {
    PyErr_SetString(PyExc_ValueError, "bind: twelve addresses expected");
    return nullptr;
  }
  for (int i = 0; i < ENTRIES; ++i) {
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
  f_mxq = reinterpret_cast<decltype(f_mxq)>(p[7]);
  f_mxd = reinterpret_cast<decltype(f_mxd)>(p[8]);
  f_mx16 = reinterpret_cast<decltype(f_mx16)>(p[9]);
  f_mxsilu = reinterpret_cast<decltype(f_mxsilu)>(p[10]);
  f_mx4 = reinterpret_cast<decltype(f_mx4)>(p[11]);
  Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(append), ENTRY(read), ENTRY(decode_int4), ENTRY(decode_window), ENTRY(mx_quantize), ENTRY(mx_dequantize),
                         ENTRY(mx_gemm16), ENTRY(mx_silu), ENTRY(mx_gemm4), ENTRY(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w4a16_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w4a16_torch(void) { return PyModule_Create(&module); }
