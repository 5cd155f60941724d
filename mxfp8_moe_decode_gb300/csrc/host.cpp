// The decoder layer's operators around the MoE step on torch tensors: argument checks, allocation of
// outputs and the call of the C ABI. A decode step's calls are 3 to 40 us of GPU
// work each, so the way to the launch counts: 2.1 to 2.3 us a call here, 5.5 with
// add_norm's three outputs allocated; by attributes and ctypes from Python 7 to 8
// and 13.
//
// Functions take positional arguments (mxfp8_moe_decode_gb300/attention.py and
// linear.py have the signatures and their documentation); a refused argument raises ValueError, an
// error code of the library is returned as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/moe_decode.h"

namespace {

using at::IntArrayRef;
using at::Tensor;

decltype(&moe_add_norm_x8) add_norm = nullptr;
decltype(&moe_kv_append_x8) append = nullptr;
decltype(&moe_attn_x8) attn = nullptr;
decltype(&moe_norm_add_norm_x8) norm_add_norm = nullptr;
decltype(&moe_rope) rope_rows = nullptr;
decltype(&moe_rope_kv_append_x8) rope_append = nullptr;
decltype(&moe_linear_x4) linear = nullptr;
decltype(&moe_linear_x4_workspace_bytes) linear_workspace = nullptr;

struct Refused {
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

std::string shown(const Tensor& t) {
  std::ostringstream s;
  s << t.scalar_type() << " " << t.sizes() << " on " << t.device();
  return s.str();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// bf16 rows of contiguous values, any row stride; returns the stride.
int64_t rows(const Tensor& t, const char* name, IntArrayRef shape, at::Device device) {
  if (t.scalar_type() != at::kBFloat16 || t.sizes() != shape || t.device() != device) {
    std::ostringstream s;
    s << name << " must be bf16 " << shape << " on " << device << ", got " << shown(t);
    refuse(s.str());
  }
  int64_t width = 1;
  bool dense = true;
  for (size_t i = shape.size() - 1; i > 0; --i) {
    dense = dense && (t.stride(i) == width || shape[i] == 1);
    width *= shape[i];
  }
  if (!dense && shape[0] > 0) refuse(std::string(name) + ": the values of a row must be contiguous");
  return shape[0] > 1 ? t.stride(0) : width;  // (one row or none: any stride)
}

void* dense(const Tensor& t, const char* name, IntArrayRef shape, at::ScalarType dtype, at::Device device) {
  if (t.sizes() != shape || t.scalar_type() != dtype || t.device() != device || !t.is_contiguous()) {
    std::ostringstream s;
    s << name << " must be a contiguous " << dtype << " " << shape << " tensor on " << device << ", got " << shown(t);
    refuse(s.str());
  }
  return t.data_ptr();
}

int as_int(int64_t v, const char* name) {
  if (v < INT_MIN || v > INT_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// A finite float, or NaN and infinity as they are (the library refuses them).
float single(PyObject* o) { return static_cast<float>(real(o)); }

// An output of rows, any row stride: the tensor that was passed (checked), or a new one.
struct RowsOut {
  PyObject* given;
  Tensor made;
  void* ptr;
  int64_t ld;
  RowsOut(PyObject* o, const char* name, IntArrayRef shape, at::Device device) : given(o) {
    if (o == Py_None) made = at::empty(shape, at::TensorOptions().dtype(at::kBFloat16).device(device));
    const Tensor& t = o == Py_None ? made : tensor(o, name);
    ld = rows(t, name, shape, device);
    ptr = t.data_ptr();
  }
  PyObject* object() const {  // a new reference
    if (given == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
  }
};

// An output: the tensor that was passed (checked), or a new one.
struct Out {
  PyObject* given;
  Tensor made;
  void* ptr;
  Out(PyObject* o, const char* name, IntArrayRef shape, at::ScalarType dtype, at::Device device) : given(o) {
    if (o == Py_None) {
      made = at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
      ptr = made.data_ptr();
    } else {
      ptr = dense(tensor(o, name), name, shape, dtype, device);
    }
  }
  PyObject* object() const {  // a new reference
    if (given == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
  }
};

PyObject* tuple_of(std::initializer_list<PyObject*> items) {  // takes the references
  bool all = true;
  for (PyObject* o : items) all = all && o != nullptr;
  PyObject* t = all ? PyTuple_New(static_cast<Py_ssize_t>(items.size())) : nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_XDECREF(o);
  }
  return t;
}

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// call(stream) on the device's current stream, with the device current
template <class Call>
int on_device(at::Device device, Call call) {
  const c10::cuda::CUDAGuard guard(device);
  return call(c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

struct Cache {
  moe_kv_cache c;
  at::Device device;
};

Cache cache_of(PyObject* pb, PyObject* pc) {
  const Tensor& b = tensor(pb, "blocks");
  if (b.dim() != 4 || !b.is_cuda() || b.scalar_type() != at::kByte || !b.is_contiguous() || b.size(2) != 2 ||
      b.size(3) % MOE_KV_PAGE_TOKENS)
    refuse("blocks must be a contiguous CUDA uint8 [pages, kv_heads, 2, 64 * head_dim] tensor");
  Cache x{{}, b.device()};
  x.c.blocks = static_cast<uint8_t*>(b.data_ptr());
  x.c.codes = static_cast<uint8_t*>(
      dense(tensor(pc, "codes"), "codes", {b.size(0), b.size(1), 2}, at::kByte, x.device));
  x.c.pages = as_int(b.size(0), "pages");
  x.c.kv_heads = as_int(b.size(1), "kv_heads");
  x.c.head_dim = as_int(b.size(3) / MOE_KV_PAGE_TOKENS, "head_dim");
  return x;
}

moe_kv_seqs seqs_of(PyObject* table, PyObject* lens, PyObject* cu_q, int64_t tokens, int64_t max_q,
                    at::Device device) {
  const Tensor& t = tensor(table, "page_table");
  if (t.dim() != 2) refuse("page_table must be an int32 [seqs, max_pages] tensor");
  const int64_t n = t.size(0);
  moe_kv_seqs s{};
  s.page_table = static_cast<const int32_t*>(dense(t, "page_table", t.sizes(), at::kInt, device));
  s.lens = static_cast<const int32_t*>(dense(tensor(lens, "lens"), "lens", {n}, at::kInt, device));
  if (cu_q != Py_None) {
    s.cu_q = static_cast<const int32_t*>(dense(tensor(cu_q, "cu_q"), "cu_q", {n + 1}, at::kInt, device));
  } else if (tokens != n) {
    std::ostringstream w;
    w << tokens << " rows for " << n << " sequences: without cu_q each has one";
    refuse(w.str());
  }
  s.seqs = as_int(n, "seqs");
  s.tokens = as_int(tokens, "tokens");
  s.max_pages = as_int(t.size(1), "max_pages");
  s.max_q = as_int(max_q, "max_q");
  return s;
}

int32_t* status_of(PyObject* o, at::Device device) {
  if (o == Py_None) return nullptr;
  return static_cast<int32_t*>(dense(tensor(o, "status"), "status", {1}, at::kInt, device));
}

// x, residual, norm_w, eps, res_out, x8, codes, normed
PyObject* add_norm_x8(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  if (x.dim() != 2 || !x.is_cuda()) refuse("x must be a CUDA bf16 [M, H] tensor");
  const int64_t shape[2] = {x.size(0), x.size(1)}, groups[2] = {shape[0], shape[1] / 32};
  const at::Device dev = x.device();
  if (shape[1] % 32) refuse("H must be a multiple of 32");
  const Tensor& r = tensor(a[1], "residual");
  const int64_t ldx = rows(x, "x", shape, dev), ldr = rows(r, "residual", shape, dev);
  const void* w = dense(tensor(a[2], "norm_w"), "norm_w", {shape[1]}, at::kBFloat16, dev);
  const float eps = static_cast<float>(real(a[3]));
  const int m = as_int(shape[0], "M"), h = as_int(shape[1], "H");
  void* normed =
      a[7] == Py_None ? nullptr : dense(tensor(a[7], "normed"), "normed", shape, at::kBFloat16, dev);
  const Out res(a[4], "res_out", shape, at::kBFloat16, dev), x8(a[5], "x8", shape, at::kByte, dev),
      codes(a[6], "codes", groups, at::kByte, dev);
  const int rc = on_device(dev, [&](cudaStream_t s) {
    return add_norm(x.data_ptr(), ldx, r.data_ptr(), ldr, w, m, h, eps, res.ptr,
                    static_cast<uint8_t*>(x8.ptr), static_cast<uint8_t*>(codes.ptr), normed, s);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({res.object(), x8.object(), codes.object(), same(a[7])});
}

// blocks, codes, k, v, page_table, start, cu_q, status
PyObject* kv_append_x8(PyObject* const* a) {
  const Cache c = cache_of(a[0], a[1]);
  const Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  if (k.dim() != 3) refuse("k must be a bf16 [tokens, kv_heads, head_dim] tensor");
  const int64_t shape[3] = {k.size(0), c.c.kv_heads, c.c.head_dim};
  const int64_t ldk = rows(k, "k", shape, c.device), ldv = rows(v, "v", shape, c.device);
  const moe_kv_seqs s = seqs_of(a[4], a[5], a[6], shape[0], 1, c.device);
  int32_t* status = status_of(a[7], c.device);
  const int rc = on_device(c.device, [&](cudaStream_t st) {
    return append(&c.c, &s, k.data_ptr(), ldk, v.data_ptr(), ldv, status, st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({same(a[0]), same(a[1])});
}

// q, blocks, codes, page_table, kv_len, cu_q, max_q, scale, window, sinks, out, lse, workspace, status
PyObject* attn_x8(PyObject* const* a) {
  const Cache c = cache_of(a[1], a[2]);
  const Tensor& q = tensor(a[0], "q");
  if (q.dim() != 3) refuse("q must be a bf16 [tokens, q_heads, head_dim] tensor");
  const int64_t shape[3] = {q.size(0), q.size(1), c.c.head_dim}, tokens = shape[0];
  const int64_t ldq = rows(q, "q", shape, c.device);
  const int64_t max_q = a[5] == Py_None ? 1 : a[6] == Py_None ? (tokens > 0 ? tokens : 1) : number(a[6]);
  const moe_kv_seqs s = seqs_of(a[3], a[4], a[5], tokens, max_q, c.device);
  const float scale = static_cast<float>(a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.c.head_dim)) : real(a[7]));
  const int heads = as_int(shape[1], "q_heads"), window = as_int(number(a[8]), "window"),
            sinks = as_int(number(a[9]), "sinks");
  float* lse = a[11] == Py_None ? nullptr
                                : static_cast<float*>(dense(tensor(a[11], "lse"), "lse", {tokens, shape[1]},
                                                            at::kFloat, c.device));
  Tensor ws;
  if (a[12] == Py_None) {
    ws = at::zeros({static_cast<int64_t>(MOE_ATTN_X8_WORKSPACE_BYTES)},
                   at::TensorOptions().dtype(at::kByte).device(c.device));
  } else {
    ws = tensor(a[12], "workspace");
    if (ws.device() != c.device || !ws.is_contiguous()) {
      std::ostringstream w;
      w << "workspace must be a contiguous tensor on " << c.device;
      refuse(w.str());
    }
  }
  int32_t* status = status_of(a[13], c.device);
  const Out out(a[10], "out", shape, at::kBFloat16, c.device);
  const int rc = on_device(c.device, [&](cudaStream_t st) {
    return attn(&c.c, &s, q.data_ptr(), ldq, heads, scale, window, sinks, out.ptr, lse, ws.data_ptr(),
                static_cast<size_t>(ws.nbytes()), status, st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({out.object(), same(a[11])});
}

// x, residual, post_w, norm_w, gate, res_scale, block_scale, eps, res_out, x8, codes, normed
PyObject* norm_add_norm_x8(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  if (x.dim() != 2 || !x.is_cuda()) refuse("x must be a CUDA bf16 [M, H] tensor");
  const int64_t shape[2] = {x.size(0), x.size(1)}, groups[2] = {shape[0], shape[1] / 32};
  const at::Device dev = x.device();
  if (shape[1] % 32) refuse("H must be a multiple of 32");
  const Tensor& r = tensor(a[1], "residual");
  const int64_t ldx = rows(x, "x", shape, dev), ldr = rows(r, "residual", shape, dev);
  const void* post =
      a[2] == Py_None ? nullptr : dense(tensor(a[2], "post_w"), "post_w", {shape[1]}, at::kBFloat16, dev);
  const void* w = dense(tensor(a[3], "norm_w"), "norm_w", {shape[1]}, at::kBFloat16, dev);
  const void* gate = nullptr;
  int64_t ldg = 0;
  if (a[4] != Py_None) {  // [H], or [M, H] with any row stride (0: the same row for all)
    const Tensor& g = tensor(a[4], "gate");
    if (g.dim() == 1) {
      gate = dense(g, "gate", {shape[1]}, at::kBFloat16, dev);
    } else {
      ldg = rows(g, "gate", shape, dev);
      gate = g.data_ptr();
    }
  }
  const float res_scale = single(a[5]), block_scale = single(a[6]), eps = single(a[7]);
  const int m = as_int(shape[0], "M"), h = as_int(shape[1], "H");
  void* normed =
      a[11] == Py_None ? nullptr : dense(tensor(a[11], "normed"), "normed", shape, at::kBFloat16, dev);
  const Out res(a[8], "res_out", shape, at::kBFloat16, dev), x8(a[9], "x8", shape, at::kByte, dev),
      codes(a[10], "codes", groups, at::kByte, dev);
  const int rc = on_device(dev, [&](cudaStream_t s) {
    return norm_add_norm(x.data_ptr(), ldx, r.data_ptr(), ldr, gate, ldg, post, w, m, h, res_scale, block_scale,
                         eps, res.ptr, static_cast<uint8_t*>(x8.ptr), static_cast<uint8_t*>(codes.ptr), normed, s);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({res.object(), x8.object(), codes.object(), same(a[11])});
}

// freqs, first, interleaved, scale
moe_rope_spec spec_of(PyObject* freqs, PyObject* first, PyObject* interleaved, PyObject* scale, at::Device device) {
  const Tensor& f = tensor(freqs, "freqs");
  if (f.dim() != 1) refuse("freqs must be an int64 [rot / 2] tensor");
  moe_rope_spec s{};
  s.freqs = static_cast<const uint64_t*>(dense(f, "freqs", f.sizes(), at::kLong, device));
  s.rot = as_int(2 * f.size(0), "rot");
  s.first = as_int(number(first), "first");
  s.interleaved = PyObject_IsTrue(interleaved);
  if (s.interleaved < 0) throw python_error();
  s.scale = single(scale);
  return s;
}

// x, positions, freqs, first, interleaved, scale, out
PyObject* rope(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  if (x.dim() != 3 || !x.is_cuda()) refuse("x must be a CUDA bf16 [tokens, heads, head_dim] tensor");
  const int64_t shape[3] = {x.size(0), x.size(1), x.size(2)};
  const at::Device dev = x.device();
  const int64_t ldx = rows(x, "x", shape, dev);
  const void* pos = dense(tensor(a[1], "positions"), "positions", {shape[0]}, at::kInt, dev);
  const moe_rope_spec spec = spec_of(a[2], a[3], a[4], a[5], dev);
  const int t = as_int(shape[0], "tokens"), h = as_int(shape[1], "heads"), d = as_int(shape[2], "head_dim");
  const RowsOut out(a[6], "out", shape, dev);
  const int rc = on_device(dev, [&](cudaStream_t s) {
    return rope_rows(&spec, x.data_ptr(), ldx, t, h, d, static_cast<const int32_t*>(pos), out.ptr, out.ld, s);
  });
  if (rc) return PyLong_FromLong(rc);
  return out.object();
}

// blocks, codes, q, k, v, page_table, start, freqs, cu_q, positions, first, interleaved, scale, q_out, status
PyObject* rope_kv_append_x8(PyObject* const* a) {
  const Cache c = cache_of(a[0], a[1]);
  const Tensor &q = tensor(a[2], "q"), &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
  if (k.dim() != 3) refuse("k must be a bf16 [tokens, kv_heads, head_dim] tensor");
  if (q.dim() != 3) refuse("q must be a bf16 [tokens, q_heads, head_dim] tensor");
  const int64_t shape[3] = {k.size(0), c.c.kv_heads, c.c.head_dim}, qshape[3] = {k.size(0), q.size(1), c.c.head_dim};
  const int64_t ldk = rows(k, "k", shape, c.device), ldv = rows(v, "v", shape, c.device),
                ldq = rows(q, "q", qshape, c.device);
  const moe_kv_seqs s = seqs_of(a[5], a[6], a[8], shape[0], 1, c.device);
  const moe_rope_spec spec = spec_of(a[7], a[10], a[11], a[12], c.device);
  const void* pos =
      a[9] == Py_None ? nullptr : dense(tensor(a[9], "positions"), "positions", {shape[0]}, at::kInt, c.device);
  int32_t* status = status_of(a[14], c.device);
  const int heads = as_int(qshape[1], "q_heads");
  const RowsOut out(a[13], "q_out", qshape, c.device);
  const int rc = on_device(c.device, [&](cudaStream_t st) {
    return rope_append(&c.c, &s, &spec, static_cast<const int32_t*>(pos), q.data_ptr(), ldq, heads, out.ptr, out.ld,
                       k.data_ptr(), ldk, v.data_ptr(), ldv, status, st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({out.object(), same(a[0]), same(a[1])});
}

// x, w, w_codes, x_codes, out, workspace, status
PyObject* linear_x4(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
  if (x.dim() != 2 || !x.is_cuda()) refuse("x must be a CUDA [M, K] tensor");
  if (w.dim() != 2) refuse("w must be a uint8 [N, K / 2] tensor");
  const at::Device dev = x.device();
  const int64_t m = x.size(0), k = x.size(1), n = w.size(0);
  if (k % 32) refuse("K must be a multiple of 32");
  const bool mx = a[3] != Py_None;
  int64_t ldx;
  const uint8_t* xc = nullptr;
  if (mx) {
    if (x.scalar_type() != at::kByte || (x.stride(1) != 1 && m > 0 && k > 1)) {
      refuse("x with x_codes must be uint8 [M, K] with contiguous rows, got " + shown(x));
    }
    ldx = m > 1 ? x.stride(0) : k;
    xc = static_cast<const uint8_t*>(dense(tensor(a[3], "x_codes"), "x_codes", {m, k / 32}, at::kByte, dev));
  } else {
    ldx = rows(x, "x", {m, k}, dev);
  }
  const uint8_t* wp = static_cast<const uint8_t*>(dense(w, "w", {n, k / 2}, at::kByte, dev));
  const uint8_t* wc = static_cast<const uint8_t*>(dense(tensor(a[2], "w_codes"), "w_codes", {n, k / 32}, at::kByte, dev));
  const int mi = as_int(m, "M"), ki = as_int(k, "K"), ni = as_int(n, "N");
  int32_t* status = status_of(a[6], dev);
  const RowsOut out(a[4], "out", {m, n}, dev);
  Tensor ws;
  if (a[5] != Py_None) {
    ws = tensor(a[5], "workspace");
    if (ws.device() != dev || !ws.is_contiguous()) {
      std::ostringstream s;
      s << "workspace must be a contiguous tensor on " << dev;
      refuse(s.str());
    }
  } else {
    const size_t need = linear_workspace(mi, ki, mx ? MOE_LINEAR_MXFP8 : MOE_LINEAR_BF16);
    if (need > 0)
      ws = at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(dev));
  }
  const int rc = on_device(dev, [&](cudaStream_t s) {
    return linear(x.data_ptr(), ldx, xc, mi, wp, wc, ni, ki, out.ptr, out.ld, ws.defined() ? ws.data_ptr() : nullptr,
                  ws.defined() ? static_cast<size_t>(ws.nbytes()) : 0, status, s);
  });
  if (rc) return PyLong_FromLong(rc);
  return out.object();
}

// addresses of the library's entry points
PyObject* bind(PyObject* const* a) {
  add_norm = reinterpret_cast<decltype(add_norm)>(static_cast<uintptr_t>(number(a[0])));
  append = reinterpret_cast<decltype(append)>(static_cast<uintptr_t>(number(a[1])));
  attn = reinterpret_cast<decltype(attn)>(static_cast<uintptr_t>(number(a[2])));
  norm_add_norm = reinterpret_cast<decltype(norm_add_norm)>(static_cast<uintptr_t>(number(a[3])));
  rope_rows = reinterpret_cast<decltype(rope_rows)>(static_cast<uintptr_t>(number(a[4])));
  rope_append = reinterpret_cast<decltype(rope_append)>(static_cast<uintptr_t>(number(a[5])));
  linear = reinterpret_cast<decltype(linear)>(static_cast<uintptr_t>(number(a[6])));
  linear_workspace = reinterpret_cast<decltype(linear_workspace)>(static_cast<uintptr_t>(number(a[7])));
  Py_RETURN_NONE;
}

template <PyObject* (*kBody)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs || (kBody != &bind && attn == nullptr)) {
    PyErr_SetString(PyExc_TypeError, n != kArgs ? "wrong number of arguments" : "the library is not bound");
    return nullptr;
  }
  try {
    return kBody(a);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*kBody)(PyObject* const*), Py_ssize_t kArgs>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kBody, kArgs>)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {
    method<add_norm_x8, 8>("add_norm_x8"), method<kv_append_x8, 8>("kv_append_x8"),
    method<attn_x8, 14>("attn_x8"),        method<norm_add_norm_x8, 12>("norm_add_norm_x8"),
    method<rope, 7>("rope"),               method<rope_kv_append_x8, 15>("rope_kv_append_x8"),
    method<linear_x4, 7>("linear_x4"),     method<bind, 8>("bind"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&module); }
