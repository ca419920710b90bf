// native.cpp — the _native module: argument marshalling of the block-scaled
// append and the _ext attentions, whose smallest calls run for less time on
// the GPU than Python spends reading a dozen tensors' attributes (17 us a call
// through ctypes, 3 us here, most of it the launch). Checks every tensor's
// device, type, shape and contiguity, raises ValueError for what does not fit,
// and calls the C entry point, whose status it returns; nothing is computed
// here. The entry points' addresses come from the loaded libpkv (bind).
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <initializer_list>

#include "../../include/pkv.h"

namespace {

decltype(&paged_attn_decode_ext) g_decode = nullptr;
decltype(&paged_attn_prefill_chunk_ext) g_prefill = nullptr;
decltype(&rope_append_block_scaled) g_append = nullptr;

// Thrown with a Python error set.
struct Raised {};

using Types = std::initializer_list<at::ScalarType>;
using Shape = std::initializer_list<int64_t>;
constexpr auto kI32 = at::kInt, kF32 = at::kFloat, kU8 = at::kByte;
constexpr auto kCodes = at::kFloat8_e4m3fn, kE8M0 = at::kFloat8_e8m0fnu;

[[noreturn]] void refuse(const char* format, const char* name) {
  PyErr_Format(PyExc_ValueError, format, name);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// A tensor of `dims` dimensions that the caller reads sizes from.
const at::Tensor& tensor_of(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != dims) refuse("%s has the wrong number of dimensions", name);
  for (int64_t s : t.sizes())
    if (s > INT_MAX) refuse("%s is too large", name);
  return t;
}

// The current CUDA device, which has to hold the call's tensors.
c10::DeviceIndex device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  const c10::DeviceIndex dev = c10::cuda::current_device();
  if (t.device().index() != dev) refuse("%s is not on the current CUDA device", name);
  return dev;
}

// The data of a dense tensor with this shape and one of these types; null for None.
void* data(PyObject* o, const char* name, Shape shape, Types types, c10::DeviceIndex dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.device().index() != dev) refuse("%s is on another device", name);
  bool typed = false;
  for (at::ScalarType k : types) typed |= t.scalar_type() == k;
  if (!typed) refuse("%s has the wrong dtype", name);
  if (t.sizes() != at::IntArrayRef(shape)) refuse("%s has the wrong shape", name);
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  return t.data_ptr();
}

void* required(PyObject* o, const char* name, Shape shape, Types types, c10::DeviceIndex dev) {
  if (o == Py_None) refuse("%s is required", name);
  return data(o, name, shape, types, dev);
}

int whole(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT_MIN || v > INT_MAX) refuse("%s does not fit 32 bits", name);
  return (int)v;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

void* stream_of(PyObject* o, c10::DeviceIndex dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
  void* s = PyLong_AsVoidPtr(o);
  if (s == nullptr && PyErr_Occurred()) throw Raised{};
  return s;
}

pkv_dtype code16(at::ScalarType t, const char* name) {
  if (t == at::kHalf) return PKV_F16;
  if (t == at::kBFloat16) return PKV_BF16;
  refuse("%s must be float16 or bfloat16", name);
}

// What decode and prefill share: out, q, caches, tables, scales.
struct Attn {
  c10::DeviceIndex dev;
  int rows, hq, d, nb, hkv, bs, n, max_blocks;
  void *out, *q, *k, *v, *tables, *lens, *ks, *vs, *slopes, *lse;
  pkv_dtype q_type, kv_type;

  Attn(PyObject* o, PyObject* q_, PyObject* k_, PyObject* v_, PyObject* tables_, PyObject* lens_,
       PyObject* ks_, PyObject* vs_, PyObject* slopes_, PyObject* lse_) {
    const at::Tensor& qt = tensor_of(q_, "q", 3);
    dev = device_of(qt, "q");
    const at::Tensor& kt = tensor_of(k_, "k_cache", 4);
    rows = qt.size(0), hq = qt.size(1), d = qt.size(2);
    nb = kt.size(0), hkv = kt.size(1), bs = kt.size(2);
    const at::Tensor& tt = tensor_of(tables_, "block_tables", 2);
    n = tensor_of(lens_, "seq_lens", 1).size(0);
    max_blocks = tt.size(1);
    const at::ScalarType qk = qt.scalar_type(), kk = kt.scalar_type();
    q_type = code16(qk, "q");
    const bool codes = kk == kU8 || kk == kCodes;
    kv_type = codes ? PKV_FP8_E4M3 : code16(kk, "k_cache");
    q = required(q_, "q", {rows, hq, d}, {qk}, dev);
    out = required(o, "out", {rows, hq, d}, {qk}, dev);
    k = required(k_, "k_cache", {nb, hkv, bs, d}, {kk}, dev);
    v = required(v_, "v_cache", {nb, hkv, bs, d}, {kk}, dev);
    tables = required(tables_, "block_tables", {n, max_blocks}, {kI32}, dev);
    lens = required(lens_, "seq_lens", {n}, {kI32}, dev);
    ks = vs = nullptr;
    const bool block = ks_ != Py_None && tensor(ks_, "k_scales").scalar_type() != kF32;
    if (block && !codes) refuse("%s: block scales go with an E4M3 cache", "k_scales");
    if (codes && block) {
      kv_type = PKV_FP8_E4M3_BLOCK;
      ks = data(ks_, "k_scales", {nb, hkv}, {kU8, kE8M0}, dev);
      vs = data(vs_, "v_scales", {nb, hkv}, {kU8, kE8M0}, dev);
    } else if (codes) {
      ks = data(ks_, "k_scales", {hkv}, {kF32}, dev);
      vs = data(vs_, "v_scales", {hkv}, {kF32}, dev);
    }
    slopes = data(slopes_, "alibi_slopes", {hq}, {kF32}, dev);
    lse = data(lse_, "out_lse", {rows, hq}, {kF32}, dev);
  }
};

// Runs f with what it throws turned into Python errors; f returns a status.
template <class F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t expected, F f) {
  if (nargs != expected) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, nargs);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (out, q, k_cache, v_cache, block_tables, seq_lens, scale, max_seq_len, k_scales, v_scales,
//  softcap, window, alibi_slopes, partition_tokens, out_lse, workspace, stream)
PyObject* decode_ext(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 17, [&]() -> long {
    const Attn t(a[0], a[1], a[2], a[3], a[4], a[5], a[8], a[9], a[12], a[14]);
    if (t.rows != t.n) refuse("%s and seq_lens differ in length", "q");
    const at::Tensor& w = tensor(a[15], "workspace");
    if (!w.is_cuda() || w.device().index() != t.dev) refuse("%s is on another device", "workspace");
    if (!w.is_contiguous()) refuse("%s must be contiguous", "workspace");
    const float scale = real(a[6]), softcap = real(a[10]);
    const int max_len = whole(a[7], "max_seq_len"), window = whole(a[11], "window");
    const int part = whole(a[13], "partition_tokens");
    void* stream = stream_of(a[16], t.dev);
    void* ws = w.data_ptr();
    const size_t ws_bytes = w.nbytes();
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_decode(t.out, t.q, t.q_type, t.k, t.v, t.kv_type, static_cast<int32_t*>(t.tables),
                  static_cast<int32_t*>(t.lens), t.n, t.hq, t.hkv, t.d, t.bs, t.max_blocks, t.nb,
                  max_len, scale, t.ks, t.vs, softcap, window, static_cast<float*>(t.slopes), part,
                  static_cast<float*>(t.lse), ws, ws_bytes, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// (out, q, k_cache, v_cache, block_tables, seq_lens, cu_q_lens, scale, max_q_len, k_scales,
//  v_scales, softcap, window, alibi_slopes, prefix_lens, out_lse, stream)
PyObject* prefill_ext(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 17, [&]() -> long {
    const Attn t(a[0], a[1], a[2], a[3], a[4], a[5], a[9], a[10], a[13], a[15]);
    void* cu = required(a[6], "cu_q_lens", {(int64_t)t.n + 1}, {kI32}, t.dev);
    void* prefix = data(a[14], "prefix_lens", {t.n}, {kI32}, t.dev);
    const float scale = real(a[7]), softcap = real(a[11]);
    const int max_q = whole(a[8], "max_q_len"), window = whole(a[12], "window");
    void* stream = stream_of(a[16], t.dev);
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_prefill(t.out, t.q, t.q_type, t.k, t.v, t.kv_type, static_cast<int32_t*>(t.tables),
                   static_cast<int32_t*>(t.lens), static_cast<int32_t*>(cu), t.n, t.rows, max_q,
                   t.hq, t.hkv, t.d, t.bs, t.max_blocks, t.nb, scale, t.ks, t.vs, softcap, window,
                   static_cast<float*>(t.slopes), static_cast<int32_t*>(prefix),
                   static_cast<float*>(t.lse), stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// (key, value, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, cu_q_lens, query,
//  query_out, cos_sin_cache, neox_style, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 14, [&]() -> long {
    const at::Tensor& kt = tensor_of(a[0], "key", 3);
    const c10::DeviceIndex dev = device_of(kt, "key");
    const int T = kt.size(0), hkv = kt.size(1), d = kt.size(2);
    const at::Tensor& ct = tensor_of(a[2], "k_cache", 4);
    const int nb = ct.size(0), bs = ct.size(2);
    const int n = tensor_of(a[7], "seq_lens", 1).size(0);
    const int max_blocks = tensor_of(a[6], "block_tables", 2).size(1);
    const at::ScalarType kk = kt.scalar_type();
    const pkv_dtype type = code16(kk, "key");
    void* key = required(a[0], "key", {T, hkv, d}, {kk}, dev);
    void* value = required(a[1], "value", {T, hkv, d}, {kk}, dev);
    void* k = required(a[2], "k_cache", {nb, hkv, bs, d}, {kU8, kCodes}, dev);
    void* v = required(a[3], "v_cache", {nb, hkv, bs, d}, {kU8, kCodes}, dev);
    void* ks = required(a[4], "k_scales", {nb, hkv}, {kU8, kE8M0}, dev);
    void* vs = required(a[5], "v_scales", {nb, hkv}, {kU8, kE8M0}, dev);
    void* tables = required(a[6], "block_tables", {n, max_blocks}, {kI32}, dev);
    void* lens = required(a[7], "seq_lens", {n}, {kI32}, dev);
    void* cu = required(a[8], "cu_q_lens", {(int64_t)n + 1}, {kI32}, dev);
    void *query = nullptr, *query_out = nullptr, *cos_sin = nullptr;
    int hq = 1, max_pos = 0, rot = 0;
    if (a[11] != Py_None) {
      const at::Tensor& c = tensor_of(a[11], "cos_sin_cache", 2);
      max_pos = c.size(0), rot = c.size(1);
      cos_sin = data(a[11], "cos_sin_cache", {max_pos, rot}, {kF32}, dev);
    }
    if (a[9] != Py_None) {
      if (cos_sin == nullptr) refuse("%s needs cos_sin_cache", "query");
      hq = tensor_of(a[9], "query", 3).size(1);
      query = data(a[9], "query", {T, hq, d}, {kk}, dev);
      query_out = a[10] == Py_None ? query : data(a[10], "query_out", {T, hq, d}, {kk}, dev);
    } else if (a[10] != Py_None) {
      refuse("%s needs query", "query_out");
    }
    const int neox = PyObject_IsTrue(a[12]);
    if (neox < 0) throw Raised{};
    void* stream = stream_of(a[13], dev);
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_append(key, value, type, k, v, static_cast<uint8_t*>(ks), static_cast<uint8_t*>(vs),
                  static_cast<int32_t*>(tables), static_cast<int32_t*>(lens),
                  static_cast<int32_t*>(cu), n, T, query_out, query, static_cast<float*>(cos_sin),
                  max_pos, rot, neox, hq, hkv, d, bs, max_blocks, nb, stream);
    Py_END_ALLOW_THREADS;
    return st;
  });
}

// Addresses of paged_attn_decode_ext, paged_attn_prefill_chunk_ext, rope_append_block_scaled.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 3, [&]() -> long {
    g_decode = reinterpret_cast<decltype(g_decode)>(PyLong_AsVoidPtr(a[0]));
    g_prefill = reinterpret_cast<decltype(g_prefill)>(PyLong_AsVoidPtr(a[1]));
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) throw Raised{};
    return 0;
  });
}

#define PKV_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {PKV_METHOD(bind), PKV_METHOD(decode_ext), PKV_METHOD(prefill_ext),
                          PKV_METHOD(append), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch, Python and machine it was compiled for, as build.py names them.
PyMODINIT_FUNC PyInit__native() {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", PKV_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
