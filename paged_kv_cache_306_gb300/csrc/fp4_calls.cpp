// fp4_calls.cpp -- the marshalling of the FP4 calls as a CPython extension.
//
// The FP4 calls on few tokens take 2 to 4 us on the GPU; checking five to eight tensors in
// Python and converting 14 to 21 arguments through ctypes takes longer than that.  This module
// does the same checks on the tensors themselves and calls the same C entry points.  A call it
// does not accept (a check that fails, an argument of another type) returns -1 without having
// done anything, and the Python path takes it: the error messages are made there only.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

decltype(&pa_reshape_and_cache_fp4) g_write;
decltype(&pa_gather_cache_fp4) g_gather;
decltype(&pa_expand_blocks_fp4) g_expand;
decltype(&pa_decode_fp4) g_decode;

PyObject* status(long st) { return PyLong_FromLong(st); }

// The tensor of an argument if it is one, contiguous and on device `dev` (any CUDA device if dev < 0).
const at::Tensor* tensor(PyObject* o, int dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || !t.is_contiguous() || (dev >= 0 && t.get_device() != dev)) return nullptr;
  return &t;
}

bool row_code(at::ScalarType t, pa_dtype* code) {
  if (t == at::kFloat) *code = PA_F32;
  else if (t == at::kHalf) *code = PA_F16;
  else if (t == at::kBFloat16) *code = PA_BF16;
  else return false;
  return true;
}

// The pools' sizes: block size from the tile's bytes (9/16 byte per element).
bool pools(const at::Tensor& k, const at::Tensor& v, int64_t heads, int64_t dims, int* bs) {
  if (k.scalar_type() != at::kByte || v.scalar_type() != at::kByte || k.dim() != 3 || k.sizes() != v.sizes() ||
      k.size(1) != heads || (dims != 64 && dims != 128))
    return false;
  const int64_t tile = k.size(2);
  if (tile != 9 * dims && tile != 18 * dims) return false;
  *bs = tile == 9 * dims ? 16 : 32;
  return true;
}

bool as_float(PyObject* o, float* f) {
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *f = static_cast<float>(d);
  return true;
}

bool as_stream(PyObject* o, int dev, void** s) {
  if (o == Py_None) {
    *s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return true;
  }
  PyObject* p = PyObject_GetAttrString(o, "cuda_stream");
  if (!p) {
    PyErr_Clear();
    return false;
  }
  *s = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

constexpr int64_t kIntMax = 0x7fffffff;

// rows(read, key, value, k_cache, v_cache, slot_mapping, k_scale, v_scale, stream)
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 9) return status(-1);
    const at::Tensor* key = tensor(a[1], -1);
    if (!key || key->dim() != 3) return status(-1);
    const int dev = key->get_device();
    if (dev != c10::cuda::current_device()) return status(-1);
    const at::Tensor *value = tensor(a[2], dev), *k = tensor(a[3], dev), *v = tensor(a[4], dev), *slots = tensor(a[5], dev);
    if (!value || !k || !v || !slots) return status(-1);
    const int64_t T = key->size(0), heads = key->size(1), dims = key->size(2);
    pa_dtype code;
    int bs = 0;
    float ks = 0.f, vs = 0.f;
    void* stream = nullptr;
    if (!row_code(key->scalar_type(), &code) || value->scalar_type() != key->scalar_type() ||
        value->sizes() != key->sizes() || slots->scalar_type() != at::kLong || slots->dim() != 1 ||
        slots->size(0) != T || heads > kIntMax || !pools(*k, *v, heads, dims, &bs) || !as_float(a[6], &ks) ||
        !as_float(a[7], &vs) || !as_stream(a[8], dev, &stream))
      return status(-1);
    const bool read = a[0] == Py_True;
    pa_status st;
    void *kp = key->data_ptr(), *vp = value->data_ptr(), *kc = k->data_ptr(), *vc = v->data_ptr();
    const auto* sp = static_cast<const int64_t*>(slots->data_ptr());
    Py_BEGIN_ALLOW_THREADS;
    if (read)
      st = g_gather(kp, vp, kc, vc, sp, T, static_cast<int>(heads), static_cast<int>(dims), bs, k->size(0), code, ks, vs,
                    stream);
    else
      st = g_write(kp, vp, kc, vc, sp, T, static_cast<int>(heads), static_cast<int>(dims), bs, k->size(0), code, ks, vs,
                   stream);
    Py_END_ALLOW_THREADS;
    return status(st);
  } catch (...) {
    return status(-1);
  }
}

// expand(k_out, v_out, k_cache, v_cache, src_dst, k_scale, v_scale, stream)
PyObject* expand(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 8) return status(-1);
    const at::Tensor* ko = tensor(a[0], -1);
    if (!ko || ko->dim() != 5) return status(-1);
    const int dev = ko->get_device();
    if (dev != c10::cuda::current_device()) return status(-1);
    const at::Tensor *vo = tensor(a[1], dev), *k = tensor(a[2], dev), *v = tensor(a[3], dev), *pairs = tensor(a[4], dev);
    if (!vo || !k || !v || !pairs || vo->dim() != 4) return status(-1);
    const int64_t blocks = vo->size(0), heads = vo->size(1), dims = vo->size(2), size = vo->size(3);
    pa_dtype code;
    int bs = 0;
    float ks = 0.f, vs = 0.f;
    void* stream = nullptr;
    if (!row_code(ko->scalar_type(), &code) || vo->scalar_type() != ko->scalar_type() || ko->size(0) != blocks ||
        ko->size(1) != heads || ko->size(2) != dims / 8 || ko->size(3) != size || ko->size(4) != 8 ||
        pairs->scalar_type() != at::kLong || pairs->dim() != 2 || pairs->size(1) != 2 || heads > kIntMax || !pools(*k, *v, heads, dims, &bs) || bs != size ||
        !as_float(a[5], &ks) || !as_float(a[6], &vs) || !as_stream(a[7], dev, &stream))
      return status(-1);
    pa_status st;
    void *kp = ko->data_ptr(), *vp = vo->data_ptr(), *kc = k->data_ptr(), *vc = v->data_ptr();
    const auto* sd = static_cast<const int64_t*>(pairs->data_ptr());
    Py_BEGIN_ALLOW_THREADS;
    st = g_expand(kp, vp, kc, vc, sd, pairs->size(0), static_cast<int>(heads), static_cast<int>(dims), bs, blocks,
                  k->size(0), code, ks, vs, stream);
    Py_END_ALLOW_THREADS;
    return status(st);
  } catch (...) {
    return status(-1);
  }
}

// decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale, max_seq_len, k_scale, v_scale, workspace, stream)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 12) return status(-1);
    const at::Tensor* q = tensor(a[1], -1);
    if (!q || q->dim() != 3) return status(-1);
    const int dev = q->get_device();
    if (dev != c10::cuda::current_device()) return status(-1);
    const at::Tensor *out = tensor(a[0], dev), *k = tensor(a[2], dev), *v = tensor(a[3], dev), *table = tensor(a[4], dev),
                     *lens = tensor(a[5], dev);
    if (!out || !k || !v || !table || !lens || k->dim() != 3) return status(-1);
    const int64_t S = q->size(0), H = q->size(1), dims = q->size(2), heads = k->size(1);
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[10] != Py_None) {
      const at::Tensor* w = tensor(a[10], dev);
      if (!w) return status(-1);
      ws = w->data_ptr();
      ws_bytes = w->nbytes();
    }
    pa_dtype code;
    int bs = 0;
    float scale = 0.f, ks = 0.f, vs = 0.f;
    void* stream = nullptr;
    const long max_len = PyLong_Check(a[7]) ? PyLong_AsLong(a[7]) : -1;
    if (max_len == -1 && PyErr_Occurred()) PyErr_Clear();
    if (max_len < 0 || max_len > kIntMax || !row_code(q->scalar_type(), &code) ||
        out->scalar_type() != q->scalar_type() || out->sizes() != q->sizes() || table->scalar_type() != at::kInt ||
        table->dim() != 2 || table->size(0) != S || table->size(1) > kIntMax || lens->scalar_type() != at::kInt ||
        lens->dim() != 1 || lens->size(0) != S || S > kIntMax || H > kIntMax || heads > kIntMax ||
        !pools(*k, *v, heads, dims, &bs) || !as_float(a[6], &scale) || !as_float(a[8], &ks) || !as_float(a[9], &vs) ||
        !as_stream(a[11], dev, &stream))
      return status(-1);
    pa_status st;
    void *op = out->data_ptr(), *qp = q->data_ptr(), *kc = k->data_ptr(), *vc = v->data_ptr();
    const auto* bt = static_cast<const int32_t*>(table->data_ptr());
    const auto* sl = static_cast<const int32_t*>(lens->data_ptr());
    Py_BEGIN_ALLOW_THREADS;
    st = g_decode(op, qp, kc, vc, bt, static_cast<int>(table->size(1)), sl, static_cast<int>(S),
                  static_cast<int>(max_len), static_cast<int>(H), static_cast<int>(heads), static_cast<int>(dims), bs,
                  k->size(0), scale, ws, ws_bytes, code, ks, vs, stream);
    Py_END_ALLOW_THREADS;
    return status(st);
  } catch (...) {
    return status(-1);
  }
}

// bind(write, gather, expand, decode): the entry points' addresses in the loaded library
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return status(-1);
  void* p[4];
  for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  g_write = reinterpret_cast<decltype(g_write)>(p[0]);
  g_gather = reinterpret_cast<decltype(g_gather)>(p[1]);
  g_expand = reinterpret_cast<decltype(g_expand)>(p[2]);
  g_decode = reinterpret_cast<decltype(g_decode)>(p[3]);
  return status(0);
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"rows", fast(rows), METH_FASTCALL, nullptr},
                         {"expand", fast(expand), METH_FASTCALL, nullptr},
                         {"decode", fast(decode), METH_FASTCALL, nullptr},
                         {"bind", fast(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp4_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp4_calls() { return PyModule_Create(&module); }
