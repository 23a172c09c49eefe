// fp4_calls.cpp -- the marshalling of the FP4, rotary and masked calls as a CPython extension.
//
// These calls on few tokens take 2 to 5 us on the GPU; checking five to ten tensors in
// Python and converting 14 to 25 arguments through ctypes takes longer than that (18 to 25 us
// measured for the rotary and masked calls).  This module
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
decltype(&pa_rope) g_rope;
decltype(&pa_rope_and_cache) g_rope_write;
decltype(&pa_decode_masked) g_decode_masked;
decltype(&pa_prefill_masked) g_prefill_masked;

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

// 16-bit, fp32 or FP8 pools: k [blocks, heads, dims / x, block size, x] and v [blocks, heads, dims, block size].
bool plain_pools(const at::Tensor& k, const at::Tensor& v, int64_t dims, pa_dtype* code) {
  const at::ScalarType t = k.scalar_type();
  if (t == at::kFloat8_e4m3fn) *code = PA_FP8_E4M3;
  else if (!row_code(t, code)) return false;
  if (v.scalar_type() != t || k.dim() != 5 || v.dim() != 4 || v.size(2) != dims) return false;
  const int64_t x = 16 / static_cast<int64_t>(k.element_size());
  return k.size(0) == v.size(0) && k.size(1) == v.size(1) && k.size(2) == dims / x && k.size(3) == v.size(3) &&
         k.size(4) == x && v.size(1) <= kIntMax && v.size(3) <= kIntMax;
}

bool as_int(PyObject* o, int* i) {
  if (!PyLong_Check(o)) return false;
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) PyErr_Clear();
  *i = static_cast<int>(x);
  return x >= 0 && x <= kIntMax;
}

// None, or a contiguous tensor of n elements of a type on the device; *p is its data.
bool maybe(PyObject* o, int dev, at::ScalarType type, int64_t n, const void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, dev);
  if (!t || t->scalar_type() != type || t->dim() != 1 || t->size(0) != n) return false;
  *p = t->data_ptr();
  return true;
}

// What decode and prefill share: q, out, pools, tables, lengths, cap, slopes, window, stream.
struct Masked {
  void *out, *q, *k, *v, *stream;
  const int32_t *table, *lens;
  const float* slopes;
  int width, seqs, rows, max_len, heads, kv_heads, dims, bs, window, dev;
  int64_t blocks;
  float scale, cap;
  pa_dtype code, cache;
};
bool masked_args(PyObject* out_o, PyObject* q_o, PyObject* k_o, PyObject* v_o, PyObject* table_o, PyObject* lens_o,
                 PyObject* scale_o, PyObject* max_o, PyObject* cap_o, PyObject* slopes_o, PyObject* window_o,
                 PyObject* stream_o, Masked* m) {
  const at::Tensor* q = tensor(q_o, -1);
  if (!q || q->dim() != 3) return false;
  const int dev = q->get_device();
  if (dev != c10::cuda::current_device()) return false;
  const at::Tensor *out = tensor(out_o, dev), *k = tensor(k_o, dev), *v = tensor(v_o, dev), *table = tensor(table_o, dev),
                   *lens = tensor(lens_o, dev);
  if (!out || !k || !v || !table || !lens || !row_code(q->scalar_type(), &m->code) ||
      out->scalar_type() != q->scalar_type() || out->sizes() != q->sizes() || !plain_pools(*k, *v, q->size(2), &m->cache) ||
      table->scalar_type() != at::kInt || table->dim() != 2 || lens->scalar_type() != at::kInt || lens->dim() != 1 ||
      table->size(0) != lens->size(0) || table->size(1) > kIntMax || lens->size(0) > kIntMax || q->size(0) > kIntMax ||
      q->size(1) > kIntMax || q->size(2) > kIntMax)
    return false;
  const void* slopes;
  if (!maybe(slopes_o, dev, at::kFloat, q->size(1), &slopes) || !as_float(scale_o, &m->scale) ||
      !as_float(cap_o, &m->cap) || !as_int(max_o, &m->max_len) || !as_int(window_o, &m->window) ||
      !as_stream(stream_o, dev, &m->stream))
    return false;
  m->out = out->data_ptr();
  m->q = q->data_ptr();
  m->k = k->data_ptr();
  m->v = v->data_ptr();
  m->table = static_cast<const int32_t*>(table->data_ptr());
  m->lens = static_cast<const int32_t*>(lens->data_ptr());
  m->slopes = static_cast<const float*>(slopes);
  m->width = static_cast<int>(table->size(1));
  m->seqs = static_cast<int>(lens->size(0));
  m->rows = static_cast<int>(q->size(0));
  m->heads = static_cast<int>(q->size(1));
  m->dims = static_cast<int>(q->size(2));
  m->kv_heads = static_cast<int>(v->size(1));
  m->bs = static_cast<int>(v->size(3));
  m->blocks = v->size(0);
  m->dev = dev;
  return true;
}

// decode_masked(out, q, k_cache, v_cache, block_tables, seq_lens, scale, max_seq_len, softcap, alibi_slopes, window,
//               k_scale, v_scale, workspace, stream)
PyObject* decode_masked(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    Masked m;
    float ks = 0.f, vs = 0.f;
    if (n != 15 || a[13] == Py_None ||
        !masked_args(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[14], &m) || m.rows != m.seqs ||
        !as_float(a[11], &ks) || !as_float(a[12], &vs))
      return status(-1);
    const at::Tensor* w = tensor(a[13], m.dev);
    if (!w) return status(-1);
    void* ws = w->data_ptr();
    const size_t ws_bytes = w->nbytes();
    pa_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_decode_masked(m.out, m.q, m.k, m.v, m.table, m.width, m.lens, m.seqs, m.max_len, m.heads, m.kv_heads, m.dims,
                         m.bs, m.blocks, m.scale, m.cap, m.slopes, m.window, ws, ws_bytes, m.code, m.cache, ks, vs,
                         m.stream);
    Py_END_ALLOW_THREADS;
    return status(st);
  } catch (...) {
    return status(-1);
  }
}

// prefill_masked(out, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, max_seq_len, softcap,
//                alibi_slopes, window, prefix_lens, stream)
PyObject* prefill_masked(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    Masked m;
    const void *starts = nullptr, *prefix = nullptr;
    if (n != 14 || a[6] == Py_None ||
        !masked_args(a[0], a[1], a[2], a[3], a[4], a[5], a[7], a[8], a[9], a[10], a[11], a[13], &m) ||
        m.cache != m.code || !maybe(a[6], m.dev, at::kInt, m.seqs + 1ll, &starts) ||
        !maybe(a[12], m.dev, at::kInt, m.seqs, &prefix))
      return status(-1);
    pa_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_prefill_masked(m.out, m.q, m.k, m.v, m.table, m.width, m.lens, static_cast<const int32_t*>(starts),
                          static_cast<const int32_t*>(prefix), m.seqs, m.rows, m.max_len, m.heads, m.kv_heads, m.dims,
                          m.bs, m.blocks, m.scale, m.cap, m.slopes, m.window, m.code, m.stream);
    Py_END_ALLOW_THREADS;
    return status(st);
  } catch (...) {
    return status(-1);
  }
}

// Rows [tokens, heads, dims] on the device, each token's contiguous; *stride: elements from one to the next.
const at::Tensor* token_rows(PyObject* o, int dev, int64_t* stride) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.dim() != 3 || (dev >= 0 && t.get_device() != dev)) return nullptr;
  const int64_t heads = t.size(1), dims = t.size(2);
  if ((dims > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != dims)) return nullptr;
  *stride = t.size(0) > 1 ? t.stride(0) : heads * dims;
  return &t;
}

// rope(q_out, key_out, q, key, value, k_cache, v_cache, positions, slot_mapping, inv_freq, layout, amplitude, k_scale,
//      v_scale, stream): with key_out None the write into the pools, else value, k_cache, v_cache and slot_mapping are None
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n != 15) return status(-1);
    int64_t sq = 0, sk = 0, sv = 0;
    const at::Tensor* q = token_rows(a[2], -1, &sq);
    if (!q) return status(-1);
    const int dev = q->get_device();
    if (dev != c10::cuda::current_device()) return status(-1);
    const at::Tensor *key = token_rows(a[3], dev, &sk), *q_out = tensor(a[0], dev), *f = tensor(a[9], dev);
    const int64_t T = q->size(0), heads = q->size(1), dims = q->size(2);
    pa_dtype code;
    int layout = 0;
    float amp = 0.f, ks = 0.f, vs = 0.f;
    void* stream = nullptr;
    const void *pos = nullptr, *slots = nullptr;
    if (!key || !q_out || !f || !row_code(q->scalar_type(), &code) || key->scalar_type() != q->scalar_type() ||
        key->size(0) != T || key->size(2) != dims || q_out->scalar_type() != q->scalar_type() ||
        q_out->sizes() != q->sizes() || f->scalar_type() != at::kDouble || f->dim() != 1 || f->size(0) > dims ||
        heads > kIntMax || key->size(1) > kIntMax || dims > kIntMax || a[7] == Py_None ||
        !maybe(a[7], dev, at::kLong, T, &pos) || !as_int(a[10], &layout) || !as_float(a[11], &amp) ||
        !as_float(a[12], &ks) || !as_float(a[13], &vs) || !as_stream(a[14], dev, &stream))
      return status(-1);
    const int64_t kv_heads = key->size(1);
    const int rotary = static_cast<int>(2 * f->size(0));
    void *qo = q_out->data_ptr(), *qp = q->data_ptr(), *kp = key->data_ptr();
    const auto* fp = static_cast<const double*>(f->data_ptr());
    const auto* pp = static_cast<const int64_t*>(pos);
    pa_status st;
    if (a[1] != Py_None) {
      const at::Tensor* key_out = tensor(a[1], dev);
      if (!key_out || key_out->scalar_type() != q->scalar_type() || key_out->sizes() != key->sizes()) return status(-1);
      void* ko = key_out->data_ptr();
      Py_BEGIN_ALLOW_THREADS;
      st = g_rope(qo, ko, qp, kp, sq, sk, pp, fp, T, static_cast<int>(heads), static_cast<int>(kv_heads),
                  static_cast<int>(dims), rotary, static_cast<pa_rope_layout>(layout), amp, code, stream);
      Py_END_ALLOW_THREADS;
      return status(st);
    }
    const at::Tensor *value = token_rows(a[4], dev, &sv), *k = tensor(a[5], dev), *v = tensor(a[6], dev);
    pa_dtype cache;
    if (!value || !k || !v || value->scalar_type() != q->scalar_type() || value->sizes() != key->sizes() ||
        !plain_pools(*k, *v, dims, &cache) || v->size(1) != kv_heads || a[8] == Py_None ||
        !maybe(a[8], dev, at::kLong, T, &slots))
      return status(-1);
    void *vp = value->data_ptr(), *kc = k->data_ptr(), *vc = v->data_ptr();
    const int bs = static_cast<int>(v->size(3));
    const int64_t blocks = v->size(0);
    Py_BEGIN_ALLOW_THREADS;
    st = g_rope_write(qo, qp, kp, vp, sq, sk, sv, kc, vc, pp, static_cast<const int64_t*>(slots), fp, T,
                      static_cast<int>(heads), static_cast<int>(kv_heads), static_cast<int>(dims), rotary, bs, blocks,
                      static_cast<pa_rope_layout>(layout), amp, code, cache, ks, vs, stream);
    Py_END_ALLOW_THREADS;
    return status(st);
  } catch (...) {
    return status(-1);
  }
}

// bind(write, gather, expand, decode, rope, rope_and_cache, decode_masked, prefill_masked): the entry points'
// addresses in the loaded library
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) return status(-1);
  void* p[8];
  for (int i = 0; i < 8; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  g_write = reinterpret_cast<decltype(g_write)>(p[0]);
  g_gather = reinterpret_cast<decltype(g_gather)>(p[1]);
  g_expand = reinterpret_cast<decltype(g_expand)>(p[2]);
  g_decode = reinterpret_cast<decltype(g_decode)>(p[3]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[4]);
  g_rope_write = reinterpret_cast<decltype(g_rope_write)>(p[5]);
  g_decode_masked = reinterpret_cast<decltype(g_decode_masked)>(p[6]);
  g_prefill_masked = reinterpret_cast<decltype(g_prefill_masked)>(p[7]);
  return status(0);
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"rows", fast(rows), METH_FASTCALL, nullptr},
                         {"expand", fast(expand), METH_FASTCALL, nullptr},
                         {"decode", fast(decode), METH_FASTCALL, nullptr},
                         {"rope", fast(rope), METH_FASTCALL, nullptr},
                         {"decode_masked", fast(decode_masked), METH_FASTCALL, nullptr},
                         {"prefill_masked", fast(prefill_masked), METH_FASTCALL, nullptr},
                         {"bind", fast(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp4_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp4_calls() { return PyModule_Create(&module); }
