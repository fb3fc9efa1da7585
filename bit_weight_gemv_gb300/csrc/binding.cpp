// Argument marshalling of the calls between the products (lowbit_kv_append,
// lowbit_paged_attention, lowbit_sample) from torch tensors to the C ABI.  These calls take eight to
// thirteen tensors and a kernel of a few microseconds; checked and unpacked in Python, the tensors
// cost more than the kernel (an append of one token: 10.9 us of host time a call, 3.8 from here;
// attention of one short request 12.0 against 6.0, sampling one row 9.5 against 8.4).  Same checks as the rest
// of the binding: TypeError or ValueError for what the library could not see (dtype, device,
// shape), the library's own status otherwise.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "../../include/lowbit.h"

namespace {

using at::ScalarType;
using at::Tensor;

decltype(&lowbit_kv_append) g_append;
decltype(&lowbit_paged_attention) g_attention;
decltype(&lowbit_sample) g_sample;

bool fail(PyObject* kind, const char* name, const char* what) {
  PyErr_Format(kind, "%s %s", name, what);
  return false;
}
bool tensor(PyObject* o, ScalarType type, const char* name, const Tensor** t) {
  if (!THPVariable_Check(o)) return fail(PyExc_TypeError, name, "must be a torch tensor");
  *t = &THPVariable_Unpack(o);
  if ((*t)->scalar_type() != type || !(*t)->is_cuda()) return fail(PyExc_TypeError, name, "must be a CUDA tensor of its declared dtype");
  return true;
}
// A dense tensor of `count` values; None gives a null pointer when `optional`.
template <class T>
bool dense(PyObject* o, ScalarType type, int64_t count, const char* name, bool optional, T** at) {
  *at = nullptr;
  if (o == Py_None && optional) return true;
  const Tensor* t;
  if (!tensor(o, type, name, &t)) return false;
  if (!t->is_contiguous()) return fail(PyExc_TypeError, name, "must be contiguous");
  if (count >= 0 && t->numel() != count) return fail(PyExc_ValueError, name, "has the wrong number of values");
  *at = static_cast<T*>(t->data_ptr());
  return true;
}
// bf16 [T][heads][dim] whose rows may be apart (a slice of a wider product).
struct Rows {
  uint16_t* at;
  int64_t T, heads, stride;
};
bool rows(PyObject* o, int64_t dim, const char* name, Rows* r) {
  const Tensor* t;
  if (!tensor(o, ScalarType::BFloat16, name, &t)) return false;
  if (t->dim() != 3 || t->size(2) != dim) return fail(PyExc_ValueError, name, "must have shape [T][heads][head_dim]");
  r->at = static_cast<uint16_t*>(t->data_ptr());
  r->T = t->size(0), r->heads = t->size(1), r->stride = t->stride(0);
  const int64_t dense_row = r->heads * dim;
  if (r->T <= 1 && (r->stride < dense_row || r->stride % 8)) r->stride = dense_row;
  if (r->stride < dense_row || t->stride(2) != 1 || (r->heads > 1 && t->stride(1) != dim))
    return fail(PyExc_ValueError, name, "must have dense heads within a row");
  return true;
}
bool batch(PyObject* cu_q, PyObject* kv_lens, PyObject* table, int64_t T, lowbit_paged_batch* b) {
  const Tensor *lens, *t;
  if (!tensor(kv_lens, ScalarType::Int, "kv_lens", &lens) || !tensor(table, ScalarType::Int, "block_table", &t)) return false;
  if (!lens->is_contiguous()) return fail(PyExc_TypeError, "kv_lens", "must be contiguous");
  const int64_t B = lens->numel();
  const int32_t* cu;
  if (!dense(cu_q, ScalarType::Int, B + 1, "cu_q [requests + 1]", false, &cu)) return false;
  if (t->dim() != 2 || t->size(0) != B || (t->size(1) > 1 && t->stride(1) != 1))
    return fail(PyExc_ValueError, "block_table", "must have shape [requests][pages] with dense rows");
  if (B > INT32_MAX || T > INT32_MAX || t->size(1) > INT32_MAX) return fail(PyExc_ValueError, "the batch", "is too large");
  const int64_t width = t->size(1);
  *b = lowbit_paged_batch{cu, static_cast<const int32_t*>(lens->data_ptr()), static_cast<const int32_t*>(t->data_ptr()),
                          B > 1 ? t->stride(0) : std::max(t->stride(0), width), (int)B, (int)T, (int)width};
  return true;
}
// Addresses (the cache's struct, a stream) come as Python integers.
bool address(PyObject* o, void** p) {
  *p = PyLong_AsVoidPtr(o);
  return !PyErr_Occurred();
}
// A stream's handle; None is torch's current stream.  Asked for after the other arguments' checks,
// which need no GPU.
bool stream_of(PyObject* o, void** s) {
  if (o != Py_None) return address(o, s);
  *s = c10::cuda::getCurrentCUDAStream().stream();
  return true;
}
bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
  return false;
}

// q, k, v, rope, cu_q, kv_lens, block_table, cache, q_out, interleaved, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void *cache_at, *stream;
  if (!count_is(n, 11) || !address(a[7], &cache_at)) return nullptr;
  const lowbit_paged_cache* cache = static_cast<const lowbit_paged_cache*>(cache_at);
  const int64_t D = cache->head_dim;
  Rows q = {nullptr, 0, 0, 0}, k, v;
  if (!rows(a[1], D, "k", &k) || !rows(a[2], D, "v", &v)) return nullptr;
  if (v.T != k.T || k.heads != cache->heads || v.heads != k.heads)
    return fail(PyExc_ValueError, "k and v", "must have the same rows and the cache's heads"), nullptr;
  uint16_t* q_out = nullptr;
  if ((a[0] == Py_None) != (a[8] == Py_None)) return fail(PyExc_ValueError, "q and q_out", "go together"), nullptr;
  if (a[0] != Py_None) {
    if (!rows(a[0], D, "q", &q) || !dense(a[8], ScalarType::BFloat16, k.T * q.heads * D, "q_out", false, &q_out)) return nullptr;
    if (q.T != k.T) return fail(PyExc_ValueError, "q", "must have k's rows"), nullptr;
  }
  const float* rope = nullptr;
  int64_t positions = 0, rot = 0;
  if (a[3] != Py_None) {
    if (!dense(a[3], ScalarType::Float, -1, "rope", false, &rope)) return nullptr;
    const Tensor& t = THPVariable_Unpack(a[3]);
    if (t.dim() != 2) return fail(PyExc_ValueError, "rope", "must have shape [positions][rot]"), nullptr;
    positions = std::min<int64_t>(t.size(0), INT32_MAX), rot = std::min<int64_t>(t.size(1), INT32_MAX);
  }
  const int interleaved = PyObject_IsTrue(a[9]);
  lowbit_paged_batch b;
  if (interleaved < 0 || !batch(a[4], a[5], a[6], k.T, &b) || !stream_of(a[10], &stream)) return nullptr;
  return PyLong_FromLong(g_append(q.at, q.stride, k.at, k.stride, v.at, v.stride, (int)q.heads, rope, (int)positions,
                                  (int)rot, interleaved, &b, cache, q_out, stream));
}

// q, cache, cu_q, kv_lens, block_table, out, workspace, scale, causal, window, lse, stream
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void *cache_at, *stream;
  if (!count_is(n, 12) || !address(a[1], &cache_at)) return nullptr;
  const lowbit_paged_cache* cache = static_cast<const lowbit_paged_cache*>(cache_at);
  Rows q;
  if (!rows(a[0], cache->head_dim, "q", &q)) return nullptr;
  uint16_t* out;
  float* lse;
  void* workspace;
  if (!dense(a[5], ScalarType::BFloat16, q.T * q.heads * cache->head_dim, "out", false, &out) ||
      !dense(a[6], ScalarType::Byte, -1, "workspace", false, &workspace) ||
      !dense(a[10], ScalarType::Float, q.T * q.heads, "lse", true, &lse))
    return nullptr;
  const double scale = PyFloat_AsDouble(a[7]);
  const int causal = PyObject_IsTrue(a[8]);
  const long window = PyLong_AsLong(a[9]);
  lowbit_paged_batch b;
  if (PyErr_Occurred() || causal < 0 || !batch(a[2], a[3], a[4], q.T, &b)) return nullptr;
  if (window < INT32_MIN || window > INT32_MAX) return fail(PyExc_ValueError, "window", "is out of range"), nullptr;
  if (!stream_of(a[11], &stream)) return nullptr;
  return PyLong_FromLong(g_attention(q.at, q.stride, (int)q.heads, &b, cache, (float)scale, causal, (int)window, out, lse,
                                     workspace, (size_t)THPVariable_Unpack(a[6]).numel(), stream));
}

// logits, u, ids, temperature, top_k, top_p, min_p, id_map, logprob, kept, stream
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* stream;
  if (!count_is(n, 11)) return nullptr;
  if (!THPVariable_Check(a[0])) return fail(PyExc_TypeError, "logits", "must be a torch tensor"), nullptr;
  const Tensor& z = THPVariable_Unpack(a[0]);
  const bool bf16 = z.scalar_type() == ScalarType::BFloat16;
  if (!z.is_cuda() || z.dim() != 2 || (!bf16 && z.scalar_type() != ScalarType::Float))
    return fail(PyExc_TypeError, "logits", "must be an fp32 or bf16 CUDA tensor [M][V]"), nullptr;
  const int64_t M = z.size(0), V = z.size(1);
  if ((V > 1 && z.stride(1) != 1) || M > INT32_MAX || V > INT32_MAX)
    return fail(PyExc_ValueError, "logits", "must have dense rows"), nullptr;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t *top_k, *id_map;
  int32_t *ids, *kept;
  float* logprob;
  const ScalarType f = ScalarType::Float, i = ScalarType::Int;
  if (!dense(a[1], f, M, "u", false, &u) || !dense(a[2], i, M, "ids", false, &ids) ||
      !dense(a[3], f, M, "temperature", true, &temperature) || !dense(a[4], i, M, "top_k", true, &top_k) ||
      !dense(a[5], f, M, "top_p", true, &top_p) || !dense(a[6], f, M, "min_p", true, &min_p) ||
      !dense(a[7], i, V, "id_map", true, &id_map) || !dense(a[8], f, M, "logprob", true, &logprob) ||
      !dense(a[9], i, M, "kept", true, &kept) || !stream_of(a[10], &stream))
    return nullptr;
  return PyLong_FromLong(g_sample(z.data_ptr(), bf16 ? LOWBIT_LOGITS_BF16 : LOWBIT_LOGITS_FP32,
                                  M > 1 ? z.stride(0) : std::max(z.stride(0), V), (int)M, (int)V, temperature, top_k,
                                  top_p, min_p, u, id_map, ids, logprob, kept, stream));
}

// The handle of torch's current stream, without a Stream object around it.
PyObject* current_stream(PyObject*, PyObject* const*, Py_ssize_t n) {
  void* stream;
  return count_is(n, 0) && stream_of(Py_None, &stream) ? PyLong_FromVoidPtr(stream) : nullptr;
}

// The three entry points' addresses in the loaded library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[3];
  if (!count_is(n, 3)) return nullptr;
  for (int i = 0; i < 3; ++i)
    if (!address(a[i], &p[i])) return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(p[0]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[1]);
  g_sample = reinterpret_cast<decltype(g_sample)>(p[2]);
  Py_RETURN_NONE;
}

// No C++ exception leaves a call (torch's accessors may throw).
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>));
}

PyMethodDef kMethods[] = {{"bind", entry<bind>(), METH_FASTCALL, nullptr},
                          {"current_stream", entry<current_stream>(), METH_FASTCALL, nullptr},
                          {"kv_append", entry<kv_append>(), METH_FASTCALL, nullptr},
                          {"paged_attention", entry<paged_attention>(), METH_FASTCALL, nullptr},
                          {"sample", entry<sample>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
