// Argument marshalling of the calls between the products (appends, attention, sampling, verification of
// drafts) from torch tensors to the C ABI.  These calls take eight to
// twenty tensors and a kernel of a few microseconds; checked and unpacked in Python, the tensors
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
decltype(&lowbit_kv_append_norm) g_append_norm;
decltype(&lowbit_paged_attention) g_attention;
decltype(&lowbit_sample) g_sample;
decltype(&lowbit_prefix_attention) g_prefix;
decltype(&lowbit_verify_drafts) g_verify;

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

// What both append calls take: q, k, v and, from `rest` on, rope, cu_q, kv_lens, block_table, cache, q_out,
// interleaved, stream.
struct Append {
  Rows q = {nullptr, 0, 0, 0}, k, v;
  const float* rope = nullptr;
  int64_t positions = 0, rot = 0;
  lowbit_paged_batch b;
  const lowbit_paged_cache* cache;
  uint16_t* q_out = nullptr;
  int interleaved;
  void* stream;
};
bool append_args(PyObject* const* a, PyObject* const* rest, Append* s) {
  void* cache_at;
  if (!address(rest[4], &cache_at)) return false;
  s->cache = static_cast<const lowbit_paged_cache*>(cache_at);
  const int64_t D = s->cache->head_dim;
  if (!rows(a[1], D, "k", &s->k) || !rows(a[2], D, "v", &s->v)) return false;
  if (s->v.T != s->k.T || s->k.heads != s->cache->heads || s->v.heads != s->k.heads)
    return fail(PyExc_ValueError, "k and v", "must have the same rows and the cache's heads");
  if ((a[0] == Py_None) != (rest[5] == Py_None)) return fail(PyExc_ValueError, "q and q_out", "go together");
  if (a[0] != Py_None) {
    if (!rows(a[0], D, "q", &s->q) || !dense(rest[5], ScalarType::BFloat16, s->k.T * s->q.heads * D, "q_out", false, &s->q_out))
      return false;
    if (s->q.T != s->k.T) return fail(PyExc_ValueError, "q", "must have k's rows");
  }
  if (rest[0] != Py_None) {
    if (!dense(rest[0], ScalarType::Float, -1, "rope", false, &s->rope)) return false;
    const Tensor& t = THPVariable_Unpack(rest[0]);
    if (t.dim() != 2) return fail(PyExc_ValueError, "rope", "must have shape [positions][rot]");
    s->positions = std::min<int64_t>(t.size(0), INT32_MAX), s->rot = std::min<int64_t>(t.size(1), INT32_MAX);
  }
  s->interleaved = PyObject_IsTrue(rest[6]);
  return s->interleaved >= 0 && batch(rest[1], rest[2], rest[3], s->k.T, &s->b) && stream_of(rest[7], &s->stream);
}

// q, k, v, rope, cu_q, kv_lens, block_table, cache, q_out, interleaved, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Append s;
  if (!count_is(n, 11) || !append_args(a, a + 3, &s)) return nullptr;
  return PyLong_FromLong(g_append(s.q.at, s.q.stride, s.k.at, s.k.stride, s.v.at, s.v.stride, (int)s.q.heads, s.rope,
                                  (int)s.positions, (int)s.rot, s.interleaved, &s.b, s.cache, s.q_out, s.stream));
}

// q, k, v, q_weight, k_weight, eps, rope, cu_q, kv_lens, block_table, cache, q_out, interleaved, stream
PyObject* kv_append_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Append s;
  const float *q_weight, *k_weight;
  if (!count_is(n, 14)) return nullptr;
  const double eps = PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred() || !append_args(a, a + 6, &s) ||
      !dense(a[3], ScalarType::Float, s.cache->head_dim, "q_weight", true, &q_weight) ||
      !dense(a[4], ScalarType::Float, s.cache->head_dim, "k_weight", true, &k_weight))
    return nullptr;
  return PyLong_FromLong(g_append_norm(s.q.at, s.q.stride, s.k.at, s.k.stride, s.v.at, s.v.stride, (int)s.q.heads,
                                       q_weight, k_weight, (float)eps, s.rope, (int)s.positions, (int)s.rot,
                                       s.interleaved, &s.b, s.cache, s.q_out, s.stream));
}

// What both attention calls take: q, cache, cu_q, kv_lens, block_table, and the rest by name.
struct Attention {
  Rows q;
  lowbit_paged_batch b;
  const lowbit_paged_cache* cache;
  uint16_t* out;
  float* lse;
  void* workspace;
  size_t bytes;
  double scale;
  int causal;
};
bool attention_args(PyObject* const* a, PyObject* out, PyObject* workspace, PyObject* scale, PyObject* causal,
                    PyObject* lse, Attention* s) {
  void* cache_at;
  if (!address(a[1], &cache_at)) return false;
  s->cache = static_cast<const lowbit_paged_cache*>(cache_at);
  const int64_t D = s->cache->head_dim;
  if (!rows(a[0], D, "q", &s->q)) return false;
  if (!dense(out, ScalarType::BFloat16, s->q.T * s->q.heads * D, "out", false, &s->out) ||
      !dense(workspace, ScalarType::Byte, -1, "workspace", false, &s->workspace) ||
      !dense(lse, ScalarType::Float, s->q.T * s->q.heads, "lse", true, &s->lse))
    return false;
  s->bytes = (size_t)THPVariable_Unpack(workspace).numel();
  s->scale = PyFloat_AsDouble(scale);
  s->causal = PyObject_IsTrue(causal);
  return !PyErr_Occurred() && s->causal >= 0 && batch(a[2], a[3], a[4], s->q.T, &s->b);
}

// q, cache, cu_q, kv_lens, block_table, out, workspace, scale, causal, window, lse, stream
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Attention s;
  void* stream;
  if (!count_is(n, 12) || !attention_args(a, a[5], a[6], a[7], a[8], a[10], &s)) return nullptr;
  const long window = PyLong_AsLong(a[9]);
  if (PyErr_Occurred()) return nullptr;
  if (window < INT32_MIN || window > INT32_MAX) return fail(PyExc_ValueError, "window", "is out of range"), nullptr;
  if (!stream_of(a[11], &stream)) return nullptr;
  return PyLong_FromLong(g_attention(s.q.at, s.q.stride, (int)s.q.heads, &s.b, s.cache, (float)s.scale, s.causal,
                                     (int)window, s.out, s.lse, s.workspace, s.bytes, stream));
}

// q, cache, cu_q, kv_lens, block_table, cu_groups, prefix_lens, out, workspace, scale, causal, lse, stream
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Attention s;
  void* stream;
  const Tensor* lens;
  const int32_t *cu_groups, *prefix_lens;
  if (!count_is(n, 13) || !attention_args(a, a[7], a[8], a[9], a[10], a[11], &s) ||
      !tensor(a[6], ScalarType::Int, "prefix_lens", &lens) ||
      !dense(a[6], ScalarType::Int, -1, "prefix_lens", false, &prefix_lens) ||
      !dense(a[5], ScalarType::Int, lens->numel() + 1, "cu_groups [groups + 1]", false, &cu_groups))
    return nullptr;
  if (lens->numel() > INT32_MAX) return fail(PyExc_ValueError, "prefix_lens", "has too many values"), nullptr;
  if (!stream_of(a[12], &stream)) return nullptr;
  return PyLong_FromLong(g_prefix(s.q.at, s.q.stride, (int)s.q.heads, &s.b, s.cache, cu_groups, prefix_lens,
                                  (int)lens->numel(), (float)s.scale, s.causal, s.out, s.lse, s.workspace, s.bytes, stream));
}

// fp32 or bf16 logits [M][V] with dense rows.
struct Logits {
  void* at;
  int64_t M, V, stride;
  int dtype;
};
bool logits_of(PyObject* o, const char* name, Logits* l) {
  if (!THPVariable_Check(o)) return fail(PyExc_TypeError, name, "must be a torch tensor");
  const Tensor& z = THPVariable_Unpack(o);
  const bool bf16 = z.scalar_type() == ScalarType::BFloat16;
  if (!z.is_cuda() || z.dim() != 2 || (!bf16 && z.scalar_type() != ScalarType::Float))
    return fail(PyExc_TypeError, name, "must be an fp32 or bf16 CUDA tensor [M][V]");
  l->M = z.size(0), l->V = z.size(1);
  if ((l->V > 1 && z.stride(1) != 1) || l->M > INT32_MAX || l->V > INT32_MAX) return fail(PyExc_ValueError, name, "must have dense rows");
  l->at = z.data_ptr();
  l->stride = l->M > 1 ? z.stride(0) : std::max(z.stride(0), l->V);
  l->dtype = bf16 ? LOWBIT_LOGITS_BF16 : LOWBIT_LOGITS_FP32;
  return true;
}

// logits, u, ids, temperature, top_k, top_p, min_p, id_map, logprob, kept, stream
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* stream;
  if (!count_is(n, 11)) return nullptr;
  Logits z;
  if (!logits_of(a[0], "logits", &z)) return nullptr;
  const int64_t M = z.M, V = z.V;
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
  return PyLong_FromLong(g_sample(z.at, z.dtype, z.stride, (int)M, (int)V, temperature, top_k, top_p, min_p, u, id_map,
                                  ids, logprob, kept, stream));
}

// A row's settings, one per request: a[0..3] temperature, top_k, top_p, min_p.
bool settings_of(PyObject* const* a, const Logits& z, int64_t B, lowbit_row_settings* r) {
  const ScalarType f = ScalarType::Float;
  *r = lowbit_row_settings{z.at, z.stride, z.dtype, (int)z.M, (int)z.V, nullptr, nullptr, nullptr, nullptr};
  return dense(a[0], f, B, "temperature", true, &r->temperature) && dense(a[1], ScalarType::Int, B, "top_k", true, &r->top_k) &&
         dense(a[2], f, B, "top_p", true, &r->top_p) && dense(a[3], f, B, "min_p", true, &r->min_p);
}

// logits, cu_drafts, drafts, u, v, n_accept, ids, workspace, draft_logits, draft_index, then temperature, top_k,
// top_p, min_p of the target and of the drafter, accept, stream
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 20)) return nullptr;
  Logits z, y = {nullptr, 0, 0, 0, 0};
  const Tensor *last, *tokens;
  if (!logits_of(a[0], "logits", &z) || !tensor(a[4], ScalarType::Float, "v", &last) || !tensor(a[2], ScalarType::Int, "drafts", &tokens)) return nullptr;
  const int64_t B = last->numel(), N = tokens->numel();
  if (B > INT32_MAX || N > INT32_MAX) return fail(PyExc_ValueError, "the batch", "is too large"), nullptr;
  const ScalarType f = ScalarType::Float, i = ScalarType::Int;
  const int32_t *cu, *drafts, *index;
  const float *u, *v;
  int32_t *n_accept, *ids;
  float* accept;
  void *workspace, *stream;
  lowbit_row_settings target, draft;
  const bool has_draft = a[8] != Py_None;
  if (!dense(a[1], i, B + 1, "cu_drafts [requests + 1]", false, &cu) || !dense(a[2], i, N, "drafts", false, &drafts) ||
      !dense(a[3], f, N, "u", false, &u) || !dense(a[4], f, B, "v", false, &v) ||
      !dense(a[5], i, B, "n_accept", false, &n_accept) || !dense(a[6], i, z.M, "ids", false, &ids) ||
      !dense(a[7], ScalarType::Byte, -1, "workspace", false, &workspace) || !dense(a[18], f, N, "accept", true, &accept) ||
      !settings_of(a + 10, z, B, &target))
    return nullptr;
  if (has_draft) {
    if (!logits_of(a[8], "draft_logits", &y) || !settings_of(a + 14, y, B, &draft)) return nullptr;
    if (y.M != N) return fail(PyExc_ValueError, "draft_logits", "must have a row for every draft"), nullptr;
  } else {
    for (int k = 14; k < 18; ++k)
      if (a[k] != Py_None) return fail(PyExc_ValueError, "the drafter's settings", "need draft_logits"), nullptr;
  }
  if (!dense(a[9], i, z.V, "draft_index", true, &index) || !stream_of(a[19], &stream)) return nullptr;
  return PyLong_FromLong(g_verify(&target, has_draft ? &draft : nullptr, (int)B, (int)N, cu, drafts, index, u, v, n_accept, ids,
                                  accept, workspace, (size_t)THPVariable_Unpack(a[7]).numel(), stream));
}

// The handle of torch's current stream, without a Stream object around it.
PyObject* current_stream(PyObject*, PyObject* const*, Py_ssize_t n) {
  void* stream;
  return count_is(n, 0) && stream_of(Py_None, &stream) ? PyLong_FromVoidPtr(stream) : nullptr;
}

// The entry points' addresses in the loaded library.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6];
  if (!count_is(n, 6)) return nullptr;
  for (int i = 0; i < 6; ++i)
    if (!address(a[i], &p[i])) return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(p[0]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[1]);
  g_sample = reinterpret_cast<decltype(g_sample)>(p[2]);
  g_append_norm = reinterpret_cast<decltype(g_append_norm)>(p[3]);
  g_prefix = reinterpret_cast<decltype(g_prefix)>(p[4]);
  g_verify = reinterpret_cast<decltype(g_verify)>(p[5]);
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
                          {"kv_append_norm", entry<kv_append_norm>(), METH_FASTCALL, nullptr},
                          {"paged_attention", entry<paged_attention>(), METH_FASTCALL, nullptr},
                          {"prefix_attention", entry<prefix_attention>(), METH_FASTCALL, nullptr},
                          {"sample", entry<sample>(), METH_FASTCALL, nullptr},
                          {"verify_drafts", entry<verify_drafts>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
