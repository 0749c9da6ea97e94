// Compiled argument marshalling of the calls around the layer: torch tensors
// in, pw_rows and device pointers out, then the C ABI of include/pw.h.
//
// These calls run for a few microseconds in a decode step; reading every
// tensor's shape, strides and address from Python and converting each argument
// took 8 to 11 us of host time a call, this takes 0.2 to 0.5 beside the launch.
// Shape, type and device errors become ValueError; the pw_status is returned.
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pw.h"

namespace pw {
bool host_sim();  // libpw.so: no kernel runs
}

namespace {

struct Bad {};  // a Python error is set

[[noreturn]] void fail(const char* what, const char* why) {
  PyErr_Format(PyExc_ValueError, "%s: %s", what, why);
  throw Bad();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) fail(what, "must be a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Bad();
  return v;
}

int small(PyObject* o, const char* what) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) fail(what, "out of range");
  return (int)v;
}

// A size that the C ABI takes in 32 bits; larger ones would arrive as others.
int size32(int64_t n, const char* what) {
  if (n > INT32_MAX) fail(what, "too large");
  return (int)n;
}

int dtype_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kHalf) return PW_F16;
  if (t.scalar_type() == at::kBFloat16) return PW_BF16;
  fail(what, "heads are float16 or bfloat16");
}

// The tensor that a call's others are compared with is on a GPU (a host address would reach a kernel as it is).
void on_gpu(const at::Tensor& t, const char* what) {
  if (!t.is_cuda() && !pw::host_sim()) fail(what, "must be on a GPU");
}

// [T][H][D] head rows of the type and on the device of `like`.
pw_rows rows(const at::Tensor& t, int64_t T, int64_t H, int64_t D, const at::Tensor& like, const char* what) {
  if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != D) fail(what, "wrong shape");
  if (t.scalar_type() != like.scalar_type()) fail(what, "wrong type");
  if (t.device() != like.device()) fail(what, "on another device");
  if (t.stride(2) != 1) fail(what, "a head's values must be contiguous");
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

// Address of a contiguous tensor of a given shape and type (n1 < 0: one dimension).
template <typename T>
T* vec(PyObject* o, at::ScalarType type, const at::Tensor& like, const char* what, int64_t n0, int64_t n1 = -1,
       int64_t n2 = -1) {
  const at::Tensor* t = maybe(o, what);
  if (!t) return nullptr;
  const int dims = n1 < 0 ? 1 : n2 < 0 ? 2 : 3;
  if (t->dim() != dims || t->size(0) != n0 || (dims > 1 && t->size(1) != n1) || (dims > 2 && t->size(2) != n2))
    fail(what, "wrong shape");
  if (t->scalar_type() != type) fail(what, type == at::kInt ? "must be int32" : "must be float32");
  if (t->device() != like.device()) fail(what, "on another device");
  if (!t->is_contiguous()) fail(what, "must be contiguous");
  return static_cast<T*>(t->data_ptr());
}

// The stream argument: None (the tensors' device's current one), a raw handle, or an object with .cuda_stream.
void* stream(PyObject* o, const at::Tensor& like) {
  if (o == Py_None) return like.is_cuda() ? c10::cuda::getCurrentCUDAStream(like.get_device()).stream() : nullptr;
  PyObject* a = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!a) throw Bad();
  void* p = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (!p && PyErr_Occurred()) throw Bad();  // before the call, which would run on the null stream
  return p;
}

// A Rotary as (address of its pw_rotary, type of its weights or -1, their length, one of its tensors or None).
const pw_rotary* rotary(PyObject* o, int dtype, int64_t D, const at::Tensor& like) {
  if (o == Py_None) return nullptr;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) fail("rotary", "must be a Rotary's key");
  const at::Tensor* some = maybe(PyTuple_GET_ITEM(o, 3), "rotary");
  if (some && some->device() != like.device()) fail("rotary", "on another device");
  const long long type = integer(PyTuple_GET_ITEM(o, 1));
  if (type >= 0 && (type != dtype || integer(PyTuple_GET_ITEM(o, 2)) != D))
    fail("rotary", "norm weights must be [head_dim] of the heads' type");
  return static_cast<const pw_rotary*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)));
}

template <pw_status (*F)(PyObject* const*)>
PyObject* call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    const long st = F(a);
    return PyErr_Occurred() ? nullptr : PyLong_FromLong(st);
  } catch (const Bad&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (cache k): whether a cache may be made of it.
pw_status check_cache(PyObject* const* a) {
  on_gpu(tensor(a[0], "k"), "k");
  return PW_OK;
}

// (rotary, q, k, positions, q_out, k_out, err, stream)
pw_status rope(PyObject* const* a) {
  const at::Tensor *q = maybe(a[1], "q"), *k = maybe(a[2], "k");
  const at::Tensor* some = q ? q : k;
  if (!some || some->dim() != 3 || (k && k->dim() != 3)) fail("q", "q or k must be [T, heads, head_dim]");
  on_gpu(*some, q ? "q" : "k");
  const int64_t T = some->size(0), D = some->size(2);
  const pw_heads heads = {dtype_of(*some, "q"), size32(some->size(1), "q"), size32((k ? k : q)->size(1), "k"), size32(D, "q")};
  const pw_rotary* r = rotary(a[0], heads.dtype, D, *some);
  pw_rows rq = {}, rk = {}, rqo = {}, rko = {};
  if (q) rq = rows(*q, T, heads.n_heads, D, *some, "q"), rqo = rows(tensor(a[4], "q_out"), T, heads.n_heads, D, *some, "q_out");
  if (k) rk = rows(*k, T, heads.n_kv_heads, D, *some, "k"), rko = rows(tensor(a[5], "k_out"), T, heads.n_kv_heads, D, *some, "k_out");
  return pw_qk_norm_rope(&heads, r, vec<const int32_t>(a[3], at::kInt, *some, "positions", T), size32(T, "q"), &rq, &rk, &rqo, &rko,
                         vec<int32_t>(a[6], at::kInt, *some, "err", 1), stream(a[7], *some));
}

// The cache's keys [pages][key heads][tokens][D] come with its calls: the library reads head rows by the handle's type, so
// every tensor of a call is held against the cache's own type and device here.

// (handle, cache k, n_heads, k, v, slots, rotary, positions, q, q_out, stream)
pw_status append(PyObject* const* a) {
  auto* kv = static_cast<pw_kv_t>(PyLong_AsVoidPtr(a[0]));
  const at::Tensor& cache = tensor(a[1], "cache");
  on_gpu(cache, "cache");
  const int64_t hq = integer(a[2]), hk = cache.size(1), D = cache.size(3);
  const at::Tensor &k = tensor(a[3], "k"), &v = tensor(a[4], "v");
  const int64_t T = k.dim() == 3 ? k.size(0) : -1;
  const pw_rows rk = rows(k, T, hk, D, cache, "k"), rv = rows(v, T, hk, D, cache, "v");
  const pw_rotary* r = rotary(a[6], dtype_of(cache, "cache"), D, cache);
  const at::Tensor* q = maybe(a[8], "q");
  pw_rows rq = {}, rqo = {};
  if (!q && a[9] != Py_None) fail("q_out", "needs q");
  if (q) rq = rows(*q, T, hq, D, cache, "q"), rqo = rows(tensor(a[9], "q_out"), T, hq, D, cache, "q_out");
  return pw_kv_append(kv, r, vec<const int32_t>(a[7], at::kInt, cache, "positions", T),
                      vec<const int32_t>(a[5], at::kInt, cache, "slots", T), size32(T, "k"), &rk, &rv, &rq, &rqo,
                      stream(a[10], cache));
}

// (handle, cache k, n_heads, q, table, lens, out, ws, q_len, scale, prefix_table, prefix_lens, group_offsets, lse, stream)
pw_status attend(PyObject* const* a) {
  auto* kv = static_cast<pw_kv_t>(PyLong_AsVoidPtr(a[0]));
  const at::Tensor& cache = tensor(a[1], "cache");
  on_gpu(cache, "cache");
  const int64_t hq = integer(a[2]), D = cache.size(3);
  const at::Tensor &q = tensor(a[3], "q"), &table = tensor(a[4], "table"), &out = tensor(a[6], "out");
  if (table.dim() != 2) fail("table", "must be [batch, pages]");
  pw_attend_desc d = {};
  const int64_t B = table.size(0);
  d.batch = size32(B, "table");
  d.q_len = small(a[8], "q_len");
  d.q = rows(q, B * d.q_len, hq, D, cache, "q");
  d.out = rows(out, B * d.q_len, hq, D, cache, "out");
  d.lse = vec<float>(a[13], at::kFloat, cache, "lse", B * d.q_len, hq);
  d.scale = (float)PyFloat_AsDouble(a[9]);
  if (PyErr_Occurred()) throw Bad();
  d.table_stride = size32(table.size(1), "table");
  d.table = vec<const int32_t>(a[4], at::kInt, cache, "table", B, d.table_stride);
  d.lens = vec<const int32_t>(a[5], at::kInt, cache, "lens", B);
  // a prefix left out by mistake would still give an answer, without it
  if ((a[10] == Py_None) != (a[11] == Py_None)) fail("prefix_table, prefix_lens", "both or neither");
  if (a[11] == Py_None && a[12] != Py_None) fail("group_offsets", "needs prefix_table and prefix_lens");
  if (a[11] != Py_None) {
    const at::Tensor& pt = tensor(a[10], "prefix_table");
    if (pt.dim() != 2) fail("prefix_table", "must be [groups, pages]");
    d.n_groups = size32(pt.size(0), "prefix_table");
    d.prefix_stride = size32(pt.size(1), "prefix_table");
    d.prefix_table = vec<const int32_t>(a[10], at::kInt, cache, "prefix_table", d.n_groups, d.prefix_stride);
    d.prefix_lens = vec<const int32_t>(a[11], at::kInt, cache, "prefix_lens", d.n_groups);
    d.group_offsets = vec<const int32_t>(a[12], at::kInt, cache, "group_offsets", d.n_groups + 1);
  }
  const at::Tensor* ws = maybe(a[7], "ws");
  if (ws && ws->device() != cache.device()) fail("ws", "on another device");
  if (ws && !ws->is_contiguous()) fail("ws", "must be contiguous");  // else it has fewer bytes than its sizes say
  return pw_kv_attend(kv, &d, ws ? ws->data_ptr() : nullptr, ws ? ws->nbytes() : 0, stream(a[14], cache));
}

// (target_p, draft_p, tokens, n_draft, u, noise, out, accepted, err, stream)
pw_status verify(PyObject* const* a) {
  const at::Tensor& p = tensor(a[0], "target_p");
  if (p.dim() != 3) fail("target_p", "must be [B, K + 1, V]");
  on_gpu(p, "target_p");
  const int64_t B = p.size(0), K = p.size(1) - 1, V = p.size(2);
  if (B > INT32_MAX || K > INT32_MAX || V > INT32_MAX) fail("target_p", "too large");
  return pw_verify_draft(vec<const float>(a[0], at::kFloat, p, "target_p", B, K + 1, V),
                         vec<const float>(a[1], at::kFloat, p, "draft_p", B, K, V),
                         vec<const int32_t>(a[2], at::kInt, p, "tokens", B, K), vec<const int32_t>(a[3], at::kInt, p, "n_draft", B),
                         vec<const float>(a[4], at::kFloat, p, "u", B, K), vec<const float>(a[5], at::kFloat, p, "noise", B, V),
                         (int)B, (int)K, (int)V, vec<int32_t>(a[6], at::kInt, p, "out", B, K + 1),
                         vec<int32_t>(a[7], at::kInt, p, "accepted", B), vec<int32_t>(a[8], at::kInt, p, "err", 1),
                         stream(a[9], p));
}

PyObject* py_check_cache(PyObject*, PyObject* const* a, Py_ssize_t n) { return call<check_cache>(a, n, 1); }
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) { return call<rope>(a, n, 8); }
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) { return call<append>(a, n, 11); }
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) { return call<attend>(a, n, 15); }
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) { return call<verify>(a, n, 10); }

PyMethodDef methods[] = {
    {"check_cache", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_check_cache)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attend)), METH_FASTCALL, nullptr},
    {"verify_draft", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_verify)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pw_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pw_torch() { return PyModule_Create(&module); }
