// The torch calls of a serving step without the interpreter between their checks: each function below takes the arguments of the Python function of its
// name, and where they are as a serving program has them (everything on the current device, contiguous, aligned, of the right types and shapes) allocates
// the results, calls the C ABI on the current stream and returns the results. It returns None for anything else, which the Python function then looks at
// in full (and refuses, copies or moves to another device or stream), and a status where the C ABI refuses. Nothing here computes.
//
// A step makes several of these calls a layer, whose kernels take 4 to 25 us. Host time of a call, us, by the Python functions alone and so: appending
// 24 tokens 20.7 / 4.9, one token over a 4-bit cache 30.8 / 10.6 (two tensor maps and two launches of it), page bounds and a selection for it
// 49.6 / 19.7.
#include <ATen/ATen.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "cqsa.h"

namespace {

using at::Tensor;

// A tensor argument; null for anything else.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A whole number held to [0, 2^31 - 1] from above; false for anything but one from 0 on.
bool count(PyObject* o, int* out) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over < 0 || (over == 0 && v < 0)) return false;
  *out = over > 0 || v > 0x7fffffffLL ? 0x7fffffff : static_cast<int>(v);
  return true;
}

bool number(PyObject* o, float* out) {
  if (o == Py_None) {
    *out = 0.0f;
    return true;
  }
  if (!PyFloat_Check(o)) return false;
  *out = static_cast<float>(PyFloat_AS_DOUBLE(o));
  return true;
}

int type_code(const Tensor& t) {
  return t.scalar_type() == at::kHalf ? CQSA_F16 : (t.scalar_type() == at::kBFloat16 ? CQSA_BF16 : -1);
}

void* address(const Tensor& t) { return t.data_ptr(); }

// A contiguous tensor on the device.
bool plain(const Tensor* t, int device) { return t && t->is_cuda() && t->get_device() == device && t->is_contiguous(); }

// [T, heads, d] of a type on a device with its heads dense, at an aligned address; *stride: elements from token to token.
bool tokens(const Tensor* t, int device, at::ScalarType type, int64_t T, int64_t heads, int64_t d, long long* stride) {
  if (!t || !t->is_cuda() || t->get_device() != device || t->scalar_type() != type || t->dim() != 3) return false;
  if (t->size(0) != T || t->size(1) != heads || t->size(2) != d || (reinterpret_cast<uintptr_t>(address(*t)) & 15)) return false;
  *stride = heads * d;
  if (t->is_contiguous()) return true;
  if (T < 2 || t->stride(2) != 1 || (t->stride(1) != d && heads > 1) || t->stride(0) < heads * d || t->stride(0) % 8) return false;
  *stride = t->stride(0);
  return true;
}

// The cache, its index tensors and its scales.
struct Cache {
  int code, device, n_seqs, max_pages, n_pages, Hkv, page;
  int64_t d;
  const Tensor *k, *v, *table, *cu, *lens;
  unsigned char *ks, *vs;

  bool scales(const Tensor* t, unsigned char** out) const {
    if (!plain(t, device) || t->element_size() != 1 || t->dim() != (code == CQSA_E4M3 ? 3 : 4)) return false;
    if (t->size(0) != n_pages || t->size(1) != Hkv || t->size(2) != page || (code == CQSA_INT4 && t->size(3) != d / 32)) return false;
    *out = static_cast<unsigned char*>(address(*t));
    return true;
  }

  // v_cache and v_scale may be null: a call that only looks at the keys. type: the tokens' (of any for bytes).
  bool take(PyObject* k_cache, PyObject* v_cache, PyObject* block_table, PyObject* cu_seqlens, PyObject* kv_lens, PyObject* k_scale,
            PyObject* v_scale, int dev, int type) {
    device = dev;
    k = tensor(k_cache);
    v = v_cache ? tensor(v_cache) : k;
    table = tensor(block_table);
    cu = tensor(cu_seqlens);
    lens = tensor(kv_lens);
    if (!plain(k, dev) || !plain(v, dev) || !plain(table, dev) || !plain(cu, dev) || !plain(lens, dev)) return false;
    if (k->dim() != 4 || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type()) return false;
    if (table->dim() != 2 || cu->dim() != 1 || lens->dim() != 1 || table->scalar_type() != at::kInt || cu->scalar_type() != at::kInt ||
        lens->scalar_type() != at::kInt || lens->size(0) != table->size(0) || cu->size(0) != table->size(0) + 1)
      return false;
    if (k->size(0) > 0x7fffffff || k->size(1) > 0x7fffffff || table->size(0) > 0x7ffffffe || table->size(1) > 0x7fffffff) return false;
    n_pages = static_cast<int>(k->size(0));
    Hkv = static_cast<int>(k->size(1));
    page = static_cast<int>(k->size(2) < 0x7fffffff ? k->size(2) : 0);
    n_seqs = static_cast<int>(table->size(0));
    max_pages = static_cast<int>(table->size(1));
    d = k->size(3);
    ks = vs = nullptr;
    if (k_scale == Py_None) {
      code = type_code(*k);
      return code >= 0 && code == type && (!v_scale || v_scale == Py_None);
    }
    const Tensor* z = tensor(k_scale);
    if (!z || (k->scalar_type() != at::kByte && k->scalar_type() != at::kFloat8_e4m3fn)) return false;
    code = z->dim() == 4 && k->scalar_type() == at::kByte ? CQSA_INT4 : CQSA_E4M3;
    if (code == CQSA_INT4) d *= 2;
    return scales(z, &ks) && (!v_scale || (v_scale == k_scale ? (vs = ks, true) : scales(tensor(v_scale), &vs)));
  }
};

// The current device if it is the tensor's, and its current stream.
bool here(const Tensor* t, int* device, cudaStream_t* stream) {
  if (!t || !t->is_cuda()) return false;
  *device = t->get_device();
  if (c10::cuda::current_device() != *device) return false;
  *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(*device)).stream();
  return true;
}

Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const Tensor& like) { return at::empty(sizes, like.options().dtype(type)); }

// The given result (like q, contiguous) or a new one.
bool result(PyObject* given, const Tensor& q, int device, Tensor* out) {
  if (given == Py_None) {
    *out = fresh(q.sizes(), q.scalar_type(), q);
    return true;
  }
  const Tensor* t = tensor(given);
  if (!plain(t, device) || t->sizes() != q.sizes() || t->scalar_type() != q.scalar_type()) return false;
  *out = *t;
  return true;
}

// The given workspace (a contiguous tensor) or a new one of `need` bytes.
bool space(PyObject* given, size_t need, const Tensor& q, int device, Tensor* ws, size_t* bytes) {
  if (given == Py_None) {
    *ws = fresh({static_cast<int64_t>(need > 16 ? need : 16)}, at::kByte, q);
    *bytes = need;
    return true;
  }
  const Tensor* t = tensor(given);
  if (!plain(t, device)) return false;
  *ws = *t;
  *bytes = t->nbytes();
  return true;
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* wrapped(const Tensor& t) { return THPVariable_Wrap(t); }

// The interpreter free for other threads; taken back whichever way the block is left (a tensor without memory of its own throws when asked for its address).
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  Released() = default;
  Released(const Released&) = delete;
  ~Released() { PyEval_RestoreThread(state); }
};

// A call of the C ABI with the interpreter free (a launch waits while the GPU's queue is full).
template <class F>
int call(F f) {
  const Released released;
  return f();
}

// Whether an argument is true; throws, the interpreter's error set, where it cannot say.
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}

// One tensor or a tuple of those that are there.
PyObject* results(std::initializer_list<const Tensor*> all) {
  Py_ssize_t n = 0;
  for (const Tensor* t : all) n += t != nullptr;
  if (n == 1) return wrapped(**all.begin());
  PyObject* r = PyTuple_New(n);
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : all) {
    if (!t) continue;
    PyObject* o = wrapped(*t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_q_len, max_kv_len, causal, scale, k_scale, v_scale, return_lse, out, workspace
PyObject* attention_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor* q = n == 15 ? tensor(a[0]) : nullptr;
  int device, max_q, max_kv;
  cudaStream_t stream;
  float scale;
  long long qs;
  Cache c;
  if (!here(q, &device, &stream) || q->dim() != 3 || !count(a[6], &max_q) || !count(a[7], &max_kv) || !number(a[9], &scale)) return none();
  const int dt = type_code(*q), causal = truth(a[8]), want_lse = truth(a[12]);
  if (dt < 0 || !c.take(a[1], a[2], a[3], a[4], a[5], a[10], a[11], device, dt)) return none();
  const int64_t T = q->size(0), Hq = q->size(1);
  if (T > 0x7fffffff || Hq > 0x7fffffff || !tokens(q, device, q->scalar_type(), T, Hq, c.d, &qs)) return none();
  if (max_q > T) max_q = static_cast<int>(T);
  Tensor out, lse, ws;
  size_t bytes;
  const size_t need = cqsa_attn_paged_workspace_size(c.n_seqs, T, Hq, c.Hkv, c.d, c.page, max_q, max_kv, dt, c.code);
  if (!result(a[13], *q, device, &out) || !space(a[14], need, *q, device, &ws, &bytes)) return none();
  if (want_lse) lse = fresh({Hq, T}, at::kFloat, *q);
  const int rc = call([&] {
    return cqsa_attn_paged_fwd(address(*q), qs, address(out), want_lse ? static_cast<float*>(address(lse)) : nullptr, address(*c.k),
                                     address(*c.v), c.ks, c.vs, static_cast<int*>(address(*c.table)), c.max_pages,
                                     static_cast<int*>(address(*c.cu)), static_cast<int*>(address(*c.lens)), c.n_seqs, T, max_q, max_kv, Hq,
                                     c.Hkv, c.d, c.page, c.n_pages, causal, scale, dt, c.code, address(ws), bytes, stream);
  });
  if (rc != CQSA_OK) return PyLong_FromLong(rc);
  return results({&out, want_lse ? &lse : nullptr});
  END_HANDLE_TH_ERRORS
}

// q, k, v, cos_sin, k_cache, v_cache, block_table, cu_seqlens, kv_lens, interleaved, k_scale, v_scale, q_out
PyObject* kv_cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *k = n == 13 ? tensor(a[1]) : nullptr, *q, *v, *turn;
  int device;
  cudaStream_t stream;
  long long qs, ks, vs;
  Cache c;
  if (!here(k, &device, &stream) || k->dim() != 3 || a[0] == Py_None) return none();
  q = tensor(a[0]);
  v = tensor(a[2]);
  turn = tensor(a[3]);
  const int dt = type_code(*k), interleaved = truth(a[9]);
  if (dt < 0 || !q || q->dim() != 3 || !c.take(a[4], a[5], a[6], a[7], a[8], a[10], a[11], device, dt)) return none();
  const int64_t T = k->size(0), Hq = q->size(1);
  const auto type = k->scalar_type();
  if (T > 0x7fffffff || Hq < 1 || Hq > 0x7fffffff || !tokens(k, device, type, T, c.Hkv, c.d, &ks) || !tokens(v, device, type, T, c.Hkv, c.d, &vs) ||
      !tokens(q, device, type, T, Hq, c.d, &qs))
    return none();
  if (!plain(turn, device) || turn->scalar_type() != at::kFloat || turn->dim() != 2 || turn->size(1) > 0x7fffffff ||
      (reinterpret_cast<uintptr_t>(address(*turn)) & 15))
    return none();
  Tensor out;
  if (!result(a[12], *q, device, &out)) return none();
  const int rc = call([&] {
    return cqsa_kv_cache_append(address(*q), address(*k), address(*v), qs, ks, vs, address(out), static_cast<float*>(address(*turn)),
                                      turn->size(0), static_cast<int>(turn->size(1)), interleaved, address(*c.k), address(*c.v), c.ks,
                                      c.vs, static_cast<int*>(address(*c.table)), c.max_pages, static_cast<int*>(address(*c.cu)),
                                      static_cast<int*>(address(*c.lens)), c.n_seqs, T, Hq, c.Hkv, c.d, c.page, c.n_pages, dt, c.code, stream);
  });
  if (rc != CQSA_OK) return PyLong_FromLong(rc);
  if (a[12] != Py_None) {  // the caller's own object
    Py_INCREF(a[12]);
    return a[12];
  }
  return wrapped(out);
  END_HANDLE_TH_ERRORS
}

// k, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens, k_scale, v_scale
PyObject* kv_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor* k = n == 9 ? tensor(a[0]) : nullptr;
  int device;
  cudaStream_t stream;
  long long ks, vs;
  Cache c;
  if (!here(k, &device, &stream) || k->dim() != 3) return none();
  const int dt = type_code(*k);
  if (dt < 0 || !c.take(a[2], a[3], a[4], a[5], a[6], a[7], a[8], device, dt)) return none();
  const int64_t T = k->size(0);
  const Tensor* v = tensor(a[1]);
  if (T > 0x7fffffff || !tokens(k, device, k->scalar_type(), T, c.Hkv, c.d, &ks) || !tokens(v, device, k->scalar_type(), T, c.Hkv, c.d, &vs)) return none();
  const int rc = call([&] {
    return cqsa_kv_cache_write(address(*k), address(*v), ks, vs, address(*c.k), address(*c.v), c.ks, c.vs, static_cast<int*>(address(*c.table)),
                                     c.max_pages, static_cast<int*>(address(*c.cu)), static_cast<int*>(address(*c.lens)), c.n_seqs, T, c.Hkv, c.d,
                                     c.page, c.n_pages, dt, c.code, stream);
  });
  return PyLong_FromLong(rc);
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, block_table, cu_seqlens, kv_lens, T, dtype's code, k_scale, v_scale
PyObject* kv_cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor* cache = n == 9 ? tensor(a[0]) : nullptr;
  int device, T, dt;
  cudaStream_t stream;
  Cache c;
  if (!here(cache, &device, &stream) || !count(a[5], &T) || !count(a[6], &dt) || !c.take(a[0], a[1], a[2], a[3], a[4], a[7], a[8], device, dt)) return none();
  const auto type = dt == CQSA_F16 ? at::kHalf : at::kBFloat16;
  const Tensor k = fresh({T, c.Hkv, c.d}, type, *cache), v = fresh({T, c.Hkv, c.d}, type, *cache);
  const int rc = call([&] {
    return cqsa_kv_cache_read(address(k), address(v), address(*c.k), address(*c.v), c.ks, c.vs, static_cast<int*>(address(*c.table)), c.max_pages,
                                    static_cast<int*>(address(*c.cu)), static_cast<int*>(address(*c.lens)), c.n_seqs, T, c.Hkv, c.d, c.page, c.n_pages,
                                    dt, c.code, stream);
  });
  if (rc != CQSA_OK) return PyLong_FromLong(rc);
  return results({&k, &v});
  END_HANDLE_TH_ERRORS
}

// k_cache, block_table, cu_seqlens, kv_lens, bounds, bounds_exp, max_q_len, k_scale
bool bounds_of(PyObject* b, PyObject* e, const Cache& c, const Tensor** bounds, const Tensor** exps) {
  *bounds = tensor(b);
  *exps = tensor(e);
  if (!plain(*bounds, c.device) || !plain(*exps, c.device) || (*bounds)->scalar_type() != at::kChar || (*exps)->scalar_type() != at::kByte) return false;
  return (*bounds)->sizes() == at::IntArrayRef({c.n_pages, c.Hkv, 2, c.d}) && (*exps)->sizes() == at::IntArrayRef({c.n_pages, c.Hkv});
}
PyObject* kv_page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *k = n == 8 ? tensor(a[0]) : nullptr, *bounds, *exps;
  int device, max_q;
  cudaStream_t stream;
  Cache c;
  if (!here(k, &device, &stream) || !count(a[6], &max_q)) return none();
  const int own = type_code(*k), dt = own < 0 ? CQSA_F16 : own;  // (bytes stand for numbers of neither type)
  if (!c.take(a[0], nullptr, a[1], a[2], a[3], a[7], nullptr, device, dt) || !bounds_of(a[4], a[5], c, &bounds, &exps)) return none();
  const int rc = call([&] {
    return cqsa_kv_page_bounds(address(*c.k), c.ks, static_cast<signed char*>(address(*bounds)), static_cast<unsigned char*>(address(*exps)),
                                     static_cast<int*>(address(*c.table)), c.max_pages, static_cast<int*>(address(*c.cu)),
                                     static_cast<int*>(address(*c.lens)), c.n_seqs, 0x7fffffff / (c.Hkv > 1 ? c.Hkv : 1), max_q, c.Hkv, c.d, c.page,
                                     c.n_pages, dt, c.code, stream);
  });
  return PyLong_FromLong(rc);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, bounds, bounds_exp, n_select, max_kv_len, scale, k_scale, v_scale, return_lse, return_pages, out,
// workspace
PyObject* attention_selected(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const Tensor *q = n == 17 ? tensor(a[0]) : nullptr, *bounds, *exps;
  int device, n_select, max_kv;
  cudaStream_t stream;
  float scale;
  long long qs;
  Cache c;
  if (!here(q, &device, &stream) || q->dim() != 3 || !count(a[8], &n_select) || !count(a[9], &max_kv) || !number(a[10], &scale)) return none();
  const int dt = type_code(*q), want_lse = truth(a[13]), want_pages = truth(a[14]);
  if (dt < 0 || !c.take(a[1], a[2], a[3], a[4], a[5], a[11], a[12], device, dt) || !bounds_of(a[6], a[7], c, &bounds, &exps)) return none();
  const int64_t T = q->size(0), Hq = q->size(1), slots = static_cast<int64_t>(c.max_pages) * c.page;
  if (T > 0x7fffffff || Hq > 0x7fffffff || !tokens(q, device, q->scalar_type(), T, Hq, c.d, &qs)) return none();
  if (n_select < 1 || static_cast<int64_t>(n_select) * c.page > 1 << 24) return none();
  if (max_kv > slots) max_kv = static_cast<int>(slots);
  Tensor out, lse, pages, ws;
  size_t bytes;
  const size_t need = cqsa_attn_selected_workspace_size(T, Hq, c.Hkv, c.d, c.page, n_select, max_kv, dt, c.code);
  if (!result(a[15], *q, device, &out) || !space(a[16], need, *q, device, &ws, &bytes)) return none();
  if (want_lse) lse = fresh({Hq, T}, at::kFloat, *q);
  if (want_pages) pages = fresh({T, c.Hkv, n_select}, at::kInt, *q);
  const int rc = call([&] {
    return cqsa_attn_selected_fwd(address(*q), qs, address(out), want_lse ? static_cast<float*>(address(lse)) : nullptr,
                                        want_pages ? static_cast<int*>(address(pages)) : nullptr, address(*c.k), address(*c.v), c.ks, c.vs,
                                        static_cast<signed char*>(address(*bounds)), static_cast<unsigned char*>(address(*exps)),
                                        static_cast<int*>(address(*c.table)), c.max_pages, static_cast<int*>(address(*c.cu)),
                                        static_cast<int*>(address(*c.lens)), c.n_seqs, T, n_select, max_kv, Hq, c.Hkv, c.d, c.page, c.n_pages, scale,
                                        dt, c.code, address(ws), bytes, stream);
  });
  if (rc != CQSA_OK) return PyLong_FromLong(rc);
  return results({&out, want_lse ? &lse : nullptr, want_pages ? &pages : nullptr});
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"attention_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attention_paged)), METH_FASTCALL, nullptr},
    {"kv_cache_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_cache_write)), METH_FASTCALL, nullptr},
    {"kv_cache_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_cache_read)), METH_FASTCALL, nullptr},
    {"kv_cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_cache_append)), METH_FASTCALL, nullptr},
    {"kv_page_bounds", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kv_page_bounds)), METH_FASTCALL, nullptr},
    {"attention_selected", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attention_selected)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "cqsa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_cqsa_torch() { return PyModule_Create(&module); }
