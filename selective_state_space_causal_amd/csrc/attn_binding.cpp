// attn_binding.cpp -- the usual case of attn.py's calls, natively (Python extension _attn_fast).
//
// A small call (a few tokens) spends longer in the interpreter than on the GPU: reading each tensor's shape, type,
// device and strides, and making the outputs.  Each function here takes the arguments of the function of its name in
// attn.py, on the current stream, and answers NotImplemented, having done nothing, whenever anything about them is not the usual
// (another type, shape or device, a missing tensor, a refusal to report): attn.py then goes
// through its own checks, which name what is wrong.  So it holds no message and no behaviour of its own.  A launch that
// fails may have done something (a call in place must not be made twice): it is raised from here.  The entry
// points of libssm.so are handed over by address (bind): this module does not load the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ssm_attn.h"

namespace {

decltype(&ssm_rope) f_rope;
decltype(&ssm_kv_write) f_kv_write;
decltype(&ssm_kv_read) f_kv_read;
decltype(&ssm_attn_prefill) f_prefill;
decltype(&ssm_attn_decode_step) f_decode;
decltype(&ssm_attn_decode_workspace_bytes) f_workspace;

PyObject* raise_status;  // attn.py's function of a name and a status that raises

PyObject* not_usual() { Py_RETURN_NOTIMPLEMENTED; }

// A Python object of a call's own, given back unless the call succeeds.  Outputs are made before the launch, so that
// nothing can go wrong after it.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* object) : p(object) {}
  Ref(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  // What to answer for the status that entry point `name` returned; every refusal comes before any launch.
  PyObject* after(int status, const char* name) {
    if (status == SSM_ERR_LAUNCH) return PyObject_CallFunction(raise_status, "si", name, status);
    if (status != SSM_OK) return not_usual();
    PyObject* r = p;
    p = nullptr;
    return r;
  }
};

// A call is usual until something is not; the device of the first tensor is that of all.
struct Call {
  bool ok = true;
  int device = -1;
  at::ScalarType dtype = at::ScalarType::Undefined;  // of the io tensors

  const at::Tensor* tensor(PyObject* o) {
    if (!ok || !THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (device < 0) device = t.get_device();
    if (t.get_device() != device) return fail();
    return &t;
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  // An io tensor [tokens, heads, dim] (a size of -1: any) as a view; the same type as the others.
  const at::Tensor* io(PyObject* o, ssm_view& v, int64_t tokens, int64_t heads, int64_t dim) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    if (dtype == at::ScalarType::Undefined) dtype = t->scalar_type();
    if (t->scalar_type() != dtype || (dtype != at::kFloat && dtype != at::kBFloat16) || t->dim() != 3) return fail();
    const auto n = t->sizes();
    const auto s = t->strides();
    if ((tokens >= 0 && n[0] != tokens) || (heads >= 0 && n[1] != heads) || (dim >= 0 && n[2] != dim)) return fail();
    if (s[2] != 1 && n[2] != 1) return fail();
    v = ssm_view{t->data_ptr(), n[0] > 1 ? s[0] : 0, n[1] > 1 ? s[1] : 0};
    return t;
  }
  // A contiguous index tensor of the given sizes (-1: any).
  const at::Tensor* index(PyObject* o, at::ScalarType type, int dims, int64_t n0, int64_t n1 = -1) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->dim() != dims || !t->is_contiguous()) return fail();
    if ((n0 >= 0 && t->size(0) != n0) || (dims > 1 && n1 >= 0 && t->size(1) != n1)) return fail();
    return t;
  }
  at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, device)));
  }
  at::Tensor fresh_io(ssm_view& v, int64_t tokens, int64_t heads, int64_t dim) const {
    at::Tensor t = fresh({tokens, heads, dim}, dtype);
    v = ssm_view{t.data_ptr(), heads * dim, dim};
    return t;
  }
  int32_t io_code() const { return dtype == at::kBFloat16 ? SSM_BF16 : SSM_F32; }
  void* stream() const { return c10::hip::getCurrentHIPStream(device).stream(); }

  // positions, freq, interleaved, mscale
  void rope(ssm_rope_desc& r, PyObject* positions, PyObject* freq, PyObject* interleaved, PyObject* mscale, int64_t tokens) {
    const at::Tensor* p = index(positions, at::kLong, 1, tokens);
    const at::Tensor* f = index(freq, at::kDouble, 1, -1);
    if (!PyBool_Check(interleaved) || !PyFloat_Check(mscale)) fail();
    if (!ok) return;
    r = ssm_rope_desc{p->const_data_ptr<int64_t>(), f->const_data_ptr<double>(), (int32_t)f->numel(), interleaved == Py_True,
                      (float)PyFloat_AS_DOUBLE(mscale)};
  }
};

PyObject* own(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}
bool put(Ref& tuple, int i, PyObject* o) {
  if (o) PyTuple_SET_ITEM(tuple.p, i, o);
  return o != nullptr;
}

const ssm_kv_cache* cache_at(PyObject* address) {
  return static_cast<const ssm_kv_cache*>(PyLong_AsVoidPtr(address));
}
bool cache_takes(PyObject* io_only_bf16, at::ScalarType dtype) {
  // io_only: None for 8-bit codes, else whether the cache is of bf16
  return io_only_bf16 == Py_None || (dtype == at::kBFloat16) == (io_only_bf16 == Py_True);
}

// rope(q, k, positions, freq, interleaved, mscale, q_out, k_out)
PyObject* rope(PyObject* const* a) {
  Call c;
  ssm_view vq, vk, vqo, vko;
  ssm_rope_desc r;
  const at::Tensor* q = c.io(a[0], vq, -1, -1, -1);
  if (!q) return not_usual();
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
  const bool has_k = a[1] != Py_None;
  if (!has_k && a[7] != Py_None) return not_usual();
  const at::Tensor* k = has_k ? c.io(a[1], vk, T, -1, D) : nullptr;
  c.rope(r, a[2], a[3], a[4], a[5], T);
  if (a[6] != Py_None) c.io(a[6], vqo, T, Hq, D);
  if (a[7] != Py_None && k) c.io(a[7], vko, T, k->size(1), D);
  if (!c.ok) return not_usual();
  const int64_t Hk = k ? k->size(1) : 0;
  if (Hq > SSM_ATTN_MAX_HEADS || Hk > SSM_ATTN_MAX_HEADS || D > SSM_ATTN_MAX_HEAD_DIM) return not_usual();
  Ref out(PyTuple_New(2));
  if (!out.p || !put(out, 0, a[6] == Py_None ? own(c.fresh_io(vqo, T, Hq, D)) : same(a[6])) ||
      !put(out, 1, k && a[7] == Py_None ? own(c.fresh_io(vko, T, Hk, D)) : same(a[7])))
    return nullptr;
  return out.after(f_rope(T, (int32_t)Hq, (int32_t)Hk, (int32_t)D, c.io_code(), &r, &vq, &vqo, k ? &vk : nullptr,
                          k ? &vko : nullptr, c.stream()),
                   "ssm_rope");
}

// kv_write(k, v, cache, device, io_only_bf16, slots, q, positions, freq, interleaved, mscale, q_out, k_out)
PyObject* kv_write(PyObject* const* a) {
  Call c;
  c.device = (int)PyLong_AsLong(a[3]);
  const ssm_kv_cache* cache = cache_at(a[2]);
  ssm_view vk, vv, vq, vqo, vko;
  ssm_rope_desc r;
  const int64_t H = cache->kv_heads, D = cache->head_dim;
  const at::Tensor* k = c.io(a[0], vk, -1, H, D);
  if (!k) return not_usual();
  const int64_t T = k->size(0);
  c.io(a[1], vv, T, H, D);
  const at::Tensor* slots = c.index(a[5], at::kLong, 1, T);
  const bool rotated = a[7] != Py_None, has_q = a[6] != Py_None;
  if (rotated != (a[8] != Py_None) || (!rotated && (has_q || a[12] != Py_None)) || (!has_q && a[11] != Py_None))
    return not_usual();
  if (rotated) c.rope(r, a[7], a[8], a[9], a[10], T);
  const at::Tensor* q = has_q ? c.io(a[6], vq, T, -1, D) : nullptr;
  if (a[11] != Py_None && q) c.io(a[11], vqo, T, q->size(1), D);
  if (a[12] != Py_None) c.io(a[12], vko, T, H, D);
  if (!c.ok || !cache_takes(a[4], c.dtype)) return not_usual();
  const int64_t Hq = q ? q->size(1) : 0;
  if (Hq > SSM_ATTN_MAX_HEADS) return not_usual();
  Ref out(q && a[11] == Py_None ? own(c.fresh_io(vqo, T, Hq, D)) : same(a[11]));
  if (!out.p) return nullptr;
  return out.after(f_kv_write(T, c.io_code(), cache, slots->const_data_ptr<int64_t>(), &vk, &vv, rotated ? &r : nullptr,
                              (int32_t)Hq, q ? &vq : nullptr, q ? &vqo : nullptr, a[12] != Py_None ? &vko : nullptr,
                              c.stream()),
                   "ssm_kv_write");
}

// kv_read(cache, device, io_only_bf16, slots, bf16, k_out, v_out)
PyObject* kv_read(PyObject* const* a) {
  Call c;
  c.device = (int)PyLong_AsLong(a[1]);
  const ssm_kv_cache* cache = cache_at(a[0]);
  ssm_view v[2];
  c.dtype = a[4] == Py_True ? at::kBFloat16 : at::kFloat;
  const at::Tensor* slots = c.index(a[3], at::kLong, 1, -1);
  if (!slots || !cache_takes(a[2], c.dtype)) return not_usual();
  const int64_t T = slots->size(0), H = cache->kv_heads, D = cache->head_dim;
  for (int i = 0; i < 2; ++i)
    if (a[5 + i] != Py_None) c.io(a[5 + i], v[i], T, H, D);
  if (!c.ok) return not_usual();
  Ref out(PyTuple_New(2));
  if (!out.p) return nullptr;
  for (int i = 0; i < 2; ++i)
    if (!put(out, i, a[5 + i] == Py_None ? own(c.fresh_io(v[i], T, H, D)) : same(a[5 + i]))) return nullptr;
  return out.after(f_kv_read(T, c.io_code(), cache, slots->const_data_ptr<int64_t>(), &v[0], &v[1], c.stream()), "ssm_kv_read");
}

// scale: a float, or None for 1 / sqrt(D)
bool scale_of(PyObject* o, int64_t D, float& s) {
  if (o != Py_None && !PyFloat_Check(o)) return false;
  s = o == Py_None ? (float)pow((double)D, -0.5) : (float)PyFloat_AS_DOUBLE(o);
  return true;
}

// attn_prefill(q, k, v, cu_q, cu_k, causal, scale, out, lse)
PyObject* attn_prefill(PyObject* const* a) {
  Call c;
  ssm_view vq, vk, vv, vo;
  ssm_attn_dims d;
  const at::Tensor* q = c.io(a[0], vq, -1, -1, -1);
  if (!q) return not_usual();
  const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
  const at::Tensor* k = c.io(a[1], vk, -1, -1, D);
  if (!k) return not_usual();
  c.io(a[2], vv, k->size(0), k->size(1), D);
  const at::Tensor* cq = c.index(a[3], at::kInt, 1, -1);
  const at::Tensor* ck = cq ? c.index(a[4], at::kInt, 1, cq->size(0)) : nullptr;
  if (a[7] != Py_None) c.io(a[7], vo, T, Hq, D);
  const at::Tensor* lse = a[8] != Py_None ? c.index(a[8], at::kFloat, 2, T, Hq) : nullptr;
  if (!c.ok || cq->size(0) < 2 || !PyBool_Check(a[5]) || D < 1 || D > SSM_ATTN_MAX_HEAD_DIM || Hq > SSM_ATTN_MAX_HEADS ||
      k->size(1) > SSM_ATTN_MAX_HEADS || !scale_of(a[6], D, d.scale))
    return not_usual();
  Ref out(a[7] == Py_None ? own(c.fresh_io(vo, T, Hq, D)) : same(a[7]));
  if (!out.p) return nullptr;
  d.batch = cq->size(0) - 1;
  d.q_tokens = T;
  d.k_tokens = k->size(0);
  d.q_heads = (int32_t)Hq;
  d.kv_heads = (int32_t)k->size(1);
  d.head_dim = (int32_t)D;
  d.io_dtype = c.io_code();
  d.causal = a[5] == Py_True;
  return out.after(f_prefill(&d, &vq, &vk, &vv, cq->const_data_ptr<int32_t>(), ck->const_data_ptr<int32_t>(), &vo,
                             lse ? lse->mutable_data_ptr<float>() : nullptr, c.stream()),
                   "ssm_attn_prefill");
}

// attn_decode_step(q, cache, device, io_only_bf16, table, lens, scale, out, lse)
PyObject* attn_decode_step(PyObject* const* a) {
  Call c;
  c.device = (int)PyLong_AsLong(a[2]);
  const ssm_kv_cache* cache = cache_at(a[1]);
  ssm_view vq, vo;
  float scale;
  const int64_t D = cache->head_dim;
  const at::Tensor* q = c.io(a[0], vq, -1, -1, D);
  if (!q) return not_usual();
  const int64_t B = q->size(0), Hq = q->size(1);
  const at::Tensor* table = c.index(a[4], at::kInt, 2, B);
  const at::Tensor* lens = c.index(a[5], at::kInt, 1, B);
  if (a[7] != Py_None) c.io(a[7], vo, B, Hq, D);
  const at::Tensor* lse = a[8] != Py_None ? c.index(a[8], at::kFloat, 2, B, Hq) : nullptr;
  if (!c.ok || !cache_takes(a[3], c.dtype) || Hq > SSM_ATTN_MAX_HEADS || !scale_of(a[6], D, scale))
    return not_usual();
  const int64_t W = table->size(1);
  Ref out(a[7] == Py_None ? own(c.fresh_io(vo, B, Hq, D)) : same(a[7]));
  if (!out.p) return nullptr;
  at::Tensor ws;
  const size_t need = f_workspace(B, (int32_t)Hq, cache, W);
  if (need) ws = c.fresh({(int64_t)need}, at::kByte);
  return out.after(f_decode(B, (int32_t)Hq, c.io_code(), scale, cache, &vq, table->const_data_ptr<int32_t>(), W,
                            lens->const_data_ptr<int32_t>(), &vo, lse ? lse->mutable_data_ptr<float>() : nullptr,
                            need ? ws.mutable_data_ptr() : nullptr, need, c.stream()),
                   "ssm_attn_decode_step");
}

// describe(address of a cache's description, k, v, k_scale, v_scale): fills it and gives (pages, heads, page_size,
// head_dim, device index, io_only_bf16)
PyObject* describe(PyObject* const* a) {
  Call c;
  const at::Tensor* k = c.tensor(a[1]);
  const at::Tensor* v = c.tensor(a[2]);
  if (!c.ok || k->dim() != 4 || v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type() || !k->is_contiguous() ||
      !v->is_contiguous())
    return not_usual();
  const at::ScalarType t = k->scalar_type();
  const bool codes = t == at::kChar || t == at::kFloat8_e4m3fn;
  if (!codes && t != at::kFloat && t != at::kBFloat16) return not_usual();
  const int64_t n[4] = {k->size(0), k->size(1), k->size(2), k->size(3)};
  for (int i = 1; i < 4; ++i)
    if (n[i] > INT32_MAX) return not_usual();
  const at::Tensor* s[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i) {
    if (!codes) {
      if (a[3 + i] != Py_None) return not_usual();
      continue;
    }
    s[i] = c.tensor(a[3 + i]);
    if (!c.ok || s[i]->scalar_type() != at::kFloat || s[i]->sizes() != k->sizes().slice(0, 3) || !s[i]->is_contiguous())
      return not_usual();
  }
  *static_cast<ssm_kv_cache*>(PyLong_AsVoidPtr(a[0])) =
      ssm_kv_cache{k->data_ptr(), v->data_ptr(), s[0] ? s[0]->mutable_data_ptr<float>() : nullptr,
                   s[1] ? s[1]->mutable_data_ptr<float>() : nullptr, n[0], (int32_t)n[2], (int32_t)n[1], (int32_t)n[3],
                   !codes ? SSM_KV_IO : t == at::kChar ? SSM_KV_I8 : SSM_KV_E4M3};
  return Py_BuildValue("LLLLiO", (long long)n[0], (long long)n[1], (long long)n[2], (long long)n[3], c.device,
                       codes ? Py_None : t == at::kBFloat16 ? Py_True : Py_False);
}

// bind(version, rope, kv_write, kv_read, attn_prefill, attn_decode_step, workspace_bytes, raise_status): the library's ABI
// version, which has to be the one that this module fills structures for, addresses, and a function
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes a version, six addresses and a function");
    return nullptr;
  }
  const long version = PyLong_AsLong(*a++);
  if (version != SSM_ABI_VERSION) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ImportError, "built for libssm ABI %d, not %ld", SSM_ABI_VERSION, version);
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  f_rope = reinterpret_cast<decltype(f_rope)>(p[0]);
  f_kv_write = reinterpret_cast<decltype(f_kv_write)>(p[1]);
  f_kv_read = reinterpret_cast<decltype(f_kv_read)>(p[2]);
  f_prefill = reinterpret_cast<decltype(f_prefill)>(p[3]);
  f_decode = reinterpret_cast<decltype(f_decode)>(p[4]);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(p[5]);
  Py_INCREF(a[6]);
  Py_XDECREF(raise_status);
  raise_status = a[6];
  Py_RETURN_NONE;
}

// No C++ exception passes into the interpreter: what went wrong (memory that ran out) goes wrong again in attn.py.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != N) return not_usual();
  try {
    return F(a);
  } catch (...) {
    return not_usual();
  }
}

PyMethodDef method(const char* name, PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return PyMethodDef{name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("bind", bind),
                         method("describe", guarded<describe, 5>),
                         method("rope", guarded<rope, 8>),
                         method("kv_write", guarded<kv_write, 13>),
                         method("kv_read", guarded<kv_read, 7>),
                         method("attn_prefill", guarded<attn_prefill, 9>),
                         method("attn_decode_step", guarded<attn_decode_step, 9>),
                         PyMethodDef{nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_fast() { return PyModule_Create(&module); }
