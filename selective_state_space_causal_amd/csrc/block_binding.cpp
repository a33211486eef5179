// block_binding.cpp -- the usual case of block.py's calls, natively (Python extension _block_fast).
//
// As attn_binding.cpp for attn.py: each function takes the arguments of the function of its name, on the current stream, and
// answers NotImplemented, having done nothing, whenever anything about them is not the usual; block.py then goes through its
// own checks, which name what is wrong.  A launch that fails is raised from here.  The entry points of libssm.so are handed
// over by address (bind).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ssm_block.h"
#include "binding.h"

namespace {

decltype(&ssm_rms_norm) f_norm;
decltype(&ssm_q4_linear) f_linear;
decltype(&ssm_q4_quantize) f_quantize;
decltype(&ssm_q4_dequantize) f_dequantize;

// A call is usual until something is not; the device of the first tensor is that of all.
struct Call {
  bool ok = true;
  int device = -1;

  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  const at::Tensor* tensor(PyObject* o) {
    if (!ok || !THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (device < 0) {
      device = t.get_device();
      if (device != c10::hip::current_device()) return fail();  // block.py makes it the current one
    }
    if (t.get_device() != device) return fail();
    return &t;
  }
  // A [T, D] tensor as rows (a size of -1: any).
  const at::Tensor* rows(PyObject* o, ssm_rows& r, int64_t tokens, int64_t width) {
    const at::Tensor* t = tensor(o);
    if (!t || t->dim() != 2) return fail();
    const int64_t n = t->size(0), d = t->size(1);
    if ((tokens >= 0 && n != tokens) || (width >= 0 && d != width) || (t->stride(1) != 1 && d != 1)) return fail();
    r = ssm_rows{t->data_ptr(), n > 1 ? t->stride(0) : 0};
    return t;
  }
  const at::Tensor* vector(PyObject* o, int64_t n) {
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) return fail();
    return t;
  }
  // A contiguous uint8 tensor of the sizes of a 4-bit weight's codes or scales.
  const at::Tensor* bytes(PyObject* o, int64_t n0, int64_t n1, int64_t n3) {
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != at::kByte || t->dim() != 4 || t->size(0) != n0 || t->size(1) != n1 || t->size(2) != 64 ||
        t->size(3) != n3 || !t->is_contiguous())
      return fail();
    return t;
  }
  // A 4-bit weight (codes, scales, out_features, in_features).
  bool weight(PyObject* o, ssm_q4_weight& q) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) return fail() != nullptr;
    PyObject* const m = PyTuple_GET_ITEM(o, 2);
    PyObject* const k = PyTuple_GET_ITEM(o, 3);
    if (!PyLong_Check(m) || !PyLong_Check(k)) return fail() != nullptr;
    int over = 0, more = 0;
    const int64_t M = PyLong_AsLongLongAndOverflow(m, &over), K = PyLong_AsLongLongAndOverflow(k, &more);
    if (over || more || M < 1 || M > SSM_Q4_MAX_FEATURES || K < 1 || K > SSM_Q4_MAX_FEATURES) return fail() != nullptr;
    const at::Tensor* codes = bytes(PyTuple_GET_ITEM(o, 0), (M + 15) / 16, (K + 127) / 128, 16);
    const at::Tensor* scales = bytes(PyTuple_GET_ITEM(o, 1), (M + 15) / 16, (K + 511) / 512, 4);
    if (!ok) return false;
    q = ssm_q4_weight{codes->data_ptr(), scales->data_ptr(), M, K};
    return true;
  }
  at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type) const {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, device)));
  }
  void* stream() const { return c10::hip::getCurrentHIPStream(device).stream(); }
};

// SSM_F32, SSM_BF16 or SSM_E4M3; -1 for another type.
int32_t code_of(at::ScalarType t) {
  return t == at::kFloat ? SSM_F32 : t == at::kBFloat16 ? SSM_BF16 : t == at::kFloat8_e4m3fn ? (int32_t)SSM_E4M3 : -1;
}

// The type that is asked for, or `otherwise` for None.
bool dtype_of(PyObject* o, at::ScalarType otherwise, at::ScalarType& type) {
  if (o == Py_None) {
    type = otherwise;
    return true;
  }
  if (!THPDtype_Check(o)) return false;
  type = reinterpret_cast<THPDtype*>(o)->scalar_type;
  return true;
}

// rms_norm(x, weight, residual, residual_out, eps, out_dtype, out, scale)
PyObject* rms_norm(PyObject* const* a) {
  Call c;
  ssm_rows x, r, ro, o;
  const at::Tensor* tx = c.rows(a[0], x, -1, -1);
  if (!tx) return not_usual();
  const int64_t T = tx->size(0), D = tx->size(1);
  const at::ScalarType type = tx->scalar_type();
  const at::Tensor* w = c.vector(a[1], D);
  const at::Tensor* tr = a[2] == Py_None ? nullptr : c.rows(a[2], r, T, D);
  const at::Tensor* tro = a[3] == Py_None ? nullptr : c.rows(a[3], ro, T, D);
  const at::Tensor* to = a[6] == Py_None ? nullptr : c.rows(a[6], o, T, D);
  at::ScalarType out_type;
  if (!c.ok || (type != at::kFloat && type != at::kBFloat16) || !PyFloat_Check(a[4])) return not_usual();
  if (!dtype_of(a[5], to ? to->scalar_type() : type, out_type) || (to && to->scalar_type() != out_type)) return not_usual();
  if (out_type != type && out_type != at::kFloat8_e4m3fn) return not_usual();
  if (tr ? (tr->scalar_type() != type && tr->scalar_type() != at::kFloat) || (tro && tro->scalar_type() != tr->scalar_type())
         : tro != nullptr)
    return not_usual();
  const bool q8 = out_type == at::kFloat8_e4m3fn;
  const at::Tensor* ts = a[7] == Py_None ? nullptr : c.vector(a[7], T);
  if (!c.ok || (!q8 && ts)) return not_usual();
  at::Tensor made, scale;
  if (!to) {
    made = c.fresh({T, D}, out_type);
    o = ssm_rows{made.data_ptr(), D};
  }
  if (q8 && !ts) {
    scale = c.fresh({T}, at::kFloat);
    ts = &scale;
  }
  float* ps = q8 ? ts->mutable_data_ptr<float>() : nullptr;
  Ref out(to ? same(a[6]) : own(std::move(made)));
  if (!out.p) return nullptr;
  if (q8) {
    PyObject* s = a[7] != Py_None ? same(a[7]) : own(std::move(scale));
    PyObject* pair = s ? PyTuple_Pack(2, out.p, s) : nullptr;
    Py_XDECREF(s);
    if (!pair) return nullptr;
    Py_DECREF(out.p);
    out.p = pair;
  }
  return out.after(f_norm(T, D, code_of(type), tr ? code_of(tr->scalar_type()) : code_of(type), code_of(out_type),
                          (float)PyFloat_AS_DOUBLE(a[4]), &x, w->const_data_ptr<float>(), tr ? &r : nullptr,
                          tr ? (tro ? &ro : &r) : nullptr, &o, ps, c.stream()),
                   "ssm_rms_norm");
}

// q4_linear(x, (codes, scales, out_features, in_features), x_scale, out_dtype, out)
PyObject* q4_linear(PyObject* const* a) {
  Call c;
  ssm_rows x, o;
  ssm_q4_weight q;
  if (!c.weight(a[1], q)) return not_usual();
  const int64_t M = q.out_features, K = q.in_features;
  const at::Tensor* tx = c.rows(a[0], x, -1, K);
  if (!tx) return not_usual();
  const int64_t T = tx->size(0);
  const at::ScalarType type = tx->scalar_type();
  const int32_t xc = code_of(type);
  const at::Tensor* xs = a[2] == Py_None ? nullptr : c.vector(a[2], T);
  const at::Tensor* to = a[4] == Py_None ? nullptr : c.rows(a[4], o, T, M);
  at::ScalarType out_type;
  if (!c.ok || xc < 0 || (xc == SSM_E4M3) != (xs != nullptr)) return not_usual();
  if (!dtype_of(a[3], to ? to->scalar_type() : xc == SSM_E4M3 ? at::kBFloat16 : type, out_type)) return not_usual();
  if ((to && to->scalar_type() != out_type) || (out_type != at::kFloat && out_type != at::kBFloat16)) return not_usual();
  at::Tensor made;
  if (!to) {
    made = c.fresh({T, M}, out_type);
    o = ssm_rows{made.data_ptr(), M};
  }
  Ref out(to ? same(a[4]) : own(std::move(made)));
  if (!out.p) return nullptr;
  return out.after(f_linear(T, xc, code_of(out_type), &x, xs ? xs->const_data_ptr<float>() : nullptr, &q, &o,
                            c.stream()),
                   "ssm_q4_linear");
}

// q4_quantize(w), without a given output: (codes, scales)
PyObject* q4_quantize(PyObject* const* a) {
  Call c;
  ssm_rows w;
  const at::Tensor* t = c.rows(a[0], w, -1, -1);
  if (!t) return not_usual();
  const int64_t M = t->size(0), K = t->size(1);
  const int32_t io = code_of(t->scalar_type());
  if ((io != SSM_F32 && io != SSM_BF16) || M < 1 || M > SSM_Q4_MAX_FEATURES || K < 16 || K > SSM_Q4_MAX_FEATURES || K % 16) return not_usual();
  at::Tensor codes = c.fresh({(M + 15) / 16, (K + 127) / 128, 64, 16}, at::kByte);
  at::Tensor scales = c.fresh({(M + 15) / 16, (K + 511) / 512, 64, 4}, at::kByte);
  const ssm_q4_weight q = {codes.data_ptr(), scales.data_ptr(), M, K};
  Ref out(PyTuple_New(2));
  if (!out.p || !put(out, 0, own(std::move(codes))) || !put(out, 1, own(std::move(scales)))) return nullptr;
  return out.after(f_quantize(io, &w, &q, c.stream()), "ssm_q4_quantize");
}

// q4_dequantize((codes, scales, out_features, in_features), dtype, out)
PyObject* q4_dequantize(PyObject* const* a) {
  Call c;
  ssm_q4_weight q;
  ssm_rows w;
  if (!c.weight(a[0], q)) return not_usual();
  const at::Tensor* to = a[2] == Py_None ? nullptr : c.rows(a[2], w, q.out_features, q.in_features);
  at::ScalarType type;
  if (!c.ok || !dtype_of(a[1], to ? to->scalar_type() : at::kBFloat16, type) || (to && to->scalar_type() != type)) return not_usual();
  if (type != at::kFloat && type != at::kBFloat16) return not_usual();
  at::Tensor made;
  if (!to) {
    made = c.fresh({q.out_features, q.in_features}, type);
    w = ssm_rows{made.data_ptr(), q.in_features};
  }
  Ref out(to ? same(a[2]) : own(std::move(made)));
  if (!out.p) return nullptr;
  return out.after(f_dequantize(code_of(type), &q, &w, c.stream()), "ssm_q4_dequantize");
}

// bind(version, rms_norm, q4_linear, q4_quantize, q4_dequantize, raise_status): the library's ABI version, which has to be the
// one that this module fills structures for, addresses, and a function
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes a version, four addresses and a function");
    return nullptr;
  }
  const long version = PyLong_AsLong(*a++);
  if (version != SSM_ABI_VERSION) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ImportError, "built for libssm ABI %d, not %ld", SSM_ABI_VERSION, version);
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  f_norm = reinterpret_cast<decltype(f_norm)>(p[0]);
  f_linear = reinterpret_cast<decltype(f_linear)>(p[1]);
  f_quantize = reinterpret_cast<decltype(f_quantize)>(p[2]);
  f_dequantize = reinterpret_cast<decltype(f_dequantize)>(p[3]);
  Py_INCREF(a[4]);
  Py_XDECREF(raise_status);
  raise_status = a[4];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {method("bind", bind), method("rms_norm", guarded<rms_norm, 8>), method("q4_linear", guarded<q4_linear, 5>),
                         method("q4_quantize", guarded<q4_quantize, 1>), method("q4_dequantize", guarded<q4_dequantize, 3>),
                         PyMethodDef{nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block_fast() { return PyModule_Create(&module); }
