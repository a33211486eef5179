// binding.h -- what the native halves of attn.py and block.py (attn_binding.cpp, block_binding.cpp) share: answers,
// references and the frame around a call.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ssm.h"

namespace {

PyObject* raise_status;  // the Python half's function of a name and a status that raises

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

PyObject* own(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}
bool put(Ref& tuple, int i, PyObject* o) {
  if (o) PyTuple_SET_ITEM(tuple.p, i, o);
  return o != nullptr;
}

// No C++ exception passes into the interpreter: what went wrong (memory that ran out) goes wrong again in the Python half.
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

}  // namespace
