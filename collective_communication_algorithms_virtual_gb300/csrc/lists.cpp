// Python extension: the arrays that vc_clip_grad_norm takes, from lists of the
// ranks' tensors, in one pass.  A tensor's pointer, size, type, device and
// contiguity asked for one by one in Python cost 0.6 us: more than its share of
// the GPU's work where tensors are small.  Nothing is kept between calls.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <vector>

#include "vc.h"

namespace {

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return VC_FLOAT32;
    case at::kBFloat16: return VC_BFLOAT16;
    case at::kHalf: return VC_FLOAT16;
    default: return -1;
  }
}

// A plain tensor (no subclass), contiguous, on CUDA device `dev`, of a type that
// the library computes on.
const at::Tensor* plain(PyObject* o, int dev, int* code) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || !t.has_storage() || t.get_device() != dev || !t.is_contiguous())
    return nullptr;
  *code = code_of(t.scalar_type());
  return *code < 0 ? nullptr : &t;
}

bool is_list(PyObject* o) { return PyList_CheckExact(o) || PyTuple_CheckExact(o); }

PyObject* bytes_of(const void* p, size_t n) { return PyBytes_FromStringAndSize(static_cast<const char*>(p), static_cast<Py_ssize_t>(n)); }

template <class F>
bool each(PyObject* ranks, Py_ssize_t n, Py_ssize_t t, F&& f) {
  if (!is_list(ranks) || PySequence_Fast_GET_SIZE(ranks) != n) return false;
  for (Py_ssize_t r = 0; r < n; ++r) {
    PyObject* mine = PySequence_Fast_GET_ITEM(ranks, r);
    if (!is_list(mine) || PySequence_Fast_GET_SIZE(mine) != t) return false;
    for (Py_ssize_t i = 0; i < t; ++i)
      if (!f(PySequence_Fast_GET_ITEM(mine, i), static_cast<size_t>(r * t + i), static_cast<size_t>(i))) return false;
  }
  return true;
}

// pack(grads, out, dev) -> (pointers, out's pointers or None, sizes, type codes),
// packed; None where anything is not as the call wants it: the caller then finds
// out what.
PyObject* pack(PyObject*, PyObject* args) {
  PyObject *grads, *out;
  int dev;
  if (!PyArg_ParseTuple(args, "OOi", &grads, &out, &dev)) return nullptr;
  try {
    if (!is_list(grads) || PySequence_Fast_GET_SIZE(grads) == 0) Py_RETURN_NONE;
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(grads);
    PyObject* first = PySequence_Fast_GET_ITEM(grads, 0);
    if (!is_list(first)) Py_RETURN_NONE;
    const Py_ssize_t t = PySequence_Fast_GET_SIZE(first);
    std::vector<uint64_t> from(n * t), to(out == Py_None ? 0 : n * t), sizes(n * t);
    std::vector<int32_t> codes(t);
    const bool fine =
        each(grads, n, t, [&](PyObject* o, size_t at, size_t i) {
          int code = -1;
          const at::Tensor* x = plain(o, dev, &code);
          if (!x || (at >= static_cast<size_t>(t) && code != codes[i])) return false;
          codes[i] = code;
          from[at] = reinterpret_cast<uint64_t>(x->data_ptr());
          sizes[at] = static_cast<uint64_t>(x->numel());
          return true;
        }) &&
        (out == Py_None || each(out, n, t, [&](PyObject* o, size_t at, size_t i) {
           int code = -1;
           const at::Tensor* x = plain(o, dev, &code);
           if (!x || code != codes[i] || static_cast<uint64_t>(x->numel()) != sizes[at]) return false;
           to[at] = reinterpret_cast<uint64_t>(x->data_ptr());
           return true;
         }));
    if (!fine) Py_RETURN_NONE;
    PyObject* outs = Py_None;
    if (out == Py_None) Py_INCREF(outs);
    else outs = bytes_of(to.data(), to.size() * 8);
    return Py_BuildValue("(NNNN)", bytes_of(from.data(), from.size() * 8), outs, bytes_of(sizes.data(), sizes.size() * 8),
                         bytes_of(codes.data(), codes.size() * 4));
  } catch (...) {  // a tensor without memory
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef methods[] = {{"pack", pack, METH_VARARGS, "pack(grads, out, dev): the arrays of vc_clip_grad_norm, or None"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lists() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch", TORCH_VERSION) < 0) Py_CLEAR(m);  // whose tensors it can read
  return m;
}
