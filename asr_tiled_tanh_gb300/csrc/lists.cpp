// lists.cpp -- tensors' data pointers and new tensors, for the Python binding.
//
// A call looks at each tensor's type, place, shape and pointer.  Through Python
// attributes that takes 0.35 us a tensor, for the lists of a small model more than the
// GPU takes; here it takes about 0.01 us in a list, 0.1 us alone.
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

// take(tensors, n, layout, device, out): the pointers of a list of dense CUDA tensors into
// the memory at `out`.  layout: the address of int64 words, for each tensor its type (0
// fp32, 1 bf16), dimensions and sizes.  Returns -1, or the place of the first that is
// not as the layout says (their number, where that differs).
PyObject* take(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 5 || !PyList_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "take(list, n, layout, device, out)");
    return nullptr;
  }
  const Py_ssize_t n = PyLong_AsSsize_t(args[1]);
  const int64_t* want = (const int64_t*)PyLong_AsVoidPtr(args[2]);
  const long device = PyLong_AsLong(args[3]);
  uint64_t* out = (uint64_t*)PyLong_AsVoidPtr(args[4]);
  if (PyErr_Occurred()) return nullptr;
  const Py_ssize_t have = PyList_GET_SIZE(args[0]);
  if (have != n) return PyLong_FromSsize_t(have < n ? have : n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyList_GET_ITEM(args[0], i);
    if (!THPVariable_Check(o)) return PyLong_FromSsize_t(i);
    const at::Tensor& t = THPVariable_Unpack(o);
    const int64_t type = *want++, dims = *want++;
    const at::ScalarType s = type ? at::kBFloat16 : at::kFloat;
    bool ok = t.defined() && t.layout() == at::kStrided && t.scalar_type() == s &&
              t.is_cuda() && t.get_device() == device && t.dim() == dims && t.is_contiguous() &&
              !t.is_neg();
    for (int64_t d = 0; ok && d < dims; ++d) ok = t.size(d) == want[d];
    if (!ok) return PyLong_FromSsize_t(i);
    want += dims;
    out[i] = (uint64_t)(uintptr_t)t.data_ptr();
  }
  return PyLong_FromLong(-1);
}

// A layout: the address of int64 words, its type (0 fp32, 1 bf16, 2 int32), dimensions,
// sizes and strides.
at::ScalarType type_of(int64_t code) {
  return code == 0 ? at::kFloat : code == 1 ? at::kBFloat16 : at::kInt;
}

// pointer(tensor, layout, device): its data pointer, or None where it is not a CUDA tensor
// as the layout says (strides of dimensions of one element do not count).
PyObject* pointer(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3) {
    PyErr_SetString(PyExc_TypeError, "pointer(tensor, layout, device)");
    return nullptr;
  }
  if (!THPVariable_Check(args[0])) Py_RETURN_NONE;
  const int64_t* want = (const int64_t*)PyLong_AsVoidPtr(args[1]);
  const long device = PyLong_AsLong(args[2]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(args[0]);
  const int64_t dims = want[1];
  if (!t.defined() || t.layout() != at::kStrided || t.scalar_type() != type_of(want[0]) ||
      !t.is_cuda() || t.get_device() != device || t.dim() != dims || t.is_neg())
    Py_RETURN_NONE;
  for (int64_t d = 0; d < dims; ++d)
    if (t.size(d) != want[2 + d] || (t.size(d) > 1 && t.stride(d) != want[2 + dims + d]))
      Py_RETURN_NONE;
  return PyLong_FromVoidPtr(t.data_ptr());
}

// empty(layout, device): a new CUDA tensor of that layout, of the current stream's memory.
PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 2) {
    PyErr_SetString(PyExc_TypeError, "empty(layout, device)");
    return nullptr;
  }
  const int64_t* want = (const int64_t*)PyLong_AsVoidPtr(args[0]);
  const long device = PyLong_AsLong(args[1]);
  if (PyErr_Occurred()) return nullptr;
  const size_t dims = (size_t)want[1];
  return THPVariable_Wrap(at::empty_strided(
      at::IntArrayRef(want + 2, dims), at::IntArrayRef(want + 2 + dims, dims),
      at::TensorOptions().dtype(type_of(want[0])).device(at::kCUDA, (at::DeviceIndex)device)));
}

// A function with its C++ exceptions (no memory, a tensor without storage) as torch's.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  return F(self, args, nargs);
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"take", (PyCFunction)(void (*)())guarded<take>, METH_FASTCALL, nullptr},
    {"pointer", (PyCFunction)(void (*)())guarded<pointer>, METH_FASTCALL, nullptr},
    {"empty", (PyCFunction)(void (*)())guarded<empty>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rnnt_lists", nullptr, -1, methods,
                      nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rnnt_lists() { return PyModule_Create(&module); }
