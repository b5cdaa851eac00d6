// lists.cpp -- tensors' data pointers, new tensors and counts of writes, for the Python
// binding.
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

// The pointers of n dense CUDA tensors of a list into `out`; want: int64 words, for each
// tensor its type (0 fp32, 1 bf16), dimensions and sizes.  Whether they are as it says.
bool take_one(PyObject* list, Py_ssize_t n, const int64_t* want, long device, uint64_t* out) {
  if (!PyList_Check(list) || PyList_GET_SIZE(list) != n) return false;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyList_GET_ITEM(list, i);
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    const int64_t type = *want++, dims = *want++;
    const at::ScalarType s = type ? at::kBFloat16 : at::kFloat;
    if (!t.defined() || t.layout() != at::kStrided || t.scalar_type() != s || !t.is_cuda() ||
        t.get_device() != device || t.dim() != dims || !t.is_contiguous() || t.is_neg())
      return false;
    for (int64_t d = 0; d < dims; ++d)
      if (t.size(d) != want[d]) return false;
    want += dims;
    out[i] = (uint64_t)(uintptr_t)t.data_ptr();
  }
  return true;
}

// take(lists, layouts, n, device, out): the pointers of lists of n tensors each, one list
// after another, into the memory at `out`.  lists, layouts (addresses of words as above):
// tuples.  Returns -1, or the place of the first list that is not as its layout says.
PyObject* take(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 5 || !PyTuple_Check(args[0]) || !PyTuple_Check(args[1]) ||
      PyTuple_GET_SIZE(args[0]) > PyTuple_GET_SIZE(args[1])) {
    PyErr_SetString(PyExc_TypeError, "take(lists, layouts, n, device, out)");
    return nullptr;
  }
  const Py_ssize_t n = PyLong_AsSsize_t(args[2]);
  const long device = PyLong_AsLong(args[3]);
  uint64_t* out = (uint64_t*)PyLong_AsVoidPtr(args[4]);
  if (PyErr_Occurred()) return nullptr;
  for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(args[0]); ++k) {
    const int64_t* want = (const int64_t*)PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[1], k));
    if (PyErr_Occurred()) return nullptr;
    if (!take_one(PyTuple_GET_ITEM(args[0], k), n, want, device, out + k * n))
      return PyLong_FromSsize_t(k);
  }
  return PyLong_FromLong(-1);
}

// A layout: the address of int64 words, its type (0 fp32, 1 bf16, 2 int32), dimensions,
// sizes and strides.
at::ScalarType type_of(int64_t code) {
  return code == 0 ? at::kFloat : code == 1 ? at::kBFloat16 : at::kInt;
}

// Tells autograd that a kernel writes this tensor (None and tensors made under inference
// mode, which have no count: nothing).
void count_write(PyObject* o) {
  if (!THPVariable_Check(o)) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// pointer(tensor, layout, device, written): its data pointer, or None where it is not a CUDA
// tensor as the layout says (strides of dimensions of one element do not count); a tensor
// that will be written is counted.
PyObject* pointer(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 4) {
    PyErr_SetString(PyExc_TypeError, "pointer(tensor, layout, device, written)");
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
  if (args[3] == Py_True) count_write(args[0]);
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

// wrote(...): counts these tensors, or lists of them.
PyObject* wrote(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  for (Py_ssize_t k = 0; k < nargs; ++k) {
    if (!PyList_Check(args[k])) {
      count_write(args[k]);
      continue;
    }
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(args[k]); ++i)
      count_write(PyList_GET_ITEM(args[k], i));
  }
  Py_RETURN_NONE;
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
    {"wrote", (PyCFunction)(void (*)())guarded<wrote>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rnnt_lists", nullptr, -1, methods,
                      nullptr,               nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rnnt_lists() { return PyModule_Create(&module); }
