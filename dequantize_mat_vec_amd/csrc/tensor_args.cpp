// Tensor arguments of the Python binding, checked without the interpreter: a
// call on six tensors spends 3.4 us on the checks in Python, as much as a short
// kernel takes, and 0.6 us on these.  sized() and rows() return what the
// functions of the same names in _lib.py return where every check passes, and
// call those for all else (other kinds of arguments, and the errors).
#include <Python.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* slow_sized = nullptr;
PyObject* slow_rows = nullptr;

// The tensor, if it is one on device dev with elements of `dtype` (None: any).
const at::Tensor* tensor_on(PyObject* dev, PyObject* obj, PyObject* dtype) {
  if (!THPVariable_CheckExact(obj)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(obj);
  if (!t.is_cuda() || t.get_device() != PyLong_AsLong(dev)) return nullptr;
  if (dtype != Py_None && (!THPDtype_Check(dtype) || t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type))
    return nullptr;
  return &t;
}

// sized(dev, obj, nbytes, what, dtype=None) -> pointer, int or None
PyObject* sized(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n >= 4 && PyLong_CheckExact(a[0]) && PyLong_CheckExact(a[2])) {
    if (a[1] == Py_None || PyLong_CheckExact(a[1])) {
      Py_INCREF(a[1]);
      return a[1];
    }
    const at::Tensor* t = tensor_on(a[0], a[1], n > 4 ? a[4] : Py_None);
    if (t && static_cast<long long>(t->nbytes()) >= PyLong_AsLongLong(a[2]) && t->is_contiguous() && !PyErr_Occurred())
      return PyLong_FromVoidPtr(t->data_ptr());
    PyErr_Clear();
  }
  return PyObject_Vectorcall(slow_sized, a, n, nullptr);
}

// rows(dev, obj, rows, width, stride, size, what, dtype) -> (pointer, stride)
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n == 8 && PyLong_CheckExact(a[0]) && PyLong_CheckExact(a[2]) && PyLong_CheckExact(a[3]) &&
      (a[4] == Py_None || PyLong_CheckExact(a[4])) && PyLong_CheckExact(a[5]) && a[7] != Py_None) {
    const at::Tensor* t = tensor_on(a[0], a[1], a[7]);
    if (t && t->dim() == 2 && (t->size(1) == 1 || t->stride(1) == 1)) {
      const long long count = PyLong_AsLongLong(a[2]), width = PyLong_AsLongLong(a[3]), size = PyLong_AsLongLong(a[5]);
      const long long stride = a[4] != Py_None ? PyLong_AsLongLong(a[4]) : (t->size(0) > 1 ? t->stride(0) : width);
      const long long most = 1LL << 40;
      if (!PyErr_Occurred() && size > 0 && count >= 0 && count < most && stride >= 0 && stride < most && width >= 0 &&
          width < most && count * (stride / 1024 + 1) < most) {
        const long long held = static_cast<long long>(t->storage().nbytes()) / size - t->storage_offset();
        if (count == 0 || (count - 1) * stride + width <= held)
          return Py_BuildValue("(NL)", PyLong_FromVoidPtr(t->data_ptr()), stride);
      }
      PyErr_Clear();
    }
  }
  return PyObject_Vectorcall(slow_rows, a, n, nullptr);
}

// place() -> (current device, its current stream's handle), None where there is no GPU
PyObject* place(PyObject*, PyObject* const*, Py_ssize_t) {
  try {
    const auto dev = c10::hip::current_device();
    return Py_BuildValue("(iN)", static_cast<int>(dev), PyLong_FromVoidPtr(c10::hip::getCurrentHIPStream(dev).stream()));
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// bind(sized, rows): the Python functions behind the fast ones
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "bind takes two functions");
    return nullptr;
  }
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(slow_sized, a[0]);
  Py_XSETREF(slow_rows, a[1]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"sized", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sized)), METH_FASTCALL, nullptr},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rows)), METH_FASTCALL, nullptr},
    {"place", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(place)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__tensor_args() { return PyModule_Create(&module); }
