// tensor_access.cpp -- Python extension `_tensors`: address, element count, type, device and
// contiguity of torch tensors in one call. The optimiser step takes lists of hundreds of
// tensors; asking each for these five things from Python costs the host some 0.4 us a tensor
// (60 us for 150 tensors, more than the step itself takes on the GPU), here some 10 ns.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

// zpp_dtype, then the other types that the wrappers know.
long kind_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::ScalarType::Half: return 0;
    case at::ScalarType::BFloat16: return 1;
    case at::ScalarType::Float: return 2;
    case at::ScalarType::Byte:
    case at::ScalarType::Char: return 3;
    case at::ScalarType::Float8_e4m3fn: return 4;
    default: return -1;
  }
}
long device_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }
int64_t address_of(const at::Tensor& t) {
  return t.numel() ? reinterpret_cast<int64_t>(t.data_ptr()) : 0;
}
// A strided tensor with storage (so that the questions above have answers).
bool plain(PyObject* o) {
  return THPVariable_Check(o) && THPVariable_Unpack(o).layout() == at::kStrided;
}

// scan(tensors, addresses, counts): writes every tensor's address and element count into the two
// writable int64 buffers and returns (kind, device), each -1 unless it is the same for all;
// device -2: a tensor is not contiguous.
PyObject* scan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3 || !PyList_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "scan(list of tensors, int64 buffer, int64 buffer)");
    return nullptr;
  }
  const Py_ssize_t count = PyList_GET_SIZE(args[0]);
  Py_buffer at, counts;
  if (PyObject_GetBuffer(args[1], &at, PyBUF_WRITABLE) != 0) return nullptr;
  if (PyObject_GetBuffer(args[2], &counts, PyBUF_WRITABLE) != 0) {
    PyBuffer_Release(&at);
    return nullptr;
  }
  PyObject* result = nullptr;
  if (at.len < count * 8 || counts.len < count * 8) {
    PyErr_SetString(PyExc_ValueError, "scan: buffers too small");
  } else {
    long kind = -1, device = -1;
    bool contiguous = true, ok = true;
    try {
      for (Py_ssize_t i = 0; i < count; ++i) {
        PyObject* o = PyList_GET_ITEM(args[0], i);
        if (!plain(o)) {
          PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
          ok = false;
          break;
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        static_cast<int64_t*>(at.buf)[i] = address_of(t);
        static_cast<int64_t*>(counts.buf)[i] = t.numel();
        contiguous = contiguous && t.is_contiguous();
        if (i == 0) {
          kind = kind_of(t);
          device = device_of(t);
        } else {
          if (kind_of(t) != kind) kind = -1;
          if (device_of(t) != device) device = -1;
        }
      }
    } catch (const std::exception& e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
      ok = false;
    }
    if (ok) result = Py_BuildValue("ll", kind, device >= 0 && !contiguous ? -2 : device);
  }
  PyBuffer_Release(&at);
  PyBuffer_Release(&counts);
  return result;
}

// probe(tensor): (address, elements, kind, device, contiguous).
PyObject* probe(PyObject*, PyObject* o) {
  if (!plain(o)) {
    PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
    return nullptr;
  }
  try {
    const at::Tensor& t = THPVariable_Unpack(o);
    return Py_BuildValue("LLlli", static_cast<long long>(address_of(t)),
                         static_cast<long long>(t.numel()), kind_of(t), device_of(t),
                         t.is_contiguous() ? 1 : 0);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"scan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(scan)), METH_FASTCALL,
     "addresses and element counts of a list of tensors; (kind, device)"},
    {"probe", probe, METH_O, "(address, elements, kind, device, contiguous) of a tensor"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
