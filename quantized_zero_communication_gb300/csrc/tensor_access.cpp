// tensor_access.cpp -- Python extension `_tensors`: what the wrappers ask of torch tensors, in one
// call. The optimiser step takes lists of hundreds of tensors; asking each for its address,
// element count, type, device and contiguity from Python costs the host some 0.4 us a tensor
// (60 us for 150 tensors, more than the step itself takes on the GPU), here some 10 ns. And a
// product for one token takes the GPU 4 us: its wrapper's common case (plain contiguous
// tensors, a new output) is one call here too, 14 us of host time otherwise. The norm of 40
// small gradients takes 8 us as one call, 22 through Python.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>
#include <zpp.h>

#include <cstdint>
#include <vector>

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
long gpu_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }
// A kernel starts on the current device, whatever device its stream belongs to.
bool current(long device) { return device >= 0 && device == c10::cuda::current_device(); }
int64_t address_of(const at::Tensor& t) {
  return t.numel() ? reinterpret_cast<int64_t>(t.data_ptr()) : 0;
}
// A strided tensor with storage (so that the questions above have answers).
bool plain(PyObject* o) {
  return THPVariable_Check(o) && THPVariable_Unpack(o).layout() == at::kStrided;
}

// Python's exception for `e`: torch's own where memory ran out, as its allocations in Python raise it.
void set_error(const std::exception& e) {
  const auto* memory = dynamic_cast<const c10::OutOfMemoryError*>(&e);
  PyObject* torch = memory ? PyImport_ImportModule("torch") : nullptr;
  PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  if (type) PyErr_SetString(type, memory->what_without_backtrace());
  else if (!memory) PyErr_SetString(PyExc_RuntimeError, e.what());
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// What a list's tensors have in common.
struct Seen {
  long kind = -1, device = -1;  // -1 unless the same for all
  bool contiguous = true;
  long place() const { return device >= 0 && !contiguous ? -2 : device; }
};
// Calls each(i, tensor) for the list's tensors; false with an error set.
template <typename F>
bool look(PyObject* list, Seen& seen, const F& each) {
  const Py_ssize_t count = PyList_GET_SIZE(list);
  try {
    for (Py_ssize_t i = 0; i < count; ++i) {
      PyObject* o = PyList_GET_ITEM(list, i);
      if (!plain(o)) {
        PyErr_Format(PyExc_TypeError, "expected a tensor, got %s", Py_TYPE(o)->tp_name);
        return false;
      }
      const at::Tensor& t = THPVariable_Unpack(o);
      const long kind = kind_of(t), device = gpu_of(t);
      seen.contiguous = seen.contiguous && t.is_contiguous();
      seen.kind = i == 0 || kind == seen.kind ? kind : -1;
      seen.device = i == 0 || device == seen.device ? device : -1;
      each(i, t);
    }
  } catch (const std::exception& e) {
    set_error(e);
    return false;
  }
  return true;
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
    Seen seen;
    if (look(args[0], seen, [&](Py_ssize_t i, const at::Tensor& t) {
          static_cast<int64_t*>(at.buf)[i] = address_of(t);
          static_cast<int64_t*>(counts.buf)[i] = t.numel();
        }))
      result = Py_BuildValue("ll", seen.kind, seen.place());
  }
  PyBuffer_Release(&at);
  PyBuffer_Release(&counts);
  return result;
}

// enter(tensors, table, column, sizes): writes every tensor's address into its row of the
// writable int64 table [.][8], at `column`; (kind, device, same), kind and device as of scan,
// same: every element count equals that in the int64 buffer `sizes`.
PyObject* enter(PyObject*, PyObject* const* args, Py_ssize_t n) {
  const long column = n == 4 ? PyLong_AsLong(args[2]) : -1;
  if (n != 4 || !PyList_Check(args[0]) || column < 0 || column > 7) {
    PyErr_SetString(PyExc_TypeError, "enter(list of tensors, int64 table, column, int64 buffer)");
    return nullptr;
  }
  const Py_ssize_t count = PyList_GET_SIZE(args[0]);
  Py_buffer table, sizes;
  if (PyObject_GetBuffer(args[1], &table, PyBUF_WRITABLE) != 0) return nullptr;
  if (PyObject_GetBuffer(args[3], &sizes, PyBUF_SIMPLE) != 0) {
    PyBuffer_Release(&table);
    return nullptr;
  }
  PyObject* result = nullptr;
  if (table.len < count * 64 || sizes.len < count * 8) {
    PyErr_SetString(PyExc_ValueError, "enter: buffers too small");
  } else {
    Seen seen;
    bool same = true;
    if (look(args[0], seen, [&](Py_ssize_t i, const at::Tensor& t) {
          static_cast<int64_t*>(table.buf)[8 * i + column] = address_of(t);
          same = same && t.numel() == static_cast<const int64_t*>(sizes.buf)[i];
        }))
      result = Py_BuildValue("lli", seen.kind, seen.place(), same ? 1 : 0);
  }
  PyBuffer_Release(&table);
  PyBuffer_Release(&sizes);
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
                         static_cast<long long>(t.numel()), kind_of(t), gpu_of(t),
                         t.is_contiguous() ? 1 : 0);
  } catch (const std::exception& e) {
    set_error(e);
    return nullptr;
  }
}

// matvec(address of zpp_matvec_blockwise, codes, scales, x, rows, block, bits, bias or None, out
// kind or -1): the product in a new tensor, a status other than ZPP_OK as an int, or None where
// something is not the plain case (the Python wrapper then finds out what).
PyObject* matvec(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 9) {
    PyErr_SetString(PyExc_TypeError, "matvec: 9 arguments");
    return nullptr;
  }
  if (!plain(args[1]) || !plain(args[2]) || !plain(args[3])) Py_RETURN_NONE;
  const bool has_bias = args[7] != Py_None;
  if (has_bias && !plain(args[7])) Py_RETURN_NONE;
  const long long rows = PyLong_AsLongLong(args[4]), block = PyLong_AsLongLong(args[5]),
                  bits = PyLong_AsLongLong(args[6]), out = PyLong_AsLongLong(args[8]);
  void* fn = PyLong_AsVoidPtr(args[0]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  try {
    const at::Tensor &codes = THPVariable_Unpack(args[1]), &scales = THPVariable_Unpack(args[2]),
                     &x = THPVariable_Unpack(args[3]);
    const long kind = kind_of(x), device = gpu_of(x);
    if (!current(device) || (kind != ZPP_F16 && kind != ZPP_BF16) || x.dim() < 1 || !x.is_contiguous())
      Py_RETURN_NONE;
    const int64_t cols = x.size(-1);
    if (cols < 1 || rows < 0 || rows > ZPP_MAX_ELEMS / cols) Py_RETURN_NONE;
    if ((bits != 4 && bits != 8) || block < ZPP_MIN_BLOCK || block > ZPP_MAX_BLOCK) Py_RETURN_NONE;
    const int64_t total = rows * cols;
    if (kind_of(codes) != 3 || kind_of(scales) != ZPP_F32 || gpu_of(codes) != device ||
        gpu_of(scales) != device || !codes.is_contiguous() || !scales.is_contiguous() ||
        codes.numel() != (bits == 8 ? total : (total + 1) / 2) ||
        scales.numel() != (total + block - 1) / block)
      Py_RETURN_NONE;
    const void* bias = nullptr;
    if (has_bias) {
      const at::Tensor& b = THPVariable_Unpack(args[7]);
      if (kind_of(b) != kind || b.numel() != rows || gpu_of(b) != device || !b.is_contiguous())
        Py_RETURN_NONE;
      bias = reinterpret_cast<const void*>(address_of(b));
    }
    const long y_kind = out < 0 ? kind : static_cast<long>(out);
    if (y_kind > ZPP_F32) Py_RETURN_NONE;
    std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = rows;
    at::Tensor y = at::empty(shape, x.options().dtype(y_kind == ZPP_F16    ? at::kHalf
                                                      : y_kind == ZPP_BF16 ? at::kBFloat16
                                                                           : at::kFloat));
    const zpp_status st = reinterpret_cast<decltype(&zpp_matvec_blockwise)>(fn)(
        reinterpret_cast<const void*>(address_of(codes)),
        reinterpret_cast<const float*>(address_of(scales)), rows, cols, static_cast<int32_t>(block),
        static_cast<int32_t>(bits), reinterpret_cast<const void*>(address_of(x)),
        static_cast<zpp_dtype>(kind), x.numel() / cols, cols, bias,
        reinterpret_cast<void*>(address_of(y)), static_cast<zpp_dtype>(y_kind), rows,
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
    if (st != ZPP_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(y));
  } catch (const std::exception& e) {
    set_error(e);
    return nullptr;
  }
}

// grad_norm(address of zpp_grad_norm, address of zpp_grad_norm_workspace, list of gradients,
// max_norm, pre_scale): (norm, factor) in a new tensor, a status other than ZPP_OK as an int, or
// None where something is not the plain case.
PyObject* grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "grad_norm: 5 arguments");
    return nullptr;
  }
  const auto number = [](PyObject* o) { return PyFloat_Check(o) || PyLong_Check(o); };
  if (!PyList_Check(args[2]) || !number(args[3]) || !number(args[4])) Py_RETURN_NONE;
  void* fn = PyLong_AsVoidPtr(args[0]);
  void* workspace = PyLong_AsVoidPtr(args[1]);
  const double max_norm = PyFloat_AsDouble(args[3]), pre_scale = PyFloat_AsDouble(args[4]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const Py_ssize_t count = PyList_GET_SIZE(args[2]);
  if (count < 1 || count > INT32_MAX) Py_RETURN_NONE;
  try {
    std::vector<const void*> at(count);
    std::vector<int64_t> counts(count);
    int64_t total = 0;
    Seen seen;
    if (!look(args[2], seen, [&](Py_ssize_t i, const at::Tensor& t) {
          at[i] = reinterpret_cast<const void*>(address_of(t));
          counts[i] = t.numel();
          total += counts[i];
        })) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    const long kind = seen.kind, device = seen.place();
    if (kind < 0 || kind > ZPP_F32 || !current(device)) Py_RETURN_NONE;
    const int64_t floats = reinterpret_cast<decltype(&zpp_grad_norm_workspace)>(workspace)(
        total, static_cast<int32_t>(count));
    if (floats < 0) Py_RETURN_NONE;
    const auto options = THPVariable_Unpack(PyList_GET_ITEM(args[2], 0)).options().dtype(at::kFloat);
    at::Tensor out = at::empty({2}, options);
    const at::Tensor work = at::empty({floats}, options);
    const zpp_status st = reinterpret_cast<decltype(&zpp_grad_norm)>(fn)(
        at.data(), counts.data(), static_cast<int32_t>(count), static_cast<zpp_dtype>(kind),
        static_cast<float>(pre_scale), static_cast<float>(max_norm),
        reinterpret_cast<float*>(address_of(work)), reinterpret_cast<float*>(address_of(out)),
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
    if (st != ZPP_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(out));
  } catch (const std::exception& e) {
    set_error(e);
    return nullptr;
  }
}

// step(address of zpp_adamw_step_counted, int64 table [tensors][8], gradients' kind, weights' kind,
// state bits, address of the zpp_adamw_params, address of the gradients' scale or 0, None or (max_norm,
// pre_scale, floats of workspace), address of the record, device): one counted step on the device's
// current stream; (norm, factor) in a new tensor, None without clipping, or a status other than
// ZPP_OK as an int; False, with nothing done, where the device is not the current one. While the stream is captured the number of the step is left to the device,
// whose count a replay moves on: hp->step is set to 0.
PyObject* step(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 10) {
    PyErr_SetString(PyExc_TypeError, "step: 10 arguments");
    return nullptr;
  }
  const auto fn = reinterpret_cast<decltype(&zpp_adamw_step_counted)>(PyLong_AsVoidPtr(args[0]));
  const long g_kind = PyLong_AsLong(args[2]), w_kind = PyLong_AsLong(args[3]),
             bits = PyLong_AsLong(args[4]), device = PyLong_AsLong(args[9]);
  auto* hp = static_cast<zpp_adamw_params*>(PyLong_AsVoidPtr(args[5]));
  const void* scale = PyLong_AsVoidPtr(args[6]);
  void* record = PyLong_AsVoidPtr(args[8]);
  double max_norm = 0.0, pre_scale = 0.0;
  long long floats = 0;
  const bool clipped = args[7] != Py_None;
  if (PyErr_Occurred() || (clipped && !PyArg_ParseTuple(args[7], "ddL", &max_norm, &pre_scale, &floats)))
    return nullptr;
  Py_buffer table;
  if (PyObject_GetBuffer(args[1], &table, PyBUF_SIMPLE) != 0) return nullptr;
  PyObject* result = nullptr;
  try {
    if (!current(device)) {
      PyBuffer_Release(&table);
      Py_RETURN_FALSE;
    }
    const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device));
    if (hp->step > 0 &&
        c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
      hp->step = 0;
    at::Tensor norm, work;
    zpp_adamw_clip clip{};
    if (clipped) {
      const auto options = at::TensorOptions().dtype(at::kFloat).device(
          at::kCUDA, static_cast<c10::DeviceIndex>(device));
      norm = at::empty({2}, options);
      work = at::empty({floats}, options);
      clip.max_norm = static_cast<float>(max_norm);
      clip.pre_scale = static_cast<float>(pre_scale);
      clip.workspace = reinterpret_cast<float*>(address_of(work));
      clip.out = reinterpret_cast<float*>(address_of(norm));
    }
    const zpp_status st =
        fn(static_cast<const zpp_adamw_tensor*>(table.buf),
           static_cast<int32_t>(table.len / static_cast<Py_ssize_t>(sizeof(zpp_adamw_tensor))),
           static_cast<zpp_dtype>(g_kind), static_cast<zpp_dtype>(w_kind), static_cast<int32_t>(bits), hp,
           static_cast<const float*>(scale), clipped ? &clip : nullptr,
           static_cast<zpp_adamw_record*>(record), stream.stream());
    if (st != ZPP_OK) result = PyLong_FromLong(st);
    else if (clipped) result = THPVariable_Wrap(std::move(norm));
    else result = Py_NewRef(Py_None);
  } catch (const std::exception& e) {
    set_error(e);
  }
  PyBuffer_Release(&table);
  return result;
}

PyMethodDef methods[] = {
    {"step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(step)), METH_FASTCALL,
     "one counted AdamW step from a table of addresses"},
    {"grad_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grad_norm)),
     METH_FASTCALL, "the norm of a list of gradients, plain case"},
    {"scan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(scan)), METH_FASTCALL,
     "addresses and element counts of a list of tensors; (kind, device)"},
    {"enter", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(enter)), METH_FASTCALL,
     "addresses of a list of tensors into a column of a table; (kind, device, same sizes)"},
    {"matvec", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matvec)), METH_FASTCALL,
     "the product with a quantised matrix, plain case"},
    {"probe", probe, METH_O, "(address, elements, kind, device, contiguous) of a tensor"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
