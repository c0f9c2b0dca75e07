// tensor_access.cpp -- Python extension `_tensors`: what the wrappers ask of torch tensors, in one
// call. The optimiser step takes lists of hundreds of tensors; asking each for its address,
// element count, type, device and contiguity from Python costs the host some 0.4 us a tensor
// (60 us for 150 tensors, more than the step itself takes on the GPU), here some 10 ns. And a
// product for one token takes the GPU 4 us: its wrapper's common case (plain contiguous
// tensors, a new output) is one call here too, 14 us of host time otherwise. The norm of 40
// small gradients takes 8 us as one call, 22 through Python. A training pass of a small linear layer
// in fp8 is six kernels of 43 us together, which took the host 600 us through Python's autograd
// functions and wrappers: here it is a C++ autograd function.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
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

// Python's exception for `e`: torch's own where memory ran out, as its allocations in Python raise it, and one that
// Python code raised on the way (a hook on saved tensors; checkpoints stop a recomputation with one) as it is.
void set_error(const std::exception& e) {
  if (const auto* raised = dynamic_cast<const python_error*>(&e)) {
    python_error(*raised).restore();
    return;
  }
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

// ------------------------------------------------------------------------------ e4m3 matrices
at::ScalarType type_of(long kind) {
  return kind == ZPP_F16 ? at::kHalf : kind == ZPP_BF16 ? at::kBFloat16 : at::kFloat;
}
using QuantFp8 = decltype(&zpp_quant_fp8);
using MatmulFp8 = decltype(&zpp_matmul_fp8);
cudaStream_t stream_of(long device) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
}
int64_t blocks_of(int64_t n) { return (n + ZPP_FP8_BLOCK - 1) / ZPP_FP8_BLOCK; }

// New codes of a matrix of `shape`, rows at multiples of 16 bytes, and its scales.
struct Coded {
  at::Tensor codes, scales;
};
at::Tensor new_codes(at::IntArrayRef shape, const at::TensorOptions& like) {
  std::vector<int64_t> strides(shape.size(), 1);
  int64_t apart = (shape.back() + 15) / 16 * 16;
  for (size_t k = shape.size() - 1; k-- > 0;) strides[k] = apart, apart *= shape[k];
  return at::empty_strided(shape, strides, like.dtype(at::kFloat8_e4m3fn));
}
Coded new_coded(at::IntArrayRef shape, int64_t rows, int64_t tile, const at::TensorOptions& like) {
  const int64_t across = blocks_of(shape.back()), down = tile == 1 ? rows : blocks_of(rows);
  const auto floats = like.dtype(at::kFloat);
  return {new_codes(shape, like), tile == 1 ? at::empty_strided({down, across}, {1, down}, floats)
                                            : at::empty({down, across}, floats)};
}
zpp_fp8_matrix matrix_of(const Coded& c, int64_t rows, int64_t cols, int64_t tile) {
  zpp_fp8_matrix m{};
  m.codes = c.codes.data_ptr();
  m.scales = static_cast<float*>(c.scales.data_ptr());
  m.rows = rows;
  m.cols = cols;
  m.stride = rows > 1 ? c.codes.stride(-2) : (cols + 15) / 16 * 16;
  m.scale_row = c.scales.stride(0);
  m.scale_block = c.scales.stride(1);
  m.tile = static_cast<int32_t>(tile);
  return m;
}
// x, contiguous with at least one row, to codes; with `turned` its transpose's too.
zpp_status quantise(QuantFp8 fn, const at::Tensor& x, int64_t tile, Coded& to, Coded* turned) {
  const int64_t cols = x.size(-1), rows = x.numel() / cols;
  to = new_coded(x.sizes(), rows, tile, x.options());
  const zpp_fp8_matrix m = matrix_of(to, rows, cols, tile);
  zpp_fp8_matrix t{};
  if (turned) {
    if (tile == 1) *turned = new_coded({cols, rows}, cols, 1, x.options());
    else *turned = {new_codes({cols, rows}, x.options()), to.scales.t()};
    t = matrix_of(*turned, cols, rows, tile);
  }
  return fn(x.data_ptr(), static_cast<zpp_dtype>(kind_of(x)), cols, &m, turned ? &t : nullptr, stream_of(gpu_of(x)));
}

// quant_fp8(address of zpp_quant_fp8, x, tile, transposed): the codes and scales as a tuple, a status
// other than ZPP_OK as an int, or None where something is not the plain case.
PyObject* quant_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "quant_fp8: 4 arguments");
    return nullptr;
  }
  if (!plain(args[1])) Py_RETURN_NONE;
  const auto fn = reinterpret_cast<QuantFp8>(PyLong_AsVoidPtr(args[0]));
  const long tile = PyLong_AsLong(args[2]);
  const int transposed = PyObject_IsTrue(args[3]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  try {
    const at::Tensor& x = THPVariable_Unpack(args[1]);
    const long kind = kind_of(x);
    if ((tile != 1 && tile != 128) || kind < 0 || kind > ZPP_F32 || !current(gpu_of(x)) || x.dim() < 1 ||
        !x.is_contiguous() || x.numel() == 0)
      Py_RETURN_NONE;
    Coded c, t;
    const zpp_status st = quantise(fn, x.detach(), tile, c, transposed ? &t : nullptr);
    if (st != ZPP_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(transposed ? 4 : 2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(c.codes)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(c.scales)));
    if (transposed) {
      PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(std::move(t.codes)));
      PyTuple_SET_ITEM(out, 3, THPVariable_Wrap(std::move(t.scales)));
    }
    return out;
  } catch (const std::exception& e) {
    set_error(e);
    return nullptr;
  }
}

// A 2-D matrix of codes as the library takes it; false where something is not the plain case.
bool coded_matrix(const at::Tensor& codes, const at::Tensor& scales, long device, zpp_fp8_matrix& m) {
  if (kind_of(codes) != 4 || kind_of(scales) != ZPP_F32 || gpu_of(codes) != device || gpu_of(scales) != device ||
      codes.dim() != 2 || scales.dim() != 2)
    return false;
  const int64_t rows = codes.size(0), cols = codes.size(1);
  if (rows < 1 || cols < 1 || (cols > 1 && codes.stride(1) != 1) || scales.size(1) != blocks_of(cols)) return false;
  const bool by_rows = scales.size(0) == rows;
  if (!by_rows && scales.size(0) != blocks_of(rows)) return false;
  m = matrix_of({codes, scales}, rows, cols, by_rows ? 1 : 128);
  return m.stride >= cols && m.stride % 16 == 0 && reinterpret_cast<uintptr_t>(m.codes) % 16 == 0;
}

// matmul_fp8(address of zpp_matmul_fp8, a, a_scales, b, b_scales, bias or None, out kind): the product in a
// new tensor, a status other than ZPP_OK as an int, or None where something is not the plain case.
PyObject* matmul_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "matmul_fp8: 7 arguments");
    return nullptr;
  }
  for (int i = 1; i <= 4; ++i)
    if (!plain(args[i])) Py_RETURN_NONE;
  const bool has_bias = args[5] != Py_None;
  if (has_bias && !plain(args[5])) Py_RETURN_NONE;
  const auto fn = reinterpret_cast<MatmulFp8>(PyLong_AsVoidPtr(args[0]));
  const long kind = PyLong_AsLong(args[6]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  try {
    const at::Tensor& a = THPVariable_Unpack(args[1]);
    const long device = gpu_of(a);
    zpp_fp8_matrix ma, mb;
    if (!current(device) || kind < 0 || kind > ZPP_F32 ||
        !coded_matrix(a, THPVariable_Unpack(args[2]), device, ma) ||
        !coded_matrix(THPVariable_Unpack(args[3]), THPVariable_Unpack(args[4]), device, mb) || ma.cols != mb.cols)
      Py_RETURN_NONE;
    const void* bias = nullptr;
    if (has_bias) {
      const at::Tensor& t = THPVariable_Unpack(args[5]);
      if (kind_of(t) != kind || t.numel() != mb.rows || gpu_of(t) != device || !t.is_contiguous()) Py_RETURN_NONE;
      bias = t.data_ptr();
    }
    at::Tensor y = at::empty({ma.rows, mb.rows}, a.options().dtype(type_of(kind)));
    const zpp_status st =
        fn(&ma, &mb, bias, y.data_ptr(), static_cast<zpp_dtype>(kind), mb.rows, stream_of(device));
    if (st != ZPP_OK) return PyLong_FromLong(st);
    return THPVariable_Wrap(std::move(y));
  } catch (const std::exception& e) {
    set_error(e);
    return nullptr;
  }
}

// The fp8 linear layer as an autograd function: see linear.py.
// Raises binding.ZppError, as the other calls do (a backward pass runs outside Python: its exception travels as one).
void demand(zpp_status st, const char* where) {
  if (st == ZPP_OK) return;
  const PyGILState_STATE gil = PyGILState_Ensure();
  PyObject* binding = PyImport_ImportModule("quantized_zero_communication_gb300.binding");
  PyObject* type = binding ? PyObject_GetAttrString(binding, "ZppError") : nullptr;
  PyObject* error = type ? PyObject_CallFunction(type, "is", static_cast<int>(st), where) : nullptr;
  if (error) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(binding);
  python_error raised;
  raised.persist();
  PyGILState_Release(gil);
  throw raised;
}
at::Tensor product(MatmulFp8 fn, const at::Tensor& a, const at::Tensor& a_scales, int64_t a_tile,
                   const at::Tensor& b, const at::Tensor& b_scales, int64_t b_tile, at::ScalarType type) {
  at::Tensor y = at::empty({a.size(0), b.size(0)}, a.options().dtype(type));
  if (y.numel() == 0) return y;
  const zpp_fp8_matrix ma = matrix_of({a, a_scales}, a.size(0), a.size(1), a_tile),
                       mb = matrix_of({b, b_scales}, b.size(0), b.size(1), b_tile);
  demand(fn(&ma, &mb, nullptr, y.data_ptr(), static_cast<zpp_dtype>(kind_of(y)), y.size(1), stream_of(gpu_of(y))),
         "zpp_matmul_fp8");
  return y;
}
// What the graph kept of a matrix [rows, cols], as a product takes it. Hooks may have put copies in its place: those of
// codes come back from the host without the padding of their rows, and are laid out again.
Coded kept(const at::Tensor& codes, const at::Tensor& scales, int64_t rows, int64_t cols, int64_t tile, long device) {
  const std::vector<int64_t> shape{rows, cols}, of_scales{tile == 1 ? rows : blocks_of(rows), blocks_of(cols)};
  TORCH_CHECK(codes.defined() && scales.defined() && kind_of(codes) == 4 && kind_of(scales) == ZPP_F32 &&
                  gpu_of(codes) == device && gpu_of(scales) == device && codes.sizes() == shape &&
                  scales.sizes() == of_scales,
              "linear_fp8: a saved tensor came back with another shape, type or device");
  const bool fits = (cols == 1 || codes.stride(1) == 1) &&
                    (rows == 1 || (codes.stride(0) >= cols && codes.stride(0) % 16 == 0)) &&
                    reinterpret_cast<uintptr_t>(codes.data_ptr()) % 16 == 0;
  if (fits) return {codes, scales};
  at::Tensor again = new_codes(shape, codes.options());
  again.copy_(codes);
  return {again, scales};
}
// A captured backward pass cannot hand a gradient to the default stream, which takes no part in captures. It
// would have to where the tensor's place in the graph was made there and is still held, by an eager
// pass of the same leaf for one; the engine's own failure at that point ends the process.
void demand_stream(torch::autograd::Node& of, size_t edge, const char* name) {
  const auto& to = of.next_edge(edge).function;
  const auto stream = to ? to->stream() : std::nullopt;
  TORCH_CHECK(!stream || c10::cuda::CUDAStream(*stream) != c10::cuda::getDefaultCUDAStream(stream->device_index()),
              "linear_fp8: this backward pass is captured, and ", name,
              "'s gradient would go to the default stream, where a graph that is still alive was made; "
              "drop that graph's outputs first, or make it on another stream");
}
struct Linear : torch::autograd::Function<Linear> {
  // held: the weight's codes, scales and those of its transpose, or none. (By pointer: a list of tensors
  // would count as inputs with gradients of their own.)
  static at::Tensor forward(torch::autograd::AutogradContext* ctx, const at::Tensor& x, const at::Tensor& weight,
                            const std::vector<at::Tensor>* held, int64_t quant, int64_t matmul, bool for_x,
                            bool for_w) {
    const c10::cuda::CUDAGuard guard(x.device());
    const auto quant_fn = reinterpret_cast<QuantFp8>(quant);
    const auto matmul_fn = reinterpret_cast<MatmulFp8>(matmul);
    const at::Tensor rows = x.reshape({-1, x.size(-1)}).contiguous();
    Coded w, wt, q, qt;
    if (!held->empty()) {
      w = {held->at(0), held->at(1)};
      if (held->size() == 4) wt = {held->at(2), held->at(3)};
    } else if (weight.numel()) {
      demand(quantise(quant_fn, weight.contiguous(), 128, w, for_x ? &wt : nullptr), "zpp_quant_fp8");
    }
    std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = weight.size(0);
    at::Tensor y;
    if (rows.size(0) && weight.size(0)) {
      demand(quantise(quant_fn, rows, 1, q, for_w ? &qt : nullptr), "zpp_quant_fp8");
      y = product(matmul_fn, q.codes, q.scales, 1, w.codes, w.scales, 128, x.scalar_type()).view(shape);
    } else {
      y = at::empty(shape, x.options());
    }
    // (to what is saved a later write is noticed)
    ctx->save_for_backward({for_x ? wt.codes : at::Tensor(), for_x ? wt.scales : at::Tensor(),
                            for_w ? qt.codes : at::Tensor(), for_w ? qt.scales : at::Tensor()});
    ctx->saved_data["fns"] = std::vector<int64_t>{quant, matmul};
    ctx->saved_data["x"] = x.sizes().vec();
    ctx->saved_data["types"] = std::vector<int64_t>{static_cast<int64_t>(x.scalar_type()),
                                                    static_cast<int64_t>(weight.scalar_type()), for_x, for_w};
    return y;
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    const auto saved = ctx->get_saved_variables();
    const auto fns = ctx->saved_data["fns"].toIntVector(), shape = ctx->saved_data["x"].toIntVector(),
               types = ctx->saved_data["types"].toIntVector();
    const auto quant_fn = reinterpret_cast<QuantFp8>(fns[0]);
    const auto matmul_fn = reinterpret_cast<MatmulFp8>(fns[1]);
    const auto x_type = static_cast<at::ScalarType>(types[0]), w_type = static_cast<at::ScalarType>(types[1]);
    torch::autograd::variable_list out(7);
    if (!grads[0].defined()) return out;
    const bool twice = at::GradMode::is_enabled();
    const bool for_x = types[2] && ctx->needs_input_grad(0), for_w = types[3] && ctx->needs_input_grad(1);
    {
      const at::NoGradGuard no_grad;
      const at::Tensor& dy = grads[0];
      const c10::cuda::CUDAGuard guard(dy.device());
      if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
        const auto node = torch::autograd::get_current_node();
        if (for_x) demand_stream(*node, 0, "x");
        if (for_w) demand_stream(*node, 1, "weight");
      }
      const int64_t n = dy.size(-1), k = shape.back();
      int64_t count = 1;
      for (size_t i = 0; i + 1 < shape.size(); ++i) count *= shape[i];
      const bool empty = count == 0 || n == 0;
      Coded q, qt;
      if (!empty)
        demand(quantise(quant_fn, dy.reshape({count, n}).contiguous(), 1, q, for_w ? &qt : nullptr), "zpp_quant_fp8");
      if (for_x && empty) out[0] = at::zeros(shape, dy.options().dtype(x_type));
      if (for_w && empty) out[1] = at::zeros({n, k}, dy.options().dtype(w_type));
      if (for_x && !empty) {
        const Coded wt = kept(saved[0], saved[1], k, n, 128, gpu_of(dy));
        out[0] = product(matmul_fn, q.codes, q.scales, 1, wt.codes, wt.scales, 128, x_type).view(shape);
      }
      if (for_w && !empty) {
        const Coded xt = kept(saved[2], saved[3], k, count, 1, gpu_of(dy));
        out[1] = product(matmul_fn, qt.codes, qt.scales, 1, xt.codes, xt.scales, 1, w_type);
      }
    }
    if (twice) {  // differentiable once: a derivative of these raises
      auto error = std::make_shared<torch::autograd::DelayedError>(
          "linear_fp8 is differentiable once, and this is its second derivative", 7);
      torch::autograd::variable_list in;
      for (int i = 0; i < 2; ++i)
        if (out[i].defined()) in.push_back(out[i].detach().requires_grad_());
      auto marked = (*error)(std::move(in));
      for (int i = 0, j = 0; i < 2; ++i)
        if (out[i].defined()) out[i] = marked[j++];
    }
    return out;
  }
};

// linear_fp8(address of zpp_quant_fp8, address of zpp_matmul_fp8, x, weight, None or a tuple of the
// weight's codes and scales): y. The arguments have been checked.
PyObject* linear_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5 || !plain(args[2]) || !plain(args[3])) {
    PyErr_SetString(PyExc_TypeError, "linear_fp8: two addresses, x, weight, codes");
    return nullptr;
  }
  const int64_t quant = reinterpret_cast<int64_t>(PyLong_AsVoidPtr(args[0])),
                matmul = reinterpret_cast<int64_t>(PyLong_AsVoidPtr(args[1]));
  if (PyErr_Occurred()) return nullptr;
  try {
    std::vector<at::Tensor> held;
    if (PyTuple_Check(args[4]))
      for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args[4]); ++i)
        held.push_back(THPVariable_Unpack(PyTuple_GET_ITEM(args[4], i)));
    const at::Tensor &x = THPVariable_Unpack(args[2]), &w = THPVariable_Unpack(args[3]);
    const bool grads = at::GradMode::is_enabled();
    return THPVariable_Wrap(
        Linear::apply(x, w, static_cast<const std::vector<at::Tensor>*>(&held), quant, matmul, grads && x.requires_grad(), grads && w.requires_grad()));
  } catch (const std::exception& e) {
    set_error(e);
    return nullptr;
  }
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
    {"quant_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quant_fp8)), METH_FASTCALL,
     "a matrix to e4m3 codes, plain case"},
    {"matmul_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matmul_fp8)), METH_FASTCALL,
     "the product of e4m3 matrices, plain case"},
    {"linear_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_fp8)), METH_FASTCALL,
     "the fp8 linear layer, differentiable"},
    {"probe", probe, METH_O, "(address, elements, kind, device, contiguous) of a tensor"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
