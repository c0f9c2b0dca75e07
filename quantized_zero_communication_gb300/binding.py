"""ctypes binding of ``libzpp.so`` (argument marshalling only).

The raw functions carry the C names and take device addresses as integers; the tensor
helpers below allocate outputs with torch on the input's device, pass pointers and the
current CUDA stream, and raise on a non-OK status. Every step of the computation runs
in the library's kernels: there is no CPU path, and a missing library or a CPU tensor
is an error.
"""
import array
import ctypes
import functools
import math
import os
import re

from . import build as _build

ZPP_OK, ZPP_ERR_INVALID_ARG, ZPP_ERR_MISALIGNED, ZPP_ERR_UNSUPPORTED, ZPP_ERR_CUDA = range(5)
ZPP_F16, ZPP_BF16, ZPP_F32 = 0, 1, 2
ZPP_STATE_BLOCK, ZPP_MAX_TENSORS = 256, 1024

HEADER = os.path.join(_build.ROOT, "include", "zpp.h")


class Topology(ctypes.Structure):
    _fields_ = [("num_nodes", ctypes.c_int32), ("gpus_per_node", ctypes.c_int32)]


class LocalRange(ctypes.Structure):
    _fields_ = [("begin", ctypes.c_int32), ("end", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    """One tensor of zpp_adamw_step (device addresses, element count)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq",
                                               "exp_avg_scale", "exp_avg_sq_scale", "weight")] + [
        ("n", ctypes.c_int64)]


class AdamwParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps",
                                               "weight_decay")] + [
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint32)]


class AdamwClip(ctypes.Structure):
    _fields_ = [("pre_scale", ctypes.c_float), ("max_norm", ctypes.c_float),
                ("workspace", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class Fp8Matrix(ctypes.Structure):
    """A matrix of e4m3 codes (zpp_fp8_matrix): device addresses, sizes and strides."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("rows", "cols", "stride", "scale_row", "scale_block")] + [
        ("tile", ctypes.c_int32)]


class NewtonSchulz(ctypes.Structure):
    """Steps, their coefficients (the address of [steps][3] doubles) and eps (zpp_newton_schulz)."""
    _fields_ = [("coefficients", ctypes.c_void_p), ("steps", ctypes.c_int32), ("eps", ctypes.c_double)]


class Matrix(ctypes.Structure):
    """One matrix of zpp_orthogonalize."""
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class MuonTensor(ctypes.Structure):
    """One matrix of zpp_muon_step (device addresses, sizes)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "momentum", "weight")] + [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MuonParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "momentum", "weight_decay")] + [
        ("nesterov", ctypes.c_int32), ("adjust", ctypes.c_int32), ("ns", NewtonSchulz)]


class ZppError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {zpp_status_string(status)}")


_lib = None


def lib_path():
    return _build.LIB


def lib():
    """Load libzpp.so (it must have been built: ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"{_build.LIB} is missing: build it with __graft_entry__.build() "
                           "(there is no fallback path)")
    L = ctypes.CDLL(_build.LIB)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    sig = {
        "zpp_quant_blockwise": [vp, i32, i64, i32, i32, vp, vp, vp],
        "zpp_dequant_blockwise": [vp, vp, i64, i32, i32, vp, i32, vp],
        "zpp_qgz_reorder_quant": [vp, i32, i64, i32, i32, Topology, vp, vp, vp],
        "zpp_dequant_reduce_requant": [vp, vp, i64, i32, i32, Topology, vp, vp, vp],
        "zpp_dequant_reduce": [vp, vp, i64, i32, i32, Topology, vp, vp],
        "zpp_dequant_reduce_scaled": [vp, vp, i64, i32, i32, Topology, ctypes.c_float, vp, i32,
                                      vp],
        "zpp_qgz_reorder_quant_range": [vp, i32, i64, i32, i32, Topology, LocalRange, vp, vp, vp],
        "zpp_qgz_reorder_quant_tensors": [vp, vp, i32, i32, i32, i32, Topology, vp, vp, vp],
        "zpp_dequant_reduce_requant_range": [vp, vp, i64, i32, i32, Topology, LocalRange, vp, vp,
                                             vp],
        "zpp_dequant_reduce_scaled_range": [vp, vp, i64, i32, i32, Topology, LocalRange,
                                            ctypes.c_float, vp, i32, vp],
        "zpp_device_copy": [vp, vp, i64, vp],
        "zpp_qgz_reorder_quant_local": [vp, i32, i64, i32, i32, Topology, LocalRange, vp, vp,
                                        vp],
        "zpp_dequant_reduce_requant_local": [vp, vp, i64, i32, i32, i32, vp, vp, vp],
        "zpp_dequant_reduce_local": [vp, vp, i64, i32, i32, i32, ctypes.c_float, vp, i32, vp],
        "zpp_device_fault": [ctypes.POINTER(ctypes.c_uint32), i32],
        "zpp_wait_selftest": [ctypes.c_uint64, vp],
        "zpp_grad_norm": [vp, vp, i32, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp],
        "zpp_adamw_step": [vp, i32, i32, i32, i32, vp, vp, vp],
        "zpp_adamw_step_counted": [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp],
        "zpp_matvec_blockwise": [vp, vp, i64, i64, i32, i32, vp, i32, i64, i64, vp, vp, i32, i64,
                                 vp],
        "zpp_quant_fp8": [vp, i32, i64, vp, vp, vp],
        "zpp_matmul_fp8": [vp, vp, vp, vp, i32, i64, vp],
        "zpp_orthogonalize": [vp, i32, i32, i32, vp, vp, vp],
        "zpp_muon_step": [vp, i32, i32, i32, vp, vp, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    L.zpp_code_bytes.argtypes = [i64, i32]
    L.zpp_code_bytes.restype = i64
    L.zpp_num_scales.argtypes = [i64, i32]
    L.zpp_num_scales.restype = i64
    L.zpp_grad_norm_workspace.argtypes = [i64, i32]
    L.zpp_grad_norm_workspace.restype = i64
    for name in ("zpp_orthogonalize_workspace", "zpp_muon_workspace"):
        getattr(L, name).argtypes = [vp, i32]
        getattr(L, name).restype = i64
    L.zpp_status_string.argtypes = [ctypes.c_int]
    L.zpp_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def declared_symbols(header=HEADER):
    """Names of the functions the public header declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"ZPP_API\s+[\w\s\*]*?\b(zpp_\w+)\s*\(", text)))


# ----------------------------------------------------------------------------- raw ABI
def zpp_quant_blockwise(x, x_dt, n, block, bits, codes, scales, stream=0):
    return lib().zpp_quant_blockwise(x, x_dt, n, block, bits, codes, scales, stream)


def zpp_dequant_blockwise(codes, scales, n, block, bits, y, y_dt, stream=0):
    return lib().zpp_dequant_blockwise(codes, scales, n, block, bits, y, y_dt, stream)


def zpp_qgz_reorder_quant(grads, g_dt, elems_per_rank, block, bits, topo, codes, scales, stream=0):
    return lib().zpp_qgz_reorder_quant(grads, g_dt, elems_per_rank, block, bits, topo, codes,
                                       scales, stream)


def zpp_qgz_reorder_quant_tensors(tensor_ptrs, sizes, g_dt, block, bits, topo, codes, scales,
                                  stream=0):
    """tensor_ptrs, sizes: Python sequences (marshalled into host arrays for the call)."""
    T = len(tensor_ptrs)
    ptrs = (ctypes.c_void_p * max(T, 1))(*tensor_ptrs)
    lens = (ctypes.c_int64 * max(T, 1))(*sizes)
    return lib().zpp_qgz_reorder_quant_tensors(ptrs, lens, T, g_dt, block, bits, topo, codes,
                                               scales, stream)


def zpp_dequant_reduce_requant(codes, scales, elems_per_rank, block, bits, topo, out_codes,
                               out_scales, stream=0):
    return lib().zpp_dequant_reduce_requant(codes, scales, elems_per_rank, block, bits, topo,
                                            out_codes, out_scales, stream)


def zpp_dequant_reduce(codes, scales, elems_per_rank, block, bits, topo, out, stream=0):
    return lib().zpp_dequant_reduce(codes, scales, elems_per_rank, block, bits, topo, out, stream)


def zpp_dequant_reduce_scaled(codes, scales, elems_per_rank, block, bits, topo, post_scale, out,
                              out_dt, stream=0):
    return lib().zpp_dequant_reduce_scaled(codes, scales, elems_per_rank, block, bits, topo,
                                           post_scale, out, out_dt, stream)


def zpp_qgz_reorder_quant_range(grads, g_dt, elems_per_rank, block, bits, topo, rng, codes,
                                scales, stream=0):
    return lib().zpp_qgz_reorder_quant_range(grads, g_dt, elems_per_rank, block, bits, topo, rng,
                                             codes, scales, stream)


def zpp_dequant_reduce_requant_range(codes, scales, elems_per_rank, block, bits, topo, rng,
                                     out_codes, out_scales, stream=0):
    return lib().zpp_dequant_reduce_requant_range(codes, scales, elems_per_rank, block, bits,
                                                  topo, rng, out_codes, out_scales, stream)


def zpp_dequant_reduce_scaled_range(codes, scales, elems_per_rank, block, bits, topo, rng,
                                    post_scale, out, out_dt, stream=0):
    return lib().zpp_dequant_reduce_scaled_range(codes, scales, elems_per_rank, block, bits,
                                                 topo, rng, post_scale, out, out_dt, stream)


def zpp_qgz_reorder_quant_local(grads, g_dt, elems_per_rank, block, bits, topo, rng, codes,
                                scales, stream=0):
    return lib().zpp_qgz_reorder_quant_local(grads, g_dt, elems_per_rank, block, bits, topo, rng,
                                             codes, scales, stream)


def zpp_dequant_reduce_requant_local(codes, scales, chunk, block, bits, sources, out_codes,
                                     out_scales, stream=0):
    return lib().zpp_dequant_reduce_requant_local(codes, scales, chunk, block, bits, sources,
                                                  out_codes, out_scales, stream)


def zpp_dequant_reduce_local(codes, scales, slice_len, block, bits, sources, post_scale, out,
                             out_dt, stream=0):
    return lib().zpp_dequant_reduce_local(codes, scales, slice_len, block, bits, sources,
                                          post_scale, out, out_dt, stream)


def zpp_device_copy(src, dst, nbytes, stream=0):
    return lib().zpp_device_copy(src, dst, nbytes, stream)


def zpp_device_fault(clear=False):
    """The device fault word (see include/zpp.h); synchronises with the device."""
    v = ctypes.c_uint32(0)
    _check(lib().zpp_device_fault(ctypes.byref(v), 1 if clear else 0), "zpp_device_fault")
    return int(v.value)


def zpp_wait_selftest(limit_ns, stream=0):
    return lib().zpp_wait_selftest(limit_ns, stream)


def zpp_grad_norm(grad_ptrs, sizes, g_dt, pre_scale, max_norm, workspace, out, stream=0):
    """grad_ptrs, sizes: Python sequences (marshalled into host arrays for the call)."""
    ptrs, lens = array.array("q", grad_ptrs), array.array("q", sizes)
    return lib().zpp_grad_norm(ptrs.buffer_info()[0], lens.buffer_info()[0], len(ptrs), g_dt,
                               pre_scale, max_norm, workspace, out, stream)


def zpp_grad_norm_workspace(total_elems, num_tensors):
    return int(lib().zpp_grad_norm_workspace(total_elems, num_tensors))


def zpp_adamw_step(tensors, g_dt, w_dt, state_bits, hp, grad_scale=0, stream=0):
    """tensors: a sequence of AdamwTensor, or an array('q') with their fields one after the
    other; hp: an AdamwParams."""
    num, at, keep = _adamw_table(tensors)
    return lib().zpp_adamw_step(at, num, g_dt, w_dt, state_bits, ctypes.addressof(hp),
                                grad_scale, stream)


def zpp_adamw_step_counted(tensors, g_dt, w_dt, state_bits, hp, grad_scale, clip, record, stream=0):
    """clip: an AdamwClip or None; the rest as zpp_adamw_step."""
    num, at, keep = _adamw_table(tensors)
    return lib().zpp_adamw_step_counted(at, num, g_dt, w_dt, state_bits, ctypes.addressof(hp),
                                        grad_scale, ctypes.addressof(clip) if clip else 0, record,
                                        stream)


def _adamw_table(tensors):
    """(number of tensors, address of their fields, what keeps it alive)."""
    if isinstance(tensors, array.array):
        return len(tensors) // 8, tensors.buffer_info()[0], tensors
    fields = (AdamwTensor * max(len(tensors), 1))(*tensors)
    return len(tensors), ctypes.addressof(fields), fields


def zpp_matvec_blockwise(codes, scales, rows, cols, block, bits, x, x_dt, vecs, x_stride, bias, y,
                         y_dt, y_stride, stream=0):
    return lib().zpp_matvec_blockwise(codes, scales, rows, cols, block, bits, x, x_dt, vecs,
                                      x_stride, bias, y, y_dt, y_stride, stream)


def zpp_quant_fp8(x, x_dt, x_stride, out, transposed=None, stream=0):
    """out, transposed: Fp8Matrix (transposed: or None)."""
    return lib().zpp_quant_fp8(x, x_dt, x_stride, ctypes.addressof(out),
                               ctypes.addressof(transposed) if transposed else 0, stream)


def zpp_matmul_fp8(a, b, bias, y, y_dt, y_stride, stream=0):
    """a, b: Fp8Matrix."""
    return lib().zpp_matmul_fp8(ctypes.addressof(a), ctypes.addressof(b), bias, y, y_dt, y_stride,
                                stream)


def _rows_of(kind, rows):
    """(address of the C array of a sequence of structures, what keeps it alive)."""
    fields = (kind * max(len(rows), 1))(*rows)
    return ctypes.addressof(fields), fields


def zpp_orthogonalize(matrices, x_dt, out_dt, ns, workspace, stream=0):
    """matrices: a sequence of Matrix; ns: a NewtonSchulz."""
    at, keep = _rows_of(Matrix, matrices)
    return lib().zpp_orthogonalize(at, len(matrices), x_dt, out_dt, ctypes.addressof(ns), workspace, stream)


def zpp_orthogonalize_workspace(matrices):
    at, keep = _rows_of(Matrix, matrices)
    return int(lib().zpp_orthogonalize_workspace(at, len(matrices)))


def zpp_muon_step(tensors, g_dt, w_dt, hp, grad_scale, workspace, stream=0):
    """tensors: a sequence of MuonTensor; hp: a MuonParams."""
    at, keep = _rows_of(MuonTensor, tensors)
    return lib().zpp_muon_step(at, len(tensors), g_dt, w_dt, ctypes.addressof(hp), grad_scale, workspace,
                               stream)


def zpp_muon_workspace(tensors):
    at, keep = _rows_of(MuonTensor, tensors)
    return int(lib().zpp_muon_workspace(at, len(tensors)))


def zpp_code_bytes(n, bits):
    return int(lib().zpp_code_bytes(n, bits))


def zpp_num_scales(n, block):
    return int(lib().zpp_num_scales(n, block))


def zpp_status_string(status):
    return lib().zpp_status_string(int(status)).decode()


# ----------------------------------------------------------------------------- tensors
# The wrappers below check every tensor's element count and dtype against what the call
# reads or writes, then that all tensors are contiguous CUDA tensors on one device, and
# raise ValueError before calling into libzpp. Sizes that the C ABI itself rejects (bad
# bits, block or topology) are left to it and raise ZppError with its status.
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_kinds = {}  # torch dtype -> zpp_dtype, filled on first use


def _dt(t):
    if not _kinds:
        torch = _torch()
        _kinds.update({torch.float16: ZPP_F16, torch.bfloat16: ZPP_BF16, torch.float32: ZPP_F32})
    return _kinds[t]


def _bytes_dtypes():
    torch = _torch()
    return (torch.uint8, torch.int8)


def _need(t, name, numel=None, dtypes=None):
    """t must hold exactly `numel` elements of one of `dtypes` (None: not checked)."""
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel}")


def _cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("zpp operates on CUDA tensors only (no CPU path)")
        if not t.is_contiguous():
            raise ValueError("zpp needs contiguous tensors")
    if any(t.device != ts[0].device for t in ts):
        raise ValueError("all tensors of a call must be on one device")


def _stream(t):
    return _torch().cuda.current_stream(t.device).cuda_stream


def _raw_stream(device):
    """The current stream's handle of a device index, without building a Stream object where
    torch offers that (a few microseconds of every call)."""
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(device) if get is not None else torch.cuda.current_stream(device).cuda_stream


def _check(status, where):
    if status != ZPP_OK:
        raise ZppError(status, where)


def _sizes_ok(n, block, bits):
    return n >= 0 and bits in (4, 8) and block in (64, 128, 256, 512, 1024, 2048, 4096)


def _qgz_sizes(E, block, bits, N, M):
    """(W, C, S) when E fits the topology (else None: the C ABI reports it)."""
    W = N * M
    if N < 1 or M < 1 or not _sizes_ok(E, block, bits) or E % (W * block):
        return None
    return W, E // M, E // W


def quant_blockwise(x, block, bits, codes=None, scales=None):
    """x (fp16/bf16, any shape) -> (codes uint8[code_bytes], scales fp32[num_scales])."""
    torch = _torch()
    n = x.numel()
    _need(x, "x", dtypes=(torch.float16, torch.bfloat16))
    ok = _sizes_ok(n, block, bits)
    if codes is not None:
        _need(codes, "codes", zpp_code_bytes(n, bits) if ok else None, _bytes_dtypes())
    if scales is not None:
        _need(scales, "scales", zpp_num_scales(n, block) if ok else None, (torch.float32,))
    _cuda(x, *(t for t in (codes, scales) if t is not None))
    if codes is None:
        codes = torch.empty(max(zpp_code_bytes(n, bits), 0), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(max(zpp_num_scales(n, block), 0), dtype=torch.float32,
                             device=x.device)
    _check(zpp_quant_blockwise(x.data_ptr(), _dt(x.dtype), n, block, bits, codes.data_ptr(),
                               scales.data_ptr(), _stream(x)), "zpp_quant_blockwise")
    return codes, scales


def dequant_blockwise(codes, scales, n, block, bits, dtype=None, y=None):
    """codes, scales -> y[n] of `dtype` (default fp16)."""
    torch = _torch()
    ok = _sizes_ok(n, block, bits)
    _need(codes, "codes", zpp_code_bytes(n, bits) if ok else None, _bytes_dtypes())
    _need(scales, "scales", zpp_num_scales(n, block) if ok else None, (torch.float32,))
    if y is not None:
        _need(y, "y", n, (torch.float16, torch.bfloat16, torch.float32))
    _cuda(codes, scales, *(t for t in (y,) if t is not None))
    if y is None:
        y = torch.empty(max(n, 0), dtype=dtype or torch.float16, device=codes.device)
    _check(zpp_dequant_blockwise(codes.data_ptr(), scales.data_ptr(), n, block, bits,
                                 y.data_ptr(), _dt(y.dtype), _stream(codes)),
           "zpp_dequant_blockwise")
    return y


def qgz_reorder_quant(grads, block, bits, N, M, codes=None, scales=None):
    """grads [W][E] (fp16/bf16) -> (codes uint8 [W][code_bytes(E)], scales fp32 [W][E/block])."""
    torch = _torch()
    W = N * M
    _need(grads, "grads", dtypes=(torch.float16, torch.bfloat16))
    if W < 1 or grads.numel() % W:
        raise ValueError(f"grads: {grads.numel()} elements do not split into {W} ranks")
    E = grads.numel() // W
    sz = _qgz_sizes(E, block, bits, N, M)
    if codes is not None:
        _need(codes, "codes", W * zpp_code_bytes(E, bits) if sz else None, _bytes_dtypes())
    if scales is not None:
        _need(scales, "scales", W * (E // block) if sz else None, (torch.float32,))
    _cuda(grads, *(t for t in (codes, scales) if t is not None))
    if codes is None:
        codes = torch.empty((W, max(zpp_code_bytes(E, bits), 0)), dtype=torch.uint8,
                            device=grads.device)
    if scales is None:
        scales = torch.empty((W, E // block if block > 0 else 0), dtype=torch.float32,
                             device=grads.device)
    _check(zpp_qgz_reorder_quant(grads.data_ptr(), _dt(grads.dtype), E, block, bits,
                                 Topology(N, M), codes.data_ptr(), scales.data_ptr(),
                                 _stream(grads)), "zpp_qgz_reorder_quant")
    return codes, scales


def qgz_reorder_quant_tensors(tensors, block, bits, N, M, codes=None, scales=None):
    """The bucket given as a list of gradient tensors, tensor t of shape [W][n_t] (the W
    ranks' copies; any shape with W * n_t elements, contiguous) -> the codes and scales
    qgz_reorder_quant gives for the bucket whose rank r concatenates row r of every tensor."""
    torch = _torch()
    if not tensors:
        raise ValueError("qgz_reorder_quant_tensors needs at least one tensor")
    W = N * M
    dt = tensors[0].dtype
    for i, t in enumerate(tensors):
        _need(t, f"tensors[{i}]", dtypes=(dt,))
    _need(tensors[0], "tensors[0]", dtypes=(torch.float16, torch.bfloat16))
    if W < 1 or any(t.numel() % W for t in tensors):
        raise ValueError("every tensor holds W equal per-rank copies")
    sizes = [t.numel() // W for t in tensors]
    E = sum(sizes)
    sz = _qgz_sizes(E, block, bits, N, M)
    if codes is not None:
        _need(codes, "codes", W * zpp_code_bytes(E, bits) if sz else None, _bytes_dtypes())
    if scales is not None:
        _need(scales, "scales", W * (E // block) if sz else None, (torch.float32,))
    _cuda(*tensors, *(t for t in (codes, scales) if t is not None))
    dev = tensors[0].device
    if codes is None:
        codes = torch.empty((W, max(zpp_code_bytes(E, bits), 0)), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((W, E // block if block > 0 else 0), dtype=torch.float32, device=dev)
    _check(zpp_qgz_reorder_quant_tensors([t.data_ptr() for t in tensors], sizes, _dt(dt), block,
                                         bits, Topology(N, M), codes.data_ptr(), scales.data_ptr(),
                                         _stream(tensors[0])), "zpp_qgz_reorder_quant_tensors")
    return codes, scales


def _hop_inputs(codes, scales, E, block, bits, N, M, hop):
    """Checks the codes / scales a hop reads: hop 1 reads the step-1 buffers ([W][E]
    elements per rank), hop 2 the hop-1 buffers ([W][C], C = E / M)."""
    torch = _torch()
    sz = _qgz_sizes(E, block, bits, N, M)
    n = None if sz is None else (E if hop == 1 else sz[1])
    W = N * M
    _need(codes, "codes", W * zpp_code_bytes(n, bits) if sz else None, _bytes_dtypes())
    _need(scales, "scales", W * (n // block) if sz else None, (torch.float32,))
    return sz


def dequant_reduce_requant(codes, scales, E, block, bits, N, M, out_codes=None, out_scales=None):
    """Intra-node hop -> (codes uint8 [W][code_bytes(E/M)], scales fp32 [W][E/M/block])."""
    torch = _torch()
    sz = _hop_inputs(codes, scales, E, block, bits, N, M, hop=1)
    W, C = N * M, E // M if M > 0 else 0
    if out_codes is not None:
        _need(out_codes, "out_codes", W * zpp_code_bytes(C, bits) if sz else None,
              _bytes_dtypes())
    if out_scales is not None:
        _need(out_scales, "out_scales", W * (C // block) if sz else None, (torch.float32,))
    _cuda(codes, scales, *(t for t in (out_codes, out_scales) if t is not None))
    if out_codes is None:
        out_codes = torch.empty((W, max(zpp_code_bytes(C, bits), 0)), dtype=torch.uint8,
                                device=codes.device)
    if out_scales is None:
        out_scales = torch.empty((W, C // block if block > 0 else 0), dtype=torch.float32,
                                 device=codes.device)
    _check(zpp_dequant_reduce_requant(codes.data_ptr(), scales.data_ptr(), E, block, bits,
                                      Topology(N, M), out_codes.data_ptr(), out_scales.data_ptr(),
                                      _stream(codes)), "zpp_dequant_reduce_requant")
    return out_codes, out_scales


def dequant_reduce(codes, scales, E, block, bits, N, M, out=None):
    """Inter-node hop -> fp32 [W][E/W], each rank's summed owner slice."""
    torch = _torch()
    sz = _hop_inputs(codes, scales, E, block, bits, N, M, hop=2)
    W = N * M
    if out is not None:
        _need(out, "out", W * (E // W) if sz else None, (torch.float32,))
    _cuda(codes, scales, *(t for t in (out,) if t is not None))
    if out is None:
        out = torch.empty((W, E // W if W > 0 else 0), dtype=torch.float32, device=codes.device)
    _check(zpp_dequant_reduce(codes.data_ptr(), scales.data_ptr(), E, block, bits, Topology(N, M),
                              out.data_ptr(), _stream(codes)), "zpp_dequant_reduce")
    return out


def dequant_reduce_scaled(codes, scales, E, block, bits, N, M, post_scale=None, dtype=None,
                          out=None):
    """Inter-node hop with the average folded in: [W][E/W] of `dtype` (default fp32) holding
    fp32(sum * post_scale); post_scale defaults to 1/W (the average over ranks)."""
    torch = _torch()
    sz = _hop_inputs(codes, scales, E, block, bits, N, M, hop=2)
    W = N * M
    if out is not None:
        _need(out, "out", W * (E // W) if sz else None,
              (torch.float16, torch.bfloat16, torch.float32))
    _cuda(codes, scales, *(t for t in (out,) if t is not None))
    if post_scale is None:
        post_scale = 1.0 / W
    if out is None:
        out = torch.empty((W, E // W if W > 0 else 0), dtype=dtype or torch.float32,
                          device=codes.device)
    _check(zpp_dequant_reduce_scaled(codes.data_ptr(), scales.data_ptr(), E, block, bits,
                                     Topology(N, M), float(post_scale), out.data_ptr(),
                                     _dt(out.dtype), _stream(codes)), "zpp_dequant_reduce_scaled")
    return out


# ------------------------------------------------------------------ one real rank's steps
def qgz_reorder_quant_local(grads, block, bits, N, M, codes=None, scales=None, chunks=None):
    """This rank's gradient bucket [E] (fp16/bf16) -> its reordered codes [code_bytes(E)]
    and scales [E/block]: chunk l' (N*S elements) goes to local peer l' in hop 1. With
    `chunks` = (begin, end) only those chunks are written (into the given buffers)."""
    torch = _torch()
    _need(grads, "grads", dtypes=(torch.float16, torch.bfloat16))
    E = grads.numel()
    sz = _qgz_sizes(E, block, bits, N, M)
    if codes is not None:
        _need(codes, "codes", zpp_code_bytes(E, bits) if sz else None, _bytes_dtypes())
    if scales is not None:
        _need(scales, "scales", E // block if sz else None, (torch.float32,))
    _cuda(grads, *(t for t in (codes, scales) if t is not None))
    if codes is None:
        codes = torch.empty(max(zpp_code_bytes(E, bits), 0), dtype=torch.uint8, device=grads.device)
    if scales is None:
        scales = torch.empty(E // block if block > 0 else 0, dtype=torch.float32,
                             device=grads.device)
    rng = LocalRange(*(chunks if chunks is not None else (0, M)))
    _check(zpp_qgz_reorder_quant_local(grads.data_ptr(), _dt(grads.dtype), E, block, bits,
                                       Topology(N, M), rng, codes.data_ptr(), scales.data_ptr(),
                                       _stream(grads)), "zpp_qgz_reorder_quant_local")
    return codes, scales


def _received(codes, scales, sources, length, block, bits):
    torch = _torch()
    ok = sources >= 1 and _sizes_ok(length, block, bits) and length % block == 0
    _need(codes, "codes", sources * zpp_code_bytes(length, bits) if ok else None, _bytes_dtypes())
    _need(scales, "scales", sources * (length // block) if ok else None, (torch.float32,))
    return ok


def dequant_reduce_requant_local(codes, scales, chunk, block, bits, sources, out_codes=None,
                                 out_scales=None):
    """The fused intra-node hop on the chunks this rank received ([sources][chunk] codes and
    scales, sources in local-index order) -> its hop-1 codes [code_bytes(chunk)] and scales."""
    torch = _torch()
    ok = _received(codes, scales, sources, chunk, block, bits)
    if out_codes is not None:
        _need(out_codes, "out_codes", zpp_code_bytes(chunk, bits) if ok else None, _bytes_dtypes())
    if out_scales is not None:
        _need(out_scales, "out_scales", chunk // block if ok else None, (torch.float32,))
    _cuda(codes, scales, *(t for t in (out_codes, out_scales) if t is not None))
    if out_codes is None:
        out_codes = torch.empty(max(zpp_code_bytes(chunk, bits), 0), dtype=torch.uint8,
                                device=codes.device)
    if out_scales is None:
        out_scales = torch.empty(chunk // block if block > 0 else 0, dtype=torch.float32,
                                 device=codes.device)
    _check(zpp_dequant_reduce_requant_local(codes.data_ptr(), scales.data_ptr(), chunk, block,
                                            bits, sources, out_codes.data_ptr(),
                                            out_scales.data_ptr(), _stream(codes)),
           "zpp_dequant_reduce_requant_local")
    return out_codes, out_scales


def dequant_reduce_local(codes, scales, slice_len, block, bits, sources, post_scale=1.0,
                         dtype=None, out=None):
    """The final inter-node hop on the slices this rank received ([sources][slice_len],
    nodes in ascending order) -> its owner slice [slice_len] of `dtype` (default fp32),
    fp32(sum * post_scale)."""
    torch = _torch()
    ok = _received(codes, scales, sources, slice_len, block, bits)
    if out is not None:
        _need(out, "out", slice_len if ok else None, (torch.float16, torch.bfloat16, torch.float32))
    _cuda(codes, scales, *(t for t in (out,) if t is not None))
    if out is None:
        out = torch.empty(max(slice_len, 0), dtype=dtype or torch.float32, device=codes.device)
    _check(zpp_dequant_reduce_local(codes.data_ptr(), scales.data_ptr(), slice_len, block, bits,
                                    sources, float(post_scale), out.data_ptr(), _dt(out.dtype),
                                    _stream(codes)), "zpp_dequant_reduce_local")
    return out


# ------------------------------------------------------------- the weights' other operators
_tensors_module = None
_KIND_NAMES = ("float16", "bfloat16", "float32", "uint8 / int8", "float8_e4m3fn")


def _tensors():
    """The extension that reads tensors' addresses, counts, types and devices."""
    global _tensors_module
    if _tensors_module is None:
        _torch()
        if not os.path.exists(_build.EXT):
            raise RuntimeError(f"{_build.EXT} is missing: build it with __graft_entry__.build() "
                               "(there is no fallback path)")
        built, here = _build.built_ext_abi(), _build.ext_abi()
        if built not in (None, here):
            raise RuntimeError(f"{_build.EXT} was built for {built}, this is {here}: "
                               "build it again with __graft_entry__.build()")
        from . import _tensors as module
        _tensors_module = module
    return _tensors_module


def _dev_list(ts, name, kinds):
    """Checks a list of tensors that one call reads or writes: one dtype among `kinds` (indices
    into _KIND_NAMES), contiguous CUDA tensors on one device. Returns (addresses, element
    counts, kind, device)."""
    ptrs = array.array("q", bytes(8 * len(ts)))
    sizes = array.array("q", ptrs)
    kind, device = _tensors().scan(ts, ptrs, sizes)
    if kind not in kinds:
        raise ValueError(f"{name}: every tensor needs one dtype of "
                         f"{tuple(_KIND_NAMES[k] for k in kinds)}")
    if device < 0:
        _cuda(*ts)
    return ptrs, sizes, kind, device


_GRAD_KINDS = (ZPP_F16, ZPP_BF16, ZPP_F32)


def grad_norm(grads, max_norm=None, pre_scale=1.0, out=None):
    """The norm of a list of gradient tensors together (one fp16 / bf16 / fp32 dtype) times
    |pre_scale|, and the factor that clips it to `max_norm` (None: no clipping) with
    pre_scale folded in -> fp32 [2] (norm, factor) on the device. The factor is NaN when the
    norm is not finite: adamw_step then skips the step."""
    torch = _torch()
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if not grads:
        raise ValueError("grad_norm needs at least one tensor")
    if out is None:
        found = _tensors().grad_norm(_address("zpp_grad_norm"), _address("zpp_grad_norm_workspace"),
                                     grads, math.inf if max_norm is None else max_norm, pre_scale)
        if found is not None:
            if type(found) is int:
                raise ZppError(found, "zpp_grad_norm")
            return found
    ptrs, sizes, kind, device = _dev_list(grads, "grads", _GRAD_KINDS)
    if out is not None:
        _need(out, "out", 2, (torch.float32,))
        _cuda(grads[0], out)
    else:
        out = grads[0].new_empty(2, dtype=torch.float32)
    work = grads[0].new_empty(zpp_grad_norm_workspace(sum(sizes), len(sizes)),
                              dtype=torch.float32)
    _launch(device, "zpp_grad_norm", ptrs.buffer_info()[0], sizes.buffer_info()[0], len(sizes), kind,
            pre_scale, math.inf if max_norm is None else max_norm, work.data_ptr(), out.data_ptr())
    return out


def _launch(device, name, *args):
    """The library function `name` on a device's current stream, with that device current: a kernel
    starts on the current device, whatever device its stream belongs to."""
    torch = _torch()
    if device == torch.cuda.current_device():
        status = getattr(lib(), name)(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = getattr(lib(), name)(*args, _raw_stream(device))
    _check(status, name)


def adamw_step(params, grads, exp_avg, exp_avg_sq, *, step, lr, betas=(0.9, 0.999), eps=1e-8,
               weight_decay=0.0, grad_scale=None, weights=None, scales=None, seed=0):
    """One AdamW step over lists of tensors (or single tensors), in place.

    params: fp32. grads: one of fp16 / bf16 / fp32. exp_avg, exp_avg_sq: fp32 states; with
    `scales` = (m scales, v scales) they are float8_e4m3fn codes (of m and of sqrt(v)) with one
    fp32 scale per 256 elements, [ceil(n / 256)] for each tensor. weights: fp16 / bf16 tensors
    that receive the rounded parameters. grad_scale: fp32 device tensor whose first element
    multiplies every gradient; if it is not finite the step changes nothing. step counts from
    1; seed (0 .. 2^32 - 1) is that of the 8-bit states' stochastic rounding."""
    torch = _torch()
    aslist = lambda v: [v] if isinstance(v, torch.Tensor) else list(v)  # noqa: E731
    f32 = (ZPP_F32,)
    params, grads = aslist(params), aslist(grads)
    lists = [("params", params, f32), ("grads", grads, _GRAD_KINDS)]
    state = f32 if scales is None else (_E4M3,)
    lists += [("exp_avg", aslist(exp_avg), state), ("exp_avg_sq", aslist(exp_avg_sq), state)]
    if scales is not None:
        lists += [("scales[0]", aslist(scales[0]), f32), ("scales[1]", aslist(scales[1]), f32)]
    if weights is not None:
        lists.append(("weights", aslist(weights), (ZPP_F16, ZPP_BF16)))
    if not params:
        raise ValueError("adamw_step needs at least one tensor")
    if not 0 <= seed < 1 << 32:
        raise ValueError("seed: 0 .. 2^32 - 1")
    tab = array.array("q", bytes(64 * len(params)))
    want, at, kinds = None, None, {}
    for column, (name, ts, allowed) in zip(_columns(scales is not None), lists):
        if len(ts) != len(params):
            raise ValueError(f"{name}: {len(ts)} tensors, expected {len(params)}")
        ptrs, sizes, kinds[name], device = _dev_list(ts, name, allowed)
        if want is None:
            want, at, blocks = sizes, device, _state_blocks(sizes)
        _same_sizes(name, sizes, blocks if name.startswith("scales") else want)
        if device != at:
            raise ValueError("all tensors of a call must be on one device")
        tab[column::8] = ptrs
    tab[7::8] = want
    hp = AdamwParams(lr, betas[0], betas[1], eps, weight_decay, step, seed)
    _adamw(tab, kinds["grads"], kinds.get("weights", ZPP_BF16), 32 if scales is None else 8, hp,
           _scale_address(grads[0], grad_scale), at)


_E4M3 = _KIND_NAMES.index("float8_e4m3fn")


def _columns(scaled):
    """Fields of AdamwTensor that params, grads, the states, the scales and weights go to."""
    return (0, 1, 2, 3, 4, 5, 6) if scaled else (0, 1, 2, 3, 6)


def _state_blocks(sizes):
    return array.array("q", [-(-n // ZPP_STATE_BLOCK) for n in sizes])


def _same_sizes(name, sizes, want):
    if sizes != want:
        i = next(i for i, (a, b) in enumerate(zip(sizes, want)) if a != b)
        raise ValueError(f"{name}[{i}]: {sizes[i]} elements, expected {want[i]}")


def _scale_address(grad, grad_scale):
    if grad_scale is None:
        return 0
    _need(grad_scale, "grad_scale", dtypes=(_torch().float32,))
    if grad_scale.numel() < 1:
        raise ValueError("grad_scale: at least one element")
    _cuda(grad, grad_scale)
    return grad_scale.data_ptr()


def _adamw(tab, g_kind, w_kind, state_bits, hp, scale, device):
    _launch(device, "zpp_adamw_step", tab.buffer_info()[0], len(tab) // 8, g_kind, w_kind, state_bits,
            ctypes.addressof(hp), scale)


@functools.cache
def _address(name):
    """The address of a library function, as the extension takes it."""
    return ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value


def matvec_blockwise(codes, scales, x, rows, block, bits, bias=None, dtype=None, y=None):
    """x [..., cols] (fp16 / bf16; rows of cols contiguous elements, any row stride) times the
    transposed [rows][cols] matrix that quant_blockwise gave (codes, scales) for -> y [..., rows]
    of `dtype` (default: x's). bias: [rows] of x's dtype. y: an output buffer, same form as x."""
    native = _tensors()
    if y is None:
        y = native.matvec(_address("zpp_matvec_blockwise"), codes, scales, x, rows, block, bits, bias,
                          -1 if dtype is None else _dt(dtype))
        if y is not None:
            if type(y) is int:
                raise ZppError(y, "zpp_matvec_blockwise")
            return y
    probe, shape = native.probe, x.shape
    x_at, x_n, x_kind, device, x_whole = probe(x)
    if x_kind not in (ZPP_F16, ZPP_BF16):
        _need(x, "x", dtypes=(_torch().float16, _torch().bfloat16))
    if not shape or shape[-1] < 1 or rows < 0:
        raise ValueError("x: [..., cols] with cols >= 1, and rows >= 0")
    cols = shape[-1]
    n = rows * cols
    c_at, c_n, c_kind, c_dev, c_whole = probe(codes)
    s_at, s_n, s_kind, s_dev, s_whole = probe(scales)
    if _sizes_ok(n, block, bits) and (c_n != (n if bits == 8 else (n + 1) // 2)
                                      or s_n != -(-n // block)):
        _need(codes, "codes", zpp_code_bytes(n, bits))
        _need(scales, "scales", zpp_num_scales(n, block))
    if c_kind != 3 or s_kind != ZPP_F32:
        _need(codes, "codes", dtypes=_bytes_dtypes())
        _need(scales, "scales", dtypes=(_torch().float32,))
    b_at, b_ok = 0, True
    if bias is not None:
        b_at, b_n, b_kind, b_dev, b_whole = probe(bias)
        if b_kind != x_kind or b_n != rows:
            _need(bias, "bias", rows, (x.dtype,))
        b_ok = b_dev == device and b_whole
    vecs, x_stride = (x_n // cols, cols) if x_whole else _rows(x, "x")
    if y is None:
        if device >= 0:
            y = x.new_empty((*shape[:-1], rows), dtype=dtype)
            y_at, _, y_kind, y_dev, _ = probe(y)
        y_stride = rows
    else:
        torch = _torch()
        _need(y, "y", vecs * rows, (torch.float16, torch.bfloat16, torch.float32))
        if y.shape != (*shape[:-1], rows) or (dtype is not None and y.dtype != dtype):
            raise ValueError(f"y: {tuple(y.shape)} of {y.dtype} does not fit the call")
        y_stride = _rows(y, "y")[1]
        y_at, _, y_kind, y_dev, _ = probe(y)
    if device < 0 or not (c_dev == s_dev == y_dev == device and c_whole and s_whole and b_ok):
        _cuda(codes, scales, *(t for t in (bias,) if t is not None))
        raise ValueError("all tensors of a call must be on one CUDA device")
    _launch(device, "zpp_matvec_blockwise", c_at, s_at, rows, cols, block, bits, x_at, x_kind, vecs,
            x_stride, b_at, y_at, y_kind, y_stride)
    return y


def _rows(t, name):
    """(rows, row stride) of a tensor seen as rows of contiguous elements."""
    cols = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols
    if t.dim() != 2 or (t.stride(1) != 1 and cols > 1) or t.stride(0) < cols:
        raise ValueError(f"{name}: rows must be contiguous and at least a row apart")
    return t.shape[0], t.stride(0)


FP8_BLOCK = 128  # columns that share a scale


def _matrix(t, name):
    """A tensor [..., cols] as rows of contiguous elements, evenly spaced: (rows, cols, row stride)."""
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name}: [..., cols] with cols >= 1")
    if not t.numel():
        return 0, t.shape[-1], t.shape[-1]
    if t.dim() != 2:
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: rows must be evenly spaced") from None
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}: rows must be at least a row apart")
    return rows, cols, t.stride(0) if rows > 1 else max(t.stride(0), cols)


def _fp8(codes, scales, name, tile=None):
    """The Fp8Matrix of a tensor of codes and its scales ([rows or row tiles, blocks], any strides). The
    scales' shape says which tiles they are for."""
    torch = _torch()
    _need(codes, name, dtypes=(torch.float8_e4m3fn,))
    _need(scales, f"{name}_scales", dtypes=(torch.float32,))
    rows, cols, stride = _matrix(codes, name)
    if rows <= 1:
        stride = -(-stride // 16) * 16  # (one row may end anywhere)
    blocks, tiles = -(-cols // FP8_BLOCK), -(-rows // FP8_BLOCK)
    shape = tuple(scales.shape)
    if shape == (rows, blocks) and tile != 128:
        tile = 1
    elif shape == (tiles, blocks) and tile != 1:
        tile = 128
    else:
        raise ValueError(f"{name}_scales: {shape}, expected one of "
                         f"{tuple(((rows, blocks), (tiles, blocks)))}")
    if stride % 16 or (rows and codes.data_ptr() % 16):
        raise ValueError(f"{name}: rows of codes start at multiples of 16 bytes, as quant_fp8 lays them")
    return Fp8Matrix(codes.data_ptr(), scales.data_ptr(), rows, cols, stride, scales.stride(0),
                     scales.stride(1), tile)


def _on_gpu(*ts):
    """The index of the CUDA device that all tensors are on."""
    if not all(t.is_cuda for t in ts):
        raise ValueError("zpp operates on CUDA tensors only (no CPU path)")
    if any(t.device != ts[0].device for t in ts):
        raise ValueError("all tensors of a call must be on one device")
    return ts[0].get_device()


def _written(*ts):
    """Marks a caller's buffers as written, so that a backward pass that kept their old contents
    raises."""
    mark = _torch().autograd.graph.increment_version
    for t in ts:
        if not t.is_inference():
            mark(t)


def _codes_like(shape, device):
    """New e4m3 codes whose rows start at multiples of 16 bytes."""
    torch = _torch()
    wide = -(-shape[-1] // 16) * 16
    return torch.empty((*shape[:-1], wide), dtype=torch.float8_e4m3fn, device=device)[..., :shape[-1]]


def quant_fp8(x, tile=1, transposed=False, out=None):
    """x [..., cols] (fp16 / bf16 / fp32; rows of contiguous elements, evenly spaced) -> (codes, scales):
    codes float8_e4m3fn of x's shape, rows at multiples of 16 bytes, and power-of-two scales fp32,
    [rows, ceil(cols / 128)] with tile 1 (a scale for each row and 128 columns: activations, gradients),
    [ceil(rows / 128), ceil(cols / 128)] with tile 128 (weights). value = code * scale.

    transposed: also (codes_t [cols, rows], scales_t) of the transposed matrix, made in the same pass.
    With tile 1 its blocks are 128 rows of a column; with tile 128 scales_t is a view of scales. out: the
    buffers to write, a tuple as an earlier call returned it. Codes and scales carry no gradient to x."""
    if out is None:
        made = _tensors().quant_fp8(_address("zpp_quant_fp8"), x, tile, transposed)
        if made is not None:
            if type(made) is int:
                raise ZppError(made, "zpp_quant_fp8")
            return made
    torch = _torch()
    _need(x, "x", dtypes=(torch.float16, torch.bfloat16, torch.float32))
    if tile not in (1, 128):
        raise ValueError("tile: 1 or 128")
    rows, cols, stride = _matrix(x, "x")
    device = _on_gpu(x)
    blocks, tiles = -(-cols // FP8_BLOCK), -(-rows // FP8_BLOCK)
    given = out is not None
    if not given:
        codes = _codes_like(x.shape, x.device)
        scales = (x.new_empty((blocks, rows), dtype=torch.float32).t() if tile == 1 else
                  x.new_empty((tiles, blocks), dtype=torch.float32))
        out = (codes, scales)
        if transposed and rows:
            out += (_codes_like((cols, rows), x.device),
                    x.new_empty((tiles, cols), dtype=torch.float32).t() if tile == 1 else scales.t())
        elif transposed:  # a matrix without rows: nothing to hold
            out += (codes.new_empty((cols, 0)), scales.new_empty((cols if tile == 1 else blocks, 0)))
    elif len(out) != (4 if transposed else 2):
        raise ValueError(f"out: {4 if transposed else 2} tensors, as an earlier call returned them")
    _on_gpu(x, *out)
    if out[0].shape != x.shape:
        raise ValueError(f"out: codes of {tuple(out[0].shape)} do not fit x")
    to = _fp8(out[0], out[1], "codes", tile)
    to_t = None
    if transposed and rows:
        if tuple(out[2].shape) != (cols, rows):
            raise ValueError(f"out: transposed codes of {tuple(out[2].shape)} do not fit x")
        to_t = _fp8(out[2], out[3], "codes_t", tile)
        if tile == 128 and (to_t.scales, to_t.scale_row, to_t.scale_block) != (
                to.scales, to.scale_block, to.scale_row):
            raise ValueError("out: with tile 128 the transposed scales are those of the codes, transposed")
    _launch(device, "zpp_quant_fp8", x.data_ptr(), _dt(x.dtype), stride, ctypes.addressof(to),
            ctypes.addressof(to_t) if to_t else 0)
    if given:
        _written(*out)
    return tuple(out)


def matmul_fp8(a, a_scales, b, b_scales, bias=None, dtype=None, y=None):
    """a [..., K] times the transpose of b [N, K], both e4m3 codes with scales as quant_fp8 gives them
    (any fp32 scales of those shapes, any strides) -> y [..., N] of `dtype` (default bf16; fp16 and
    fp32 too). bias: [N] of y's dtype. y: an output buffer, rows of contiguous elements evenly spaced.
    Not differentiable: an operand that requires a gradient is refused where gradients are recorded
    (linear_fp8 is the layer; a bias that is trained is added to its result)."""
    torch = _torch()
    if torch.is_grad_enabled():
        for name, t in (("bias", bias), ("a", a), ("a_scales", a_scales), ("b", b), ("b_scales", b_scales)):
            if getattr(t, "requires_grad", False):
                raise ValueError(f"{name}: requires a gradient, and matmul_fp8 is not differentiable (detach it, or "
                                 "call under torch.no_grad())")
    if y is None and (dtype is None or dtype in (torch.float16, torch.bfloat16, torch.float32)):
        made = _tensors().matmul_fp8(_address("zpp_matmul_fp8"), a, a_scales, b, b_scales, bias,
                                     ZPP_BF16 if dtype is None else _dt(dtype))
        if made is not None:
            if type(made) is int:
                raise ZppError(made, "zpp_matmul_fp8")
            return made
    pa, pb = _fp8(a, a_scales, "a"), _fp8(b, b_scales, "b")
    if b.dim() != 2 or pa.cols != pb.cols:
        raise ValueError(f"b: {tuple(b.shape)}, expected [N, {pa.cols}]")
    shape = (*a.shape[:-1], pb.rows)
    tensors = [a, a_scales, b, b_scales]
    given = y is not None
    if given:
        if tuple(y.shape) != shape or (dtype is not None and y.dtype != dtype):
            raise ValueError(f"y: {tuple(y.shape)} of {y.dtype} does not fit the call")
        _need(y, "y", dtypes=(torch.float16, torch.bfloat16, torch.float32))
        tensors.append(y)
    else:
        if dtype is None:
            dtype = torch.bfloat16
        if dtype not in (torch.float16, torch.bfloat16, torch.float32):
            raise ValueError(f"dtype: {dtype}, expected float16, bfloat16 or float32")
    if bias is not None:
        _need(bias, "bias", pb.rows, (dtype if y is None else y.dtype,))
        if not bias.is_contiguous():
            raise ValueError("zpp needs contiguous tensors")
        tensors.append(bias)
    device = _on_gpu(*tensors)
    if y is None:
        y = torch.empty(shape, dtype=dtype, device=a.device)
    y_stride = _matrix(y, "y")[2] if pb.rows else 0
    _launch(device, "zpp_matmul_fp8", ctypes.addressof(pa), ctypes.addressof(pb),
            0 if bias is None else bias.data_ptr(), y.data_ptr(), _dt(y.dtype), y_stride)
    if given:
        _written(y)
    return y


NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _steps(steps, coefficients, eps):
    """(NewtonSchulz, what keeps its coefficients alive): one triple for every step, or one for each."""
    rows = list(coefficients)
    if rows and not hasattr(rows[0], "__len__"):
        rows = [rows] * steps
    if len(rows) != steps or steps < 1 or any(len(r) != 3 for r in rows):
        raise ValueError("coefficients: (a, b, c), or one such triple for each of the steps (at least 1)")
    held = array.array("d", [float(v) for r in rows for v in r])
    return NewtonSchulz(held.buffer_info()[0], steps, eps), held


def _sides(ts, name):
    for i, t in enumerate(ts):
        if t.dim() != 2:
            raise ValueError(f"{name}[{i}]: {tuple(t.shape)}, expected a matrix")


def orthogonalize(x, steps=5, coefficients=NS_COEFFICIENTS, eps=1e-7, dtype=None, out=None):
    """Newton-Schulz steps on a matrix, or on every matrix of a list (contiguous, one of fp16 / bf16 /
    fp32): X = x / max(|x|, eps), then steps of A = X X^T, X = a X + (b A + c A A) X, which brings every
    singular value near 1 (of the transpose where there are more rows than columns). coefficients:
    (a, b, c) for all steps, or a triple for each. Returns new matrices of `dtype`, fp16 or bf16 (default:
    x's, bf16 for fp32), or fills `out` (which may be x). An update's arithmetic, without a gradient to x."""
    torch = _torch()
    single = isinstance(x, torch.Tensor)
    xs = [x] if single else list(x)
    if not xs:
        raise ValueError("orthogonalize needs at least one matrix")
    ns, held = _steps(steps, coefficients, eps)
    ptrs, _, kind, device = _dev_list(xs, "x", _GRAD_KINDS)
    _sides(xs, "x")
    given = out is not None
    if given:
        outs = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(outs) != len(xs) or any(o.shape != t.shape for o, t in zip(outs, xs)):
            raise ValueError("out: matrices of x's shapes")
        if dtype is not None and any(o.dtype != dtype for o in outs):
            raise ValueError("out: matrices of the given dtype")
    else:
        if dtype is None:
            dtype = torch.bfloat16 if kind == ZPP_F32 else xs[0].dtype
        if dtype not in (torch.float16, torch.bfloat16):
            raise ValueError(f"dtype: {dtype}, expected float16 or bfloat16")
        outs = [torch.empty(t.shape, dtype=dtype, device=t.device) for t in xs]
    out_ptrs, _, out_kind, out_device = _dev_list(outs, "out", (ZPP_F16, ZPP_BF16))
    if out_device != device:
        raise ValueError("all tensors of a call must be on one device")
    table = [Matrix(p, o, *t.shape) for p, o, t in zip(ptrs, out_ptrs, xs)]
    at, keep = _rows_of(Matrix, table)
    need = int(lib().zpp_orthogonalize_workspace(at, len(table)))
    work = torch.empty(max(need, 0), dtype=torch.uint8, device=xs[0].device)
    _launch(device, "zpp_orthogonalize", at, len(table), kind, out_kind, ctypes.addressof(ns),
            work.data_ptr())
    if given:
        _written(*outs)
    return outs[0] if single else outs


class QgzBuffers:
    """Device buffers of one qgZ exchange: reordered codes/scales (c0, s0), hop-1
    codes/scales (c1, s1) and the owner slices (out)."""

    def __init__(self, c0, s0, c1, s1, out):
        self.c0, self.s0, self.c1, self.s1, self.out = c0, s0, c1, s1, out

    @classmethod
    def allocate(cls, W, E, block, bits, M, device, out_dtype=None):
        torch = _torch()
        C = E // M
        return cls(torch.empty((W, zpp_code_bytes(E, bits)), dtype=torch.uint8, device=device),
                   torch.empty((W, E // block), dtype=torch.float32, device=device),
                   torch.empty((W, zpp_code_bytes(C, bits)), dtype=torch.uint8, device=device),
                   torch.empty((W, C // block), dtype=torch.float32, device=device),
                   torch.empty((W, E // W), dtype=out_dtype or torch.float32, device=device))

    def check(self, W, E, block, bits, M):
        """Raise ValueError unless every buffer has the size and dtype of an exchange of W
        ranks of E elements (the layouts of allocate())."""
        torch = _torch()
        C = E // M
        _need(self.c0, "bufs.c0", W * zpp_code_bytes(E, bits), _bytes_dtypes())
        _need(self.s0, "bufs.s0", W * (E // block), (torch.float32,))
        _need(self.c1, "bufs.c1", W * zpp_code_bytes(C, bits), _bytes_dtypes())
        _need(self.s1, "bufs.s1", W * (C // block), (torch.float32,))
        _need(self.out, "bufs.out", W * (E // W), (torch.float16, torch.bfloat16, torch.float32))


def qgz_pipelined(grads, block, bits, N, M, post_scale=1.0, bufs=None, streams=None,
                  n_streams=2, chunks=None):
    """The whole qgZ exchange as independent local-index sub-pipelines (reorder + quantise
    of chunks l, hop 1 for receivers (n, l), hop 2 for ranks (n, l)), joined back into the
    caller's stream. `chunks` local indices form one sub-pipeline (default: one per l).

    Schedules: with a list of `streams`, whole sub-pipelines go round robin over them;
    with ``streams=("split", low, high)`` every reorder + quantise runs on the `low`
    stream and each sub-pipeline's two hops on the `high` stream, gated by an event, so
    hop work fills the SMs that reorder work frees (give `high` the higher priority).
    Returns the buffers (owner slices in ``bufs.out``; fp32 by default)."""
    torch = _torch()
    W = N * M
    _need(grads, "grads", dtypes=(torch.float16, torch.bfloat16))
    if W < 1 or grads.numel() % W:
        raise ValueError(f"grads: {grads.numel()} elements do not split into {W} ranks")
    E = grads.numel() // W
    if _qgz_sizes(E, block, bits, N, M) is None:
        raise ValueError("elements per rank must be a multiple of W * block (bits 4 or 8, "
                         "block a power of two in [64, 4096])")
    if bufs is not None:
        bufs.check(W, E, block, bits, M)
        _cuda(grads, bufs.c0, bufs.s0, bufs.c1, bufs.s1, bufs.out)
    else:
        _cuda(grads)
        bufs = QgzBuffers.allocate(W, E, block, bits, M, grads.device)
    main = torch.cuda.current_stream(grads.device)
    if streams is None:
        streams = [torch.cuda.Stream(grads.device) for _ in range(min(n_streams, M))]
    split = len(streams) == 3 and streams[0] == "split"
    side = list(streams[1:]) if split else list(streams)
    chunks = chunks or 1
    fork = torch.cuda.Event()
    fork.record(main)
    topo = Topology(N, M)
    gdt, odt = _dt(grads.dtype), _dt(bufs.out.dtype)
    for st in side:
        st.wait_event(fork)
    for i, l0 in enumerate(range(0, M, chunks)):
        rng = LocalRange(l0, min(M, l0 + chunks))
        st_q = side[0] if split else side[i % len(side)]
        st_h = side[1] if split else st_q
        _check(zpp_qgz_reorder_quant_range(grads.data_ptr(), gdt, E, block, bits, topo, rng,
                                           bufs.c0.data_ptr(), bufs.s0.data_ptr(),
                                           st_q.cuda_stream), "zpp_qgz_reorder_quant_range")
        if split:
            ready = torch.cuda.Event()
            ready.record(st_q)
            st_h.wait_event(ready)
        _check(zpp_dequant_reduce_requant_range(bufs.c0.data_ptr(), bufs.s0.data_ptr(), E, block,
                                                bits, topo, rng, bufs.c1.data_ptr(),
                                                bufs.s1.data_ptr(), st_h.cuda_stream),
               "zpp_dequant_reduce_requant_range")
        _check(zpp_dequant_reduce_scaled_range(bufs.c1.data_ptr(), bufs.s1.data_ptr(), E, block,
                                               bits, topo, rng, float(post_scale),
                                               bufs.out.data_ptr(), odt, st_h.cuda_stream),
               "zpp_dequant_reduce_scaled_range")
    for st in side:
        join = torch.cuda.Event()
        join.record(st)
        main.wait_event(join)
    return bufs


def device_copy(src, dst):
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError(f"dst holds {dst.numel() * dst.element_size()} bytes, src {nbytes}")
    _cuda(src, dst)
    _check(zpp_device_copy(src.data_ptr(), dst.data_ptr(), nbytes, _stream(src)), "zpp_device_copy")
    return dst
