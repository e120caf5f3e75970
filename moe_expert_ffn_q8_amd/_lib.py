"""ctypes binding of libq8moe.so: the same names as the C ABI (include/q8moe.h).

Argument marshalling only: every computation happens in the HIP kernels of the
library.  Tensors are torch tensors on the GPU; Q8_0 data is a uint8 tensor
whose last dimension is (k/32)*34 bytes.  Work is enqueued on torch's current
stream of the tensors' device.  A negative status raises Q8Error.

There is no fallback: if libq8moe.so is missing or cannot be loaded, importing
this module raises.
"""
import ctypes
import os
from typing import NamedTuple, Optional

import torch

QK = 32
BLOCK_BYTES = 34

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq8moe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                      "python moe_expert_ffn_q8_amd/build.py")

_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_size = ctypes.c_size_t


class Q8MatmulDesc(ctypes.Structure):
    _fields_ = [("w", _vp), ("x", _vp), ("y", _vp),
                ("n", _i64), ("k", _i64), ("m", _i64), ("batch", _i64),
                ("w_batch_stride", _i64), ("x_row_stride", _i64), ("x_batch_stride", _i64),
                ("y_row_stride", _i64), ("y_batch_stride", _i64)]


class Q8R8Desc(ctypes.Structure):
    _fields_ = [("w_r8", _vp), ("x", _vp), ("y", _vp),
                ("n", _i64), ("k", _i64), ("batch", _i64),
                ("w_batch_stride", _i64), ("x_batch_stride", _i64), ("y_batch_stride", _i64)]


class Q8R8F32Desc(ctypes.Structure):
    _fields_ = [("w_r8", _vp), ("x", _vp), ("y", _vp),
                ("n", _i64), ("k", _i64), ("batch", _i64),
                ("w_batch_stride", _i64), ("x_batch_stride", _i64), ("y_batch_stride", _i64)]


class Q8R8MmDesc(ctypes.Structure):
    _fields_ = [("w_r8", _vp), ("x", _vp), ("y", _vp),
                ("n", _i64), ("k", _i64), ("m", _i64), ("batch", _i64),
                ("w_batch_stride", _i64), ("x_row_stride", _i64), ("x_batch_stride", _i64),
                ("y_row_stride", _i64), ("y_batch_stride", _i64)]


class MoeR8FfnDesc(ctypes.Structure):
    _fields_ = [("w_up_gate_r8", _vp), ("w_down_r8", _vp), ("x", _vp), ("ids", _vp), ("cw", _vp),
                ("h", _vp), ("out", _vp), ("ws", _vp), ("ws_bytes", ctypes.c_size_t)]


class KqMatvecDesc(ctypes.Structure):
    _fields_ = [("w", _vp), ("x", _vp), ("y", _vp),
                ("n", _i64), ("k", _i64), ("batch", _i64),
                ("w_batch_stride", _i64), ("x_batch_stride", _i64), ("y_batch_stride", _i64)]


class Q8UpGateDesc(ctypes.Structure):
    _fields_ = [("w", _vp), ("x", _vp), ("h", _vp),
                ("n_ff", _i64), ("n_embd", _i64), ("m", _i64), ("batch", _i64),
                ("w_batch_stride", _i64), ("x_row_stride", _i64), ("x_batch_stride", _i64),
                ("h_row_stride", _i64), ("h_batch_stride", _i64)]


class Q8MatmulF32Desc(ctypes.Structure):
    _fields_ = [("w", _vp), ("x", _vp), ("y", _vp),
                ("n", _i64), ("k", _i64), ("m", _i64), ("batch", _i64),
                ("w_batch_stride", _i64), ("x_row_stride", _i64), ("x_batch_stride", _i64),
                ("y_row_stride", _i64), ("y_batch_stride", _i64)]


class ResidualNormDesc(ctypes.Structure):
    _fields_ = [("x", _vp), ("residual", _vp), ("residual_out", _vp), ("gate", _vp),
                ("post_weight", _vp), ("post_bias", _vp), ("weight", _vp), ("bias", _vp), ("y", _vp),
                ("y_scale", _vp), ("x_row_stride", _i64), ("residual_row_stride", _i64),
                ("residual_out_row_stride", _i64), ("gate_row_stride", _i64), ("y_row_stride", _i64),
                ("x_type", _int), ("residual_type", _int), ("gate_type", _int), ("y_type", _int),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float), ("layer", _int)]


class MoeUpGateDesc(ctypes.Structure):
    _fields_ = [("w_up_gate", _vp), ("x", _vp), ("ids", _vp), ("h", _vp), ("ws", _vp),
                ("ws_bytes", _size)]


class MoeDownDesc(ctypes.Structure):
    _fields_ = [("w_down", _vp), ("h", _vp), ("ids", _vp), ("cw", _vp), ("out", _vp),
                ("ws", _vp), ("ws_bytes", _size)]


_SIGS = {
    "q8_status_str": (ctypes.c_char_p, [_int]),
    "q8_version": (ctypes.c_char_p, []),
    "q8_0_quantize_rows": (_int, [_vp, _i64, _vp, _i64, _i64, _vp]),
    "q8_0_matvec": (_int, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "q8_0_matmul": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "q8_0_matmul_batched": (_int, [ctypes.POINTER(Q8MatmulDesc), _i64, _vp]),
    "q8_0_matmul_f32_batched": (_int, [ctypes.POINTER(Q8MatmulF32Desc), _i64, _vp]),
    "q8_0_up_gate_swiglu_batched": (_int, [ctypes.POINTER(Q8UpGateDesc), _i64, _vp]),
    "q8_0_matmul_f32_step_ws_bytes": (_i64, [ctypes.POINTER(Q8MatmulF32Desc), _i64]),
    "q8_0_matmul_f32_step": (_int, [ctypes.POINTER(Q8MatmulF32Desc), _i64, _vp, _i64, _vp]),
    "moe_workspace_bytes": (_size, [_i64, _i64, _i64, _i64, _i64]),
    "moe_up_gate_swiglu": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                                  _size, _vp]),
    "moe_down_combine": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                                _size, _vp]),
    "moe_up_gate_swiglu_batched": (_int, [ctypes.POINTER(MoeUpGateDesc), _i64, _i64, _i64, _i64,
                                          _i64, _i64, _vp]),
    "moe_down_combine_batched": (_int, [ctypes.POINTER(MoeDownDesc), _i64, _i64, _i64, _i64, _i64,
                                        _i64, _vp]),
    "q8_0_matmul_blocksums": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "q8v_matvec_r8_batched_blocksums": (_int, [ctypes.POINTER(Q8R8Desc), _i64,
                                               ctypes.POINTER(_vp), _vp]),
    "q8v_matvec_r8_f32_batched_blocksums": (_int, [ctypes.POINTER(Q8R8F32Desc), _i64,
                                                   ctypes.POINTER(_vp), _vp]),
    "q8v_matmul_r8_batched_blocksums": (_int, [ctypes.POINTER(Q8R8MmDesc), _i64,
                                               ctypes.POINTER(_vp), _vp]),
    "moe_route": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _size, _vp]),
    "q8v_moe_up_gate": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                               _i64, _vp, _size, _vp]),
    "q8v_moe_hq": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                          _size, _vp]),
    "q8v_moe_r8_ffn": (_int, [ctypes.POINTER(MoeR8FfnDesc), _i64, _i64, _i64, _i64, _i64, _vp,
                              _vp, _vp, _vp, _vp, _vp, _vp]),
    "q8_read_probe": (_int, [_vp, _i64, _vp, _i64, _vp]),
    "q8_0_r8_bytes": (_i64, [_i64, _i64]),
    "q8_0_repack_r8": (_int, [_vp, _vp, _i64, _i64, _vp]),
    "q8_0_matvec_r8": (_int, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "q8_0_matvec_r8_batched": (_int, [ctypes.POINTER(Q8R8Desc), _i64, _vp]),
    "q8_0_matvec_r8_f32_batched": (_int, [ctypes.POINTER(Q8R8F32Desc), _i64, _vp]),
    "q8_0_matmul_r8_batched": (_int, [ctypes.POINTER(Q8R8MmDesc), _i64, _vp]),
    "q8_1_quantize_rows": (_int, [_vp, _i64, _vp, _i64, _i64, _vp]),
    "moe_r8_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, _i64, _i64]),
    "moe_r8_ffn_batched": (_int, [ctypes.POINTER(MoeR8FfnDesc), _i64, _i64, _i64, _i64, _i64,
                                  _i64, _vp]),
    "moe_r8_ffn_batched_noalloc": (_int, [ctypes.POINTER(MoeR8FfnDesc), _i64, _i64, _i64, _i64,
                                          _i64, _i64, _vp]),
    "moe_r8_fused_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, _i64]),
    "moe_r8_ffn_fused": (_int, [ctypes.POINTER(MoeR8FfnDesc), _i64, _i64, _i64, _i64, _vp]),
    "kq_matvec_batched": (_int, [_int, ctypes.POINTER(KqMatvecDesc), _i64, _vp]),
    "q4_k_matvec": (_int, [_vp, _vp, _vp, _i64, _i64, _vp]),
    "i8_quantize_rows": (_int, [_vp, _int, _i64, _vp, _i64, _vp, _i64, _i64, _vp]),
    "i8_workspace_bytes": (_size, [_i64, _i64]),
    "i8_matmul": (_int, [_vp, _int, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _int, _i64, _i64, _i64,
                         _i64, _vp, _size, _vp]),
    "i8_up_gate_swiglu": (_int, [_vp, _int, _i64, _vp, _vp, _i64, _vp, _vp, _int, _i64, _i64,
                                 _i64, _i64, _vp, _size, _vp]),
    "i8_matmul_act": (_int, [_vp, _int, _i64, _vp, _vp, _i64, _vp, _vp, _int, _vp, _i64, _vp, _int,
                             _i64, _i64, _i64, _i64, _vp, _size, _vp]),
    "embed_rows": (_int, [_vp, _int, _i64, _vp, _vp, ctypes.c_float, _vp, _int, _i64, _i64, _i64, _i64,
                          _vp]),
    "q8_0_embed_rows": (_int, [_vp, _int, _vp, ctypes.c_float, _vp, _int, _i64, _i64, _i64, _i64, _vp]),
    "norm_rows": (_int, [_vp, _int, _i64, _vp, _vp, ctypes.c_float, _int, _vp, _int, _i64, _vp, _i64,
                         _i64, _vp]),
    "residual_norm_rows": (_int, [ctypes.POINTER(ResidualNormDesc), _i64, _i64, _vp]),
    "sample_workspace_bytes": (_size, [_i64, _i64]),
    "sample_rows": (_int, [_vp, _int, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp,
                           _size, _vp]),
    "q8v_i8_form": (_int, [_i64, _i64, _i64, _int]),
    "q8v_i8_act_form": (_int, [_i64, _i64, _i64]),
    "logprob_workspace_bytes": (_size, [_i64, _i64, _i64]),
    "logprob_rows": (_int, [_vp, _int, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                            _vp, _size, _vp]),
    "q5_k_matvec": (_int, [_vp, _vp, _vp, _i64, _i64, _vp]),
}

EXPORTS = tuple(_SIGS)

for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

STATUS = {0: "Q8_OK", -1: "Q8_E_NULL", -2: "Q8_E_SHAPE", -3: "Q8_E_ALIGN",
          -4: "Q8_E_UNSUPPORTED", -5: "Q8_E_WORKSPACE", -6: "Q8_E_HIP"}


class Q8Error(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = _lib.q8_status_str(status).decode()
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")


def _check(fn, rc):
    if rc != 0:
        raise Q8Error(fn, rc)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(t):
    if t is None or not t.is_cuda:
        return None
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t, dtype, name):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")


def _nbytes(t):
    return t.numel() * t.element_size()


def _fit(t, nbytes, name):
    """A contiguous GPU tensor that holds at least nbytes (the extent the
    kernels touch for the shape arguments of the call)."""
    if t is None:
        return
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    if nbytes > _nbytes(t):
        raise ValueError(f"{name}: the shape arguments need {nbytes} bytes, the tensor holds "
                         f"{_nbytes(t)}")


def _one_device(*ts):
    """Every tensor (or (tensor, offset) pair) of a call on one device."""
    devs = {(t[0] if isinstance(t, tuple) else t).device for t in ts if t is not None}
    if len(devs) > 1:
        raise ValueError(f"tensors on several devices: {sorted(map(str, devs))}")


def _addr(t, unit, nbytes, name):
    """Address of a descriptor operand: t is a tensor or a (tensor, offset)
    pair with the offset in `unit` bytes; the tensor must hold nbytes from
    that address on."""
    base, off = (t if isinstance(t, tuple) else (t, 0))
    if not base.is_contiguous() or not base.is_cuda:
        raise ValueError(f"{name}: must be a contiguous GPU tensor")
    if off < 0:
        raise ValueError(f"{name}: negative offset")
    avail = _nbytes(base) - off * unit
    if nbytes > 0 and nbytes > avail:
        raise ValueError(f"{name}: the descriptor needs {nbytes} bytes from its start, the "
                         f"tensor holds {max(avail, 0)}")
    return base.data_ptr() + off * unit


def _span(batch, bstride, rows, rstride, last):
    """Elements from the first to one past the last one touched: `batch`
    entries `bstride` apart, each `rows` rows `rstride` apart of `last`
    elements (0 when nothing is touched)."""
    if batch <= 0 or rows <= 0 or last <= 0:
        return 0
    return (batch - 1) * bstride + (rows - 1) * rstride + last


def _r8_bytes_py(n, k):
    return (n + 7) // 8 * 272 * (k // QK)


def status_str(status):
    return _lib.q8_status_str(int(status)).decode()


def version():
    return _lib.q8_version().decode()


def q8_empty(rows, k, device):
    """Uninitialised Q8_0 storage for [rows][k] values (uint8 [rows][k/32*34])."""
    return torch.empty((rows, k // QK * BLOCK_BYTES), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------

def q8_0_quantize_rows(x, y=None, k=None):
    """x: fp32 [n_rows][stride] (or [k]) -> y: uint8 [n_rows][k/32*34]."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dtype != torch.float32 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x: GPU fp32 with unit column stride")
    n_rows = x.shape[0]
    k = x.shape[1] if k is None else k
    if x.shape[1] < k:
        raise ValueError(f"x: rows of {x.shape[1]} values, k = {k}")
    if y is None:
        y = q8_empty(n_rows, k, x.device)
    _need(y, torch.uint8, "y")
    _one_device(x, y)
    _fit(y, n_rows * (k // QK) * BLOCK_BYTES, "y")
    _check("q8_0_quantize_rows", _lib.q8_0_quantize_rows(
        _ptr(x), x.stride(0) if n_rows > 1 else k, _ptr(y), n_rows, k, _stream(x)))
    return y


def q8_0_matvec(w, x, n, k, y=None):
    _need(w, torch.uint8, "w")
    _need(x, torch.uint8, "x")
    if y is None:
        y = torch.empty(n, dtype=torch.float32, device=w.device)
    _need(y, torch.float32, "y")
    _one_device(w, x, y)
    nb = k // QK
    _fit(w, n * nb * BLOCK_BYTES, "w")
    _fit(x, nb * BLOCK_BYTES, "x")
    _fit(y, n * 4, "y")
    _check("q8_0_matvec", _lib.q8_0_matvec(_ptr(w), _ptr(x), _ptr(y), n, k, _stream(w)))
    return y


def q8_0_r8_bytes(n, k):
    v = _lib.q8_0_r8_bytes(n, k)
    _check("q8_0_r8_bytes", v if v < 0 else 0)
    return int(v)


def q8_0_repack_r8(w, n, k, out=None):
    """Native Q8_0 rows (uint8 GPU tensor) -> the row-interleaved (R8) layout."""
    _need(w, torch.uint8, "w")
    if out is None:
        out = torch.empty(q8_0_r8_bytes(n, k), dtype=torch.uint8, device=w.device)
    _need(out, torch.uint8, "out")
    _one_device(w, out)
    _fit(w, n * (k // QK) * BLOCK_BYTES, "w")
    _fit(out, q8_0_r8_bytes(n, k), "out")
    _check("q8_0_repack_r8", _lib.q8_0_repack_r8(_ptr(w), _ptr(out), n, k, _stream(w)))
    return out


def q8_0_matvec_r8(w_r8, x, n, k, y=None):
    _need(w_r8, torch.uint8, "w_r8")
    _need(x, torch.uint8, "x")
    if y is None:
        y = torch.empty(n, dtype=torch.float32, device=w_r8.device)
    _need(y, torch.float32, "y")
    _one_device(w_r8, x, y)
    _fit(w_r8, q8_0_r8_bytes(n, k), "w_r8")
    _fit(x, (k // QK) * BLOCK_BYTES, "x")
    _fit(y, n * 4, "y")
    _check("q8_0_matvec_r8", _lib.q8_0_matvec_r8(_ptr(w_r8), _ptr(x), _ptr(y), n, k,
                                                 _stream(w_r8)))
    return y


def make_r8_desc(w_r8, x, y, n, k, batch=1, w_batch_stride=0, x_batch_stride=0,
                 y_batch_stride=0):
    """One q8_0_r8_desc.  w_r8 (bytes), x (blocks), y (floats) are (tensor,
    element offset) pairs or tensors; w_batch_stride in bytes, x_batch_stride
    in blocks, y_batch_stride in floats."""
    _one_device(w_r8, x, y)
    nb = k // QK
    wb = _span(batch, w_batch_stride, 1, 0, _r8_bytes_py(n, k)) if n > 0 else 0
    return Q8R8Desc(_addr(w_r8, 1, wb, "w_r8"),
                    _addr(x, BLOCK_BYTES, _span(batch, x_batch_stride, 1, 0, nb) * BLOCK_BYTES, "x"),
                    _addr(y, 4, _span(batch, y_batch_stride, 1, 0, n) * 4, "y"), n, k, batch,
                    w_batch_stride, x_batch_stride, y_batch_stride)


def q8_0_matvec_r8_batched(descs, stream_of):
    """descs: list of Q8R8Desc; stream_of: a tensor on the target device."""
    arr = (Q8R8Desc * max(1, len(descs)))(*descs)
    _check("q8_0_matvec_r8_batched",
           _lib.q8_0_matvec_r8_batched(arr, len(descs), _stream(stream_of)))


def make_r8_f32_desc(w_r8, x, y, n, k, batch=1, w_batch_stride=0, x_batch_stride=0,
                     y_batch_stride=0):
    """One q8_0_r8_f32_desc.  w_r8 (bytes), x (floats), y (floats) are (tensor,
    element offset) pairs or tensors; w_batch_stride in bytes, the others in
    floats."""
    _one_device(w_r8, x, y)
    wb = _span(batch, w_batch_stride, 1, 0, _r8_bytes_py(n, k)) if n > 0 else 0
    return Q8R8F32Desc(_addr(w_r8, 1, wb, "w_r8"),
                       _addr(x, 4, _span(batch, x_batch_stride, 1, 0, k) * 4 if n > 0 else 0, "x"),
                       _addr(y, 4, _span(batch, y_batch_stride, 1, 0, n) * 4, "y"), n, k, batch,
                       w_batch_stride, x_batch_stride, y_batch_stride)


def _sum_ptrs(sums):
    for i, t in enumerate(sums):
        _need(t, torch.int32, f"sums[{i}]")
    return (_vp * max(1, len(sums)))(*[t.data_ptr() for t in sums])


def q8v_matvec_r8_batched_blocksums(descs, sums, stream_of):
    """q8_0_matvec_r8_batched plus the int32 block sums of descriptor i in
    sums[i] (a GPU int32 tensor of batch*n*(k/32) elements)."""
    for d, t in zip(descs, sums):
        _fit(t, max(d.batch, 0) * max(d.n, 0) * (d.k // QK) * 4, "sums")
    arr = (Q8R8Desc * max(1, len(descs)))(*descs)
    _check("q8v_matvec_r8_batched_blocksums", _lib.q8v_matvec_r8_batched_blocksums(
        arr, len(descs), _sum_ptrs(sums), _stream(stream_of)))


def q8v_matvec_r8_f32_batched_blocksums(descs, sums, stream_of):
    """q8_0_matvec_r8_f32_batched plus the int32 block sums of descriptor i in
    sums[i] (batch*n*(k/32) elements)."""
    for d, t in zip(descs, sums):
        _fit(t, max(d.batch, 0) * max(d.n, 0) * (d.k // QK) * 4, "sums")
    arr = (Q8R8F32Desc * max(1, len(descs)))(*descs)
    _check("q8v_matvec_r8_f32_batched_blocksums", _lib.q8v_matvec_r8_f32_batched_blocksums(
        arr, len(descs), _sum_ptrs(sums), _stream(stream_of)))


def q8v_matmul_r8_batched_blocksums(descs, sums, stream_of):
    """q8_0_matmul_r8_batched plus the int32 block sums of descriptor i in
    sums[i] (batch*m*n*(k/32) elements)."""
    for d, t in zip(descs, sums):
        _fit(t, max(d.batch, 0) * max(d.m, 0) * max(d.n, 0) * (d.k // QK) * 4, "sums")
    arr = (Q8R8MmDesc * max(1, len(descs)))(*descs)
    _check("q8v_matmul_r8_batched_blocksums", _lib.q8v_matmul_r8_batched_blocksums(
        arr, len(descs), _sum_ptrs(sums), _stream(stream_of)))


def q8_0_matvec_r8_f32_batched(descs, stream_of):
    """descs: list of Q8R8F32Desc; stream_of: a tensor on the target device."""
    arr = (Q8R8F32Desc * max(1, len(descs)))(*descs)
    _check("q8_0_matvec_r8_f32_batched",
           _lib.q8_0_matvec_r8_f32_batched(arr, len(descs), _stream(stream_of)))


def make_r8_mm_desc(w_r8, x, y, n, k, m=1, batch=1, w_batch_stride=0, x_row_stride=None,
                    x_batch_stride=0, y_row_stride=None, y_batch_stride=0):
    """One q8_0_r8_mm_desc.  w_r8 (bytes), x (blocks), y (floats) are (tensor,
    element offset) pairs or tensors; w_batch_stride in bytes, x strides in
    blocks, y strides in floats."""
    nb = k // QK
    xrs = nb if x_row_stride is None else x_row_stride
    yrs = n if y_row_stride is None else y_row_stride
    _one_device(w_r8, x, y)
    live = n > 0 and m > 0
    wb = _span(batch, w_batch_stride, 1, 0, _r8_bytes_py(n, k)) if live else 0
    xb = _span(batch, x_batch_stride, m, xrs, nb) * BLOCK_BYTES if live else 0
    return Q8R8MmDesc(_addr(w_r8, 1, wb, "w_r8"), _addr(x, BLOCK_BYTES, xb, "x"),
                      _addr(y, 4, _span(batch, y_batch_stride, m, yrs, n) * 4, "y"), n, k, m,
                      batch, w_batch_stride, xrs, x_batch_stride, yrs, y_batch_stride)


def q8_0_matmul_r8_batched(descs, stream_of):
    arr = (Q8R8MmDesc * max(1, len(descs)))(*descs)
    _check("q8_0_matmul_r8_batched",
           _lib.q8_0_matmul_r8_batched(arr, len(descs), _stream(stream_of)))


Q8_1_BLOCK_BYTES = 36
KQ_BLOCK_BYTES = {4: 144, 5: 176}


def q8_1_quantize_rows(x, k=None, y=None):
    """x: fp32 [n_rows][stride] (or [k]) -> y: uint8 [n_rows][k/32*36] (Q8_1)."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dtype != torch.float32 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x: GPU fp32 with unit column stride")
    n_rows = x.shape[0]
    k = x.shape[1] if k is None else k
    if x.shape[1] < k:
        raise ValueError(f"x: rows of {x.shape[1]} values, k = {k}")
    if y is None:
        y = torch.empty((n_rows, k // QK * Q8_1_BLOCK_BYTES), dtype=torch.uint8, device=x.device)
    _need(y, torch.uint8, "y")
    _one_device(x, y)
    _fit(y, n_rows * (k // QK) * Q8_1_BLOCK_BYTES, "y")
    _check("q8_1_quantize_rows", _lib.q8_1_quantize_rows(
        _ptr(x), x.stride(0) if n_rows > 1 else k, _ptr(y), n_rows, k, _stream(x)))
    return y


def kq_matvec(t, w, x, n, k, y=None):
    """One product over K-quant weights (t = 4: Q4_K, t = 5: Q5_K) and a Q8_1 row."""
    _need(w, torch.uint8, "w")
    _need(x, torch.uint8, "x")
    if y is None:
        y = torch.empty(n, dtype=torch.float32, device=w.device)
    _need(y, torch.float32, "y")
    fn = {4: _lib.q4_k_matvec, 5: _lib.q5_k_matvec}.get(t)
    if fn is None:
        raise ValueError(f"unknown K-quant type {t}")
    _one_device(w, x, y)
    _fit(w, n * (k // 256) * KQ_BLOCK_BYTES[t], "w")
    _fit(x, (k // QK) * Q8_1_BLOCK_BYTES, "x")
    _fit(y, n * 4, "y")
    _check("q4_k_matvec" if t == 4 else "q5_k_matvec",
           fn(_ptr(w), _ptr(x), _ptr(y), n, k, _stream(w)))
    return y


def make_kq_desc(w, x, y, n, k, batch=1, w_batch_stride=0, x_batch_stride=0, y_batch_stride=0,
                 t=4):
    """One kq_matvec_desc for K-quant type t (4: Q4_K, 5: Q5_K).  w (bytes), x
    (bytes), y (floats) are (tensor, element offset) pairs or tensors; strides
    in super-blocks, Q8_1 blocks, floats."""
    _one_device(w, x, y)
    bb = KQ_BLOCK_BYTES[t]
    live = n > 0
    wb = _span(batch, w_batch_stride, 1, 0, n * (k // 256)) * bb if live else 0
    xb = _span(batch, x_batch_stride, 1, 0, k // QK) * Q8_1_BLOCK_BYTES if live else 0
    return KqMatvecDesc(_addr(w, 1, wb, "w"), _addr(x, 1, xb, "x"),
                        _addr(y, 4, _span(batch, y_batch_stride, 1, 0, n) * 4, "y"), n, k, batch,
                        w_batch_stride, x_batch_stride, y_batch_stride)


def kq_matvec_batched(t, descs, stream_of):
    arr = (KqMatvecDesc * max(1, len(descs)))(*descs)
    _check("kq_matvec_batched", _lib.kq_matvec_batched(t, arr, len(descs), _stream(stream_of)))


def q8_0_matmul(w, x, n, k, m, y=None):
    _need(w, torch.uint8, "w")
    _need(x, torch.uint8, "x")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=w.device)
    _need(y, torch.float32, "y")
    _one_device(w, x, y)
    nb = k // QK
    _fit(w, n * nb * BLOCK_BYTES, "w")
    _fit(x, m * nb * BLOCK_BYTES, "x")
    _fit(y, m * n * 4, "y")
    _check("q8_0_matmul", _lib.q8_0_matmul(_ptr(w), _ptr(x), _ptr(y), n, k, m, _stream(w)))
    return y


def make_desc(w, x, y, n, k, m=1, batch=1, w_batch_stride=0, x_row_stride=None,
              x_batch_stride=0, y_row_stride=None, y_batch_stride=0):
    """One q8_0_matmul_desc.  w, x, y are (tensor, element offset) pairs or tensors;
    strides are in blocks (w, x) and floats (y)."""
    nb = k // QK
    xrs = nb if x_row_stride is None else x_row_stride
    yrs = n if y_row_stride is None else y_row_stride
    _one_device(w, x, y)
    live = n > 0 and m > 0
    wb = _span(batch, w_batch_stride, 1, 0, n * nb) * BLOCK_BYTES if live else 0
    xb = _span(batch, x_batch_stride, m, xrs, nb) * BLOCK_BYTES if live else 0
    return Q8MatmulDesc(_addr(w, BLOCK_BYTES, wb, "w"), _addr(x, BLOCK_BYTES, xb, "x"),
                        _addr(y, 4, _span(batch, y_batch_stride, m, yrs, n) * 4, "y"), n, k, m,
                        batch, w_batch_stride, xrs, x_batch_stride, yrs, y_batch_stride)


def make_up_gate_desc(w, x, h, n_ff, n_embd, m=1, batch=1, w_batch_stride=0, x_row_stride=None,
                      x_batch_stride=0, h_row_stride=None, h_batch_stride=0):
    """One q8_0_up_gate_desc.  w (combined [2*n_ff][n_embd/32] blocks, gate rows
    first), x (Q8_0 rows), h are (tensor, element offset) pairs or tensors;
    strides are in blocks (w, x) and floats (h)."""
    nb = n_embd // QK
    xrs = nb if x_row_stride is None else x_row_stride
    hrs = n_ff if h_row_stride is None else h_row_stride
    _one_device(w, x, h)
    live = n_ff > 0 and m > 0
    wb = _span(batch, w_batch_stride, 1, 0, 2 * n_ff * nb) * BLOCK_BYTES if live else 0
    xb = _span(batch, x_batch_stride, m, xrs, nb) * BLOCK_BYTES if live else 0
    return Q8UpGateDesc(_addr(w, BLOCK_BYTES, wb, "w"), _addr(x, BLOCK_BYTES, xb, "x"),
                        _addr(h, 4, _span(batch, h_batch_stride, m, hrs, n_ff) * 4, "h"), n_ff,
                        n_embd, m, batch, w_batch_stride, xrs, x_batch_stride, hrs,
                        h_batch_stride)


def q8_0_up_gate_swiglu_batched(descs, stream_of):
    """descs: list of Q8UpGateDesc; stream_of: a tensor on the target device."""
    arr = (Q8UpGateDesc * max(1, len(descs)))(*descs)
    _check("q8_0_up_gate_swiglu_batched",
           _lib.q8_0_up_gate_swiglu_batched(arr, len(descs), _stream(stream_of)))


def q8_0_matmul_batched(descs, stream_of):
    """descs: list of Q8MatmulDesc; stream_of: a tensor on the target device."""
    arr = (Q8MatmulDesc * len(descs))(*descs)
    _check("q8_0_matmul_batched", _lib.q8_0_matmul_batched(arr, len(descs), _stream(stream_of)))


def make_f32_desc(w, x, y, n, k, m=1, batch=1, w_batch_stride=0, x_row_stride=None,
                  x_batch_stride=0, y_row_stride=None, y_batch_stride=0):
    """One q8_0_matmul_f32_desc (fp32 activations, quantized inside).  w, x, y
    are (tensor, element offset) pairs or tensors; strides are in blocks (w)
    and floats (x, y)."""
    xrs = k if x_row_stride is None else x_row_stride
    yrs = n if y_row_stride is None else y_row_stride
    _one_device(w, x, y)
    live = n > 0 and m > 0
    wb = _span(batch, w_batch_stride, 1, 0, n * (k // QK)) * BLOCK_BYTES if live else 0
    xb = _span(batch, x_batch_stride, m, xrs, k) * 4 if live else 0
    return Q8MatmulF32Desc(_addr(w, BLOCK_BYTES, wb, "w"), _addr(x, 4, xb, "x"),
                           _addr(y, 4, _span(batch, y_batch_stride, m, yrs, n) * 4, "y"), n, k,
                           m, batch, w_batch_stride, xrs, x_batch_stride, yrs, y_batch_stride)


def q8_0_matmul_f32_batched(descs, stream_of):
    """descs: list of Q8MatmulF32Desc; stream_of: a tensor on the target device."""
    arr = (Q8MatmulF32Desc * len(descs))(*descs)
    _check("q8_0_matmul_f32_batched",
           _lib.q8_0_matmul_f32_batched(arr, len(descs), _stream(stream_of)))


def q8_0_matmul_f32_step_ws_bytes(descs):
    """Workspace bytes q8_0_matmul_f32_step needs for these descriptors."""
    arr = (Q8MatmulF32Desc * max(1, len(descs)))(*descs)
    n = int(_lib.q8_0_matmul_f32_step_ws_bytes(arr, len(descs)))
    if n < 0:
        raise Q8Error("q8_0_matmul_f32_step_ws_bytes", n)
    return n


def q8_0_matmul_f32_step_workspace(descs, device):
    """A zero-filled workspace for q8_0_matmul_f32_step (uint8 tensor)."""
    n = q8_0_matmul_f32_step_ws_bytes(descs)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def q8_0_matmul_f32_step(descs, ws, stream_of=None):
    """descs: list of Q8MatmulF32Desc (m <= 2); ws: the zero-filled uint8
    workspace tensor (reused across calls)."""
    _need(ws, torch.uint8, "ws")
    arr = (Q8MatmulF32Desc * max(1, len(descs)))(*descs)
    _check("q8_0_matmul_f32_step", _lib.q8_0_matmul_f32_step(
        arr, len(descs), _ptr(ws), ws.numel(), _stream(ws if stream_of is None else stream_of)))


def q8_0_matmul_blocksums(w, x, n, k, m):
    _need(w, torch.uint8, "w")
    _need(x, torch.uint8, "x")
    _one_device(w, x)
    _fit(w, n * (k // QK) * BLOCK_BYTES, "w")
    _fit(x, m * (k // QK) * BLOCK_BYTES, "x")
    y = torch.empty((m, n), dtype=torch.float32, device=w.device)
    s = torch.empty((m, n, k // QK), dtype=torch.int32, device=w.device)
    _check("q8_0_matmul_blocksums", _lib.q8_0_matmul_blocksums(
        _ptr(w), _ptr(x), _ptr(y), _ptr(s), n, k, m, _stream(w)))
    return y, s


def _ids_shape(ids):
    if ids.dim() != 2:
        raise ValueError(f"ids: expected [n_tok][n_used], got shape {tuple(ids.shape)}")
    return int(ids.shape[0]), int(ids.shape[1])


def _check_up_gate(w, x, ids, h, n_tok, n_used, n_embd, n_ff, n_expert, r8=False):
    """Extents of one expert-FFN up_gate layer (native rows, or R8 with r8=True)."""
    _one_device(w, x, ids, h)
    if tuple(ids.shape) != (n_tok, n_used):
        raise ValueError(f"ids: shape {tuple(ids.shape)}, expected {(n_tok, n_used)}")
    rows = n_expert * 2 * n_ff
    _fit(w, _r8_bytes_py(rows, n_embd) if r8 else rows * (n_embd // QK) * BLOCK_BYTES,
         "w_up_gate_r8" if r8 else "w_up_gate")
    _fit(x, n_tok * n_embd * 4, "x")
    _fit(h, n_tok * n_used * n_ff * 4, "h")


def _check_down(w, h, ids, cw, out, n_tok, n_used, n_ff, n_embd, n_expert, r8=False):
    """Extents of one expert-FFN down + combine layer."""
    _one_device(w, h, ids, cw, out)
    if tuple(ids.shape) != (n_tok, n_used):
        raise ValueError(f"ids: shape {tuple(ids.shape)}, expected {(n_tok, n_used)}")
    rows = n_expert * n_embd
    _fit(w, _r8_bytes_py(rows, n_ff) if r8 else rows * (n_ff // QK) * BLOCK_BYTES,
         "w_down_r8" if r8 else "w_down")
    _fit(h, n_tok * n_used * n_ff * 4, "h")
    _fit(cw, n_tok * n_used * 4, "cw")
    _fit(out, n_tok * n_embd * 4, "out")


def moe_workspace_bytes(n_tok, n_embd, n_ff, n_expert, n_used):
    return int(_lib.moe_workspace_bytes(n_tok, n_embd, n_ff, n_expert, n_used))


def moe_workspace(n_tok, n_embd, n_ff, n_expert, n_used, device):
    nbytes = moe_workspace_bytes(n_tok, n_embd, n_ff, n_expert, n_used)
    if nbytes == 0:
        raise Q8Error("moe_workspace_bytes", -4)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def moe_up_gate_swiglu(w_up_gate, x, ids, n_embd, n_ff, n_expert, ws, h=None):
    """h[t][u][j] = silu(gate) * up from fp32 token rows x [n_tok][n_embd]
    (quantized inside); returns h fp32 [n_tok][n_used][n_ff]."""
    _need(w_up_gate, torch.uint8, "w_up_gate")
    _need(x, torch.float32, "x")
    _need(ids, torch.int32, "ids")
    _need(ws, torch.uint8, "ws")
    n_tok, n_used = _ids_shape(ids)
    if h is None:
        h = torch.empty((n_tok, n_used, n_ff), dtype=torch.float32, device=ids.device)
    _need(h, torch.float32, "h")
    _check_up_gate(w_up_gate, x, ids, h, n_tok, n_used, n_embd, n_ff, n_expert)
    _one_device(ids, ws)
    _check("moe_up_gate_swiglu", _lib.moe_up_gate_swiglu(
        _ptr(w_up_gate), _ptr(x), _ptr(ids), _ptr(h), n_tok, n_embd, n_ff, n_expert, n_used,
        _ptr(ws), ws.numel(), _stream(ids)))
    return h


def moe_down_combine(w_down, h, ids, cw, n_ff, n_embd, n_expert, ws, out=None):
    """out[t] = sum_u cw[t][u] * down_e(q(h[t][u])); returns fp32 [n_tok][n_embd]."""
    _need(w_down, torch.uint8, "w_down")
    _need(h, torch.float32, "h")
    _need(ids, torch.int32, "ids")
    _need(cw, torch.float32, "cw")
    _need(ws, torch.uint8, "ws")
    n_tok, n_used = _ids_shape(ids)
    if out is None:
        out = torch.empty((n_tok, n_embd), dtype=torch.float32, device=ids.device)
    _need(out, torch.float32, "out")
    _check_down(w_down, h, ids, cw, out, n_tok, n_used, n_ff, n_embd, n_expert)
    _one_device(ids, ws)
    _check("moe_down_combine", _lib.moe_down_combine(
        _ptr(w_down), _ptr(h), _ptr(ids), _ptr(cw), _ptr(out), n_tok, n_ff, n_embd, n_expert,
        n_used, _ptr(ws), ws.numel(), _stream(ids)))
    return out


def moe_up_gate_swiglu_batched(layers, n_embd, n_ff, n_expert):
    """Grouped up_gate over independent layers of one shape.  layers: list of
    dicts with w_up_gate, x, ids, h (written), ws; returns the list of h."""
    if not layers:
        return []
    for d in layers:
        _need(d["w_up_gate"], torch.uint8, "w_up_gate")
        _need(d["x"], torch.float32, "x")
        _need(d["ids"], torch.int32, "ids")
        _need(d["h"], torch.float32, "h")
        _need(d["ws"], torch.uint8, "ws")
    n_tok, n_used = _ids_shape(layers[0]["ids"])
    for d in layers:
        _check_up_gate(d["w_up_gate"], d["x"], d["ids"], d["h"], n_tok, n_used, n_embd, n_ff,
                       n_expert)
        _one_device(layers[0]["ids"], d["ids"], d["ws"])
    arr = (MoeUpGateDesc * len(layers))(*[
        MoeUpGateDesc(_ptr(d["w_up_gate"]), _ptr(d["x"]), _ptr(d["ids"]), _ptr(d["h"]),
                      _ptr(d["ws"]), d["ws"].numel()) for d in layers])
    _check("moe_up_gate_swiglu_batched", _lib.moe_up_gate_swiglu_batched(
        arr, len(layers), n_tok, n_embd, n_ff, n_expert, n_used, _stream(layers[0]["ids"])))
    return [d["h"] for d in layers]


def moe_down_combine_batched(layers, n_ff, n_embd, n_expert):
    """Grouped down projection + combine over independent layers of one shape.
    layers: list of dicts with w_down, h, ids, cw, out (written), ws."""
    if not layers:
        return []
    for d in layers:
        _need(d["w_down"], torch.uint8, "w_down")
        _need(d["h"], torch.float32, "h")
        _need(d["ids"], torch.int32, "ids")
        _need(d["cw"], torch.float32, "cw")
        _need(d["out"], torch.float32, "out")
        _need(d["ws"], torch.uint8, "ws")
    n_tok, n_used = _ids_shape(layers[0]["ids"])
    for d in layers:
        _check_down(d["w_down"], d["h"], d["ids"], d["cw"], d["out"], n_tok, n_used, n_ff, n_embd,
                    n_expert)
        _one_device(layers[0]["ids"], d["ids"], d["ws"])
    arr = (MoeDownDesc * len(layers))(*[
        MoeDownDesc(_ptr(d["w_down"]), _ptr(d["h"]), _ptr(d["ids"]), _ptr(d["cw"]), _ptr(d["out"]),
                    _ptr(d["ws"]), d["ws"].numel()) for d in layers])
    _check("moe_down_combine_batched", _lib.moe_down_combine_batched(
        arr, len(layers), n_tok, n_ff, n_embd, n_expert, n_used, _stream(layers[0]["ids"])))
    return [d["out"] for d in layers]


def q8v_moe_up_gate(w_up_gate, x, ids, n_embd, n_ff, n_expert, ws, sums=True, route=True):
    """moe_up_gate_swiglu plus its validation outputs: returns (h, sums, counts,
    offsets, pairs) -- sums int32 [n_tok*n_used][2*n_ff][n_embd/32] and the
    expert-major grouping the kernels served (None where not asked for)."""
    _need(w_up_gate, torch.uint8, "w_up_gate")
    _need(x, torch.float32, "x")
    _need(ids, torch.int32, "ids")
    _need(ws, torch.uint8, "ws")
    n_tok, n_used = _ids_shape(ids)
    dev = ids.device
    h = torch.full((n_tok, n_used, n_ff), float("nan"), dtype=torch.float32, device=dev)
    _check_up_gate(w_up_gate, x, ids, h, n_tok, n_used, n_embd, n_ff, n_expert)
    _one_device(ids, ws)
    slots = n_tok * n_used
    s = (torch.full((slots, 2 * n_ff, n_embd // QK), -(1 << 31), dtype=torch.int32, device=dev)
         if sums else None)
    c = torch.full((n_expert,), -1, dtype=torch.int32, device=dev) if route else None
    o = torch.full((n_expert + 1,), -1, dtype=torch.int32, device=dev) if route else None
    p = torch.full((max(slots, 1),), -1, dtype=torch.int32, device=dev) if route else None
    _check("q8v_moe_up_gate", _lib.q8v_moe_up_gate(
        _ptr(w_up_gate), _ptr(x), _ptr(ids), _ptr(h), _ptr(s), _ptr(c), _ptr(o), _ptr(p), n_tok,
        n_embd, n_ff, n_expert, n_used, _ptr(ws), ws.numel(), _stream(ids)))
    return h, s, c, o, (p[:slots] if p is not None else None)


def q8v_moe_hq(w_down, h, ids, cw, n_ff, n_embd, n_expert, ws, sums=True):
    """moe_down_combine plus its validation outputs: returns (out, hq, sums) --
    hq uint8 [n_tok*n_used][n_ff/32*34] (the Q8_0 bytes of h the down products
    used), sums int32 [n_tok*n_used][n_embd][n_ff/32] (None if not asked)."""
    _need(w_down, torch.uint8, "w_down")
    _need(h, torch.float32, "h")
    _need(ids, torch.int32, "ids")
    _need(cw, torch.float32, "cw")
    _need(ws, torch.uint8, "ws")
    n_tok, n_used = _ids_shape(ids)
    dev = ids.device
    out = torch.full((n_tok, n_embd), float("nan"), dtype=torch.float32, device=dev)
    _check_down(w_down, h, ids, cw, out, n_tok, n_used, n_ff, n_embd, n_expert)
    _one_device(ids, ws)
    slots = n_tok * n_used
    hq = torch.zeros((slots, n_ff // QK * BLOCK_BYTES), dtype=torch.uint8, device=dev)
    s = (torch.full((slots, n_embd, n_ff // QK), -(1 << 31), dtype=torch.int32, device=dev)
         if sums else None)
    _check("q8v_moe_hq", _lib.q8v_moe_hq(
        _ptr(w_down), _ptr(h), _ptr(ids), _ptr(cw), _ptr(out), _ptr(hq), _ptr(s), n_tok, n_ff,
        n_embd, n_expert, n_used, _ptr(ws), ws.numel(), _stream(ids)))
    return out, hq, s


def q8v_moe_r8_ffn(layer, n_embd, n_ff, n_expert, route=False):
    """moe_r8_ffn_batched for one layer (a dict as for moe_r8_ffn_batched) plus
    the validation outputs: returns (ug_sums, dn_sums, hq, counts, offsets,
    pairs); the routing only with route=True (grouped path only)."""
    arr, n_tok, n_used = _r8_ffn_descs([layer], n_embd, n_ff, n_expert, True)
    dev = layer["ids"].device
    slots = n_tok * n_used
    ug = torch.full((slots, 2 * n_ff, n_embd // QK), -(1 << 31), dtype=torch.int32, device=dev)
    dn = torch.full((slots, n_embd, n_ff // QK), -(1 << 31), dtype=torch.int32, device=dev)
    hq = torch.zeros((slots, n_ff // QK * BLOCK_BYTES), dtype=torch.uint8, device=dev)
    c = torch.full((n_expert,), -1, dtype=torch.int32, device=dev) if route else None
    o = torch.full((n_expert + 1,), -1, dtype=torch.int32, device=dev) if route else None
    p = torch.full((max(slots, 1),), -1, dtype=torch.int32, device=dev) if route else None
    _check("q8v_moe_r8_ffn", _lib.q8v_moe_r8_ffn(
        arr, n_tok, n_embd, n_ff, n_expert, n_used, _ptr(ug), _ptr(dn), _ptr(hq), _ptr(c), _ptr(o),
        _ptr(p), _stream(layer["ids"])))
    return ug, dn, hq, c, o, (p[:slots] if p is not None else None)


def moe_route(ids, n_expert, ws):
    _need(ids, torch.int32, "ids")
    _need(ws, torch.uint8, "ws")
    _one_device(ids, ws)
    n_tok, n_used = _ids_shape(ids)
    dev = ids.device
    counts = torch.empty(n_expert, dtype=torch.int32, device=dev)
    offsets = torch.empty(n_expert + 1, dtype=torch.int32, device=dev)
    pairs = torch.empty(max(n_tok * n_used, 1), dtype=torch.int32, device=dev)
    _check("moe_route", _lib.moe_route(_ptr(ids), _ptr(counts), _ptr(offsets), _ptr(pairs),
                                       n_tok, n_expert, n_used, _ptr(ws), ws.numel(),
                                       _stream(ids)))
    return counts, offsets, pairs[: n_tok * n_used]


def q8_read_probe(buf, sink):
    """Stream-read the bytes of `buf` (a GPU tensor); sink: int32 GPU tensor."""
    _need(sink, torch.int32, "sink")
    _fit(buf, 0, "buf")
    _one_device(buf, sink)
    _check("q8_read_probe", _lib.q8_read_probe(_ptr(buf), buf.numel() * buf.element_size(),
                                               _ptr(sink), sink.numel(), _stream(buf)))


def moe_r8_workspace(n_tok, n_embd, n_ff, n_expert, n_used, device):
    nbytes = _lib.moe_r8_workspace_bytes(n_tok, n_embd, n_ff, n_expert, n_used)
    if nbytes == 0:
        raise Q8Error("moe_r8_workspace_bytes", -4)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _r8_ffn_descs(layers, n_embd, n_ff, n_expert, with_ws):
    for d in layers:
        _need(d["w_up_gate_r8"], torch.uint8, "w_up_gate_r8")
        _need(d["w_down_r8"], torch.uint8, "w_down_r8")
        _need(d["x"], torch.float32, "x")
        _need(d["ids"], torch.int32, "ids")
        _need(d["cw"], torch.float32, "cw")
        _need(d["h"], torch.float32, "h")
        _need(d["out"], torch.float32, "out")
        if with_ws:
            _need(d["ws"], torch.uint8, "ws")
    n_tok, n_used = _ids_shape(layers[0]["ids"])
    for d in layers:
        _check_up_gate(d["w_up_gate_r8"], d["x"], d["ids"], d["h"], n_tok, n_used, n_embd, n_ff,
                       n_expert, r8=True)
        _check_down(d["w_down_r8"], d["h"], d["ids"], d["cw"], d["out"], n_tok, n_used, n_ff,
                    n_embd, n_expert, r8=True)
        _one_device(layers[0]["ids"], d["ids"], d["ws"] if with_ws else None)
    arr = (MoeR8FfnDesc * len(layers))(*[
        MoeR8FfnDesc(_ptr(d["w_up_gate_r8"]), _ptr(d["w_down_r8"]), _ptr(d["x"]), _ptr(d["ids"]),
                     _ptr(d["cw"]), _ptr(d["h"]), _ptr(d["out"]),
                     _ptr(d["ws"]) if with_ws else None, d["ws"].numel() if with_ws else 0)
        for d in layers])
    return arr, n_tok, n_used


def moe_r8_ffn_batched(layers, n_embd, n_ff, n_expert):
    """The expert FFN over R8 expert weights for independent layers of one
    shape (decode kernels up to 16 tokens, the grouped matrix-core path above).
    layers: list of dicts with w_up_gate_r8, w_down_r8, x, ids, cw, h
    (written), out (written), ws."""
    if not layers:
        return
    arr, n_tok, n_used = _r8_ffn_descs(layers, n_embd, n_ff, n_expert, True)
    _check("moe_r8_ffn_batched", _lib.moe_r8_ffn_batched(
        arr, len(layers), n_tok, n_embd, n_ff, n_expert, n_used, _stream(layers[0]["ids"])))


def moe_r8_ffn_batched_noalloc(layers, n_embd, n_ff, n_expert):
    """moe_r8_ffn_batched without a caller workspace (the library's own
    per-device array; decode shapes, up to 16 tokens).  layers: dicts as for
    moe_r8_ffn_batched; a "ws" entry, if present, is ignored."""
    if not layers:
        return
    arr, n_tok, n_used = _r8_ffn_descs(layers, n_embd, n_ff, n_expert, False)
    _check("moe_r8_ffn_batched_noalloc", _lib.moe_r8_ffn_batched_noalloc(
        arr, len(layers), n_tok, n_embd, n_ff, n_expert, n_used, _stream(layers[0]["ids"])))


def moe_r8_fused_workspace(n_embd, n_ff, n_expert, n_used, device):
    """A workspace for moe_r8_ffn_fused (zeroed: its counters must start at
    zero; every call leaves them zero)."""
    nbytes = _lib.moe_r8_fused_workspace_bytes(n_embd, n_ff, n_expert, n_used)
    if nbytes == 0:
        raise Q8Error("moe_r8_fused_workspace_bytes", -4)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def moe_r8_ffn_fused(layer, n_embd, n_ff, n_expert):
    """One token through one layer of the expert FFN over R8 weights in one
    launch.  layer: a dict as for moe_r8_ffn_batched (one token) whose ws comes
    from moe_r8_fused_workspace."""
    arr, n_tok, n_used = _r8_ffn_descs([layer], n_embd, n_ff, n_expert, True)
    if n_tok != 1:
        raise Q8Error("moe_r8_ffn_fused", -4)
    _check("moe_r8_ffn_fused", _lib.moe_r8_ffn_fused(arr, n_embd, n_ff, n_expert, n_used,
                                                     _stream(layer["ids"])))


def moe_error_word(ws):
    """The int32 error word at the start of a MoE workspace (1 = an id was out of range)."""
    return int(ws[:4].view(torch.int32).item())


# ---------------------------------------------------------------------------
# 8-bit products with one scale per token and per output channel, and log
# probabilities of logit rows.

_FLOATS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_INT8 = {torch.int8: 3}
_ACTS = {**_FLOATS, **_INT8}


def _rows(t, name, types):
    """(type, row stride, rows, columns) of a 2-D tensor whose rows are
    contiguous (where it lies: _on)."""
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: {t.dtype}, expected one of {[str(d) for d in types]}")
    try:
        rows, cols = t.shape
        stride, step = t.stride()
    except ValueError:
        raise ValueError(f"{name}: expected 2 dimensions, got shape {tuple(t.shape)}") from None
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return code, stride, rows, cols


def _vector(t, n, dtype, name):
    """Address of a contiguous tensor of n elements (where it lies: _on)."""
    if t.dtype is not dtype or not t.is_contiguous():
        _need(t, dtype, name)
    if t.numel() != n:
        raise ValueError(f"{name}: {t.numel()} elements, expected {n}")
    return t.data_ptr()


def _on(x, name, *ts):
    """The device of x, a GPU, where every other tensor of the call has to be."""
    device = x.device
    if not x.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    for t in ts:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on several devices: {device}, {t.device}")
    return device


# The device that is current and the handle of a device's current stream.
# (torch.cuda.current_stream() builds a Stream object at 2 us a call; these take
# 0.1.)  A call for another device makes it current and starts again.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def i8_quantize_rows(x, q=None, scale=None):
    """x: fp32, fp16 or bf16 [n_rows][k] (or [k]) -> (q int8 [n_rows][k],
    scale fp32 [n_rows]): codes by row with scale = max|x| / 127.  Rows may
    have a stride.  For a weight matrix [n][k], once at load, and for tokens
    whose codes serve several products."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    xt, xs, n_rows, k = _rows(x, "x", _FLOATS)
    if q is None:
        q = torch.empty((n_rows, k), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(n_rows, dtype=torch.float32, device=x.device)
    _, qs, q_rows, q_k = _rows(q, "q", _INT8)
    if (q_rows, q_k) != (n_rows, k):
        raise ValueError(f"q: shape {(q_rows, q_k)}, expected {(n_rows, k)}")
    scale_p = _vector(scale, n_rows, torch.float32, "scale")
    index = _on(x, "x", q, scale).index
    if index != _current_device():
        with torch.cuda.device(index):
            return i8_quantize_rows(x, q, scale)
    rc = _lib.i8_quantize_rows(x.data_ptr(), xt, xs, q.data_ptr(), qs, scale_p, n_rows, k,
                               _raw_stream(index))
    if rc != 0:
        raise Q8Error("i8_quantize_rows", rc)
    return q, scale


def i8_workspace_bytes(m, k):
    return int(_lib.i8_workspace_bytes(m, k))


def i8_workspace(m, k, device):
    """Workspace of a product whose m activation rows are not codes."""
    n = i8_workspace_bytes(m, k)
    if n == 0:
        raise Q8Error("i8_workspace_bytes", -4)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _i8_product(name, fn, x, w, w_scale, x_scale, bias, out, dtype, ws, gated, act=None, residual=None):
    xt, xs, m, k = _rows(x, "x", _ACTS)
    _, wst, n, wk = _rows(w, "w", _INT8)
    if wk != k:
        raise ValueError(f"w: rows of {wk} codes, x has {k}")
    w_scale_p = _vector(w_scale, n, torch.float32, "w_scale")
    x_scale_p = bias_p = ws_p = None
    ws_bytes = 0
    if xt == 3:
        if x_scale is None:
            raise ValueError("x_scale: needed with int8 codes")
        x_scale_p = _vector(x_scale, m, torch.float32, "x_scale")
    else:
        if x_scale is not None:
            raise ValueError("x_scale: given with rows that are not int8 codes")
        if ws is not None:
            ws_bytes = ws.numel()
            ws_p = _vector(ws, ws_bytes, torch.uint8, "ws")
    if gated:
        if n % 2:
            raise ValueError(f"w: {n} rows, expected gate and up rows of one number")
        n //= 2
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=x.device)
    yt, ys, y_rows, y_cols = _rows(out, "h" if gated else "y", _FLOATS)
    if y_rows != m or y_cols != n:
        raise ValueError(f"{'h' if gated else 'y'}: shape {(y_rows, y_cols)}, expected {(m, n)}")
    if bias is not None:
        bias_p = _vector(bias, n, torch.float32, "bias")
    rs, residual_p = 0, None
    if residual is not None:
        rt, rs, r_rows, r_cols = _rows(residual, "residual", _FLOATS)
        if rt != yt:
            raise TypeError(f"residual: {residual.dtype}, expected {out.dtype} as y")
        if r_rows != m or r_cols != n:
            raise ValueError(f"residual: shape {(r_rows, r_cols)}, expected {(m, n)}")
        residual_p = residual.data_ptr()
    index = _on(x, "x", w, w_scale, x_scale, bias, out, ws if ws_p else None, residual).index
    if index != _current_device():
        with torch.cuda.device(index):
            return _i8_product(name, fn, x, w, w_scale, x_scale, bias, out, dtype, ws, gated, act,
                               residual)
    if act is not None:
        rc = fn(x.data_ptr(), xt, xs, x_scale_p, w.data_ptr(), wst, w_scale_p, bias_p, act, residual_p,
                rs, out.data_ptr(), yt, ys, n, k, m, ws_p, ws_bytes, _raw_stream(index))
    elif gated:
        rc = fn(x.data_ptr(), xt, xs, x_scale_p, w.data_ptr(), wst, w_scale_p, out.data_ptr(), yt, ys,
                n, k, m, ws_p, ws_bytes, _raw_stream(index))
    else:
        rc = fn(x.data_ptr(), xt, xs, x_scale_p, w.data_ptr(), wst, w_scale_p, bias_p,
                out.data_ptr(), yt, ys, n, k, m, ws_p, ws_bytes, _raw_stream(index))
    if rc != 0:
        raise Q8Error(name, rc)
    return out


def i8_matmul(x, w, w_scale, x_scale=None, bias=None, y=None, dtype=torch.float32, ws=None):
    """y[t][j] = (sum_i x[t][i] w[j][i]) * x_scale[t] * w_scale[j] (+ bias[j]).
    x: int8 codes [m][k] with x_scale, or fp32 / fp16 / bf16 rows, quantized
    inside (ws: i8_workspace(m, k)); w: int8 [n][k]; w_scale, bias: fp32 [n].
    y: fp32, fp16 or bf16 [m][n] (made with `dtype` if not given)."""
    return _i8_product("i8_matmul", _lib.i8_matmul, x, w, w_scale, x_scale, bias, y, dtype, ws,
                       False)


_ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "gelu": 3, "gelu_tanh": 4, "silu": 5}


def i8_matmul_act(x, w, w_scale, x_scale=None, bias=None, act="none", residual=None, y=None,
                  dtype=None, ws=None):
    """y = act(i8_matmul(...)) + residual, with act one of "none", "relu",
    "relu2" (its square), "gelu", "gelu_tanh", "silu"; residual: rows of y's
    type [m][n], may be y itself (in place); y is made, if not given, with
    `dtype`, or of the residual's type, or fp32; the rest as for i8_matmul."""
    code = _ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act: {act!r}, expected one of {list(_ACTIVATIONS)}")
    if dtype is None:
        dtype = torch.float32 if residual is None else residual.dtype
    return _i8_product("i8_matmul_act", _lib.i8_matmul_act, x, w, w_scale, x_scale, bias, y, dtype, ws,
                       False, code, residual)


def i8_up_gate_swiglu(x, w, w_scale, x_scale=None, h=None, dtype=torch.float32, ws=None):
    """h[t][j] = silu(g) * u with g, u the products of rows j and n_ff + j of
    the combined weight w int8 [2*n_ff][k] (gate rows first); x, x_scale, ws
    as for i8_matmul; h: fp32, fp16 or bf16 [m][n_ff]."""
    return _i8_product("i8_up_gate_swiglu", _lib.i8_up_gate_swiglu, x, w, w_scale, x_scale, None, h,
                       dtype, ws, True)


class LogprobOut(NamedTuple):
    """Outputs of logprob_rows; top_ids and top_logprobs are None without
    alternatives, logprob without given tokens.  In an `out`, lse and entropy
    may be None where they are not wanted."""
    logprob: Optional[torch.Tensor]        # fp32 [m][n_given]
    lse: Optional[torch.Tensor]            # fp32 [m]
    entropy: Optional[torch.Tensor]        # fp32 [m]
    top_ids: Optional[torch.Tensor]        # int32 [m][n_top]
    top_logprobs: Optional[torch.Tensor]   # fp32 [m][n_top]


def logprob_outputs(m, n_given, n_top, device):
    """Output tensors for logprob_rows (its `out`)."""
    def new(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=device)
    return LogprobOut(new(m, n_given) if n_given else None, new(m), new(m),
                      new(m, n_top, dtype=torch.int32) if n_top else None,
                      new(m, n_top) if n_top else None)


def logprob_workspace_bytes(m, n_vocab, n_top):
    return int(_lib.logprob_workspace_bytes(m, n_vocab, n_top))


def logprob_workspace(m, n_vocab, n_top, device):
    """Workspace of logprob_rows for up to m rows (also of fewer logits and
    alternatives)."""
    n = logprob_workspace_bytes(m, n_vocab, n_top)
    if n == 0:
        raise Q8Error("logprob_workspace_bytes", -4)
    return torch.empty(n, dtype=torch.uint8, device=device)


def logprob_rows(logits, tokens=None, n_top=0, ws=None, out=None):
    """Log probabilities of the given tokens (int32 [m] or [m][n_given]), log
    sum exp, entropy and the n_top largest logits (ties to the lowest index)
    of each row of logits, fp32 / fp16 / bf16 [m][n_vocab].  ws:
    logprob_workspace of this many rows or more.  Returns a LogprobOut (`out` if
    given)."""
    t, stride, m, n_vocab = _rows(logits, "logits", _FLOATS)
    if n_top < 0:
        raise Q8Error("logprob_rows", -2)
    n_given = 0
    if tokens is not None:
        _need(tokens, torch.int32, "tokens")
        shape = tokens.shape
        if len(shape) not in (1, 2) or shape[0] != m:
            raise ValueError(f"tokens: shape {tuple(shape)}, expected [{m}] or [{m}][n_given]")
        n_given = 1 if len(shape) == 1 else shape[1]
    if out is None:
        out = logprob_outputs(m, n_given, n_top, logits.device)
    given_p = ids_p = top_p = ws_p = None
    ws_bytes = 0
    if (n_given and out.logprob is None) or (n_top and (out.top_ids is None or out.top_logprobs is None)):
        raise ValueError("out: lacks an output that this call has")
    if n_given:
        given_p = _vector(out.logprob, m * n_given, torch.float32, "logprob")
    lse_p = None if out.lse is None else _vector(out.lse, m, torch.float32, "lse")
    entropy_p = None if out.entropy is None else _vector(out.entropy, m, torch.float32, "entropy")
    if n_top:
        ids_p = _vector(out.top_ids, m * n_top, torch.int32, "top_ids")
        top_p = _vector(out.top_logprobs, m * n_top, torch.float32, "top_logprobs")
    if ws is not None:
        ws_bytes = ws.numel()
        ws_p = _vector(ws, ws_bytes, torch.uint8, "ws")
    index = _on(logits, "logits", tokens, ws, *out).index
    if index != _current_device():
        with torch.cuda.device(index):
            return logprob_rows(logits, tokens, n_top, ws, out)
    rc = _lib.logprob_rows(logits.data_ptr(), t, stride, None if tokens is None else tokens.data_ptr(),
                           n_given, given_p, lse_p, entropy_p, ids_p, top_p, m, n_vocab, n_top, ws_p,
                           ws_bytes, _raw_stream(index))
    if rc != 0:
        raise Q8Error("logprob_rows", rc)
    return out


# ---------------------------------------------------------------------------
# Around the products of a token step: embedding rows, norms with the residual
# stream, sampling.

def _embed_out(tokens, k, y, dtype, device):
    if tokens.dim() != 1:
        raise ValueError(f"tokens: shape {tuple(tokens.shape)}, expected [m]")
    m = tokens.shape[0]
    _vector(tokens, m, torch.int32, "tokens")
    if y is None:
        y = torch.empty((m, k), dtype=dtype, device=device)
    yt, ys, y_rows, y_cols = _rows(y, "y", _FLOATS)
    if y_rows != m or y_cols != k:
        raise ValueError(f"y: shape {(y_rows, y_cols)}, expected {(m, k)}")
    return y, yt, ys, m


def embed_rows(table, tokens, scale=1.0, table_scale=None, y=None, dtype=torch.float32):
    """y[t] = scale * table[tokens[t]]: table fp32, fp16, bf16 [n][k], or int8
    codes [n][k] with table_scale fp32 [n]; tokens int32 [m] (outside [0, n): a
    row of NaN); y: fp32, fp16 or bf16 [m][k] (made with `dtype` if not given)."""
    tt, ts, n, k = _rows(table, "table", _ACTS)
    scale_p = None
    if tt == 3:
        if table_scale is None:
            raise ValueError("table_scale: needed with int8 codes")
        scale_p = _vector(table_scale, n, torch.float32, "table_scale")
    elif table_scale is not None:
        raise ValueError("table_scale: given with a table that is not int8 codes")
    y, yt, ys, m = _embed_out(tokens, k, y, dtype, table.device)
    index = _on(table, "table", table_scale, tokens, y).index
    if index != _current_device():
        with torch.cuda.device(index):
            return embed_rows(table, tokens, scale, table_scale, y)
    rc = _lib.embed_rows(table.data_ptr(), tt, ts, scale_p, tokens.data_ptr(), scale, y.data_ptr(), yt,
                         ys, m, n, k, _raw_stream(index))
    if rc != 0:
        raise Q8Error("embed_rows", rc)
    return y


def q8_0_embed_rows(w, tokens, n, k, scale=1.0, r8=False, y=None, dtype=torch.float32):
    """y[t] = scale * row tokens[t] of n Q8_0 rows of k values, or of their R8
    layout (r8); tokens and y as for embed_rows."""
    if n > 0 and k > 0:
        _fit(w, q8_0_r8_bytes(n, k) if r8 else n * (k // QK) * BLOCK_BYTES, "w")
    y, yt, ys, m = _embed_out(tokens, k, y, dtype, w.device)
    index = _on(w, "w", tokens, y).index
    if index != _current_device():
        with torch.cuda.device(index):
            return q8_0_embed_rows(w, tokens, n, k, scale, r8, y)
    rc = _lib.q8_0_embed_rows(w.data_ptr(), bool(r8), tokens.data_ptr(), scale, y.data_ptr(), yt, ys, m,
                              n, k, _raw_stream(index))
    if rc != 0:
        raise Q8Error("q8_0_embed_rows", rc)
    return y


class NormOut(NamedTuple):
    """Outputs of norm_rows and residual_norm_rows."""
    y: torch.Tensor                        # float rows, or int8 codes
    y_scale: Optional[torch.Tensor]        # fp32 [m], of codes
    residual: Optional[torch.Tensor]       # the updated stream


def _norm_out(x, y, y_scale, dtype, m, n):
    if y is None:
        y = torch.empty((m, n), dtype=dtype, device=x.device)
    yt, ys, y_rows, y_cols = _rows(y, "y", _ACTS)
    if y_rows != m or y_cols != n:
        raise ValueError(f"y: shape {(y_rows, y_cols)}, expected {(m, n)}")
    if yt == 3:
        if y_scale is None:
            y_scale = torch.empty(m, dtype=torch.float32, device=x.device)
        return y, yt, ys, y_scale, _vector(y_scale, m, torch.float32, "y_scale")
    if y_scale is not None:
        raise ValueError("y_scale: given with a y that is not int8 codes")
    return y, yt, ys, None, None


def norm_rows(x, weight, bias=None, eps=1e-5, layer=False, y=None, y_scale=None, dtype=torch.float32):
    """y = norm(x) * weight (+ bias) of rows x, fp32 / fp16 / bf16 [m][n]: the root
    mean square norm, or with mean and variance (layer).  weight, bias: fp32
    [n].  y: fp32, fp16, bf16, or int8 codes with y_scale fp32 [m] (made with
    `dtype` if not given).  Returns a NormOut."""
    xt, xs, m, n = _rows(x, "x", _FLOATS)
    weight_p = _vector(weight, n, torch.float32, "weight")
    bias_p = None if bias is None else _vector(bias, n, torch.float32, "bias")
    y, yt, ys, y_scale, scale_p = _norm_out(x, y, y_scale, dtype, m, n)
    index = _on(x, "x", weight, bias, y, y_scale).index
    if index != _current_device():
        with torch.cuda.device(index):
            return norm_rows(x, weight, bias, eps, layer, y, y_scale)
    rc = _lib.norm_rows(x.data_ptr(), xt, xs, weight_p, bias_p, eps, layer, y.data_ptr(), yt, ys, scale_p,
                        m, n, _raw_stream(index))
    if rc != 0:
        raise Q8Error("norm_rows", rc)
    return NormOut(y, y_scale, None)


def residual_norm_rows(x, residual, weight, bias=None, post_weight=None, post_bias=None, gate=None,
                       residual_scale=1.0, eps=1e-5, layer=False, residual_out=None, y=None,
                       y_scale=None, dtype=torch.float32):
    """A block's output x into the residual stream, and the next norm:
    residual_out = gate * x + residual_scale * residual (x normed with
    post_weight and post_bias first, if given), y = norm(residual_out) * weight
    (+ bias).  x, residual: float rows [m][n], each of its own type;
    residual_out: of residual's type, may be residual itself; gate: float [n] or
    [m][n]; the rest as for norm_rows.  Returns a NormOut."""
    d = ResidualNormDesc()
    d.x_type, d.x_row_stride, m, n = _rows(x, "x", _FLOATS)
    d.x = x.data_ptr()
    if residual_out is None:
        residual_out = torch.empty((m, n), dtype=residual.dtype, device=x.device)
    for t, name in ((residual, "residual"), (residual_out, "residual_out")):
        rt, rs, rows, cols = _rows(t, name, _FLOATS)
        if rows != m or cols != n:
            raise ValueError(f"{name}: shape {(rows, cols)}, expected {(m, n)}")
        if t is residual:
            d.residual_type, d.residual_row_stride = rt, rs
        elif rt != d.residual_type:
            raise TypeError(f"residual_out: {t.dtype}, expected {residual.dtype} as residual")
        else:
            d.residual_out_row_stride = rs
    if residual_out is residual:
        d.residual_out_row_stride = d.residual_row_stride
    d.residual, d.residual_out = residual.data_ptr(), residual_out.data_ptr()
    if gate is not None:
        if gate.dim() == 1:
            d.gate_type = _FLOATS.get(gate.dtype, -1)
            if d.gate_type < 0:
                raise TypeError(f"gate: {gate.dtype}, expected a float type")
            d.gate = _vector(gate, n, gate.dtype, "gate")
        else:
            d.gate_type, d.gate_row_stride, rows, cols = _rows(gate, "gate", _FLOATS)
            if rows != m or cols != n:
                raise ValueError(f"gate: shape {(rows, cols)}, expected {(n,)} or {(m, n)}")
            d.gate = gate.data_ptr()
    if post_weight is not None:
        d.post_weight = _vector(post_weight, n, torch.float32, "post_weight")
    if post_bias is not None:
        if post_weight is None:
            raise ValueError("post_bias: given without post_weight")
        d.post_bias = _vector(post_bias, n, torch.float32, "post_bias")
    d.weight = _vector(weight, n, torch.float32, "weight")
    if bias is not None:
        d.bias = _vector(bias, n, torch.float32, "bias")
    y, d.y_type, d.y_row_stride, y_scale, d.y_scale = _norm_out(x, y, y_scale, dtype, m, n)
    d.y = y.data_ptr()
    d.residual_scale, d.eps, d.layer = residual_scale, eps, layer
    index = _on(x, "x", residual, residual_out, gate, post_weight, post_bias, weight, bias, y,
                y_scale).index
    if index != _current_device():
        with torch.cuda.device(index):
            return residual_norm_rows(x, residual, weight, bias, post_weight, post_bias, gate,
                                      residual_scale, eps, layer, residual_out, y, y_scale)
    rc = _lib.residual_norm_rows(d, m, n, _raw_stream(index))
    if rc != 0:
        raise Q8Error("residual_norm_rows", rc)
    return NormOut(y, y_scale, residual_out)


class SampleOut(NamedTuple):
    """Outputs of sample_rows."""
    ids: torch.Tensor                      # int32 [m], -1 for a row that is no distribution
    logprob: torch.Tensor                  # fp32 [m], of the token among what is kept
    kept: torch.Tensor                     # int32 [m]


def sample_outputs(m, device):
    """Output tensors for sample_rows (its `out`)."""
    return SampleOut(torch.empty(m, dtype=torch.int32, device=device),
                     torch.empty(m, dtype=torch.float32, device=device),
                     torch.empty(m, dtype=torch.int32, device=device))


def sample_workspace_bytes(m, n_vocab):
    return int(_lib.sample_workspace_bytes(m, n_vocab))


def sample_workspace(m, n_vocab, device):
    """Workspace of sample_rows for up to m rows of up to n_vocab logits."""
    n = sample_workspace_bytes(m, n_vocab)
    if n == 0:
        raise Q8Error("sample_workspace_bytes", -4)
    return torch.empty(n, dtype=torch.uint8, device=device)


def sample_rows(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, ws=None, out=None):
    """A token per row of logits, fp32 / fp16 / bf16 [m][n_vocab], from random
    numbers u fp32 [m] in [0, 1), after temperature, top-k, top-p and min-p
    (fp32 [m], top_k int32 [m], each may be None; temperature 0: the largest
    logit).  ws: sample_workspace of this many rows and logits or more.
    Returns a SampleOut (`out` if given)."""
    t, stride, m, n_vocab = _rows(logits, "logits", _FLOATS)
    u_p = _vector(u, m, torch.float32, "u")
    temp_p = None if temperature is None else _vector(temperature, m, torch.float32, "temperature")
    k_p = None if top_k is None else _vector(top_k, m, torch.int32, "top_k")
    p_p = None if top_p is None else _vector(top_p, m, torch.float32, "top_p")
    min_pp = None if min_p is None else _vector(min_p, m, torch.float32, "min_p")
    if out is None:
        out = sample_outputs(m, logits.device)
    ids_p = _vector(out.ids, m, torch.int32, "ids")
    logprob_p = _vector(out.logprob, m, torch.float32, "logprob")
    kept_p = _vector(out.kept, m, torch.int32, "kept")
    ws_p, ws_bytes = None, 0
    if ws is not None:
        ws_bytes = ws.numel()
        ws_p = _vector(ws, ws_bytes, torch.uint8, "ws")
    index = _on(logits, "logits", u, temperature, top_k, top_p, min_p, ws, *out).index
    if index != _current_device():
        with torch.cuda.device(index):
            return sample_rows(logits, u, temperature, top_k, top_p, min_p, ws, out)
    rc = _lib.sample_rows(logits.data_ptr(), t, stride, u_p, temp_p, k_p, p_p, min_pp, ids_p, logprob_p,
                          kept_p, m, n_vocab, ws_p, ws_bytes, _raw_stream(index))
    if rc != 0:
        raise Q8Error("sample_rows", rc)
    return out


# Raw access for tests of the argument checks (no tensors needed).
raw = _lib
