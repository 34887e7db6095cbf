"""Python binding of libbsmm.so, the block-scaled low-precision GEMM library.

Argument marshalling only: every function here checks what the library
cannot see through raw pointers (each tensor's shape, element type and size,
and that all are contiguous CUDA tensors on the current device), allocates
its outputs with torch (device memory is the caller's, as the C ABI
requires), passes raw device pointers and the current torch stream to the C
entry point of the same name, and raises :class:`BsmmError` on a non-zero
status.  Everything else (divisibility, formats, alignment, workspace size)
is the library's to check.  All computation happens in the
library's CUDA kernels; there is no CPU path.  The library is loaded on first
use and its absence is an error.

Entry points (see ``include/bsmm.h`` for the full contract):

* :func:`quantize`        absmax block quantizer (E4M3/E5M2/E2M1/INT8 codes,
                          FP32/UE8M0/UE4M3 scales, optional transposed output)
* :func:`gemm`            batched block-scaled GEMM, MXFP8 or NVFP4
* :func:`gemm_grouped`    FP8 GEMM with 1x128 / 128x128 FP32 scales
* :func:`int8_channel`    INT8 per-channel matmul with exact INT32 sums
* :func:`linear_backward` MXFP8 dX / dW of a linear layer
* :func:`gated_act`, :func:`gated_act_backward`  act(gate) * up, its inputs
                          kept for the backward pass in 8 bits
* :func:`linear_backward_checkpoint`  :func:`linear_backward` from an 8-bit X
* :func:`adapters`, :func:`adapters_backward`  low-rank adapters of many
                          requests beside a shared projection
* :func:`route`, :func:`expert_gemm`, :func:`expert_combine` and their
                          backward calls: a mixture of MXFP8 experts
* :func:`adamw`           AdamW over many tensors, states in 32 or 8 bits
"""

from __future__ import annotations

import ctypes
import functools
import os
from array import array

import torch

__all__ = [
    "BsmmError", "lib", "library_path", "quantize", "quantize_batch", "gemm", "gemm_noalloc", "gemm_grouped", "int8_channel",
    "linear_backward", "gemm_workspace_size", "int8_channel_workspace_size",
    "linear_backward_workspace_size", "check_device_status", "selftest_wait_timeout", "selftest_quotient", "trace",
    "scale_atoms_size", "quantize_atoms", "gemm_atoms", "linear_backward_quantized",
    "gated_act", "gated_act_backward", "linear_backward_checkpoint", "adapters", "adapters_backward",
    "adapters_workspace_size", "adapters_backward_workspace_size",
    "route", "route_backward", "expert_gemm", "expert_backward", "expert_combine", "expert_combine_backward", "adamw",
    "route_workspace_size", "expert_gemm_workspace_size", "expert_backward_workspace_size",
    "set_wait_timeout_ns", "version",
    "F32", "BF16", "E4M3", "E5M2", "E2M1", "INT8", "SCALE_F32", "SCALE_UE8M0", "SCALE_UE4M3",
]

# bsmm_status
OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGNMENT, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(8)
STATUS_NAMES = ["OK", "INVALID_ARG", "SHAPE", "ALIGNMENT", "UNSUPPORTED", "CUDA", "TIMEOUT", "WORKSPACE"]
# bsmm_dtype
F32, BF16, E4M3, E5M2, E2M1, INT8 = range(6)
# bsmm_scale_type
SCALE_F32, SCALE_UE8M0, SCALE_UE4M3 = range(3)

# bsmm_act
SILU, GELU = range(2)

_ACT_NAMES = {"silu": SILU, "gelu": GELU}
_CODE_NAMES = {"e4m3": E4M3, "e5m2": E5M2, "e2m1": E2M1, "int8": INT8}
_SCALE_NAMES = {"f32": SCALE_F32, "ue8m0": SCALE_UE8M0, "ue4m3": SCALE_UE4M3}

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbsmm.so")
_LIB = None


class BsmmError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{where}: BSMM_ERR_{name}: {msg}")


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_SZ = ctypes.c_size_t
_F64 = ctypes.c_double


class _QuantizeJob(ctypes.Structure):
    """bsmm_quantize_job (include/bsmm.h)."""
    _fields_ = [("x", _P), ("x_type", _INT), ("rows", _I64), ("cols", _I64), ("ld_x", _I64),
                ("block_rows", _INT), ("block_cols", _INT), ("code_type", _INT), ("scale_type", _INT),
                ("transpose_out", _INT), ("codes", _P), ("ld_codes", _I64), ("scales", _P), ("ld_scales", _I64)]


_SIGS = {
    "bsmm_version": ([], _INT),
    "bsmm_last_error": ([], ctypes.c_char_p),
    "bsmm_set_wait_timeout_ns": ([ctypes.c_uint64], None),
    "bsmm_check_device_status": ([_P, ctypes.POINTER(_INT)], _INT),
    "bsmm_selftest_wait_timeout": ([ctypes.c_uint64, _P], _INT),
    "bsmm_selftest_quotient": ([ctypes.c_uint64, ctypes.c_uint64, _P, _P], _INT),
    "bsmm_trace_start": ([], _INT),
    "bsmm_trace_stop": ([], _INT),
    "bsmm_trace_count": ([], _INT),
    "bsmm_trace_read": ([_INT, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float),
                         ctypes.POINTER(ctypes.c_float)], _INT),
    "bsmm_quantize": ([_P, _INT, _I64, _I64, _I64, _INT, _INT, _INT, _INT, _INT, _P, _I64, _P, _I64, _P], _INT),
    "bsmm_quantize_batch": ([ctypes.POINTER(_QuantizeJob), _INT, _P], _INT),
    "bsmm_gemm_workspace_size": ([_I64, _I64, _I64, _I64, _INT], _SZ),
    "bsmm_gemm": ([_I64, _I64, _I64, _I64, _P, _INT, _P, _INT, _P, _I64, _P, _I64, _INT, _P, _INT, _P, _SZ, _P],
                  _INT),
    "bsmm_gemm_noalloc": ([_I64, _I64, _I64, _I64, _P, _INT, _P, _INT, _P, _I64, _P, _I64, _INT, _P, _INT, _P],
                          _INT),
    "bsmm_gemm_grouped": ([_I64, _I64, _I64, _P, _INT, _P, _INT, _P, _P, _INT, _INT, _P, _P], _INT),
    "bsmm_int8_channel_workspace_size": ([_I64, _I64, _I64], _SZ),
    "bsmm_int8_channel": ([_P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _INT),
    "bsmm_linear_backward_workspace_size": ([_I64, _I64, _I64], _SZ),
    "bsmm_linear_backward": ([_P, _P, _P, _I64, _I64, _I64, _INT, _P, _P, _P, _SZ, _P], _INT),
    "bsmm_scale_atoms_size": ([_I64, _I64, _I64, _INT, _INT], _SZ),
    "bsmm_quantize_atoms": ([_P, _INT, _I64, _I64, _I64, _INT, _INT, _INT, _P, _P, _SZ, _P], _INT),
    "bsmm_gemm_atoms": ([_I64, _I64, _I64, _I64, _P, _INT, _P, _INT, _P, _P, _INT, _P, _INT, _P, _SZ, _P], _INT),
    "bsmm_linear_backward_quantized_workspace_size": ([_I64, _I64, _I64, _INT], _SZ),
    "bsmm_linear_backward_quantized": ([_I64, _I64, _I64, _INT, _P, _P, _P, _P, _P, _P, _P, _P, _INT, _P, _P, _P,
                                        _SZ, _P], _INT),
    "bsmm_gated_act": ([_P, _INT, _I64, _I64, _I64, _INT, _INT, _P, _P, _INT, _INT, _INT, _P, _P, _P], _INT),
    "bsmm_gated_act_backward": ([_P, _INT, _I64, _I64, _INT, _P, _INT, _P, _INT, _P, _P, _P], _INT),
    "bsmm_linear_backward_checkpoint": ([_P, _P, _P, _INT, _P, _INT, _I64, _I64, _I64, _INT, _P, _P, _P, _SZ, _P],
                                        _INT),
    "bsmm_adapters_workspace_size": ([_I64, _I64, _I64], _SZ),
    "bsmm_adapters": ([_I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, _P, _I64, _INT, _P, _P, _SZ,
                       _P], _INT),
    "bsmm_adapters_backward_workspace_size": ([_I64, _I64, _I64], _SZ),
    "bsmm_adapters_backward": ([_I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _I64, _INT, _P, _P, _P, _P, _P, _P, _P,
                                _I64, _P, _P, _P, _INT, _P, _SZ, _P], _INT),
    "bsmm_route_workspace_size": ([_I64, _I64], _SZ),
    "bsmm_route": ([_I64, _I64, _INT, _P, _INT, _I64, _INT, _P, _P, _P, _P, _P, _P, _SZ, _P], _INT),
    "bsmm_route_backward": ([_I64, _I64, _INT, _P, _INT, _I64, _INT, _P, _P, _P, _P, _P], _INT),
    "bsmm_expert_gemm_workspace_size": ([_I64, _I64, _I64, _INT], _SZ),
    "bsmm_expert_gemm": ([_I64, _I64, _I64, _I64, _I64, _P, _INT, _P, _P, _INT, _P, _P, _P, _P, _P, _SZ, _P], _INT),
    "bsmm_expert_backward_workspace_size": ([_I64, _I64, _I64, _I64], _SZ),
    "bsmm_expert_backward": ([_I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _INT, _P, _P, _P, _SZ, _P], _INT),
    "bsmm_expert_combine": ([_I64, _I64, _INT, _I64, _P, _P, _P, _P, _INT, _P], _INT),
    "bsmm_expert_combine_backward": ([_I64, _I64, _INT, _I64, _P, _INT, _P, _P, _P, _P, _P, _P], _INT),
    "bsmm_adamw": ([_I64, _P, _P, _INT, _P, _INT, _P, _P, _INT, _P, _P, _P, _F64, _F64, _F64, _F64, _F64, _I64, _F64, _P,
                    _P], _INT),
}


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(library_path):
            raise RuntimeError(f"{library_path} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        h = ctypes.CDLL(library_path)
        for name, (args, res) in _SIGS.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = res
        _LIB = h
    return _LIB


def _check(status: int, where: str) -> None:
    if status != OK:
        raise BsmmError(status, where, lib().bsmm_last_error().decode())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_FLOATS = (torch.float32, torch.bfloat16)


def _want(t, name: str, shape=None, dtypes=None, itemsize=None, min_bytes=None) -> torch.Tensor:
    """Checks a tensor argument's shape, dtype and size before its pointer is
    passed on: the library sees raw pointers only, so a buffer that is too
    small, or of another element type, would be read or written out of
    bounds on the device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if itemsize is not None and t.element_size() != itemsize:
        raise ValueError(f"{name} must have {itemsize}-byte elements, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(int(s) for s in shape):
        raise ValueError(f"{name} must have shape {tuple(int(s) for s in shape)}, got {tuple(t.shape)}")
    if min_bytes is not None and t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, {min_bytes} needed")
    return t


def _on_device(**named) -> torch.device:
    """All tensor arguments are contiguous CUDA tensors on the current device
    (the library launches on the current device); returns that device."""
    dev = None
    for name, t in named.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other arguments on {dev}")
    if dev is not None and dev.index != torch.cuda.current_device():
        raise ValueError(f"the arguments are on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _empty(shape, dtype, dev, stream):
    """An output of a call on `stream`.  It comes from that stream's own pool:
    memory of the current stream's may still be in use there by earlier work,
    which nothing makes `stream` wait for.  The caller goes on with it on the
    current stream, so the allocator is told of that one too."""
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(dev.index):
        return torch.empty(shape, dtype=dtype, device=dev)
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=dev)
    if t.numel():
        t.record_stream(here)
    return t


def _scratch(nbytes, dev, stream):
    """A workspace, from the pool of the one stream that uses it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _lists():
    """The compiled part of the binding."""
    global _LISTS
    if _LISTS is None:
        try:
            from . import _tensor_lists
        except ImportError as e:
            raise RuntimeError("_tensor_lists.so cannot be loaded: build it for this torch and Python first "
                               f"(python -c 'import __graft_entry__ as g; g.build()'): {e}") from e
        _LISTS = _tensor_lists
    return _LISTS


_LISTS = None


def _match(pattern, *tensors):
    """The tensors' addresses and sizes, where they fit the pattern
    (tensor_lists.cpp) on the current device; else None, and the caller's own
    checks say what is wrong.  A tenth of the time of those."""
    first = tensors[0]
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        return None
    return _lists().match(pattern, torch._C._cuda_getDevice(), *tensors)


def _empties(dev, stream, *specs):
    """Several outputs, ``specs`` being type, shape, type, shape, ...: in one call
    where they come from the current stream's pool (see :func:`_empty`)."""
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(dev.index):
        return _lists().empties(dev.index, *specs)
    return [_empty(shape, dtype, dev, stream) for dtype, shape in zip(specs[::2], specs[1::2])]


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _code(c) -> int:
    return _CODE_NAMES[c] if isinstance(c, str) else int(c)


def _scale(s) -> int:
    return _SCALE_NAMES[s] if isinstance(s, str) else int(s)


def version() -> int:
    return lib().bsmm_version()


def set_wait_timeout_ns(ns: int) -> None:
    lib().bsmm_set_wait_timeout_ns(int(ns))


def check_device_status(stream=None):
    """Synchronizes the stream; returns (status, site) of the device status word."""
    where = ctypes.c_int(0)
    st = lib().bsmm_check_device_status(_stream(stream), ctypes.byref(where))
    return st, where.value


def selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(lib().bsmm_selftest_wait_timeout(int(timeout_ns), _stream(stream)), "bsmm_selftest_wait_timeout")


# --------------------------------------------------------------------------- #
# quantize                                                                    #
# --------------------------------------------------------------------------- #

def selftest_quotient(pairs: int, seed: int = 0, device=None) -> int:
    """Pairs on which the quantizers' block quotient disagrees with the
    hardware division (bsmm_selftest_quotient); 0 is the expected answer."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    bad = torch.zeros(1, dtype=torch.int64, device=dev)
    with torch.cuda.device(dev):
        _check(lib().bsmm_selftest_quotient(int(pairs), int(seed) & (2**64 - 1), _ptr(bad), _stream(None)),
               "bsmm_selftest_quotient")
        return int(bad.item())


class trace:
    """Per-kernel timing of everything the library launches inside the block
    (bsmm_trace_*): ``with trace() as launches: ...`` leaves in ``launches``
    one ``(kernel, start_ms, ms)`` per launch, in launch order, start
    relative to the first launch.  Reading them waits for those kernels."""

    def __enter__(self):
        self.launches = []
        _check(lib().bsmm_trace_start(), "bsmm_trace_start")
        return self.launches

    def __exit__(self, exc_type, exc, tb):
        L = lib()
        L.bsmm_trace_stop()
        if exc_type is not None:  # leave the records unread; the block's exception propagates
            return False
        for i in range(L.bsmm_trace_count()):
            name, t0, ms = ctypes.c_char_p(), ctypes.c_float(), ctypes.c_float()
            _check(L.bsmm_trace_read(i, ctypes.byref(name), ctypes.byref(t0), ctypes.byref(ms)), "bsmm_trace_read")
            self.launches.append((name.value.decode(), t0.value, ms.value))
        return False


def _quantize_job(x, block, code, scale, transpose, codes, scales, stream):
    """Checked arguments of one quantization, its outputs (allocated where
    not given) and the C job that describes it."""
    _want(x, "x", dtypes=_FLOATS)
    if x.dim() != 2:
        raise ValueError("x must be a 2-D float32 or bfloat16 tensor")
    br, bc = int(block[0]), int(block[1])
    c, s = _code(code), _scale(scale)
    rows, cols = x.shape
    orows, ocols = (cols, rows) if transpose else (rows, cols)
    srows, scols = ((cols // bc, rows // br) if transpose else (rows // br, cols // bc)) if br > 0 and bc > 0 else (0, 0)
    width = ocols // 2 if c == E2M1 else ocols
    scale_dtype = torch.float32 if s == SCALE_F32 else torch.uint8
    if codes is not None:
        _want(codes, "codes", (orows, width), itemsize=1)
    if scales is not None:
        _want(scales, "scales", (srows, scols), itemsize=scale_dtype.itemsize)
    dev = _on_device(x=x, codes=codes, scales=scales)
    if codes is None:
        codes = _empty((orows, width), torch.int8 if c == INT8 else torch.uint8, dev, stream)
    if scales is None:
        scales = _empty((srows, scols), scale_dtype, dev, stream)
    job = _QuantizeJob(_ptr(x), BF16 if x.dtype == torch.bfloat16 else F32, rows, cols, cols, br, bc, c, s,
                       1 if transpose else 0, _ptr(codes), ocols, _ptr(scales), scols)
    return job, codes, scales


def quantize(x: torch.Tensor, block, code="e4m3", scale="f32", transpose=False, codes=None, scales=None,
             stream=None):
    """Block-quantize a 2-D float32/bfloat16 CUDA tensor.

    Returns ``(codes, scales)``: codes uint8 (int8 for INT8; E2M1 packed two
    per byte) of shape [rows, cols] (or [cols, rows] transposed), scales
    float32 or uint8 of shape [rows/br, cols/bc] (or transposed)."""
    j, codes, scales = _quantize_job(x, block, code, scale, transpose, codes, scales, stream)
    _check(lib().bsmm_quantize(j.x, j.x_type, j.rows, j.cols, j.ld_x, j.block_rows, j.block_cols, j.code_type,
                               j.scale_type, j.transpose_out, j.codes, j.ld_codes, j.scales, j.ld_scales,
                               _stream(stream)), "bsmm_quantize")
    return codes, scales


def quantize_batch(jobs, stream=None):
    """Several independent quantizations in one call (bsmm_quantize_batch).

    ``jobs`` is a list of dicts with the arguments of :func:`quantize`
    (``x`` and ``block`` required; ``code``, ``scale``, ``transpose``,
    ``codes``, ``scales`` optional).  Returns the ``(codes, scales)`` pairs in
    job order."""
    prepared = [_quantize_job(j["x"], j["block"], j.get("code", "e4m3"), j.get("scale", "f32"),
                              j.get("transpose", False), j.get("codes"), j.get("scales"), stream) for j in jobs]
    arr = (_QuantizeJob * max(len(prepared), 1))(*[p[0] for p in prepared])
    _check(lib().bsmm_quantize_batch(arr, len(prepared), _stream(stream)), "bsmm_quantize_batch")
    return [(p[1], p[2]) for p in prepared]


# --------------------------------------------------------------------------- #
# GEMMs                                                                       #
# --------------------------------------------------------------------------- #

def gemm_workspace_size(B, M, N, K, a_type) -> int:
    return lib().bsmm_gemm_workspace_size(B, M, N, K, _code(a_type))


def gemm(a, b, a_scales, b_scales, a_type="e4m3", b_type="e4m3", scale="ue8m0", out_dtype=torch.float32, y=None,
         workspace=None, K=None, stream=None):
    """Batched block-scaled GEMM ``(B,M,K) x (B,N,K) -> (B,M,N)``.

    ``a``/``b`` hold codes (uint8 or float8 tensors; E2M1 packed, so their last
    dimension is K/2 and ``K`` is inferred as twice it), ``a_scales``
    (B,M,K_a) / ``b_scales`` (B,N,K_b) hold scale bytes."""
    at, bt = _code(a_type), _code(b_type)
    a, b, a_scales, b_scales, Bn, M, N, K = _gemm_operands(a, b, a_scales, b_scales, at, bt, K)
    if y is not None:
        _want(y, "y", (Bn, M, N), dtypes=_FLOATS)
    if workspace is not None:
        _want(workspace, "workspace")
    dev = _on_device(a=a, b=b, a_scales=a_scales, b_scales=b_scales, y=y, workspace=workspace)
    if y is None:
        y = _empty((Bn, M, N), out_dtype, dev, stream)
    if workspace is None:
        workspace = _scratch(max(gemm_workspace_size(Bn, M, N, K, at), 1), dev, stream)
    _check(lib().bsmm_gemm(Bn, M, N, K, _ptr(a), at, _ptr(b), bt, _ptr(a_scales), a_scales.shape[-1],
                           _ptr(b_scales), b_scales.shape[-1], _scale(scale), _ptr(y),
                           BF16 if y.dtype == torch.bfloat16 else F32, _ptr(workspace), _nbytes(workspace),
                           _stream(stream)), "bsmm_gemm")
    return y


def _code_bytes(t: int, K: int) -> int:
    """Bytes of K codes of type t in a row (E2M1 packs two per byte)."""
    return K // 2 if t == E2M1 else K


def _gemm_operands(a, b, a_scales, b_scales, at, bt, K):
    """Batched GEMM operands: codes (B,M,K) and (B,N,K) bytes (E2M1: K/2),
    scales (B,M,K_a) and (B,N,K_b) bytes; 2-D operands are one batch."""
    for t, n in ((a, "a"), (b, "b")):
        _want(t, n, itemsize=1)
    if a.dim() == 2 and b.dim() == 2:
        a, b = a[None], b[None]
        a_scales = a_scales[None] if a_scales is not None and a_scales.dim() == 2 else a_scales
        b_scales = b_scales[None] if b_scales is not None and b_scales.dim() == 2 else b_scales
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b must be (B, M, K) and (B, N, K) code tensors")
    Bn, M, ka = a.shape
    N = b.shape[1]
    if K is None:
        K = ka * 2 if at == E2M1 else ka
    _want(a, "a", (Bn, M, _code_bytes(at, K)))
    _want(b, "b", (Bn, N, _code_bytes(bt, K)))
    if a_scales is not None:  # row-major scales (the atom entry points pass None)
        for t, n, rows in ((a_scales, "a_scales", M), (b_scales, "b_scales", N)):
            _want(t, n, itemsize=1)
            if t.dim() != 3:
                raise ValueError(f"{n} must be (B, rows, K / block)")
            _want(t, n, (Bn, rows, t.shape[-1]))
    return a, b, a_scales, b_scales, Bn, M, N, K


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def gemm_noalloc(a, b, a_scales, b_scales, a_type="e4m3", b_type="e4m3", scale="ue8m0", y=None, K=None,
                 stream=None):
    """:func:`gemm` through the entry point that allocates nothing: its
    scratch is a static device array of NOALLOC_SCRATCH_BYTES inside the
    library (for callers that cannot allocate device memory).  ``y`` must be
    given; this wrapper allocates nothing either."""
    at, bt = _code(a_type), _code(b_type)
    a, b, a_scales, b_scales, Bn, M, N, K = _gemm_operands(a, b, a_scales, b_scales, at, bt, K)
    if y is None:
        raise ValueError("gemm_noalloc needs y")
    _want(y, "y", (Bn, M, N), dtypes=_FLOATS)
    _on_device(a=a, b=b, a_scales=a_scales, b_scales=b_scales, y=y)
    _check(lib().bsmm_gemm_noalloc(Bn, M, N, K, _ptr(a), at, _ptr(b), bt, _ptr(a_scales), a_scales.shape[-1],
                                   _ptr(b_scales), b_scales.shape[-1], _scale(scale), _ptr(y),
                                   BF16 if y.dtype == torch.bfloat16 else F32, _stream(stream)),
           "bsmm_gemm_noalloc")
    return y


def gemm_grouped(a, b, a_scales, b_scales, group_n=128, group_k=128, a_type="e4m3", b_type="e4m3", y=None,
                 stream=None):
    """``y[m,n] = sum_kb a_scales[m,kb] * b_scales[n//group_n,kb] * (a.b over block kb)``."""
    for t, n in ((a, "a"), (b, "b")):
        _want(t, n, itemsize=1)
        if t.dim() != 2:
            raise ValueError(f"{n} must be a 2-D code tensor")
    M, K = a.shape
    N = b.shape[0]
    _want(b, "b", (N, K))
    for t, n in ((a_scales, "a_scales"), (b_scales, "b_scales")):
        _want(t, n, dtypes=(torch.float32,))
    # an empty output reads no scales; indivisible groups: the library says why
    if M and N and group_n > 0 and group_k > 0 and N % group_n == 0 and K % group_k == 0:
        _want(a_scales, "a_scales", (M, K // group_k))
        _want(b_scales, "b_scales", (N // group_n, K // group_k))
    if y is not None:
        _want(y, "y", (M, N), dtypes=(torch.float32,))
    dev = _on_device(a=a, b=b, a_scales=a_scales, b_scales=b_scales, y=y)
    if y is None:
        y = _empty((M, N), torch.float32, dev, stream)
    _check(lib().bsmm_gemm_grouped(M, N, K, _ptr(a), _code(a_type), _ptr(b), _code(b_type), _ptr(a_scales),
                                   _ptr(b_scales), group_n, group_k, _ptr(y), _stream(stream)),
           "bsmm_gemm_grouped")
    return y


def int8_channel_workspace_size(B, D_in, D_out) -> int:
    return lib().bsmm_int8_channel_workspace_size(B, D_in, D_out)


def int8_channel(x, w, return_acc=False, out=None, workspace=None, stream=None) -> dict:
    """INT8 per-channel matmul; returns the dict of the page (w_q, w_scales,
    x_q, x_scales, y) plus ``acc`` (int32 sums) when ``return_acc``."""
    for t, n in ((x, "x"), (w, "w")):
        _want(t, n, dtypes=(torch.float32,))
        if t.dim() != 2:
            raise ValueError(f"{n} must be a 2-D float32 tensor")
    Bn, D_in = x.shape
    D_out = w.shape[1]
    _want(w, "w", (D_in, D_out))
    want = {"x_q": ((Bn, D_in), (torch.int8,)), "x_scales": ((Bn,), (torch.float32,)),
            "w_q": ((D_in, D_out), (torch.int8,)), "w_scales": ((D_out,), (torch.float32,)),
            "y": ((Bn, D_out), (torch.float32,)), "acc": ((Bn, D_out), (torch.int32,))}
    o = dict(out) if out else {}
    for k, t in o.items():
        if k not in want:
            raise ValueError(f"out has an unknown key {k!r}")
        _want(t, f"out[{k!r}]", *want[k])
    if workspace is not None:
        _want(workspace, "workspace")
    dev = _on_device(x=x, w=w, workspace=workspace, **{f"out_{k}": t for k, t in o.items()})
    for k in ("x_q", "x_scales", "w_q", "w_scales", "y") + (("acc",) if return_acc else ()):
        if k not in o:
            o[k] = _empty(want[k][0], want[k][1][0], dev, stream)
    if workspace is None:
        workspace = _scratch(max(int8_channel_workspace_size(Bn, D_in, D_out), 1), dev, stream)
    _check(lib().bsmm_int8_channel(_ptr(x), _ptr(w), Bn, D_in, D_out, _ptr(o["x_q"]), _ptr(o["x_scales"]),
                                   _ptr(o["w_q"]), _ptr(o["w_scales"]), _ptr(o["y"]), _ptr(o.get("acc")),
                                   _ptr(workspace), _nbytes(workspace), _stream(stream)), "bsmm_int8_channel")
    if out is not None:  # the caller's dict gets the outputs allocated here too
        out.update(o)
        return out
    return o


def linear_backward_workspace_size(M, N, K) -> int:
    return lib().bsmm_linear_backward_workspace_size(M, N, K)


def linear_backward(dY, W, X, fp8="e5m2", dX=None, dW=None, workspace=None, stream=None):
    """MXFP8 backward of ``Y = X @ W^T``: returns ``(dX, dW)`` in bfloat16."""
    bf16 = (torch.bfloat16,)
    for t, n in ((dY, "dY"), (W, "W"), (X, "X")):
        _want(t, n, dtypes=bf16)
        if t.dim() != 2:
            raise ValueError(f"{n} must be a 2-D bfloat16 tensor")
    M, N = dY.shape
    K = W.shape[1]
    _want(W, "W", (N, K))
    _want(X, "X", (M, K))
    if dX is not None:
        _want(dX, "dX", (M, K), dtypes=bf16)
    if dW is not None:
        _want(dW, "dW", (N, K), dtypes=bf16)
    if workspace is not None:
        _want(workspace, "workspace")
    dev = _on_device(dY=dY, W=W, X=X, dX=dX, dW=dW, workspace=workspace)
    if dX is None:
        dX = _empty((M, K), torch.bfloat16, dev, stream)
    if dW is None:
        dW = _empty((N, K), torch.bfloat16, dev, stream)
    if workspace is None:
        workspace = _scratch(max(linear_backward_workspace_size(M, N, K), 1), dev, stream)
    _check(lib().bsmm_linear_backward(_ptr(dY), _ptr(W), _ptr(X), M, N, K, _code(fp8), _ptr(dX), _ptr(dW),
                                      _ptr(workspace), _nbytes(workspace), _stream(stream)), "bsmm_linear_backward")
    return dX, dW


# --------------------------------------------------------------------------- #
# Scales in the tensor cores' atom layout                                     #
# --------------------------------------------------------------------------- #

def scale_atoms_size(B, rows, K, code="e4m3", scale="ue8m0") -> int:
    return lib().bsmm_scale_atoms_size(B, rows, K, _code(code), _scale(scale))


def quantize_atoms(x, code="e4m3", scale="ue8m0", batches=1, transpose=False, codes=None, atoms=None, stream=None):
    """Quantize a GEMM operand with its scales written in the atom layout.

    ``x`` is [batches * rows, K] (or [K, rows] with ``transpose``); returns
    ``(codes, atoms)``: codes [batches * rows, K] (E2M1 packed: K/2 bytes a
    row) and the atoms as a flat uint8 tensor."""
    _want(x, "x", dtypes=_FLOATS)
    if x.dim() != 2:
        raise ValueError("x must be a 2-D float32 or bfloat16 tensor")
    c, s = _code(code), _scale(scale)
    batches = int(batches)
    if batches < 1:
        raise ValueError("batches must be positive")
    if transpose:
        K, rows = x.shape
    else:
        total, K = x.shape
        if total % batches:
            raise ValueError(f"x's {total} rows do not split into {batches} batches")
        rows = total // batches
    if codes is not None:
        _want(codes, "codes", (batches * rows, _code_bytes(c, K)), itemsize=1)
    if atoms is not None:
        _want(atoms, "atoms")
    dev = _on_device(x=x, codes=codes, atoms=atoms)
    if codes is None:
        codes = _empty((batches * rows, _code_bytes(c, K)), torch.uint8, dev, stream)
    if atoms is None:
        atoms = _empty(max(scale_atoms_size(batches, rows, K, c, s), 1), torch.uint8, dev, stream)
    _check(lib().bsmm_quantize_atoms(_ptr(x), BF16 if x.dtype == torch.bfloat16 else F32, batches, rows, K,
                                     1 if transpose else 0, c, s, _ptr(codes), _ptr(atoms), _nbytes(atoms),
                                     _stream(stream)), "bsmm_quantize_atoms")
    return codes, atoms


def gemm_atoms(a, b, a_atoms, b_atoms, a_type="e4m3", b_type="e4m3", scale="ue8m0", out_dtype=torch.float32,
               y=None, workspace=None, K=None, stream=None):
    """:func:`gemm` with both operands' scales in the atom layout."""
    at, bt, sc = _code(a_type), _code(b_type), _scale(scale)
    a, b, _, _, Bn, M, N, K = _gemm_operands(a, b, None, None, at, bt, K)
    _want(a_atoms, "a_atoms", min_bytes=scale_atoms_size(Bn, M, K, at, sc))
    _want(b_atoms, "b_atoms", min_bytes=scale_atoms_size(Bn, N, K, bt, sc))
    if y is not None:
        _want(y, "y", (Bn, M, N), dtypes=_FLOATS)
    if workspace is not None:
        _want(workspace, "workspace")
    dev = _on_device(a=a, b=b, a_atoms=a_atoms, b_atoms=b_atoms, y=y, workspace=workspace)
    if y is None:
        y = _empty((Bn, M, N), out_dtype, dev, stream)
    if workspace is None and at == E2M1:
        workspace = _scratch(max(gemm_workspace_size(Bn, M, N, K, at), 1), dev, stream)
    _check(lib().bsmm_gemm_atoms(Bn, M, N, K, _ptr(a), at, _ptr(b), bt, _ptr(a_atoms), _ptr(b_atoms),
                                 sc, _ptr(y), BF16 if y.dtype == torch.bfloat16 else F32,
                                 _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "bsmm_gemm_atoms")
    return y


def linear_backward_quantized(dy_n, dy_n_scales, w_t, w_t_scales, dy_t, dy_t_scales, x_t, x_t_scales,
                              fp8="e5m2", scales_are_atoms=False, dX=None, dW=None, workspace=None, stream=None):
    """The backward's two GEMMs from pre-quantized operands: dY along N
    [M, N], W^T [K, N], dY^T [N, M], X^T [K, M] with their scales (row-major,
    or atoms).  Returns ``(dX, dW)`` in bfloat16."""
    c = _code(fp8)
    _want(dy_n, "dy_n", itemsize=1)
    if dy_n.dim() != 2:
        raise ValueError("dy_n must be a 2-D code tensor [M, N]")
    M, N = dy_n.shape
    _want(w_t, "w_t", itemsize=1)
    if w_t.dim() != 2:
        raise ValueError("w_t must be a 2-D code tensor [K, N]")
    K = w_t.shape[0]
    # (codes, scales, rows, contraction) of each operand
    operands = (("dy_n", dy_n, dy_n_scales, M, N), ("w_t", w_t, w_t_scales, K, N),
                ("dy_t", dy_t, dy_t_scales, N, M), ("x_t", x_t, x_t_scales, K, M))
    for n, codes, scales, rows, kc in operands:
        _want(codes, n, (rows, kc), itemsize=1)
        if scales_are_atoms:
            _want(scales, f"{n}_scales", min_bytes=scale_atoms_size(1, rows, kc, c, SCALE_UE8M0))
        elif kc % 32 == 0:  # else the library says why
            _want(scales, f"{n}_scales", (rows, kc // 32), itemsize=1)
    bf16 = (torch.bfloat16,)
    if dX is not None:
        _want(dX, "dX", (M, K), dtypes=bf16)
    if dW is not None:
        _want(dW, "dW", (N, K), dtypes=bf16)
    if workspace is not None:
        _want(workspace, "workspace")
    dev = _on_device(dy_n=dy_n, dy_n_scales=dy_n_scales, w_t=w_t, w_t_scales=w_t_scales, dy_t=dy_t,
                     dy_t_scales=dy_t_scales, x_t=x_t, x_t_scales=x_t_scales, dX=dX, dW=dW, workspace=workspace)
    if dX is None:
        dX = _empty((M, K), torch.bfloat16, dev, stream)
    if dW is None:
        dW = _empty((N, K), torch.bfloat16, dev, stream)
    need = lib().bsmm_linear_backward_quantized_workspace_size(M, N, K, 1 if scales_are_atoms else 0)
    if workspace is None and need:
        workspace = _scratch(need, dev, stream)
    _check(lib().bsmm_linear_backward_quantized(M, N, K, c, _ptr(dy_n), _ptr(dy_n_scales), _ptr(w_t),
                                                _ptr(w_t_scales), _ptr(dy_t), _ptr(dy_t_scales), _ptr(x_t),
                                                _ptr(x_t_scales), 1 if scales_are_atoms else 0, _ptr(dX), _ptr(dW),
                                                _ptr(workspace), _nbytes(workspace),
                                                _stream(stream)), "bsmm_linear_backward_quantized")
    return dX, dW


# --------------------------------------------------------------------------- #
# Activation checkpoints in 8 bits                                            #
# --------------------------------------------------------------------------- #

def _raw_stream(stream, dev) -> int:
    """The stream's handle; the current stream's through torch's raw query,
    which builds no Stream object (a tenth of its time)."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev.index)


def _fits(t, dtype, shape, dev) -> bool:
    """Whether a tensor is all that its checks ask for.  A call whose tensors
    all fit skips the checks that say what is wrong; one that does not goes
    through them (small calls spend most of their time on the host)."""
    try:
        return t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and t.is_contiguous()
    except AttributeError:  # not a tensor
        return False


def _current(t) -> bool:
    return isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == torch._C._cuda_getDevice()


def _at(t):
    return None if t is None else t.data_ptr()


def _act(a) -> int:
    return _ACT_NAMES[a] if isinstance(a, str) else int(a)


def _checkpoint_scales(s: int):
    """Block along the rows and scale dtype of a checkpoint's scale type."""
    return (128, torch.float32) if s == SCALE_F32 else (32, torch.uint8)


def gated_act(gate_up, act="silu", h_type="e4m3", code="int8", scale="f32", h_scales_are_atoms=False, h=None,
              h_scales=None, codes=None, scales=None, stream=None):
    """``h = act(gate) * up`` of ``gate_up`` [M, 2 I] (gate first), quantized
    as the next GEMM's MXFP8 operand (``h_type`` "e4m3" / "e5m2") or bfloat16
    ("bf16"), with ``gate_up`` kept for the backward pass as 8-bit codes
    (``code``, ``scale`` as :func:`quantize` names them; ``code=None`` keeps
    nothing).

    Returns ``(h, h_scales, codes, scales)``; ``h_scales`` is None for
    bfloat16, ``codes`` and ``scales`` are None when nothing is kept."""
    ht = BF16 if h_type == "bf16" else _code(h_type)
    quantized = ht != BF16
    c, s = (-1 if code is None else _code(code)), _scale(scale)
    block, scale_dtype = _checkpoint_scales(s)
    if (h is None and h_scales is None and codes is None and scales is None and _current(gate_up) and gate_up.dim() == 2
            and gate_up.dtype in _FLOATS and gate_up.is_contiguous() and gate_up.shape[1] % 2 == 0):
        dev, (M, I) = gate_up.device, gate_up.shape
        I //= 2
    else:
        _want(gate_up, "gate_up", dtypes=_FLOATS)
        if gate_up.dim() != 2 or gate_up.shape[1] % 2:
            raise ValueError("gate_up must be a 2-D float32 or bfloat16 tensor [M, 2 I]")
        M, I = gate_up.shape
        I //= 2
        if h is not None:
            _want(h, "h", (M, I), dtypes=(torch.bfloat16,) if not quantized else None, itemsize=1 if quantized else None)
        if h_scales is not None:
            if h_scales_are_atoms:
                _want(h_scales, "h_scales", min_bytes=scale_atoms_size(1, M, I, ht, SCALE_UE8M0))
            else:
                _want(h_scales, "h_scales", (M, I // 32), itemsize=1)
        if code is None:
            codes = scales = None
        if codes is not None:
            _want(codes, "codes", (M, 2 * I), itemsize=1)
        if scales is not None:
            _want(scales, "scales", (M, 2 * I // block), itemsize=scale_dtype.itemsize)
        dev = _on_device(gate_up=gate_up, h=h, h_scales=h_scales, codes=codes, scales=scales)
    if h is None:
        h = _empty((M, I), torch.uint8 if quantized else torch.bfloat16, dev, stream)
    if quantized and h_scales is None:
        n = max(scale_atoms_size(1, M, I, ht, SCALE_UE8M0), 1) if h_scales_are_atoms else 0
        h_scales = _empty((n,) if h_scales_are_atoms else (M, I // 32), torch.uint8, dev, stream)
    if code is not None:
        if codes is None:
            codes = _empty((M, 2 * I), torch.int8 if c == INT8 else torch.uint8, dev, stream)
        if scales is None:
            scales = _empty((M, 2 * I // block), scale_dtype, dev, stream)
    _check(lib().bsmm_gated_act(gate_up.data_ptr(), BF16 if gate_up.dtype == torch.bfloat16 else F32, M, I, 2 * I,
                                _act(act), ht, h.data_ptr(), h_scales.data_ptr() if quantized else None,
                                1 if h_scales_are_atoms else 0, c, s, _at(codes), _at(scales), _raw_stream(stream, dev)),
           "bsmm_gated_act")
    return h, (h_scales if quantized else None), codes, scales


def gated_act_backward(dh, codes, scales, act="silu", code="int8", scale="f32", return_h=False, d_gate_up=None, h=None,
                       stream=None):
    """Backward of :func:`gated_act` from its checkpoint: returns
    ``(d_gate_up, h)``, ``d_gate_up`` [M, 2 I] of ``dh``'s type and ``h`` the
    recomputed bfloat16 activation (None without ``return_h``)."""
    c, s = _code(code), _scale(scale)
    block, scale_dtype = _checkpoint_scales(s)
    fit = False
    if (d_gate_up is None and h is None and _current(dh) and dh.dim() == 2 and dh.dtype in _FLOATS and dh.is_contiguous()
            and isinstance(codes, torch.Tensor) and codes.element_size() == 1
            and isinstance(scales, torch.Tensor) and scales.element_size() == scale_dtype.itemsize):
        dev, (M, I) = dh.device, dh.shape
        fit = (_fits(codes, codes.dtype, (M, 2 * I), dev) and _fits(scales, scales.dtype, (M, 2 * I // block), dev))
    if not fit:
        _want(dh, "dh", dtypes=_FLOATS)
        if dh.dim() != 2:
            raise ValueError("dh must be a 2-D float32 or bfloat16 tensor [M, I]")
        M, I = dh.shape
        _want(codes, "codes", (M, 2 * I), itemsize=1)
        _want(scales, "scales", (M, 2 * I // block), itemsize=scale_dtype.itemsize)
        if d_gate_up is not None:
            _want(d_gate_up, "d_gate_up", (M, 2 * I), dtypes=(dh.dtype,))
        if h is not None:
            _want(h, "h", (M, I), dtypes=(torch.bfloat16,))
        dev = _on_device(dh=dh, codes=codes, scales=scales, d_gate_up=d_gate_up, h=h)
    if d_gate_up is None:
        d_gate_up = _empty((M, 2 * I), dh.dtype, dev, stream)
    if return_h and h is None:
        h = _empty((M, I), torch.bfloat16, dev, stream)
    _check(lib().bsmm_gated_act_backward(dh.data_ptr(), BF16 if dh.dtype == torch.bfloat16 else F32, M, I, _act(act),
                                         codes.data_ptr(), c, scales.data_ptr(), s, d_gate_up.data_ptr(), _at(h),
                                         _raw_stream(stream, dev)), "bsmm_gated_act_backward")
    return d_gate_up, h


def linear_backward_checkpoint(dY, W, x_codes, x_scales, x_code="e4m3", x_scale="ue8m0", fp8="e5m2", dX=None, dW=None,
                               workspace=None, stream=None):
    """:func:`linear_backward` with X kept in 8 bits (:func:`quantize` with
    blocks of 1 x 32 UE8M0 or 1 x 128 F32): returns ``(dX, dW)`` in bfloat16."""
    bf16 = (torch.bfloat16,)
    c, s = _code(x_code), _scale(x_scale)
    block, scale_dtype = _checkpoint_scales(s)
    fit = False
    if (dX is None and dW is None and workspace is None and _current(dY) and dY.dim() == 2 and isinstance(W, torch.Tensor)
            and W.dim() == 2 and isinstance(x_codes, torch.Tensor) and x_codes.element_size() == 1
            and isinstance(x_scales, torch.Tensor) and x_scales.element_size() == scale_dtype.itemsize):
        dev, (M, N), K = dY.device, dY.shape, W.shape[1]
        fit = (K % block == 0 and _fits(dY, torch.bfloat16, (M, N), dev) and _fits(W, torch.bfloat16, (N, K), dev)
               and _fits(x_codes, x_codes.dtype, (M, K), dev) and _fits(x_scales, x_scales.dtype, (M, K // block), dev))
    if not fit:
        for t, n in ((dY, "dY"), (W, "W")):
            _want(t, n, dtypes=bf16)
            if t.dim() != 2:
                raise ValueError(f"{n} must be a 2-D bfloat16 tensor")
        M, N = dY.shape
        K = W.shape[1]
        _want(W, "W", (N, K))
        _want(x_codes, "x_codes", (M, K), itemsize=1)
        if K % block == 0:  # else the library says why
            _want(x_scales, "x_scales", (M, K // block), itemsize=scale_dtype.itemsize)
        if dX is not None:
            _want(dX, "dX", (M, K), dtypes=bf16)
        if dW is not None:
            _want(dW, "dW", (N, K), dtypes=bf16)
        if workspace is not None:
            _want(workspace, "workspace")
        dev = _on_device(dY=dY, W=W, x_codes=x_codes, x_scales=x_scales, dX=dX, dW=dW, workspace=workspace)
    if dX is None:
        dX = _empty((M, K), torch.bfloat16, dev, stream)
    if dW is None:
        dW = _empty((N, K), torch.bfloat16, dev, stream)
    if workspace is None:
        workspace = _scratch(max(linear_backward_workspace_size(M, N, K), 1), dev, stream)
    _check(lib().bsmm_linear_backward_checkpoint(dY.data_ptr(), W.data_ptr(), x_codes.data_ptr(), c, x_scales.data_ptr(),
                                                 s, M, N, K, _code(fp8), dX.data_ptr(), dW.data_ptr(),
                                                 workspace.data_ptr(), _nbytes(workspace), _raw_stream(stream, dev)),
           "bsmm_linear_backward_checkpoint")
    return dX, dW


# --------------------------------------------------------------------------- #
# Low-rank adapters of many requests                                          #
# --------------------------------------------------------------------------- #

def _rows(t, name, shape, dtypes):
    """A 2-D argument whose rows are contiguous at any pitch; returns the pitch."""
    _want(t, name, shape, dtypes=dtypes)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    pitch, step = t.stride()
    if (step != 1 and t.shape[1] > 1) or (pitch < t.shape[1] and t.shape[0] > 1):
        raise ValueError(f"{name} must have contiguous rows")
    return max(pitch, t.shape[1])


def _adapter_weights(a, b, ids, scaling, T):
    bf16 = (torch.bfloat16,)
    _want(a, "a", dtypes=bf16)
    _want(b, "b", dtypes=bf16)
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b must be (L, R, K) and (L, N, R) bfloat16 tensors")
    L, R, K = a.shape
    N = b.shape[1]
    _want(b, "b", (L, N, R))
    _want(ids, "ids", (T,), dtypes=(torch.int32,))
    if scaling is not None:
        _want(scaling, "scaling", (L,), dtypes=(torch.float32,))
    return L, R, K, N


def adapters_workspace_size(T, R, L) -> int:
    return lib().bsmm_adapters_workspace_size(T, R, L)


def adapters(x, a, b, ids, y=None, scaling=None, out=None, u=None, out_dtype=torch.bfloat16, workspace=None,
             stream=None):
    """``out = y + scaling[id] * (x @ a[id].T) @ b[id].T`` for every token's
    adapter ``id = ids[t]`` (outside ``[0, L)``: none).

    ``x`` [T, K] bfloat16, ``a`` [L, R, K], ``b`` [L, N, R] bfloat16, ``ids``
    [T] int32, ``y`` [T, N] float32 or bfloat16, the shared projection's
    product (None: 0).  Rows of ``x``, ``y`` and ``out`` may lie at any pitch;
    ``out`` may be ``y``.  Returns ``(out, u)``: ``u`` [T, R] float32 is
    ``x @ a[id].T``, which :func:`adapters_backward` takes."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor [T, K]")
    T = x.shape[0]
    dtype = y.dtype if y is not None else out.dtype if out is not None else out_dtype
    bf16, dev = torch.bfloat16, x.device
    if (_current(x) and isinstance(a, torch.Tensor) and a.dim() == 3 and isinstance(b, torch.Tensor) and b.dim() == 3
            and dtype in _FLOATS):
        (L, R, K), N = a.shape, b.shape[1]
        fit = (_fits(x, bf16, (T, K), dev) and _fits(a, bf16, (L, R, K), dev) and _fits(b, bf16, (L, N, R), dev)
               and _fits(ids, torch.int32, (T,), dev)
               and (scaling is None or _fits(scaling, torch.float32, (L,), dev))
               and (y is None or _fits(y, dtype, (T, N), dev)) and (out is None or _fits(out, dtype, (T, N), dev))
               and (u is None or _fits(u, torch.float32, (T, R), dev)) and workspace is None)
    else:
        fit = False
    if fit:
        ld_x, ld_y, ld_out = K, N, N
    else:
        L, R, K, N = _adapter_weights(a, b, ids, scaling, T)
        ld_x = _rows(x, "x", (T, K), (bf16,))
        ld_y = _rows(y, "y", (T, N), _FLOATS) if y is not None else N
        ld_out = _rows(out, "out", (T, N), (dtype,)) if out is not None else N
        if dtype not in _FLOATS:
            raise ValueError(f"out must be torch.float32 or torch.bfloat16, got {dtype}")
        if u is not None:
            _want(u, "u", (T, R), dtypes=(torch.float32,))
        if workspace is not None:
            _want(workspace, "workspace")
        dev = _on_device(a=a, b=b, ids=ids, scaling=scaling, u=u, workspace=workspace)
        for n, t in (("x", x), ("y", y), ("out", out)):
            if t is not None and t.device != dev:
                raise ValueError(f"{n} is on {t.device}, the other arguments on {dev}")
    if out is None:
        out = _empty((T, N), dtype, dev, stream)
    if u is None:
        u = _empty((T, R), torch.float32, dev, stream)
    if workspace is None:
        need = adapters_workspace_size(T, R, L)
        if need:
            workspace = _scratch(need, dev, stream)
    _check(lib().bsmm_adapters(T, K, N, R, L, x.data_ptr(), ld_x, a.data_ptr(), b.data_ptr(), ids.data_ptr(),
                               _at(scaling), _at(y), ld_y, out.data_ptr(), ld_out, BF16 if dtype is bf16 else F32,
                               u.data_ptr(), _at(workspace), _nbytes(workspace), _raw_stream(stream, dev)),
           "bsmm_adapters")
    return out, u


def adapters_backward_workspace_size(T, R, L) -> int:
    return lib().bsmm_adapters_backward_workspace_size(T, R, L)


def adapters_backward(dy, x, a, b, ids, u, scaling=None, dx_base=None, x_scales=None, x_code="e4m3",
                      grad_dtype=torch.float32, dx=None, da=None, db=None, workspace=None, stream=None):
    """Backward of :func:`adapters` from ``dy`` [T, N] bfloat16 and the
    forward's ``u``: returns ``(dx, da, db)``.

    ``x`` is the forward's bfloat16 input, or with ``x_scales`` its MXFP8
    checkpoint (codes [T, K] of type ``x_code``, scales [T, K / 32]).  ``dx``
    [T, K] bfloat16 adds to ``dx_base`` (the shared projection's own dX; may
    be the same tensor); ``da`` and ``db`` are of ``grad_dtype``."""
    if not isinstance(dy, torch.Tensor) or dy.dim() != 2:
        raise ValueError("dy must be a 2-D bfloat16 tensor [T, N]")
    T = dy.shape[0]
    if (_current(dy) and isinstance(a, torch.Tensor) and a.dim() == 3 and isinstance(b, torch.Tensor) and b.dim() == 3
            and grad_dtype in _FLOATS and isinstance(x, torch.Tensor)):
        one, dev = torch.bfloat16, dy.device
        (L, R, K), N = a.shape, b.shape[1]
        fit = (_fits(dy, one, (T, N), dev) and _fits(a, one, (L, R, K), dev) and _fits(b, one, (L, N, R), dev)
               and _fits(ids, torch.int32, (T,), dev) and _fits(u, torch.float32, (T, R), dev)
               and (scaling is None or _fits(scaling, torch.float32, (L,), dev))
               and (_fits(x, one, (T, K), dev) if x_scales is None else
                    K % 32 == 0 and x.element_size() == 1 and _fits(x, x.dtype, (T, K), dev)
                    and _fits(x_scales, torch.uint8, (T, K // 32), dev))
               and (dx_base is None or _fits(dx_base, one, (T, K), dev)) and (dx is None or _fits(dx, one, (T, K), dev))
               and da is None and db is None and workspace is None)
    else:
        fit = False
    if fit:
        ld_dy, ld_x, xt = N, K, (BF16 if x_scales is None else _code(x_code))
    else:
        L, R, K, N = _adapter_weights(a, b, ids, scaling, T)
        bf16 = (torch.bfloat16,)
        ld_dy = _rows(dy, "dy", (T, N), bf16)
        if x_scales is not None:
            _want(x, "x", (T, K), itemsize=1)
            if K % 32 == 0:  # else the library says why
                _want(x_scales, "x_scales", (T, K // 32), itemsize=1)
            ld_x, xt = K, _code(x_code)
        else:
            ld_x, xt = _rows(x, "x", (T, K), bf16), BF16
        _want(u, "u", (T, R), dtypes=(torch.float32,))
        if grad_dtype not in _FLOATS:
            raise ValueError("grad_dtype must be float32 or bfloat16")
        for t, n, shape in ((dx_base, "dx_base", (T, K)), (dx, "dx", (T, K))):
            if t is not None:
                _want(t, n, shape, dtypes=bf16)
        for t, n, shape in ((da, "da", (L, R, K)), (db, "db", (L, N, R))):
            if t is not None:
                _want(t, n, shape, dtypes=(grad_dtype,))
        if workspace is not None:
            _want(workspace, "workspace")
        dev = _on_device(a=a, b=b, ids=ids, scaling=scaling, u=u, x_scales=x_scales, dx_base=dx_base, dx=dx, da=da, db=db,
                         workspace=workspace, **({"x": x} if x_scales is not None else {}))
        for n, t in (("dy", dy), ("x", x)):
            if t.device != dev:
                raise ValueError(f"{n} is on {t.device}, the other arguments on {dev}")
    if dx is None:
        dx = _empty((T, K), torch.bfloat16, dev, stream)
    if da is None:
        da = _empty((L, R, K), grad_dtype, dev, stream)
    if db is None:
        db = _empty((L, N, R), grad_dtype, dev, stream)
    if workspace is None:
        workspace = _scratch(max(adapters_backward_workspace_size(T, R, L), 1), dev, stream)
    _check(lib().bsmm_adapters_backward(T, K, N, R, L, dy.data_ptr(), ld_dy, x.data_ptr(), ld_x, xt, _at(x_scales),
                                        a.data_ptr(), b.data_ptr(), ids.data_ptr(), _at(scaling), u.data_ptr(),
                                        _at(dx_base), K, dx.data_ptr(), da.data_ptr(), db.data_ptr(),
                                        BF16 if grad_dtype == torch.bfloat16 else F32, workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), _raw_stream(stream, dev)),
           "bsmm_adapters_backward")
    return dx, da, db


# --------------------------------------------------------------------------- #
# Mixture of experts                                                          #
# --------------------------------------------------------------------------- #

_I32 = (torch.int32,)
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)


def _same_device(dev, **named):
    for n, t in named.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{n} is on {t.device}, the other arguments on {dev}")


# The sizes below depend on their arguments alone, which a model repeats: asked
# for once each, they cost a call 0.1 us instead of 0.6 to 0.9.

@functools.lru_cache(maxsize=4096)
def _atoms_size(E, N, K, code) -> int:
    return scale_atoms_size(E, N, K, code, SCALE_UE8M0)


@functools.lru_cache(maxsize=4096)
def route_workspace_size(T, E) -> int:
    return lib().bsmm_route_workspace_size(T, E)


def route(logits, k, renormalize=True, weights=None, ids=None, offsets=None, rows=None, slots=None, workspace=None,
          stream=None):
    """The ``k`` experts of each token and the tokens' layout by expert.

    ``logits`` [T, E] float32 or bfloat16, rows at any pitch.  Returns
    ``(weights, ids, offsets, rows, slots)``: the softmax of the ``k`` largest
    logits [T, k] float32 (over those, or without ``renormalize`` over all E),
    their experts [T, k] int32 (-1 where nothing is left to choose), and the
    (token, choice) pairs by expert: ``offsets`` [E + 1], ``rows`` [T k] (the
    token of each slot) and ``slots`` [T, k] (the slot of each pair) int32."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a 2-D float32 or bfloat16 tensor [T, E]")
    (T, E), k = logits.shape, int(k)
    dev = logits.device
    ld = E if _match("F:TE", logits) else _rows(logits, "logits", (T, E), _FLOATS)
    if not _current(logits):
        raise ValueError(f"logits is on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    if k < 0:
        raise ValueError("k must not be negative")
    shapes = (torch.float32, (T, k), torch.int32, (T, k), torch.int32, (E + 1,), torch.int32, (T * k,), torch.int32, (T, k))
    if weights is ids is offsets is rows is slots is workspace is None:
        weights, ids, offsets, rows, slots = _empties(dev, stream, *shapes)
    else:
        outs = {"weights": weights, "ids": ids, "offsets": offsets, "rows": rows, "slots": slots}
        for (n, t), dtype, shape in zip(outs.items(), shapes[::2], shapes[1::2]):
            if t is not None:
                _want(t, n, shape, dtypes=(dtype,))
        if workspace is not None:
            _want(workspace, "workspace")
        _same_device(dev, **outs, workspace=workspace)
        _on_device(**outs, workspace=workspace)
        weights, ids, offsets, rows, slots = (_empty(shape, dtype, dev, stream) if t is None else t
                                              for t, dtype, shape in zip(outs.values(), shapes[::2], shapes[1::2]))
    if workspace is None:
        need = route_workspace_size(T, E)
        if need:
            workspace = _scratch(need, dev, stream)
    _check(lib().bsmm_route(T, E, k, logits.data_ptr(), BF16 if logits.dtype is torch.bfloat16 else F32, ld,
                            1 if renormalize else 0, ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(),
                            rows.data_ptr(), slots.data_ptr(), _at(workspace), _nbytes(workspace),
                            _raw_stream(stream, dev)), "bsmm_route")
    return weights, ids, offsets, rows, slots


def route_backward(d_weights, logits, ids, weights, renormalize=True, d_logits=None, stream=None):
    """Backward of :func:`route`: ``d_logits`` [T, E] of the logits' type."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a 2-D float32 or bfloat16 tensor [T, E]")
    T, E = logits.shape
    fit = _match("F:TE i:Tk f:Tk f:Tk", logits, ids, weights, d_weights) if d_logits is None else None
    if fit:
        k, dev = fit[6], logits.device
        d_logits = _empty((T, E), logits.dtype, dev, stream)
        return _route_backward(T, E, k, logits, E, renormalize, fit[3], fit[1], fit[2], d_logits, dev, stream)
    ld = _rows(logits, "logits", (T, E), _FLOATS)
    _want(ids, "ids", dtypes=_I32)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids must be an int32 tensor [{T}, k]")
    k = ids.shape[1]
    _want(weights, "weights", (T, k), dtypes=_F32)
    _want(d_weights, "d_weights", (T, k), dtypes=_F32)
    if d_logits is not None:
        _want(d_logits, "d_logits", (T, E), dtypes=(logits.dtype,))
    dev = _on_device(ids=ids, weights=weights, d_weights=d_weights, d_logits=d_logits)
    _same_device(dev, logits=logits)
    if d_logits is None:
        d_logits = _empty((T, E), logits.dtype, dev, stream)
    return _route_backward(T, E, k, logits, ld, renormalize, d_weights.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                           d_logits, dev, stream)


def _route_backward(T, E, k, logits, ld, renormalize, d_weights, ids, weights, d_logits, dev, stream):
    _check(lib().bsmm_route_backward(T, E, k, logits.data_ptr(), BF16 if logits.dtype is torch.bfloat16 else F32, ld,
                                     1 if renormalize else 0, d_weights, ids, weights, d_logits.data_ptr(),
                                     _raw_stream(stream, dev)), "bsmm_route_backward")
    return d_logits


@functools.lru_cache(maxsize=4096)
def expert_gemm_workspace_size(S, E, K, by_rows=True) -> int:
    return lib().bsmm_expert_gemm_workspace_size(S, E, K, 1 if by_rows else 0)


def expert_gemm(x, x_scales, w, w_atoms, offsets, rows=None, x_type="e4m3", w_type="e4m3", y=None, workspace=None,
                stream=None):
    """``y[s] = w[e] @ x[rows[s]]`` for the slots ``offsets[e] <= s <
    offsets[e + 1]`` of every expert ``e``, MXFP8: y [S, N] bfloat16.

    ``x`` [X, K] codes with scale bytes ``x_scales`` [X, K / 32]; ``w``
    [E, N, K] codes with ``w_atoms`` as :func:`quantize_atoms` writes them for
    E batches; ``offsets`` [E + 1] and ``rows`` [S] int32 (None: slot s is row
    s of x).  Slots of no expert are left as they are in ``y``."""
    xt, wt = _code(x_type), _code(w_type)
    fit = _match("c:XK c:XB c:ENK .:# i:O i?:S", x, x_scales, w, w_atoms, offsets, rows)
    if fit:
        X, K, B, E, N, atoms, slots = fit[6:13]
        S = X if rows is None else fit[13]
        if K != 32 * B or slots != E + 1 or atoms < _atoms_size(E, N, K, wt):
            fit = None
    if not fit:
        _want(x, "x", itemsize=1)
        _want(w, "w", itemsize=1)
        if x.dim() != 2 or w.dim() != 3:
            raise ValueError("x and w must be code tensors [X, K] and [E, N, K]")
        (X, K), (E, N) = x.shape, w.shape[:2]
        _want(w, "w", (E, N, K))
        _want(x_scales, "x_scales", itemsize=1)
        if K % 32 == 0:  # else the library says why
            _want(x_scales, "x_scales", (X, K // 32))
            _want(w_atoms, "w_atoms", min_bytes=_atoms_size(E, N, K, wt))
        S = _expert_slots(offsets, rows, E, X)
    if y is not None:
        _want(y, "y", (S, N), dtypes=_BF16)
    if workspace is not None:
        _want(workspace, "workspace")
    if fit and y is None and workspace is None:
        dev = x.device
    else:
        dev = _on_device(x=x, x_scales=x_scales, w=w, w_atoms=w_atoms, offsets=offsets, rows=rows, y=y,
                         workspace=workspace)
    if y is None:
        y = _empty((S, N), torch.bfloat16, dev, stream)
    if workspace is None and rows is not None:
        need = expert_gemm_workspace_size(S, E, K)
        if need:
            workspace = _scratch(need, dev, stream)
    _check(lib().bsmm_expert_gemm(S, X, E, N, K, x.data_ptr(), xt, x_scales.data_ptr(), w.data_ptr(), wt,
                                  w_atoms.data_ptr(), offsets.data_ptr(), _at(rows), y.data_ptr(), _at(workspace),
                                  _nbytes(workspace), _raw_stream(stream, dev)), "bsmm_expert_gemm")
    return y


def _expert_slots(offsets, rows, E, X) -> int:
    _want(offsets, "offsets", (E + 1,), dtypes=_I32)
    if rows is None:
        return X
    _want(rows, "rows", dtypes=_I32)
    if rows.dim() != 1:
        raise ValueError("rows must be a 1-D int32 tensor [S]")
    return rows.shape[0]


@functools.lru_cache(maxsize=4096)
def expert_backward_workspace_size(S, E, N, K) -> int:
    return lib().bsmm_expert_backward_workspace_size(S, E, N, K)


def expert_backward(dY, W, X, offsets, rows=None, fp8="e5m2", dX=None, dW=None, workspace=None, stream=None):
    """:func:`linear_backward` by expert, from bfloat16 ``dY`` [S, N], ``W``
    [E, N, K] and ``X`` [rows of x, K]: returns ``(dX, dW)``, ``dX`` [S, K] by
    slot (:func:`expert_combine` without weights sums it by token) and ``dW``
    [E, N, K], bfloat16."""
    fit = _match("b:SN b:ENK b:RK i:O i?:S", dY, W, X, offsets, rows)
    if fit:
        S, N, E, K, R, slots = fit[5:11]
        if slots != E + 1 or (rows is None and R != S):
            fit = None
    if not fit:
        for t, n, dims in ((dY, "dY", 2), (W, "W", 3), (X, "X", 2)):
            _want(t, n, dtypes=_BF16)
            if t.dim() != dims:
                raise ValueError("dY, W and X must be bfloat16 tensors [S, N], [E, N, K] and [rows, K]")
        E, N, K = W.shape
        _want(X, "X", (X.shape[0], K))
        S = _expert_slots(offsets, rows, E, X.shape[0])
        _want(dY, "dY", (S, N))
    if dX is not None:
        _want(dX, "dX", (S, K), dtypes=_BF16)
    if dW is not None:
        _want(dW, "dW", (E, N, K), dtypes=_BF16)
    if workspace is not None:
        _want(workspace, "workspace")
    if fit and dX is dW is workspace is None:
        dev = dY.device
    else:
        dev = _on_device(dY=dY, W=W, X=X, offsets=offsets, rows=rows, dX=dX, dW=dW, workspace=workspace)
    if dX is None and dW is None:
        dX, dW = _empties(dev, stream, torch.bfloat16, (S, K), torch.bfloat16, (E, N, K))
    if dX is None:
        dX = _empty((S, K), torch.bfloat16, dev, stream)
    if dW is None:
        dW = _empty((E, N, K), torch.bfloat16, dev, stream)
    if workspace is None:
        workspace = _scratch(max(expert_backward_workspace_size(S, E, N, K), 1), dev, stream)
    _check(lib().bsmm_expert_backward(S, X.shape[0], E, N, K, dY.data_ptr(), W.data_ptr(), X.data_ptr(),
                                      offsets.data_ptr(), _at(rows), _code(fp8), dX.data_ptr(), dW.data_ptr(),
                                      workspace.data_ptr(), _nbytes(workspace), _raw_stream(stream, dev)),
           "bsmm_expert_backward")
    return dX, dW


def _combined(y, slots, weights):
    _want(y, "y", dtypes=_BF16)
    _want(slots, "slots", dtypes=_I32)
    if y.dim() != 2 or slots.dim() != 2:
        raise ValueError("y and slots must be a bfloat16 tensor [S, N] and an int32 tensor [T, k]")
    (S, N), (T, k) = y.shape, slots.shape
    if weights is not None:
        _want(weights, "weights", (T, k), dtypes=_F32)
    return S, N, T, k


def expert_combine(y, slots, weights=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """``out[t] = sum over j of weights[t, j] * y[slots[t, j]]`` (weights None:
    1; a slot outside y has no part): ``out`` [T, N] float32 or bfloat16."""
    fit = _match("b:SN i:Tk f?:Tk", y, slots, weights)
    S, N, T, k = fit[3:] if fit else _combined(y, slots, weights)
    dtype = out_dtype if out is None else out.dtype
    if dtype not in _FLOATS:
        raise ValueError(f"out must be torch.float32 or torch.bfloat16, got {dtype}")
    if out is not None:
        _want(out, "out", (T, N))
    dev = y.device if fit and out is None else _on_device(y=y, slots=slots, weights=weights, out=out)
    if out is None:
        out = _empty((T, N), dtype, dev, stream)
    _check(lib().bsmm_expert_combine(T, S, k, N, y.data_ptr(), slots.data_ptr(), _at(weights), out.data_ptr(),
                                     BF16 if dtype is torch.bfloat16 else F32, _raw_stream(stream, dev)),
           "bsmm_expert_combine")
    return out


def expert_combine_backward(d_out, y, slots, weights=None, dy=None, d_weights=None, stream=None):
    """Backward of :func:`expert_combine`: returns ``(dy, d_weights)``, ``dy``
    [S, N] bfloat16 (slots that do not occur are left as they are) and
    ``d_weights`` [T, k] float32 (None without weights)."""
    fit = _match("b:SN i:Tk f?:Tk F:TN b?:SN f?:Tk", y, slots, weights, d_out, dy, d_weights)
    if fit:
        (S, N, T, k), dev = fit[6:], y.device
    else:
        S, N, T, k = _combined(y, slots, weights)
        _want(d_out, "d_out", (T, N), dtypes=_FLOATS)
        if dy is not None:
            _want(dy, "dy", (S, N), dtypes=_BF16)
        if d_weights is not None:
            _want(d_weights, "d_weights", (T, k), dtypes=_F32)
        dev = _on_device(y=y, slots=slots, weights=weights, d_out=d_out, dy=dy, d_weights=d_weights)
    if dy is d_weights is None and weights is not None:
        dy, d_weights = _empties(dev, stream, torch.bfloat16, (S, N), torch.float32, (T, k))
    if dy is None:
        dy = _empty((S, N), torch.bfloat16, dev, stream)
    if d_weights is None and weights is not None:
        d_weights = _empty((T, k), torch.float32, dev, stream)
    _check(lib().bsmm_expert_combine_backward(T, S, k, N, d_out.data_ptr(),
                                              BF16 if d_out.dtype is torch.bfloat16 else F32, y.data_ptr(),
                                              slots.data_ptr(), _at(weights), dy.data_ptr(), _at(d_weights),
                                              _raw_stream(stream, dev)), "bsmm_expert_combine_backward")
    return dy, d_weights


# --------------------------------------------------------------------------- #
# AdamW                                                                       #
# --------------------------------------------------------------------------- #

def _tensor_list(ts, name, sizes, per=1, dtypes=None, itemsize=None, gaps=False):
    """A list of contiguous CUDA tensors of one type, on the current device:
    their addresses and sizes (64-bit words) and that type.  ``sizes``: those of
    another list, of which each tensor holds ceil(size / per) numbers.  ``gaps``:
    None may stand in a tensor's place (address 0)."""
    ts = list(ts)
    first = next((t for t in ts if t is not None), None) if gaps else ts[0] if ts else None
    dev = first.get_device() if isinstance(first, torch.Tensor) else -1
    found = None
    if not ts or (dev >= 0 and dev == torch._C._cuda_getDevice()) or (gaps and first is None):
        found = _lists().addresses(ts, dev, sizes, per, gaps)
    if found is None or (found[2] is not None and not _list_type(found[2], dtypes, itemsize)):
        _explain_list(ts, name, sizes, per, dtypes, itemsize, gaps)
    return found


def _list_type(dtype, dtypes, itemsize) -> bool:
    return (dtypes is None or dtype in dtypes) and (itemsize is None or dtype.itemsize == itemsize)


def _explain_list(ts, name, sizes, per, dtypes, itemsize, gaps):
    """Raises for what is wrong with a list of tensors."""
    given = [t for t in ts if t is not None] if gaps else ts
    for t in given:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must hold torch.Tensors")
    kinds = {t.dtype for t in given}
    if len(kinds) > 1:
        raise ValueError(f"{name} must be of one type, got {' and '.join(sorted(str(k) for k in kinds))}")
    for dtype in kinds:
        if not _list_type(dtype, dtypes, None):
            raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {dtype}")
        if not _list_type(dtype, None, itemsize):
            raise ValueError(f"{name} must have {itemsize}-byte elements, got {dtype}")
    if sizes is not None:
        want = [(n + per - 1) // per for n in array("q", sizes)]
        if len(ts) != len(want):
            raise ValueError(f"{name} holds {len(ts)} tensors, {len(want)} needed")
        for i, (t, n) in enumerate(zip(ts, want)):
            if t is not None and t.numel() != n:
                raise ValueError(f"{name}[{i}] holds {t.numel()} numbers, {n} needed")
    if not all(t.is_cuda and t.get_device() == torch._C._cuda_getDevice() for t in given):
        raise ValueError(f"{name} must be CUDA tensors on the current device")
    if not all(t.layout is torch.strided and t.is_contiguous() for t in given):
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be tensors with memory of their own")


def adamw(params, grads, m, v, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=1.0, m_scales=None,
          v_scales=None, copies=None, hyper=None, stream=None):
    """One AdamW step on lists of tensors, in place, in one launch per 384.

    ``params`` and ``grads`` float32 or bfloat16.  ``m`` and ``v`` float32, or
    with ``m_scales`` and ``v_scales`` (float32, one per 128 numbers) E4M3 codes
    of ``m`` and of ``sqrt(v)``, rounded to nearest for betas up to (0.944,
    0.9558) and dithered by ``step`` above, where nearest would not follow; zeros
    start a run.  ``copies`` receives the updated parameters in bfloat16,
    where its entry is not None.
    ``hyper``, a float32 tensor ``(lr, step, grad_scale)`` on the device, takes the
    place of those arguments when the kernels run (a captured step's schedule).

    The versions of ``params`` and ``copies`` rise, so that a backward pass
    through what autograd has saved of them raises, as after torch's own
    in-place changes (a graph's replay changes them without that)."""
    params = list(params)
    copies = None if copies is None else list(copies)
    if (m_scales is None) != (v_scales is None):
        raise ValueError("m_scales and v_scales go together")
    bits8 = m_scales is not None
    pp, n, pt = _tensor_list(params, "params", None, dtypes=_FLOATS)
    gg, _, gt = _tensor_list(grads, "grads", n, dtypes=_FLOATS)
    mm, _, _ = _tensor_list(m, "m", n, dtypes=None if bits8 else _F32, itemsize=1 if bits8 else None)
    vv, _, _ = _tensor_list(v, "v", n, dtypes=None if bits8 else _F32, itemsize=1 if bits8 else None)
    ms = vs = cc = None
    if bits8:
        ms, _, _ = _tensor_list(m_scales, "m_scales", n, 128, dtypes=_F32)
        vs, _, _ = _tensor_list(v_scales, "v_scales", n, 128, dtypes=_F32)
    if copies is not None:
        cc, _, _ = _tensor_list(copies, "copies", n, dtypes=_BF16, gaps=True)
    if hyper is not None:
        _want(hyper, "hyper", (3,), dtypes=_F32)
        _on_device(hyper=hyper)
    if not params:
        return
    _check(lib().bsmm_adamw(len(params), n, pp, BF16 if pt is torch.bfloat16 else F32, gg,
                            BF16 if gt is torch.bfloat16 else F32, mm, vv, E4M3 if bits8 else F32, ms, vs, cc,
                            lr, betas[0], betas[1], eps, weight_decay, int(step), grad_scale, _at(hyper),
                            _raw_stream(stream, params[0].device)), "bsmm_adamw")
    _lists().changed(params, copies)
