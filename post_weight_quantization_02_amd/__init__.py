"""GPTQ per-layer quantization solver on AMD gfx950 (MI355X).

A thin ctypes binding of ``libgptq.so`` (C ABI in ``include/gptq.h``).  The
functions keep the C names; PyTorch only provides device memory and the HIP
stream.  Every step of the solver runs in the library's HIP kernels; there is
no Python or CPU fallback, and loading fails loudly if the library is missing.

    H = torch.zeros(d, d, device="cuda")
    gptq_hessian_accumulate(H, X_chunk)            # once per calibration chunk
    U, lam, info = gptq_prepare_hinv(H, 0.01)
    codes, scales, zeros, err = gptq_quantize_layer(W, U, lam, bits=4, group_size=128)

``quantize_layer`` chains the three calls.
"""
from __future__ import annotations

import ctypes
import os
from typing import Iterable, Optional

__all__ = [
    "GPTQ_F32", "GPTQ_F16", "GPTQError", "NotPositiveDefinite", "library", "lib_path",
    "gptq_hessian_accumulate", "gptq_hessian_accumulate_workspace_size",
    "gptq_prepare_hinv", "gptq_prepare_hinv_workspace_size",
    "gptq_quantize_layer", "gptq_quantize_layer_workspace_size", "gptq_quantize_layer_noalloc",
    "GPTQ_NOALLOC_SCRATCH_BYTES",
    "gptq_act_order_perm", "gptq_prepare_hinv_perm", "gptq_quantize_layer_perm",
    "gptq_packed_words_per_row", "gptq_pack_codes", "gptq_dequant_matmul", "gptq_dequantize",
    "gptq2d_quantize", "gptq2d_quantize_workspace_size",
    "GPTQ_BF16", "GPTQ_MAX_TOP", "gptq_fp8_quantize", "gptq_fp8_matmul", "gptq_fp8_matmul_workspace_size",
    "gptq_token_logprobs", "gptq_token_logprobs_workspace_size",
    "gptq_int8_quantize", "gptq_int8_matmul", "gptq_int8_matmul_workspace_size", "gptq_int8_matmul_grouped",
    "gptq_distill_loss", "gptq_distill_loss_workspace_size",
    "gptq_launch_timing", "gptq_launch_timing_read", "TIMING_PANEL", "TIMING_PRODUCT",
    "gptq_status_string", "gptq_version", "quantize_layer",
]

GPTQ_F32 = 0
GPTQ_F16 = 1
GPTQ_BF16 = 2                           # the fp8, int8, log-probability and distillation calls only
GPTQ_MAX_TOP = 64                       # include/gptq.h
GPTQ_NOALLOC_SCRATCH_BYTES = 96 << 20   # include/gptq.h
TIMING_PANEL, TIMING_PRODUCT = 0, 1     # kinds of gptq_launch_timing_read

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


def lib_path() -> str:
    """The in-tree libgptq.so, or the library named by GPTQ_LIBRARY (the
    sanitizer build of the host code is tested that way)."""
    return os.environ.get("GPTQ_LIBRARY") or os.path.join(_HERE, "_lib", "libgptq.so")


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status}: {gptq_status_string(status)}")
        self.status = status


class NotPositiveDefinite(GPTQError):
    def __init__(self, info: int):
        RuntimeError.__init__(self, f"damped Hessian is not positive definite (info={info})")
        self.status = -1
        self.info = info


def library() -> ctypes.CDLL:
    """Load libgptq.so once; raise if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(python -m post_weight_quantization_02_amd._build)")
    lib = ctypes.CDLL(path)
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
    lib.gptq_hessian_accumulate.argtypes = [vp, i64, vp, i32, i64, i64, vp, sz, vp]
    lib.gptq_hessian_accumulate.restype = i32
    lib.gptq_hessian_accumulate_workspace_size.argtypes = [i64, i64, i32]
    lib.gptq_hessian_accumulate_workspace_size.restype = sz
    lib.gptq_prepare_hinv.argtypes = [vp, i64, ctypes.c_float, vp, vp, vp, vp, sz, vp]
    lib.gptq_prepare_hinv.restype = i32
    lib.gptq_prepare_hinv_workspace_size.argtypes = [i64]
    lib.gptq_prepare_hinv_workspace_size.restype = sz
    lib.gptq_quantize_layer.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, i64, i64, vp, vp, vp,
                                        vp, vp, sz, vp]
    lib.gptq_quantize_layer.restype = i32
    lib.gptq_quantize_layer_noalloc.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, i64, i64, vp, vp,
                                                vp, vp, vp]
    lib.gptq_quantize_layer_noalloc.restype = i32
    lib.gptq_quantize_layer_workspace_size.argtypes = [i64, i64, i64]
    lib.gptq_quantize_layer_workspace_size.restype = sz
    lib.gptq_act_order_perm.argtypes = [vp, i64, vp, vp]
    lib.gptq_act_order_perm.restype = i32
    lib.gptq_prepare_hinv_perm.argtypes = [vp, i64, vp, ctypes.c_float, vp, vp, vp, vp, sz, vp]
    lib.gptq_prepare_hinv_perm.restype = i32
    lib.gptq_quantize_layer_perm.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, i32, i64, i64, vp,
                                             vp, vp, vp, vp, vp, sz, vp]
    lib.gptq_quantize_layer_perm.restype = i32
    lib.gptq_packed_words_per_row.argtypes = [i64, i32]
    lib.gptq_packed_words_per_row.restype = i64
    lib.gptq_pack_codes.argtypes = [vp, i64, i64, i64, i32, vp, vp, i64, vp]
    lib.gptq_pack_codes.restype = i32
    lib.gptq_dequant_matmul.argtypes = [vp, i64, i32, vp, vp, i64, vp, i64, i64, vp, i32, i64, i64, vp,
                                        i64, vp]
    lib.gptq_dequant_matmul.restype = i32
    lib.gptq2d_quantize_workspace_size.argtypes = [i64, i64]
    lib.gptq2d_quantize_workspace_size.restype = sz
    lib.gptq2d_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, vp, i64, vp, vp, vp, vp, sz, vp]
    lib.gptq2d_quantize.restype = i32
    lib.gptq_dequantize.argtypes = [vp, i64, i64, i64, vp, vp, i64, vp, vp, i32, i64, vp]
    lib.gptq_dequantize.restype = i32
    lib.gptq_fp8_quantize.argtypes = [vp, i32, i64, i64, i64, i64, vp, i64, vp, i64, vp]
    lib.gptq_fp8_quantize.restype = i32
    lib.gptq_fp8_matmul_workspace_size.argtypes = [i64, i64, i64]
    lib.gptq_fp8_matmul_workspace_size.restype = sz
    lib.gptq_fp8_matmul.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, vp, i32, i64, vp, sz, vp]
    lib.gptq_fp8_matmul.restype = i32
    lib.gptq_token_logprobs_workspace_size.argtypes = [i64, i64, i64]
    lib.gptq_token_logprobs_workspace_size.restype = sz
    lib.gptq_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.gptq_token_logprobs.restype = i32
    lib.gptq_int8_quantize.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, vp]
    lib.gptq_int8_quantize.restype = i32
    lib.gptq_int8_matmul_workspace_size.argtypes = [i64, i64, i64]
    lib.gptq_int8_matmul_workspace_size.restype = sz
    lib.gptq_int8_matmul.argtypes = [vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, vp, i32, i64, vp, sz, vp]
    lib.gptq_int8_matmul.restype = i32
    lib.gptq_int8_matmul_grouped.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, vp, vp, i32,
                                             i64, vp]
    lib.gptq_int8_matmul_grouped.restype = i32
    lib.gptq_distill_loss_workspace_size.argtypes = [i64, i64]
    lib.gptq_distill_loss_workspace_size.restype = sz
    lib.gptq_distill_loss.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, ctypes.c_float, i32, vp, vp, vp, i64, vp, sz, vp]
    lib.gptq_distill_loss.restype = i32
    lib.gptq_launch_timing.argtypes = [i32]
    lib.gptq_launch_timing.restype = i32
    lib.gptq_launch_timing_read.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64),
                                            ctypes.POINTER(ctypes.c_double)]
    lib.gptq_launch_timing_read.restype = i32
    lib.gptq_status_string.argtypes = [i32]
    lib.gptq_status_string.restype = ctypes.c_char_p
    lib.gptq_version.argtypes = []
    lib.gptq_version.restype = ctypes.c_char_p
    _LIB = lib
    return lib


_CALLS = None


class _NoCalls:
    """In the place of the extension where there is none: leaves every call to the binding's own path."""
    int8_quantize = int8_matmul = int8_matmul_grouped = distill_loss = staticmethod(lambda *args: None)


def _load_calls(path: str):
    """The extension at ``path``, if it was built for this torch (its functions take tensors apart)."""
    import importlib.machinery
    import importlib.util
    torch = _torch()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with __graft_entry__.build() "
                          "(python -m post_weight_quantization_02_amd._build)")
    loader = importlib.machinery.ExtensionFileLoader("_calls", path)
    calls = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
    loader.exec_module(calls)
    here = f"{torch.__version__} {torch.version.git_version}"
    if calls.torch_version != here:
        raise ImportError(f"{path} was built for torch {calls.torch_version}, this is {here}")
    lib = library()
    names = ("gptq_int8_quantize", "gptq_int8_matmul_workspace_size", "gptq_int8_matmul", "gptq_int8_matmul_grouped",
             "gptq_distill_loss_workspace_size", "gptq_distill_loss")
    calls.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names}, torch._C._get_tracing_state,
               torch.autograd.forward_ad, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    return calls


def _calls():
    """The extension that does the ordinary forms of some calls in one step (csrc/calls.cpp):
    its functions return None where a call is not such a one.  Built with the library; where it
    is missing or another torch's, that is said once and the binding's own path takes all calls."""
    global _CALLS
    if _CALLS is None:
        try:
            _CALLS = _load_calls(os.path.join(_HERE, "_lib", "_calls.so"))
        except ImportError as e:
            import warnings
            _CALLS = _NoCalls
            warnings.warn(f"the int8 and distillation calls take 3 to 7 us more of the host each: {e}", RuntimeWarning, stacklevel=3)
    return _CALLS


def gptq_status_string(status: int) -> str:
    return library().gptq_status_string(int(status)).decode()


def gptq_version() -> str:
    return library().gptq_version().decode()


# --------------------------------------------------------------------------- helpers
def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream, *tensors) -> Optional[int]:
    """The HIP stream handle to launch on.

    With no stream, or torch's current stream, nothing else happens.  With any
    other stream, that stream first waits for the work already queued on the
    current stream (the producer of the inputs, in torch's usual stream
    semantics), and every tensor the call touches (inputs, outputs and the
    workspace) is recorded as in use on that stream, so the caching allocator
    does not hand its memory out again before the launched kernels are done."""
    torch = _torch()
    cur = torch.cuda.current_stream()
    if stream is None or stream == cur:
        return cur.cuda_stream
    stream.wait_stream(cur)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return GPTQ_F16
    if t.dtype == torch.float32:
        return GPTQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _rowmajor(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def _workspace(nbytes: int, device, ws=None):
    torch = _torch()
    if ws is not None:
        return ws
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _check(status: int, where: str):
    if status != 0:
        raise GPTQError(status, where)


_ELEM = {}


def _elem_code(t, name) -> int:
    """Element type of the calls that take fp32, fp16 and bf16."""
    if not _ELEM:
        torch = _torch()
        _ELEM.update({torch.float32: GPTQ_F32, torch.float16: GPTQ_F16, torch.bfloat16: GPTQ_BF16})
    code = _ELEM.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _expect(t, name, shape, dtypes, device):
    """A tensor of that shape and one of those dtypes on that device, its last
    dimension contiguous and its rows not overlapping."""
    if t.shape == shape and t.dtype in dtypes and t.device == device and t.is_contiguous():
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    if len(shape) == 2 and shape[0] > 1 and t.stride(0) < shape[1]:
        raise ValueError(f"{name} has overlapping rows")


def _end(t, start) -> int:
    """Address behind the last element of a tensor that starts at ``start``."""
    if t.is_contiguous():
        return start + t.numel() * t.element_size()
    return start + (sum((d - 1) * st for d, st in zip(t.shape, t.stride())) + 1) * t.element_size()


def _share_rows(t, o) -> bool:
    """Whether two tensors whose address ranges meet share an element.  Rows of one pitch are
    told apart by their columns; of other layouts the ranges alone are looked at."""
    def rows(v):             # number of rows, bytes of a row, bytes from row to row
        z = v.element_size()
        if v.dim() == 2 and v.shape[0] > 1 and v.stride(1) == 1:
            return v.shape[0], v.shape[1] * z, v.stride(0) * z
        return (1, v.numel() * z, 0) if v.is_contiguous() else None

    a, b = rows(t), rows(o)
    if a is None or b is None or (a[2] and b[2] and a[2] != b[2]):
        return True
    pitch = max(a[2], b[2])
    if pitch == 0 or a[1] > pitch or b[1] > pitch:
        return True
    down, right = divmod(o.data_ptr() - t.data_ptr(), pitch)      # o's row 0 against t's
    return (right < a[1] and down < a[0] and down + b[0] > 0 or
            right + b[1] > pitch and down + 1 < a[0] and down + 1 + b[0] > 0)


def _apart(t, name, *others):
    """An output given by the caller shares no memory with the other tensors of the call."""
    lo = t.data_ptr()
    hi = _end(t, lo)
    for o in others:
        if o is not None:
            a = o.data_ptr()
            if a < hi and (a >= lo or _end(o, a) > lo) and o.numel() > 0 and t.numel() > 0 and _share_rows(t, o):
                raise ValueError(f"{name} overlaps another tensor of the call")


_AUTOGRAD = None


def _forward_only(torch, where, *tensors):
    """Refuses what autograd or a trace would lose without a word: the calls run outside torch."""
    global _AUTOGRAD
    if _AUTOGRAD is None:
        _AUTOGRAD = torch._C._get_tracing_state, torch.autograd.forward_ad
    tracing, forward = _AUTOGRAD
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{where} has no backward pass: detach its inputs or call it under torch.no_grad()")
    if tracing() is not None:
        raise RuntimeError(f"{where} cannot be traced: its kernels run outside torch's operators")
    if forward._current_level >= 0:
        for t in tensors:
            if t is not None and forward.unpack_dual(t).tangent is not None:
                raise ValueError(f"{where} has no forward-mode derivative: call it on the primals")


def _launch(torch, device, stream, fn, args, tensors, where):
    """fn(*args, stream handle) on ``device``: on its current stream, or on ``stream``,
    which has to belong to it (ordered as in _stream)."""
    index = device.index
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _launch(torch, device, stream, fn, args, tensors, where)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)     # current_stream() without the Python object
    elif stream.device != device:
        raise ValueError(f"{where}: the stream belongs to {stream.device}, the tensors to {device}")
    else:
        handle = _stream(stream, *tensors)
    status = fn(*args, handle)
    if status != 0:
        raise GPTQError(status, where)


def _pitch(t) -> int:
    """Leading dimension: the row stride, also of a matrix of one row or none."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _ws_ptr(torch, nbytes: int, device, ws, *inputs):
    """(tensor, address, bytes) of a workspace; a given one shares no memory with the inputs."""
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return ws, ws.data_ptr(), nbytes
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {device}")
    _apart(ws, "ws", *inputs)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


# --------------------------------------------------------------------------- C names
def gptq_hessian_accumulate_workspace_size(d_col: int, n_rows: int, x_dtype: int) -> int:
    return int(library().gptq_hessian_accumulate_workspace_size(d_col, n_rows, x_dtype))


def gptq_prepare_hinv_workspace_size(d_col: int) -> int:
    return int(library().gptq_prepare_hinv_workspace_size(d_col))


def gptq_quantize_layer_workspace_size(d_row: int, d_col: int, block_size: int) -> int:
    return int(library().gptq_quantize_layer_workspace_size(d_row, d_col, block_size))


def gptq_hessian_accumulate(H, X, ws=None, stream=None):
    """H += 2 X^T X on the device (H [d x d] fp32, X [n x d] fp16/fp32 row-major)."""
    _rowmajor(X, "X")
    d = H.shape[0]
    n = X.shape[0]
    code = _dtype_code(X)
    need = gptq_hessian_accumulate_workspace_size(d, n, code)
    ws = _workspace(need, X.device, ws)
    st = library().gptq_hessian_accumulate(H.data_ptr(), d, X.data_ptr(), code, n, X.stride(0),
                                           ws.data_ptr(), ws.numel(), _stream(stream, H, X, ws))
    _check(st, "gptq_hessian_accumulate")
    return H


def gptq_prepare_hinv(H, percdamp: float = 0.01, U=None, lam=None, info=None, ws=None,
                      stream=None):
    """Damping and U (upper, U^T U = (H + lambda I)^-1).  Returns (U, lambda, info) as
    device tensors; ``info`` is nonzero if the damped H was not positive definite."""
    torch = _torch()
    d = H.shape[0]
    dev = H.device
    U = U if U is not None else torch.empty(d, d, dtype=torch.float32, device=dev)
    lam = lam if lam is not None else torch.empty(1, dtype=torch.float32, device=dev)
    info = info if info is not None else torch.empty(1, dtype=torch.int32, device=dev)
    ws = _workspace(gptq_prepare_hinv_workspace_size(d), dev, ws)
    st = library().gptq_prepare_hinv(H.data_ptr(), d, float(percdamp), U.data_ptr(),
                                     lam.data_ptr(), info.data_ptr(), ws.data_ptr(), ws.numel(),
                                     _stream(stream, H, U, lam, info, ws))
    _check(st, "gptq_prepare_hinv")
    return U, lam, info


def gptq_quantize_layer(W0, U, lam=None, bits: int = 4, group_size: int = 0,
                        block_size: int = 128, codes=None, scales=None, zeros=None,
                        out_err=None, ws=None, stream=None):
    """The lazy-batch loop.  Returns (codes uint8, scales fp32, zeros int32, err fp64)."""
    torch = _torch()
    _rowmajor(W0, "W0")
    d_row, d_col = W0.shape
    dev = W0.device
    ng = -(-d_col // group_size) if group_size else 1
    codes = codes if codes is not None else torch.empty(d_row, d_col, dtype=torch.uint8, device=dev)
    scales = scales if scales is not None else torch.empty(d_row, ng, dtype=torch.float32, device=dev)
    zeros = zeros if zeros is not None else torch.empty(d_row, ng, dtype=torch.int32, device=dev)
    out_err = out_err if out_err is not None else torch.empty(1, dtype=torch.float64, device=dev)
    ws = _workspace(gptq_quantize_layer_workspace_size(d_row, d_col, block_size), dev, ws)
    st = library().gptq_quantize_layer(W0.data_ptr(), _dtype_code(W0), d_row, d_col, W0.stride(0),
                                       U.data_ptr(), _ptr(lam), int(bits), int(group_size),
                                       int(block_size), codes.data_ptr(), scales.data_ptr(),
                                       zeros.data_ptr(), out_err.data_ptr(), ws.data_ptr(),
                                       ws.numel(), _stream(stream, W0, U, lam, codes, scales, zeros,
                                                           out_err, ws))
    _check(st, "gptq_quantize_layer")
    return codes, scales, zeros, out_err


def gptq_quantize_layer_noalloc(W0, U, lam=None, bits: int = 4, group_size: int = 0,
                                block_size: int = 128, codes=None, scales=None, zeros=None,
                                out_err=None, stream=None):
    """gptq_quantize_layer without a workspace: the library's fixed per-device
    array (GPTQ_NOALLOC_SCRATCH_BYTES) serves as one.  Pass every output to keep
    the call free of allocations (e.g. under graph capture).  Calls that may
    overlap on one device race on that array."""
    torch = _torch()
    _rowmajor(W0, "W0")
    d_row, d_col = W0.shape
    dev = W0.device
    ng = -(-d_col // group_size) if group_size else 1
    codes = codes if codes is not None else torch.empty(d_row, d_col, dtype=torch.uint8, device=dev)
    scales = scales if scales is not None else torch.empty(d_row, ng, dtype=torch.float32, device=dev)
    zeros = zeros if zeros is not None else torch.empty(d_row, ng, dtype=torch.int32, device=dev)
    out_err = out_err if out_err is not None else torch.empty(1, dtype=torch.float64, device=dev)
    st = library().gptq_quantize_layer_noalloc(W0.data_ptr(), _dtype_code(W0), d_row, d_col, W0.stride(0),
                                               U.data_ptr(), _ptr(lam), int(bits), int(group_size),
                                               int(block_size), codes.data_ptr(), scales.data_ptr(),
                                               zeros.data_ptr(), out_err.data_ptr(),
                                               _stream(stream, W0, U, lam, codes, scales, zeros, out_err))
    _check(st, "gptq_quantize_layer_noalloc")
    return codes, scales, zeros, out_err


def gptq_act_order_perm(H, perm=None, stream=None):
    """Act-order quantization order: int32 [d] with perm[i] the column quantized at
    position i (descending diag(H), equal diagonals in ascending index order)."""
    torch = _torch()
    d = H.shape[0]
    perm = perm if perm is not None else torch.empty(d, dtype=torch.int32, device=H.device)
    st = library().gptq_act_order_perm(H.data_ptr(), d, perm.data_ptr(), _stream(stream, H, perm))
    _check(st, "gptq_act_order_perm")
    return perm


def gptq_prepare_hinv_perm(H, perm, percdamp: float = 0.01, U=None, lam=None, info=None,
                           ws=None, stream=None):
    """gptq_prepare_hinv for H with rows and columns in the order ``perm``; U is in
    that order.  Returns (U, lambda, info)."""
    torch = _torch()
    d = H.shape[0]
    dev = H.device
    U = U if U is not None else torch.empty(d, d, dtype=torch.float32, device=dev)
    lam = lam if lam is not None else torch.empty(1, dtype=torch.float32, device=dev)
    info = info if info is not None else torch.empty(1, dtype=torch.int32, device=dev)
    ws = _workspace(gptq_prepare_hinv_workspace_size(d), dev, ws)
    st = library().gptq_prepare_hinv_perm(H.data_ptr(), d, perm.data_ptr(), float(percdamp),
                                          U.data_ptr(), lam.data_ptr(), info.data_ptr(),
                                          ws.data_ptr(), ws.numel(),
                                          _stream(stream, H, perm, U, lam, info, ws))
    _check(st, "gptq_prepare_hinv_perm")
    return U, lam, info


def gptq_quantize_layer_perm(W0, U, lam, perm, bits: int = 4, group_size: int = 0,
                             block_size: int = 128, codes=None, scales=None, zeros=None,
                             g_idx=None, out_err=None, ws=None, stream=None):
    """The loop over the columns in the order ``perm`` (U from gptq_prepare_hinv_perm).
    Returns (codes in the original column order, scales, zeros, g_idx, err)."""
    torch = _torch()
    _rowmajor(W0, "W0")
    d_row, d_col = W0.shape
    dev = W0.device
    ng = -(-d_col // group_size) if group_size else 1
    codes = codes if codes is not None else torch.empty(d_row, d_col, dtype=torch.uint8, device=dev)
    scales = scales if scales is not None else torch.empty(d_row, ng, dtype=torch.float32, device=dev)
    zeros = zeros if zeros is not None else torch.empty(d_row, ng, dtype=torch.int32, device=dev)
    g_idx = g_idx if g_idx is not None else torch.empty(d_col, dtype=torch.int32, device=dev)
    out_err = out_err if out_err is not None else torch.empty(1, dtype=torch.float64, device=dev)
    ws = _workspace(gptq_quantize_layer_workspace_size(d_row, d_col, block_size), dev, ws)
    st = library().gptq_quantize_layer_perm(W0.data_ptr(), _dtype_code(W0), d_row, d_col,
                                            W0.stride(0), U.data_ptr(), _ptr(lam), perm.data_ptr(),
                                            int(bits), int(group_size), int(block_size),
                                            codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                            g_idx.data_ptr(), out_err.data_ptr(), ws.data_ptr(),
                                            ws.numel(), _stream(stream, W0, U, lam, perm, codes, scales,
                                                                zeros, g_idx, out_err, ws))
    _check(st, "gptq_quantize_layer_perm")
    return codes, scales, zeros, g_idx, out_err


def gptq_packed_words_per_row(d_col: int, bits: int) -> int:
    return int(library().gptq_packed_words_per_row(d_col, bits))


def gptq_pack_codes(codes, bits: int, perm=None, packed=None, stream=None):
    """Pack uint8 codes [d_row x d_col] into 32-bit words (position i holds column
    perm[i] when perm is given).  Returns the packed int32 tensor (bit patterns)."""
    torch = _torch()
    _rowmajor(codes, "codes")
    d_row, d_col = codes.shape
    words = gptq_packed_words_per_row(d_col, bits)
    packed = packed if packed is not None else torch.empty(d_row, words, dtype=torch.int32,
                                                             device=codes.device)
    st = library().gptq_pack_codes(codes.data_ptr(), d_row, d_col, codes.stride(0), int(bits),
                                   _ptr(perm), packed.data_ptr(), packed.stride(0),
                                   _stream(stream, codes, perm, packed))
    _check(st, "gptq_pack_codes")
    return packed


def gptq2d_quantize_workspace_size(m: int, n: int) -> int:
    return int(library().gptq2d_quantize_workspace_size(m, n))


def gptq2d_quantize(X, U_Q, U_P, bits: int, codes=None, scale=None, zero=None, out_err=None, ws=None,
                    stream=None):
    """Two-sided adaptive rounding of X [m x n] (fp16/fp32) with the upper factors
    U_Q [m x m] and U_P [n x n].  Returns (codes uint8, scale fp32 [1], zero int32 [1],
    err fp64 [1])."""
    torch = _torch()
    _rowmajor(X, "X")
    m, n = X.shape
    dev = X.device
    codes = codes if codes is not None else torch.empty(m, n, dtype=torch.uint8, device=dev)
    scale = scale if scale is not None else torch.empty(1, dtype=torch.float32, device=dev)
    zero = zero if zero is not None else torch.empty(1, dtype=torch.int32, device=dev)
    out_err = out_err if out_err is not None else torch.empty(1, dtype=torch.float64, device=dev)
    ws = _workspace(gptq2d_quantize_workspace_size(m, n), dev, ws)
    st = library().gptq2d_quantize(X.data_ptr(), _dtype_code(X), m, n, X.stride(0), U_Q.data_ptr(),
                                   U_P.data_ptr(), int(bits), codes.data_ptr(), codes.stride(0), scale.data_ptr(),
                                   zero.data_ptr(), out_err.data_ptr(), ws.data_ptr(), ws.numel(),
                                   _stream(stream, X, U_Q, U_P, codes, scale, zero, out_err, ws))
    _check(st, "gptq2d_quantize")
    return codes, scale, zero, out_err


def gptq_dequantize(codes, scales, zeros, group_size: int, g_idx=None, out=None, out_dtype=None,
                    stream=None):
    """What [d_row x d_col] = scales * (codes - zeros) per group (through g_idx if
    given), fp32 unless out / out_dtype say fp16."""
    torch = _torch()
    _rowmajor(codes, "codes")
    d_row, d_col = codes.shape
    if out is None:
        out = torch.empty(d_row, d_col, dtype=out_dtype or torch.float32, device=codes.device)
    _rowmajor(out, "out")
    st = library().gptq_dequantize(codes.data_ptr(), d_row, d_col, codes.stride(0), scales.data_ptr(),
                                   zeros.data_ptr(), int(group_size), _ptr(g_idx), out.data_ptr(),
                                   _dtype_code(out), out.stride(0),
                                   _stream(stream, codes, scales, zeros, g_idx, out))
    _check(st, "gptq_dequantize")
    return out


def gptq_dequant_matmul(packed, bits: int, scales, zeros, group_size: int, X, d_col: int,
                        perm=None, Y=None, stream=None):
    """Y [m x d_row] fp32 = X What^T from packed codes (1 <= m <= 8)."""
    torch = _torch()
    _rowmajor(X, "X")
    d_row = packed.shape[0]
    m = X.shape[0]
    Y = Y if Y is not None else torch.empty(m, d_row, dtype=torch.float32, device=X.device)
    st = library().gptq_dequant_matmul(packed.data_ptr(), packed.stride(0), int(bits), scales.data_ptr(),
                                       zeros.data_ptr(), int(group_size), _ptr(perm), d_row, d_col,
                                       X.data_ptr(), _dtype_code(X), m, X.stride(0), Y.data_ptr(),
                                       Y.stride(0), _stream(stream, packed, scales, zeros, perm, X, Y))
    _check(st, "gptq_dequant_matmul")
    return Y


def gptq_fp8_quantize(X, block_rows: int = 1, codes=None, scales=None, stream=None):
    """e4m3 codes of X [m x k] (fp32, fp16 or bf16) with one power-of-two fp32 scale
    per row and 128 columns (``block_rows=1``, activations) or per 128 x 128 tile
    (``block_rows=128``, weights).  Returns (codes float8_e4m3fn [m x k], scales):
    scales [ceil(k/128) x m], or [ceil(m/128) x ceil(k/128)] for tiles.  The codes
    made here have rows a multiple of 128 bytes apart."""
    torch = _torch()
    _rowmajor(X, "X")
    _forward_only(torch, "gptq_fp8_quantize", X)
    code = _elem_code(X, "X")
    m, k = X.shape
    dev = X.device
    kb = (k + 127) // 128
    rows, cols = (kb, m) if block_rows == 1 else ((m + 127) // 128, kb)
    if codes is None:
        ldc = kb * 128
        codes = torch.empty_strided((m, k), (ldc, 1), dtype=torch.float8_e4m3fn, device=dev)
    else:
        _expect(codes, "codes", (m, k), (torch.float8_e4m3fn, torch.uint8), dev)
        _apart(codes, "codes", X, scales)
        ldc = _pitch(codes)
    if scales is None:
        scales, lds = torch.empty(rows, cols, dtype=torch.float32, device=dev), max(cols, 1)
    else:
        _expect(scales, "scales", (rows, cols), (torch.float32,), dev)
        _apart(scales, "scales", X)
        lds = _pitch(scales)
    _launch(torch, dev, stream, library().gptq_fp8_quantize,
            (X.data_ptr(), code, m, k, X.stride(0) if m > 1 else k, int(block_rows), codes.data_ptr(), max(ldc, k),
             scales.data_ptr(), lds), (X, codes, scales), "gptq_fp8_quantize")
    return codes, scales


def gptq_fp8_matmul_workspace_size(m: int, n: int, k: int) -> int:
    return int(library().gptq_fp8_matmul_workspace_size(m, n, k))


def gptq_fp8_matmul(x_codes, x_scales, w_codes, w_scales, bias=None, Y=None, out_dtype=None, ws=None,
                    stream=None):
    """Y [m x n] = X W^T (+ bias) from e4m3 codes (float8_e4m3fn or uint8 bit patterns)
    x_codes [m x k], w_codes [n x k] and fp32 scales x_scales [ceil(k/128) x m],
    w_scales [ceil(n/128) x ceil(k/128)], rounded once to Y's dtype (``out_dtype``: fp32,
    fp16 or bf16; fp32 if not given).  bias: n values of that dtype.  fp32 outputs are
    fp32 sums.  fp16 and bf16 outputs of more than a few rows take the 8-bit matrix
    instruction's sum inside each block of 128 columns, off by up to 7 * 2^-13 sum |x w|
    before the rounding (1e-5 to 5e-5 of Y's norm on random codes)."""
    torch = _torch()
    _rowmajor(x_codes, "x_codes")
    m, k = x_codes.shape
    dev = x_codes.device
    if w_codes.dim() != 2:
        raise ValueError("w_codes must be a 2-D tensor")
    n, kb = w_codes.shape[0], (k + 127) // 128
    nb = (n + 127) // 128
    fp8, f32 = (torch.float8_e4m3fn, torch.uint8), torch.float32
    _expect(x_codes, "x_codes", (m, k), fp8, dev)
    _expect(w_codes, "w_codes", (n, k), fp8, dev)
    _expect(x_scales, "x_scales", (kb, m), (f32,), dev)
    _expect(w_scales, "w_scales", (nb, kb), (f32,), dev)
    _forward_only(torch, "gptq_fp8_matmul", x_scales, w_scales, bias, Y)
    if Y is None:
        Y, ldy = torch.empty(m, n, dtype=out_dtype or f32, device=dev), n
    else:
        _expect(Y, "Y", (m, n), (out_dtype or Y.dtype,), dev)
        _apart(Y, "Y", x_codes, x_scales, w_codes, w_scales, bias, ws)
        ldy = _pitch(Y)
    y_code = _elem_code(Y, "Y")
    b_ptr = None
    if bias is not None:
        _expect(bias, "bias", (n,), (Y.dtype,), dev)
        b_ptr = bias.data_ptr()
    lib = library()
    need = lib.gptq_fp8_matmul_workspace_size(m, n, k)
    ws_ptr, ws_bytes = None, 0
    if need > 0 or ws is not None:
        ws, ws_ptr, ws_bytes = _ws_ptr(torch, need, dev, ws, x_codes, x_scales, w_codes, w_scales, bias)
    _launch(torch, dev, stream, lib.gptq_fp8_matmul,
            (x_codes.data_ptr(), x_codes.stride(0) if m > 1 else k, x_scales.data_ptr(),
             x_scales.stride(0) if kb > 1 else max(m, 1), w_codes.data_ptr(), w_codes.stride(0) if n > 1 else k,
             w_scales.data_ptr(), w_scales.stride(0) if nb > 1 else kb, m, n, k, b_ptr, Y.data_ptr(), y_code, ldy,
             ws_ptr, ws_bytes), (x_codes, x_scales, w_codes, w_scales, bias, Y, ws), "gptq_fp8_matmul")
    return Y


def gptq_token_logprobs_workspace_size(n: int, v: int, top_k: int = 0) -> int:
    return int(library().gptq_token_logprobs_workspace_size(n, v, top_k))


def gptq_token_logprobs(logits, tokens, top_k: int = 0, logprobs=None, entropy=None, top_ids=None,
                        top_logprobs=None, ws=None, stream=None):
    """Per row of logits [n x v] (fp32, fp16 or bf16): the log probability of
    tokens[i] (int64 [n]; 0 where the token is negative: none there), the entropy in
    nats, and the top_k <= 64 most probable tokens (equal logits: lower index first).
    Returns (logprobs [n], entropy [n], top_ids int32 [n x top_k], top_logprobs
    [n x top_k]), fp32 but for the ids."""
    torch = _torch()
    _rowmajor(logits, "logits")
    _forward_only(torch, "gptq_token_logprobs", logits)
    code = _elem_code(logits, "logits")
    n, v = logits.shape
    dev = logits.device
    top_k = int(top_k)
    f32, cols = torch.float32, max(top_k, 0)
    _expect(tokens, "tokens", (n,), (torch.int64,), dev)
    contiguous = [("tokens", tokens)]
    if logprobs is None:
        logprobs = torch.empty(n, dtype=f32, device=dev)
    else:
        _expect(logprobs, "logprobs", (n,), (f32,), dev)
        contiguous.append(("logprobs", logprobs))
    if entropy is None:
        entropy = torch.empty(n, dtype=f32, device=dev)
    else:
        _expect(entropy, "entropy", (n,), (f32,), dev)
        contiguous.append(("entropy", entropy))
    if top_ids is None:
        top_ids = torch.empty(n, cols, dtype=torch.int32, device=dev)
    else:
        _expect(top_ids, "top_ids", (n, cols), (torch.int32,), dev)
        contiguous.append(("top_ids", top_ids))
    if top_logprobs is None:
        top_logprobs = torch.empty(n, cols, dtype=f32, device=dev)
    else:
        _expect(top_logprobs, "top_logprobs", (n, cols), (f32,), dev)
        contiguous.append(("top_logprobs", top_logprobs))
    for i, (name, t) in enumerate(contiguous):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if i > 0:
            _apart(t, name, logits, ws, *(o for _, o in contiguous[:i]))
    lib = library()
    need = lib.gptq_token_logprobs_workspace_size(n, v, top_k)
    ws_ptr, ws_bytes = None, 0
    if need > 0 or ws is not None:
        ws, ws_ptr, ws_bytes = _ws_ptr(torch, need, dev, ws, logits, tokens)
    _launch(torch, dev, stream, lib.gptq_token_logprobs,
            (logits.data_ptr(), code, n, v, logits.stride(0) if n > 1 else v, tokens.data_ptr(), top_k,
             logprobs.data_ptr(), entropy.data_ptr(), top_ids.data_ptr(), top_logprobs.data_ptr(), ws_ptr, ws_bytes),
            (logits, tokens, logprobs, entropy, top_ids, top_logprobs, ws), "gptq_token_logprobs")
    return logprobs, entropy, top_ids, top_logprobs


def gptq_int8_quantize(X, codes=None, scales=None, stream=None):
    """int8 codes of X [m x k] (fp32, fp16 or bf16) with one fp32 scale per row: a row is a
    token's activations or a channel's weights.  Returns (codes int8 [m x k], scales [m]),
    X ~ scales[:, None] * codes.  A row with a NaN or an infinity has scale NaN.  The codes
    made here have rows a multiple of 128 bytes apart."""
    if codes is None and scales is None and stream is None:
        done = (_CALLS or _calls()).int8_quantize(X)
        if done is not None:
            return done
    torch = _torch()
    _rowmajor(X, "X")
    _forward_only(torch, "gptq_int8_quantize", X)
    code = _elem_code(X, "X")
    m, k = X.shape
    dev = X.device
    if codes is None:
        ldc = (k + 127) // 128 * 128
        codes = torch.empty_strided((m, k), (ldc, 1), dtype=torch.int8, device=dev)
    else:
        _expect(codes, "codes", (m, k), (torch.int8,), dev)
        _apart(codes, "codes", X, scales)
        ldc = _pitch(codes)
    if scales is None:
        scales = torch.empty(m, dtype=torch.float32, device=dev)
    else:
        _expect(scales, "scales", (m,), (torch.float32,), dev)
        _apart(scales, "scales", X)
    _launch(torch, dev, stream, library().gptq_int8_quantize,
            (X.data_ptr(), code, m, k, X.stride(0) if m > 1 else k, codes.data_ptr(), max(ldc, k), scales.data_ptr()),
            (X, codes, scales), "gptq_int8_quantize")
    return codes, scales


def gptq_int8_matmul_workspace_size(m: int, n: int, k: int) -> int:
    return int(library().gptq_int8_matmul_workspace_size(m, n, k))


def gptq_int8_matmul(x_codes, x_scales, w_codes, w_scales, bias=None, Y=None, out_dtype=None, ws=None, stream=None):
    """Y [m x n] = X W^T (+ bias) from int8 codes x_codes [m x k], w_codes [n x k] (k < 2^17)
    and fp32 scales x_scales [m], w_scales [n], rounded once to Y's dtype (``out_dtype``: fp32,
    fp16 or bf16; fp32 if not given).  bias: n values of that dtype.  The sums are exact, so
    a row's result depends neither on the other rows nor on the layout."""
    if Y is None and ws is None and stream is None:
        done = (_CALLS or _calls()).int8_matmul(x_codes, x_scales, w_codes, w_scales, bias, out_dtype)
        if done is not None:
            return done
    torch = _torch()
    _rowmajor(x_codes, "x_codes")
    m, k = x_codes.shape
    dev = x_codes.device
    if w_codes.dim() != 2:
        raise ValueError("w_codes must be a 2-D tensor")
    n = w_codes.shape[0]
    i8, f32 = (torch.int8,), torch.float32
    _expect(x_codes, "x_codes", (m, k), i8, dev)
    _expect(w_codes, "w_codes", (n, k), i8, dev)
    _expect(x_scales, "x_scales", (m,), (f32,), dev)
    _expect(w_scales, "w_scales", (n,), (f32,), dev)
    _forward_only(torch, "gptq_int8_matmul", x_scales, w_scales, bias, Y)
    if Y is None:
        Y, ldy = torch.empty(m, n, dtype=out_dtype or f32, device=dev), n
    else:
        _expect(Y, "Y", (m, n), (out_dtype or Y.dtype,), dev)
        _apart(Y, "Y", x_codes, x_scales, w_codes, w_scales, bias, ws)
        ldy = _pitch(Y)
    y_code = _elem_code(Y, "Y")
    b_ptr = None
    if bias is not None:
        _expect(bias, "bias", (n,), (Y.dtype,), dev)
        b_ptr = bias.data_ptr()
    lib = library()
    need = lib.gptq_int8_matmul_workspace_size(m, n, k)
    ws_ptr, ws_bytes = None, 0
    if need > 0 or ws is not None:
        ws, ws_ptr, ws_bytes = _ws_ptr(torch, need, dev, ws, x_codes, x_scales, w_codes, w_scales, bias)
    _launch(torch, dev, stream, lib.gptq_int8_matmul,
            (x_codes.data_ptr(), x_codes.stride(0) if m > 1 else k, x_scales.data_ptr(), w_codes.data_ptr(),
             w_codes.stride(0) if n > 1 else k, w_scales.data_ptr(), m, n, k, b_ptr, Y.data_ptr(), y_code, ldy, ws_ptr,
             ws_bytes), (x_codes, x_scales, w_codes, w_scales, bias, Y, ws), "gptq_int8_matmul")
    return Y


def gptq_int8_matmul_grouped(x_codes, x_scales, w_codes, w_scales, offsets, rows=None, bias=None, Y=None, out_dtype=None,
                             stream=None):
    """The product by expert: for positions i with offsets[e] <= i < offsets[e + 1] (offsets
    int32 [experts + 1] on the device, not decreasing) row i of Y is row rows[i] of X (int32,
    or row i without ``rows``) times the weights of expert e, w_codes [experts x n x k] and
    w_scales [experts x n], plus bias[e] (bias [experts x n] of Y's dtype).  Y has a row per
    position: as many as ``rows``, or x_codes, has.  Rows of Y that belong to no expert are left
    as they are (in a tensor made here: undefined); a row of X out of range gives NaN."""
    if Y is None and stream is None:
        done = (_CALLS or _calls()).int8_matmul_grouped(x_codes, x_scales, w_codes, w_scales, offsets, rows, bias, out_dtype)
        if done is not None:
            return done
    torch = _torch()
    _rowmajor(x_codes, "x_codes")
    rows_x, k = x_codes.shape
    dev = x_codes.device
    if w_codes.dim() != 3:
        raise ValueError("w_codes must be a 3-D tensor")
    experts, n = w_codes.shape[:2]
    i8, f32, i32 = (torch.int8,), torch.float32, (torch.int32,)
    _expect(x_codes, "x_codes", (rows_x, k), i8, dev)
    _expect(w_codes, "w_codes", (experts, n, k), i8, dev)
    ld_w = w_codes.stride(1) if n > 1 else k
    stride_w = w_codes.stride(0) if experts > 1 else n * ld_w
    if ld_w < k or stride_w < n * ld_w:
        raise ValueError("w_codes has overlapping rows")
    _expect(x_scales, "x_scales", (rows_x,), (f32,), dev)
    _expect(w_scales, "w_scales", (experts, n), (f32,), dev)
    _expect(offsets, "offsets", (experts + 1,), i32, dev)
    m, r_ptr = rows_x, None
    if rows is not None:
        if rows.dim() != 1:
            raise ValueError("rows must be a 1-D tensor")
        m = rows.shape[0]
        _expect(rows, "rows", (m,), i32, dev)
        r_ptr = rows.data_ptr()
    _forward_only(torch, "gptq_int8_matmul_grouped", x_scales, w_scales, bias, Y)
    if Y is None:
        Y, ldy = torch.empty(m, n, dtype=out_dtype or f32, device=dev), n
    else:
        _expect(Y, "Y", (m, n), (out_dtype or Y.dtype,), dev)
        _apart(Y, "Y", x_codes, x_scales, w_codes, w_scales, offsets, rows, bias)
        ldy = _pitch(Y)
    y_code = _elem_code(Y, "Y")
    b_ptr = None
    if bias is not None:
        _expect(bias, "bias", (experts, n), (Y.dtype,), dev)
        b_ptr = bias.data_ptr()
    for t, name in ((w_scales, "w_scales"), (bias, "bias")):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _launch(torch, dev, stream, library().gptq_int8_matmul_grouped,
            (x_codes.data_ptr(), x_codes.stride(0) if rows_x > 1 else k, x_scales.data_ptr(), rows_x, r_ptr, m,
             offsets.data_ptr(), experts, w_codes.data_ptr(), ld_w, stride_w, w_scales.data_ptr(), n, k, b_ptr,
             Y.data_ptr(), y_code, ldy), (x_codes, x_scales, w_codes, w_scales, offsets, rows, bias, Y),
            "gptq_int8_matmul_grouped")
    return Y


def gptq_distill_loss_workspace_size(n: int, v: int) -> int:
    return int(library().gptq_distill_loss_workspace_size(n, v))


def gptq_distill_loss(logits, ids, logprobs, temperature: float = 1.0, tail: bool = False, weights=None,
                      want_grad: bool = False, loss=None, grad=None, ws=None, stream=None):
    """Per row of logits [n x v] (fp32, fp16 or bf16) the divergence from a teacher's top
    tokens, ids int32 [n x top] (negative: no entry) and logprobs fp32 [n x top] as
    gptq_token_logprobs gives them: sum_j q_j (log q_j - log p(ids_j)), p = softmax(logits /
    temperature).  q is softmax(logprobs / temperature); with ``tail`` exp(logprobs), log
    probabilities at that temperature already, and, for all other tokens together, what is
    missing to 1.  Returns (loss fp32 [n], grad): grad, of
    logits' shape and dtype, is the loss's gradient times weights (fp32 [n]; 1 if not given)
    where ``want_grad`` or a tensor for it is given, else None.  Rows without entries have loss
    and gradient 0, rows of weight 0 gradient 0.  Rounding can leave rows of models that agree
    a loss just below 0.  pipeline.distill_loss is the same for
    autograd."""
    if loss is None and grad is None and ws is None and stream is None:
        done = (_CALLS or _calls()).distill_loss(logits, ids, logprobs, temperature, tail, weights, want_grad)
        if done is not None:
            return done
    torch = _torch()
    _rowmajor(logits, "logits")
    _forward_only(torch, "gptq_distill_loss", logits, logprobs, weights)
    code = _elem_code(logits, "logits")
    n, v = logits.shape
    dev = logits.device
    f32 = (torch.float32,)
    if ids.dim() != 2:
        raise ValueError("ids must be a 2-D tensor")
    top = ids.shape[1]
    _expect(ids, "ids", (n, top), (torch.int32,), dev)
    _expect(logprobs, "logprobs", (n, top), f32, dev)
    if not (ids.is_contiguous() and logprobs.is_contiguous()):
        raise ValueError("ids and logprobs must be contiguous")
    w_ptr = None
    if weights is not None:
        _expect(weights, "weights", (n,), f32, dev)
        w_ptr = weights.data_ptr()
    if loss is None:
        loss = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _expect(loss, "loss", (n,), f32, dev)
        _apart(loss, "loss", logits, ids, logprobs, weights, grad, ws)
    g_ptr, ldg = None, v
    if grad is not None:
        _expect(grad, "grad", (n, v), (logits.dtype,), dev)
        _apart(grad, "grad", logits, ids, logprobs, weights, ws)
        g_ptr, ldg = grad.data_ptr(), _pitch(grad)
    elif want_grad:
        grad = torch.empty(n, v, dtype=logits.dtype, device=dev)
        g_ptr = grad.data_ptr()
    lib = library()
    need = lib.gptq_distill_loss_workspace_size(n, v)
    ws_ptr, ws_bytes = None, 0
    if need > 0 or ws is not None:
        ws, ws_ptr, ws_bytes = _ws_ptr(torch, need, dev, ws, logits, ids, logprobs, weights)
    _launch(torch, dev, stream, lib.gptq_distill_loss,
            (logits.data_ptr(), code, n, v, logits.stride(0) if n > 1 else v, ids.data_ptr(), logprobs.data_ptr(), top,
             float(temperature), 1 if tail else 0, w_ptr, loss.data_ptr(), g_ptr, ldg, ws_ptr, ws_bytes),
            (logits, ids, logprobs, weights, loss, grad, ws), "gptq_distill_loss")
    return loss, grad


def gptq_launch_timing(enable: bool) -> None:
    """Switch per-launch timing of the loop's panel and product launches on or
    off for the calling thread (a measurement aid)."""
    _check(library().gptq_launch_timing(1 if enable else 0), "gptq_launch_timing")


def gptq_launch_timing_read(kind: int):
    """(milliseconds, launches, work) summed over the recorded launches of
    ``kind`` (TIMING_PANEL: work in bytes; TIMING_PRODUCT: work in flop), which
    are then forgotten.  Waits for the recorded events."""
    ms, n, work = ctypes.c_double(), ctypes.c_int64(), ctypes.c_double()
    _check(library().gptq_launch_timing_read(int(kind), ctypes.byref(ms), ctypes.byref(n), ctypes.byref(work)),
           "gptq_launch_timing_read")
    return ms.value, n.value, work.value


def quantize_layer(W0, x_chunks: Iterable, bits: int = 4, group_size: int = 0,
                   block_size: int = 128, percdamp: float = 0.01, act_order: bool = False,
                   stream=None):
    """All three calls for one layer (natural order, or act-order with
    ``act_order=True``); raises NotPositiveDefinite after synchronising if the
    damped Hessian could not be factored.  Returns a dict of device tensors."""
    torch = _torch()
    d_col = W0.shape[1]
    H = torch.zeros(d_col, d_col, dtype=torch.float32, device=W0.device)
    for xc in x_chunks:
        gptq_hessian_accumulate(H, xc, stream=stream)
    out = {"H": H}
    if act_order:
        perm = gptq_act_order_perm(H, stream=stream)
        U, lam, info = gptq_prepare_hinv_perm(H, perm, percdamp, stream=stream)
        codes, scales, zeros, g_idx, err = gptq_quantize_layer_perm(
            W0, U, lam, perm, bits, group_size, block_size, stream=stream)
        out.update(perm=perm, g_idx=g_idx)
    else:
        U, lam, info = gptq_prepare_hinv(H, percdamp, stream=stream)
        codes, scales, zeros, err = gptq_quantize_layer(W0, U, lam, bits, group_size, block_size,
                                                        stream=stream)
    (stream or torch.cuda.current_stream()).synchronize()
    if int(info.item()) != 0:
        raise NotPositiveDefinite(int(info.item()))
    out.update(U=U, codes=codes, scales=scales, zeros=zeros, err=err)
    out["lambda"] = lam
    return out
