"""Thin Python binding of the C ABI in include/awq.h (ctypes; argument marshalling only).

Every computation happens in the CUDA library: this module checks dtypes and
shapes, takes data pointers and the current CUDA stream from torch tensors, and
calls the entry point of the same name.  It raises if the library is missing:
there is no CPU fallback.

Results and scratch that a call allocates belong to the stream that it runs on (`stream`, or the current
one): before another stream uses a result it waits for that stream, and tells the allocator
(`Tensor.record_stream`), as for any tensor made there.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple, Optional, Tuple

import torch

from .build import LIB

AWQ_OK = 0
AWQ_OP_QUANTIZE_PACK, AWQ_OP_SCALE_SEARCH, AWQ_OP_GEMV, AWQ_OP_GEMM = 0, 1, 2, 3
STATUS_NAMES = {0: "AWQ_OK", 1: "AWQ_ERR_INVALID_ARG", 2: "AWQ_ERR_UNSUPPORTED", 3: "AWQ_ERR_WORKSPACE",
                4: "AWQ_ERR_CUDA", 5: "AWQ_ERR_TIMEOUT", 6: "AWQ_ERR_RANGE"}
(AWQ_ERR_INVALID_ARG, AWQ_ERR_UNSUPPORTED, AWQ_ERR_WORKSPACE, AWQ_ERR_CUDA, AWQ_ERR_TIMEOUT,
 AWQ_ERR_RANGE) = 1, 2, 3, 4, 5, 6

# Every symbol the header declares, with its ctypes signature.
_u16p = ctypes.c_void_p
_u32p = ctypes.c_void_p


class QuantConfig(ctypes.Structure):
    """awq_quant_config: the pages' quant_config {w_bit, q_group_size, zero_point}."""
    _fields_ = [("w_bit", ctypes.c_int32), ("q_group_size", ctypes.c_int32), ("zero_point", ctypes.c_int32)]


SIGNATURES = {
    "awq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "awq_abi_version": (ctypes.c_int32, []),
    "awq_quantize_pack": (ctypes.c_int, [_u16p, _u16p, ctypes.c_int32, ctypes.c_int32, QuantConfig,
                                         _u32p, _u16p, _u32p, ctypes.c_void_p]),
    "awq_scale_search": (ctypes.c_int, [_u16p, ctypes.c_int32, _u16p, ctypes.c_int32, ctypes.c_int32,
                                        QuantConfig, ctypes.c_int32, _u16p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "awq_scale_search_duo": (ctypes.c_int, [_u16p, ctypes.c_int32, _u16p, ctypes.c_int32, ctypes.c_int32,
                                            QuantConfig, ctypes.c_int32, _u16p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "awq_scale_search_noalloc": (ctypes.c_int, [_u16p, ctypes.c_int32, _u16p, ctypes.c_int32, ctypes.c_int32,
                                                QuantConfig, ctypes.c_int32, _u16p, ctypes.c_void_p,
                                                ctypes.c_void_p, ctypes.c_void_p]),
    "awq_fold_inverse_scale": (ctypes.c_int, [_u16p, _u16p, ctypes.c_int32, ctypes.c_int32, _u16p,
                                              ctypes.c_void_p]),
    "awq_linear_gemv": (ctypes.c_int, [_u16p, ctypes.c_int32, _u32p, _u16p, _u32p, ctypes.c_int32,
                                       ctypes.c_int32, QuantConfig, _u16p, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "awq_linear_gemm": (ctypes.c_int, [_u16p, ctypes.c_int32, _u32p, _u16p, _u32p, ctypes.c_int32,
                                       ctypes.c_int32, QuantConfig, _u16p, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "awq_apply_clip": (ctypes.c_int, [_u16p, ctypes.c_int32, _u16p, _u16p, ctypes.c_int32, ctypes.c_int32,
                                      QuantConfig, ctypes.c_int32, ctypes.c_int32, _u32p, _u16p, _u32p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p]),
    "awq_apply_clip_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                         QuantConfig, ctypes.c_int32]),
    "awq_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                              QuantConfig]),
    "awq_linear_fused": (ctypes.c_int, [_u16p, ctypes.c_int32, ctypes.c_int64, _u32p, _u16p, _u32p, ctypes.c_int32,
                                        ctypes.c_int32, QuantConfig, _u16p, ctypes.c_int32, ctypes.c_int32, _u16p,
                                        ctypes.c_int64, _u16p, ctypes.c_int64, ctypes.c_void_p]),
    "awq_linear_grouped": (ctypes.c_int, [_u16p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
                                          ctypes.c_void_p, ctypes.c_int32, _u32p, _u16p, _u32p, ctypes.c_int32,
                                          ctypes.c_int32, QuantConfig, _u16p, ctypes.c_int32, ctypes.c_int32, _u16p,
                                          ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "awq_linear_grouped_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    "awq_moe_route": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                     ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "awq_moe_route_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "awq_moe_combine": (ctypes.c_int, [_u16p, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _u16p, ctypes.c_int64, _u16p,
                                       ctypes.c_int64, ctypes.c_void_p]),
    "awq_device_error": (ctypes.c_int, [ctypes.c_void_p]),
    "awq_check_bounded_wait": (ctypes.c_int, [ctypes.c_void_p]),
}

_lib = None


def load_library(path: str = LIB) -> ctypes.CDLL:
    """Load libawq_b200.so and attach the signatures (raises if it is not built)."""
    global _lib
    if _lib is not None and path == LIB:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing "
                           "(run `python -m bit_weight_only_linear_b200.build`)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB:
        _lib = lib
    return lib


class AWQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = load_library().awq_status_string(status).decode()
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}: {msg}")


def _check(fn: str, status: int) -> None:
    if status != AWQ_OK:
        raise AWQError(fn, status)


def config(group_size: int = 128, zero_point: bool = True, w_bit: int = 4) -> QuantConfig:
    return QuantConfig(int(w_bit), int(group_size), 1 if zero_point else 0)


_CONFIGS = {}


def _config(group_size: int, zero_point: bool) -> QuantConfig:
    c = _CONFIGS.get((group_size, zero_point))
    if c is None:
        c = _CONFIGS[(group_size, zero_point)] = config(group_size, zero_point)
    return c


def _dev(t: Optional[torch.Tensor], name: str, dtypes) -> int:
    if t is None:
        return 0
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.data_ptr()


_F16 = (torch.float16,)
_W32 = (torch.int32, torch.uint32)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_CURRENT = contextlib.nullcontext()
_LEGACY = 1             # cudaStreamLegacy: the handle that names the default stream explicitly


def _on(stream, device):
    """Context in which the tensors made for a call belong to the stream that the call runs on.

    The allocator hands a freed block out again at once, for work that follows on the stream the block was
    made on.  A block made on the current stream and written on another could still be read, or be
    written, by work queued before."""
    if stream is None:
        return _CURRENT
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(0 if handle == _LEGACY else handle, device=device)
    return torch.cuda.stream(stream)


def packed_shapes(N: int, K: int, group_size: int, zero_point: bool):
    ng = K // group_size
    return (N, K // 8), (N, ng), ((N, (ng + 7) // 8) if zero_point else None)


def quantize_pack(W: torch.Tensor, s: Optional[torch.Tensor] = None, group_size: int = 128,
                  zero_point: bool = True, out=None, stream=None):
    """awq_quantize_pack: W [N][K] fp16, s [K] fp16 or None -> (qweight int32 [N][K/8],
    scales fp16 [N][K/G], qzeros int32 [N][ceil(K/G/8)] or None)."""
    N, K = W.shape
    qs, ss, zs = packed_shapes(N, K, group_size, zero_point)
    if out is None:
        with _on(stream, W.device):
            qweight = torch.empty(qs, dtype=torch.int32, device=W.device)
            scales = torch.empty(ss, dtype=torch.float16, device=W.device)
            qzeros = torch.empty(zs, dtype=torch.int32, device=W.device) if zero_point else None
    else:
        qweight, scales, qzeros = out
    st = load_library().awq_quantize_pack(
        _dev(W, "W", _F16), _dev(s, "s", _F16), N, K, config(group_size, zero_point),
        _dev(qweight, "qweight", _W32), _dev(scales, "scales", _F16), _dev(qzeros, "qzeros", _W32),
        _stream(stream))
    _check("awq_quantize_pack", st)
    return qweight, scales, qzeros


def fold_inverse_scale(X: torch.Tensor, s: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """awq_fold_inverse_scale: X' = fp16(X / s) per input channel."""
    M, K = X.shape
    if out is None:
        with _on(stream, X.device):
            out = torch.empty_like(X)
    st = load_library().awq_fold_inverse_scale(_dev(X, "X", _F16), _dev(s, "s", _F16), M, K,
                                               _dev(out, "out", _F16), _stream(stream))
    _check("awq_fold_inverse_scale", st)
    return out


def _linear(fn_name: str, X, qweight, scales, qzeros, group_size, zero_point, out, workspace, stream):
    M, K = X.shape
    N = qweight.shape[0]
    if qweight.shape[1] * 8 != K:
        raise ValueError("qweight must be [N][K/8]")
    if out is None:
        with _on(stream, X.device):
            out = torch.empty((M, N), dtype=torch.float16, device=X.device)
    ws_ptr, ws_bytes = 0, 0
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    fn = getattr(load_library(), fn_name)
    st = fn(_dev(X, "X", _F16), M, _dev(qweight, "qweight", _W32), _dev(scales, "scales", _F16),
            _dev(qzeros, "qzeros", _W32), N, K, _config(group_size, zero_point), _dev(out, "Y", _F16),
            ws_ptr, ws_bytes, _stream(stream))
    _check(fn_name, st)
    return out


def linear_gemv(X, qweight, scales, qzeros, group_size=128, zero_point=True, out=None, workspace=None,
                stream=None) -> torch.Tensor:
    """awq_linear_gemv: Y [M][N] = X [M][K] . deq(W)^T, decode form (M <= 8)."""
    return _linear("awq_linear_gemv", X, qweight, scales, qzeros, group_size, zero_point, out, workspace, stream)


_GEMM_WS = {}


def gemm_workspace(M: int, N: int, K: int, group_size: int = 128, zero_point: bool = True, device=None, stream=None):
    """A device workspace large enough for awq_linear_gemm at these sizes (the split-K
    partial sums), cached per device and stream (two streams' calls may overlap) and grown on
    demand; None when none is needed.  A capture gets one of its own from the graph's pool."""
    need = workspace_bytes(AWQ_OP_GEMM, M, N, K, group_size, zero_point)
    if need == 0:
        return None
    dev = device if isinstance(device, torch.device) else torch.device("cuda" if device is None else device)
    with _on(stream, dev):
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(need, dtype=torch.uint8, device=dev)
        index = torch.cuda.current_device() if dev.index is None else dev.index
        key = index, torch._C._cuda_getCurrentRawStream(index)
        ws = _GEMM_WS.get(key)
        if ws is None or ws.numel() < need:
            ws = _GEMM_WS[key] = torch.empty(need, dtype=torch.uint8, device=dev)
    return ws


def linear_gemm(X, qweight, scales, qzeros, group_size=128, zero_point=True, out=None, workspace=None,
                stream=None) -> torch.Tensor:
    """awq_linear_gemm: Y [M][N] = X [M][K] . deq(W)^T, tcgen05 tensor-core form (any M).  A
    batch too small to fill the GPU splits K over a workspace (the cached one of
    gemm_workspace() unless one is given)."""
    if workspace is None:
        workspace = gemm_workspace(X.shape[0], qweight.shape[0], X.shape[1], group_size, zero_point, X.device, stream)
    return _linear("awq_linear_gemm", X, qweight, scales, qzeros, group_size, zero_point, out, workspace, stream)


def workspace_bytes(op: int, M: int, N: int, K: int, group_size: int = 128, zero_point: bool = True) -> int:
    return int(load_library().awq_workspace_bytes(op, M, N, K, _config(group_size, zero_point)))


def _search_outputs(X: torch.Tensor, n_grid: int, stream):
    with _on(stream, X.device):
        return (torch.empty(X.shape[1], dtype=torch.float16, device=X.device),
                torch.empty(n_grid, dtype=torch.float64, device=X.device),
                torch.empty(1, dtype=torch.int32, device=X.device))


def scale_search(X: torch.Tensor, W: torch.Tensor, group_size: int = 128, zero_point: bool = True,
                 n_grid: int = 20, workspace: Optional[torch.Tensor] = None, stream=None, out=None,
                 duo_scaling: bool = False) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """awq_scale_search (awq_scale_search_duo with duo_scaling): returns (s* fp16 [K], losses
    fp64 [n_grid], best index int32 [1]), all on device (into `out` = (s, losses, best) when
    given)."""
    M, K = X.shape
    N = W.shape[0]
    if workspace is None:
        need = workspace_bytes(AWQ_OP_SCALE_SEARCH, M, N, K, group_size, zero_point)
        with _on(stream, X.device):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=X.device)
    s_out, losses, best = _search_outputs(X, n_grid, stream) if out is None else out
    name = "awq_scale_search_duo" if duo_scaling else "awq_scale_search"
    st = getattr(load_library(), name)(
        _dev(X, "X", _F16), M, _dev(W, "W", _F16), N, K, config(group_size, zero_point), n_grid,
        _dev(s_out, "s_out", _F16), losses.data_ptr(), best.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(name, st)
    return s_out, losses, best


def scale_search_noalloc(X: torch.Tensor, W: torch.Tensor, group_size: int = 128, zero_point: bool = True,
                         n_grid: int = 20, stream=None, out=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """awq_scale_search_noalloc: the scale search on the library's fixed scratch (for
    callers that cannot allocate device memory).  Returns (s*, losses, best index) on
    device, into `out` when given (otherwise torch allocates them here, for convenience)."""
    M, K = X.shape
    N = W.shape[0]
    s_out, losses, best = _search_outputs(X, n_grid, stream) if out is None else out
    st = load_library().awq_scale_search_noalloc(
        _dev(X, "X", _F16), M, _dev(W, "W", _F16), N, K, config(group_size, zero_point), n_grid,
        _dev(s_out, "s_out", _F16), losses.data_ptr(), best.data_ptr(), _stream(stream))
    _check("awq_scale_search_noalloc", st)
    return s_out, losses, best


def check_bounded_wait(stream=None) -> None:
    """awq_check_bounded_wait: enqueue a kernel whose wait can never complete (it gives up
    after the library's 2 s limit and flags a timeout, read by device_error())."""
    _check("awq_check_bounded_wait", load_library().awq_check_bounded_wait(_stream(stream)))


def device_error(stream=None) -> None:
    """Synchronise and raise AWQError if a bounded device wait ran out."""
    _check("awq_device_error", load_library().awq_device_error(_stream(stream)))


def apply_clip(X: torch.Tensor, W: torch.Tensor, s: Optional[torch.Tensor], group_size: int = 128,
               zero_point: bool = True, n_grid: int = 20, n_clip: int = 10, out=None,
               workspace: Optional[torch.Tensor] = None, stream=None, errors: bool = False):
    """awq_apply_clip: per-group clip ratio chosen by the group's output error, then the
    packed clipped weights.  Returns (qweight, scales, qzeros or None, clip index uint8
    [N][K/G]), plus the errors fp64 [N][K/G][n_clip] when `errors`."""
    M, K = X.shape
    N = W.shape[0]
    lib = load_library()
    if workspace is None:
        need = int(lib.awq_apply_clip_workspace_bytes(M, N, K, config(group_size, zero_point), n_clip))
        with _on(stream, X.device):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=X.device)
    qs, ss, zs = packed_shapes(N, K, group_size, zero_point)
    with _on(stream, W.device):
        if out is None:
            qweight = torch.empty(qs, dtype=torch.int32, device=W.device)
            scales = torch.empty(ss, dtype=torch.float16, device=W.device)
            qzeros = torch.empty(zs, dtype=torch.int32, device=W.device) if zero_point else None
            idx = torch.empty((N, K // group_size), dtype=torch.uint8, device=W.device)
        else:
            qweight, scales, qzeros, idx = out
        err = torch.empty((N, K // group_size, n_clip), dtype=torch.float64, device=W.device) if errors else None
    st = lib.awq_apply_clip(
        _dev(X, "X", _F16), M, _dev(W, "W", _F16), _dev(s, "s", _F16), N, K, config(group_size, zero_point),
        n_grid, n_clip, _dev(qweight, "qweight", _W32), _dev(scales, "scales", _F16), _dev(qzeros, "qzeros", _W32),
        0 if idx is None else idx.data_ptr(), 0 if err is None else err.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("awq_apply_clip", st)
    if errors:
        return qweight, scales, qzeros, idx, err
    return qweight, scales, qzeros, idx


# ---------------------------------------------------------------------------
# Fused and expert-grouped linears, routing and combination.  These four take strided rows and
# run on the inputs' device (and on its current stream unless one is given), whichever device is
# current.  What they allocate, results and scratch, belongs to the stream that they run on: with a
# `stream` of its own, other streams wait for it before they use a result, as with any tensor made there.
# ---------------------------------------------------------------------------

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
SCORINGS = {"softmax": 0, "sigmoid": 1}


def _refuse(t, name, index, shape, dtypes, what):
    """Raise the ValueError that says which of a tensor's properties is wrong."""
    if t.get_device() != index or t.dtype not in dtypes:
        raise ValueError(f"{name} must be on cuda:{index} with dtype one of {dtypes}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must {what}")


def _rows(t: Optional[torch.Tensor], name: str, index: int, rows: int, cols: int, dtype=torch.float16):
    """(data pointer, distance of rows in elements) of a [rows][cols] tensor with contiguous rows."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype or t.get_device() != index or t.shape != (rows, cols):
        _refuse(t, name, index, (rows, cols), (dtype,), "")
    ld, inner = t.stride()
    if rows <= 1:
        ld = (cols + 7) // 8 * 8       # one row or none: any distance does
    if ld < cols or (inner != 1 and cols > 1):
        _refuse(t, name, index, (rows, cols), (dtype,), "have contiguous rows that do not overlap")
    return t.data_ptr(), ld


def _flat(t: Optional[torch.Tensor], name: str, index: int, shape, dtypes) -> int:
    """Data pointer of a contiguous tensor of the given shape."""
    if t is None:
        return 0
    if t.dtype not in dtypes or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, index, shape, dtypes, "be contiguous")
    return t.data_ptr()


def _entry(fn_name: str):
    """The entry point as f(index, stream, *args): called with device `index` current, on `stream` or the
    device's current stream."""
    def call(index, stream, *args):
        fn = getattr(_lib or load_library(), fn_name)
        st = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
        if torch._C._cuda_getDevice() == index:
            status = fn(*args, st)
        else:
            with torch.cuda.device(index):
                status = fn(*args, st)
        if status:
            raise AWQError(fn_name, status)
    return call


_linear_fused, _linear_grouped, _moe_route, _moe_combine = map(
    _entry, ("awq_linear_fused", "awq_linear_grouped", "awq_moe_route", "awq_moe_combine"))


def _empty(like: torch.Tensor, shape, stream, dtype=None) -> torch.Tensor:
    with _on(stream, like.device):
        return like.new_empty(shape, dtype=dtype)


def _cuda(t: torch.Tensor, name: str, dims: int = 2):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.get_device()


def _activation(activation) -> int:
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation {activation!r} is not one of {sorted(k for k in ACTIVATIONS if k)}")
    return code


def _weights(lead, qweight, scales, qzeros, K, group_size, zero_point, index):
    """(N, data pointers) of packed weights with the leading axes `lead` (() or (E,))."""
    shape = qweight.shape
    if len(shape) != len(lead) + 2 or shape[-1] * 8 != K:
        raise ValueError(f"qweight has shape {tuple(shape)}, expected {[*lead, 'N', K // 8]}")
    if zero_point == (qzeros is None):
        raise ValueError("qzeros must be given with zero_point and left out without")
    if group_size not in _GROUP_SIZES or K % group_size:
        raise ValueError(f"group_size {group_size} is not 32, 64, 128 or 256, or does not divide K = {K}")
    N, ng = shape[-2], K // group_size
    return (N, _flat(qweight, "qweight", index, shape, _W32), _flat(scales, "scales", index, (*lead, N, ng), _F16),
            0 if qzeros is None else _flat(qzeros, "qzeros", index, (*lead, N, (ng + 7) // 8), _W32))


_GROUP_SIZES = frozenset((32, 64, 128, 256))


def linear_fused(X, qweight, scales, qzeros, group_size=128, zero_point=True, bias=None, activation=None,
                 gated=False, residual=None, out=None, stream=None) -> torch.Tensor:
    """awq_linear_fused: Y = act(X [M][K] . deq(W)^T + bias) + residual in one launch, any M >= 0.

    gated: W holds the gate's N/2 rows, then the other half's; Y [M][N/2] = act(gate) * other
    (+ residual).  activation: None/"none", "relu", "silu", "gelu" (erf) or "gelu_tanh".
    X, residual and out may have strided rows (X: 16-byte aligned rows); residual may be out."""
    dev = _cuda(X, "X")
    M, K = X.shape
    N, pq, ps, pz = _weights((), qweight, scales, qzeros, K, group_size, zero_point, dev)
    act = _activation(activation)
    if gated and N & 1:
        raise ValueError("a gated linear needs an even number of weight rows")
    n_out = N // 2 if gated else N
    px, ldx = _rows(X, "X", dev, M, K)
    pr, ldr = _rows(residual, "residual", dev, M, n_out)
    if out is None:
        out = X.new_empty((M, n_out)) if stream is None else _empty(X, (M, n_out), stream)
        py, ldy = out.data_ptr(), n_out
    else:
        py, ldy = _rows(out, "out", dev, M, n_out)
    _linear_fused(dev, stream, px, M, ldx, pq, ps, pz, N, K, _config(group_size, zero_point),
                  _flat(bias, "bias", dev, (N,), _F16), act, 1 if gated else 0, pr, ldr, py, ldy)
    return out


_I32 = (torch.int32,)
_GATHER_MIN_SHARE = 64   # kGatherMinShare: rows per expert below which a grouped call needs no workspace


def _workspace(t: Optional[torch.Tensor], index: int):
    """(data pointer, bytes) of a workspace of any type."""
    if t is None:
        return 0, 0
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{index}")
    return t.data_ptr(), t.numel() * t.element_size()


def linear_grouped(X, qweight, scales, qzeros, offsets, rows=None, group_size=128, zero_point=True, bias=None,
                   activation=None, gated=False, out=None, workspace=None, stream=None) -> torch.Tensor:
    """awq_linear_grouped: the fused linear with one matrix per expert (qweight [E][N][K/8], scales
    [E][N][K/G], qzeros [E][N][..], bias [E][N]).  Rows offsets[e]..offsets[e+1]-1 of the result
    [R][N or N/2] use expert e; offsets is an int32 [E+1] CUDA tensor, never read by the host.

    Row p reads row rows[p] of X (int32 [R]; R = len(rows)), or row p where rows is None (R = len(X)).
    Rows that no expert owns are left as they are in `out` (uninitialised without one).  Large gathered
    calls copy their rows into a workspace first (allocated here unless one is given)."""
    dev = _cuda(X, "X")
    T, K = X.shape
    E = qweight.shape[0]
    N, pq, ps, pz = _weights((E,), qweight, scales, qzeros, K, group_size, zero_point, dev)
    act = _activation(activation)
    if gated and N & 1:
        raise ValueError("a gated linear needs an even number of weight rows")
    n_out = N // 2 if gated else N
    R = T if rows is None else rows.shape[0]
    px, ldx = _rows(X, "X", dev, T, K)
    if out is None:
        out = X.new_empty((R, n_out)) if stream is None else _empty(X, (R, n_out), stream)
        py, ldy = out.data_ptr(), n_out
    else:
        py, ldy = _rows(out, "out", dev, R, n_out)
    if workspace is None and R >= _GATHER_MIN_SHARE * E and rows is not None:
        need = (_lib or load_library()).awq_linear_grouped_workspace_bytes(R, E, K)
        if need:
            workspace = _empty(X, need, stream, torch.uint8)
    ws, ws_bytes = _workspace(workspace, dev)
    _linear_grouped(dev, stream, px, T, ldx, _flat(rows, "rows", dev, (R,), _I32), R,
        _flat(offsets, "offsets", dev, (E + 1,), _I32), E, pq, ps, pz, N, K, _config(group_size, zero_point),
        _flat(bias, "bias", dev, (E, N), _F16), act, 1 if gated else 0, py, ldy, ws, ws_bytes)
    return out


class MoeRoute(NamedTuple):
    """What moe_route returns: weights fp32 [T][k], experts int32 [T][k] (-1: none), offsets int32
    [E+1], rows int32 [T k] (token of each expert-sorted row, -1 behind the last), positions int32
    [T][k] (row of each slot, -1: none)."""
    weights: torch.Tensor
    experts: torch.Tensor
    offsets: torch.Tensor
    rows: torch.Tensor
    positions: torch.Tensor


def moe_route(logits, top_k: int, scoring: str = "softmax", renormalize: bool = True, out: Optional[MoeRoute] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> MoeRoute:
    """awq_moe_route: each token's top_k experts by logits [T][E] (fp32 or fp16; -inf masks an
    expert), their weights, and the order of the rows by expert for linear_grouped / moe_combine."""
    dev = _cuda(logits, "logits")
    T, E = logits.shape
    half = logits.dtype is torch.float16
    score = SCORINGS.get(scoring)
    if not 1 <= top_k <= E:                  # before tensors of that size are made
        raise AWQError("awq_moe_route", AWQ_ERR_INVALID_ARG)
    if score is None:
        raise ValueError(f"scoring {scoring!r} is not one of {sorted(SCORINGS)}")
    pl, ld = _rows(logits, "logits", dev, T, E, torch.float16 if half else torch.float32)
    if out is None:
        slots = T * top_k                    # one allocation for the four of that size: most of this call's time
        with _on(stream, dev):
            made = logits.new_empty_strided((4, T, top_k), (slots, top_k, 1), dtype=torch.int32)
            offsets = logits.new_empty_strided((E + 1,), (1,), dtype=torch.int32)
        weights, experts, positions, rows = made.unbind()
        out = MoeRoute(weights.view(torch.float32), experts, offsets, rows.flatten(), positions)
        p, step = made.data_ptr(), 4 * slots
        pointers = p, p + step, offsets.data_ptr(), p + 3 * step, p + 2 * step
    else:
        weights, experts, offsets, rows, positions = out
        slots = (T, top_k)
        pointers = (_flat(weights, "weights", dev, slots, _F32), _flat(experts, "experts", dev, slots, _I32),
                    _flat(offsets, "offsets", dev, (E + 1,), _I32), _flat(rows, "rows", dev, (T * top_k,), _I32),
                    _flat(positions, "positions", dev, slots, _I32))
    if workspace is None:
        need = _route_need(T, E, dev)
        if need:
            workspace = _empty(logits, need, stream, torch.uint8)
    ws, ws_bytes = _workspace(workspace, dev)
    _moe_route(dev, stream, pl, 1 if half else 0, T, ld, E, top_k, score, 1 if renormalize else 0, *pointers, ws,
               ws_bytes)
    return out


_F32 = (torch.float32,)
_ROUTE_SINGLE = 32      # kRouteSingle: tokens up to which routing is one block and needs no workspace


def _route_need(T: int, E: int, index: int) -> int:
    if T <= _ROUTE_SINGLE:
        return 0
    lib = _lib or load_library()
    if torch._C._cuda_getDevice() == index:
        return lib.awq_moe_route_workspace_bytes(T, E)
    with torch.cuda.device(index):
        return lib.awq_moe_route_workspace_bytes(T, E)


def moe_combine(Y, weights, positions, residual=None, out=None, stream=None) -> torch.Tensor:
    """awq_moe_combine: out[t] = residual[t] + sum_j weights[t][j] Y[positions[t][j]] (positions
    outside Y contribute nothing).  Y [R][N], weights fp32 / positions int32 [T][k]; Y, residual and
    out may have strided rows; residual may be out."""
    dev = _cuda(Y, "Y")
    R, N = Y.shape
    if positions.dim() != 2:
        raise ValueError("positions must have 2 dimensions")
    T, k = slots = positions.shape
    py, ldy = _rows(Y, "Y", dev, R, N)
    pr, ldr = _rows(residual, "residual", dev, T, N)
    if out is None:
        out = Y.new_empty((T, N)) if stream is None else _empty(Y, (T, N), stream)
        po, ldo = out.data_ptr(), N
    else:
        po, ldo = _rows(out, "out", dev, T, N)
    _moe_combine(dev, stream, py, R, ldy, _flat(weights, "weights", dev, slots, _F32),
        _flat(positions, "positions", dev, slots, _I32), T, k, N, pr, ldr, po, ldo)
    return out
