"""Thin Python binding of libiq.so (see include/iq.h, include/iq_run.h and include/iq_train.h).

Argument marshalling only: every step runs in the HIP library.  Each wrapper
checks the shape, dtype and device of every tensor it is given (IQError before
any launch), allocates missing outputs and the call's workspace with torch
(the library itself allocates nothing), and enqueues the work on torch's
current stream.  If libiq.so is missing this module raises -- there is no CPU
fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch
from torch.autograd import forward_ad

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libiq.so")

FORMATS = ("IQ2_XXS", "IQ2_XS", "IQ2_S", "IQ1_S", "IQ1_M")
FMT = {n: i for i, n in enumerate(FORMATS)}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}

STATUS_NONFINITE, STATUS_OVERFLOW, STATUS_BADCHOICE, STATUS_BADIMP, STATUS_BADID = 1, 2, 4, 8, 16
STATUS_ROUNDED = 32  # linear, moe: a codebook value times a multiplier is not exact in fp16
ERRORS = {-1: "IQ_ERR_FMT", -2: "IQ_ERR_DTYPE", -3: "IQ_ERR_NULL", -4: "IQ_ERR_SHAPE", -5: "IQ_ERR_ARG",
          -6: "IQ_ERR_HIP", -7: "IQ_ERR_WORKSPACE"}

# C ABI signatures, by exported name
_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "iq_format_info": ([_I, _P], _I),
    "iq_imatrix_collect_workspace_size": ([_I64, _I64, _I, _I, _I, _P], _I),
    "iq_imatrix_collect": ([_P, _I, _I64, _I64, _P, _I, _I, _I, _P, _P, _P, _SZ, _P, _P], _I),
    "iq_hessian_collect_workspace_size": ([_I64, _I64, _I, _I, _I, _P], _I),
    "iq_hessian_collect": ([_P, _I, _I64, _I64, _P, _I, _I, _I, _P, _P, _SZ, _P, _P], _I),
    "iq_imatrix_merge": ([_P, _P, _I, _I64, _P, _P, _P, _P], _I),
    "iq_imatrix_importance": ([_P, _P, _I, _I64, _F, _P, _P, _P], _I),
    "iq_quantize_workspace_size": ([_I, _I64, _I64, _I64, _I, _P], _I),
    "iq_quantize": ([_I, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "iq_quantize_noalloc": ([_I, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P], _I),
    "iq_quantize_timed": ([_I, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P, _P, _P, _P], _I),
    "iq_quantize_every_choice": ([_I, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _SZ, _P, _P], _I),
    "iq_choice_search_workspace_size": ([_I, _I64, _I64, _I64, _I, _P], _I),
    "iq_choice_search": ([_I, _P, _I, _I64, _I64, _I64, _P, _P, _P, _F, _P, _P, _P, _SZ, _P, _P], _I),
    "iq_dequantize": ([_I, _P, _I64, _I64, _P, _P, _I, _P], _I),
    "iq_error_string": ([_I], ctypes.c_char_p),
    # include/iq_run.h
    "iq_linear_workspace_size": ([_I, _I64, _I64, _I, _I64, _I, _P], _I),
    "iq_linear": ([_I, _P, _I64, _I64, _P, _P, _I, _I64, _P, _P, _P, _P, _I, _I, _P, _P, _SZ, _P, _P], _I),
    "iq_moe_workspace_size": ([_I, _I, _I64, _I64, _I, _I, _I64, _I, _P], _I),
    "iq_moe": ([_I, _I, _P, _P, _P, _I64, _I64, _I, _P, _P, _P, _I, _I64, _P, _I, _I, _I, _P, _P, _P, _P, _SZ, _P,
                _P], _I),
    # include/iq_train.h
    "iq_checkpoint": ([_P, _I, _I64, _I64, _P, _P, _P, _P], _I),
    "iq_restore": ([_P, _P, _I64, _I64, _P, _I, _P], _I),
    "iq_glu_workspace_size": ([_I, _I64, _I64, _I, _I64, _P], _I),
    "iq_glu": ([_I, _P, _P, _I64, _I64, _P, _P, _I, _I64, _I, _P, _P, _SZ, _P, _P], _I),
    "iq_glu_backward_workspace_size": ([_I, _I64, _I64, _I, _I64, _P], _I),
    "iq_glu_backward": ([_I, _P, _P, _I64, _I64, _P, _P, _P, _P, _I, _I64, _I, _P, _P, _SZ, _P, _P], _I),
    "iq_linear_backward_workspace_size": ([_I, _I64, _I64, _I, _I64, _I, _I, _P], _I),
    "iq_linear_backward": ([_I, _P, _I64, _I64, _P, _P, _P, _P, _I, _I64, _P, _P, _P, _P, _I, _I, _P, _P, _P, _P, _SZ,
                            _P, _P], _I),
}


class IQError(RuntimeError):
    pass


class _FormatInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("block_values", "block_bytes", "grid_size", "choice_groups", "num_choices", "groups_per_choice")]


_lib = None


def lib():
    """Load libiq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise IQError(f"{LIB_PATH} is missing: build it with `python -m ggml_iq_codebook_imatrix_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        raise IQError(f"{what}: {ERRORS.get(rc, rc)} ({lib().iq_error_string(rc).decode()})")


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        if fmt not in FMT:
            raise IQError(f"unknown format {fmt!r}")
        return FMT[fmt]
    if int(fmt) not in range(len(FORMATS)):
        raise IQError(f"unknown format {fmt!r}")
    return int(fmt)


# --------------------------------------------------------------------------
# Argument checks: shape and dtype first (no device needed), then placement.
# --------------------------------------------------------------------------
def _need(t, name: str, shape=None, dtype=None):
    """t must be a tensor of `shape` (a tuple, None entries free) and dtype."""
    if not isinstance(t, torch.Tensor):
        raise IQError(f"{name} must be a tensor")
    if shape is not None and (t.dim() != len(shape) or
                              any(s is not None and int(d) != int(s) for d, s in zip(t.shape, shape))):
        want = "[" + ", ".join("*" if s is None else str(s) for s in shape) + "]"
        raise IQError(f"{name} has shape {list(t.shape)}, expected {want}")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise IQError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t


def _ptr(t, name: str, device):
    """Device pointer of t, which must be a contiguous tensor on `device`."""
    if t is None:
        return None
    if not t.is_cuda:
        raise IQError(f"{name} must be a device tensor")
    if t.device != device:
        raise IQError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise IQError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _device_of(t: torch.Tensor):
    """The device of the call's main tensor; it must be the current device,
    since the library launches on the current device."""
    if not t.is_cuda:
        raise IQError("tensors must be device tensors")
    if t.device.index != torch.cuda.current_device():
        raise IQError(f"tensors are on {t.device} but the current device is cuda:{torch.cuda.current_device()}")
    return t.device


def _status_ok(status):
    if status is not None:
        _need(status, "status", (None,), torch.int32)
        if status.numel() < 1:
            raise IQError("status must hold at least one int32")


def _workspace(nbytes: int, device, workspace):
    """The caller's workspace (a uint8 device tensor of at least nbytes) or a
    new one from torch's allocator; returns (tensor, pointer, size)."""
    if nbytes == 0:
        return None, None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _need(workspace, "workspace", None, torch.uint8)
    if workspace.numel() < nbytes:
        raise IQError(f"workspace holds {workspace.numel()} bytes, the call needs {nbytes}")
    return workspace, _ptr(workspace, "workspace", device), workspace.numel()


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def format_info(fmt) -> dict:
    info = _FormatInfo()
    _check(lib().iq_format_info(_fmt(fmt), ctypes.byref(info)), "iq_format_info")
    return {n: getattr(info, n) for n, _ in _FormatInfo._fields_}


def new_status(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def read_status(status: torch.Tensor) -> int:
    torch.cuda.synchronize(status.device)
    return int(status.item())


def _size_query(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(getattr(lib(), fn)(*args, ctypes.byref(out)), fn)
    return int(out.value)


# --------------------------------------------------------------------------
# Workspace queries
# --------------------------------------------------------------------------
def collect_workspace_size(T: int, K: int, top_k: int = 0, num_experts: int = 1, chunk_rows: int = 1024) -> int:
    return _size_query("iq_imatrix_collect_workspace_size", int(T), int(K), int(top_k), int(num_experts),
                       int(chunk_rows))


def hessian_workspace_size(T: int, K: int, top_k: int = 0, num_experts: int = 1, chunk_rows: int = 1024) -> int:
    return _size_query("iq_hessian_collect_workspace_size", int(T), int(K), int(top_k), int(num_experts),
                       int(chunk_rows))


def quantize_workspace_size(fmt, rows: int, cols: int, rows_per_expert: int | None = None,
                            weighted: bool = True) -> int:
    rpe = (rows or 1) if rows_per_expert is None else int(rows_per_expert)
    return _size_query("iq_quantize_workspace_size", _fmt(fmt), int(rows), int(cols), rpe, int(bool(weighted)))


def choice_search_workspace_size(fmt, rows: int, cols: int, rows_per_expert: int | None = None,
                                 weighted: bool = True) -> int:
    rpe = (rows or 1) if rows_per_expert is None else int(rows_per_expert)
    return _size_query("iq_choice_search_workspace_size", _fmt(fmt), int(rows), int(cols), rpe,
                       int(bool(weighted)))


# --------------------------------------------------------------------------
# Collection
# --------------------------------------------------------------------------
def _collect_args(x, ids):
    _need(x, "x", (None, None), tuple(DTYPE))
    T, K = x.shape
    top_k = 0
    if ids is not None:
        _need(ids, "ids", (T, None), torch.int32)
        top_k = ids.shape[1]
    return T, K, top_k


def imatrix_collect(x: torch.Tensor, ids: torch.Tensor | None = None, num_experts: int = 1,
                    chunk_rows: int = 1024, sums: torch.Tensor | None = None,
                    counts: torch.Tensor | None = None, status: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None):
    """Accumulate per-expert sum of x^2 and token counts. Returns (sums [E,K] f32, counts [E] i64)."""
    T, K, top_k = _collect_args(x, ids)
    E = int(num_experts)
    if sums is not None:
        _need(sums, "sums", (E, K), torch.float32)
    if counts is not None:
        _need(counts, "counts", (E,), torch.int64)
    _status_ok(status)
    dev = _device_of(x)
    if sums is None:
        sums = torch.zeros((E, K), dtype=torch.float32, device=dev)
    if counts is None:
        counts = torch.zeros((E,), dtype=torch.int64, device=dev)
    ws, wp, wn = _workspace(collect_workspace_size(T, K, top_k if ids is not None else 0, E, chunk_rows), dev,
                            workspace)
    rc = lib().iq_imatrix_collect(_ptr(x, "x", dev), DTYPE[x.dtype], T, K, _ptr(ids, "ids", dev), top_k, E,
                                  int(chunk_rows), _ptr(sums, "sums", dev), _ptr(counts, "counts", dev), wp, wn,
                                  _ptr(status, "status", dev), _stream())
    _check(rc, "iq_imatrix_collect")
    return sums, counts


def hessian_collect(x: torch.Tensor, ids: torch.Tensor | None = None, num_experts: int = 1,
                    chunk_rows: int = 1024, hess: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Accumulate each expert's 256-column diagonal blocks of X^T X -> hess [E, K/256, 256, 256] f32."""
    T, K, top_k = _collect_args(x, ids)
    E = int(num_experts)
    if K % 256:
        raise IQError("K must be a multiple of 256")
    if hess is not None:
        _need(hess, "hess", (E, K // 256, 256, 256), torch.float32)
    _status_ok(status)
    dev = _device_of(x)
    if hess is None:
        hess = torch.zeros((E, K // 256, 256, 256), dtype=torch.float32, device=dev)
    ws, wp, wn = _workspace(hessian_workspace_size(T, K, top_k if ids is not None else 0, E, chunk_rows), dev,
                            workspace)
    rc = lib().iq_hessian_collect(_ptr(x, "x", dev), DTYPE[x.dtype], T, K, _ptr(ids, "ids", dev), top_k, E,
                                  int(chunk_rows), _ptr(hess, "hess", dev), wp, wn, _ptr(status, "status", dev),
                                  _stream())
    _check(rc, "iq_hessian_collect")
    return hess


def imatrix_merge(src_sums: torch.Tensor, src_counts: torch.Tensor, sums: torch.Tensor, counts: torch.Tensor,
                  status: torch.Tensor | None = None):
    """Add one collection's statistics into another's in place: sums += src_sums,
    counts += src_counts.  Returns (sums, counts)."""
    _need(src_sums, "src_sums", (None, None), torch.float32)
    E, K = src_sums.shape
    _need(src_counts, "src_counts", (E,), torch.int64)
    _need(sums, "sums", (E, K), torch.float32)
    _need(counts, "counts", (E,), torch.int64)
    _status_ok(status)
    dev = _device_of(sums)
    rc = lib().iq_imatrix_merge(_ptr(src_sums, "src_sums", dev), _ptr(src_counts, "src_counts", dev), E, K,
                                _ptr(sums, "sums", dev), _ptr(counts, "counts", dev), _ptr(status, "status", dev),
                                _stream())
    _check(rc, "iq_imatrix_merge")
    return sums, counts


def imatrix_importance(sums: torch.Tensor, counts: torch.Tensor, floor_rel: float = 1e-6,
                       out: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """a = sqrt(max(sums/count, floor_rel * mean)) per expert; idle experts get ones."""
    _need(sums, "sums", (None, None), torch.float32)
    E, K = sums.shape
    _need(counts, "counts", (E,), torch.int64)
    if out is not None:
        _need(out, "out", (E, K), torch.float32)
    _status_ok(status)
    dev = _device_of(sums)
    if out is None:
        out = torch.empty((E, K), dtype=torch.float32, device=dev)
    rc = lib().iq_imatrix_importance(_ptr(sums, "sums", dev), _ptr(counts, "counts", dev), E, K, float(floor_rel),
                                     _ptr(out, "out", dev), _ptr(status, "status", dev), _stream())
    _check(rc, "iq_imatrix_importance")
    return out


# --------------------------------------------------------------------------
# Encode / decode
# --------------------------------------------------------------------------
def _encode_args(fmt, w, grid, importance, rows_per_expert):
    f = _fmt(fmt)
    _need(w, "w", (None, None), tuple(DTYPE))
    rows, cols = w.shape
    if cols % 256:
        raise IQError(f"w has {cols} columns, not a multiple of 256")
    info = format_info(f)
    _need(grid, "grid", (info["grid_size"], 8), torch.float32)
    rpe = (rows or 1) if rows_per_expert is None else int(rows_per_expert)
    if rpe < 1 or rows % rpe:
        raise IQError(f"rows_per_expert {rpe} does not divide rows {rows}")
    if importance is not None:
        _need(importance, "importance", (rows // rpe, cols), torch.float32)
    return f, rows, cols, rpe, info


def quantize(fmt, w: torch.Tensor, grid: torch.Tensor, importance: torch.Tensor | None = None,
             rows_per_expert: int | None = None, choices: torch.Tensor | None = None,
             out: torch.Tensor | None = None, status: torch.Tensor | None = None,
             check: bool = False, workspace: torch.Tensor | None = None, events=None) -> torch.Tensor:
    """Encode w [rows, cols] -> uint8 [rows, cols/256, block_bytes].
    events: optional (start, stop) torch.cuda.Event pair recorded around the
    search kernel alone (iq_quantize_timed)."""
    f, rows, cols, rpe, info = _encode_args(fmt, w, grid, importance, rows_per_expert)
    nb = cols // 256
    if choices is not None:
        _need(choices, "choices", (rows, nb, info["choice_groups"]), torch.uint8)
    if out is not None:
        _need(out, "out", (rows, nb, info["block_bytes"]), torch.uint8)
    _status_ok(status)
    dev = _device_of(w)
    if out is None:
        out = torch.empty((rows, nb, info["block_bytes"]), dtype=torch.uint8, device=dev)
    if check and status is None:
        status = new_status(dev)
    ws, wp, wn = _workspace(quantize_workspace_size(f, rows, cols, rpe, importance is not None), dev, workspace)
    args = (f, _ptr(w, "w", dev), DTYPE[w.dtype], rows, cols, rpe, _ptr(grid, "grid", dev),
            _ptr(importance, "importance", dev), _ptr(choices, "choices", dev), _ptr(out, "out", dev), wp, wn,
            _ptr(status, "status", dev))
    if events is None:
        rc = lib().iq_quantize(*args, _stream())
        _check(rc, "iq_quantize")
    else:
        start, stop = events
        for e in (start, stop):
            e.record()  # materialises the event on the current device
        rc = lib().iq_quantize_timed(*args, ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(stop.cuda_event),
                                     _stream())
        _check(rc, "iq_quantize_timed")
    if check:
        st = read_status(status)
        if st:
            raise IQError(f"iq_quantize device status {st:#x}")
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20  # IQ_NOALLOC_SCRATCH_BYTES


def quantize_noalloc(fmt, w: torch.Tensor, grid: torch.Tensor, importance: torch.Tensor | None = None,
                     rows_per_expert: int | None = None, choices: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """quantize() through iq_quantize_noalloc: the library works in its static
    device scratch, so apart from `out` when it is not given nothing is
    allocated.  Calls that overlap on one GPU race (they share the scratch)."""
    f, rows, cols, rpe, info = _encode_args(fmt, w, grid, importance, rows_per_expert)
    nb = cols // 256
    if choices is not None:
        _need(choices, "choices", (rows, nb, info["choice_groups"]), torch.uint8)
    if out is not None:
        _need(out, "out", (rows, nb, info["block_bytes"]), torch.uint8)
    _status_ok(status)
    dev = _device_of(w)
    if out is None:
        out = torch.empty((rows, nb, info["block_bytes"]), dtype=torch.uint8, device=dev)
    rc = lib().iq_quantize_noalloc(f, _ptr(w, "w", dev), DTYPE[w.dtype], rows, cols, rpe, _ptr(grid, "grid", dev),
                                   _ptr(importance, "importance", dev), _ptr(choices, "choices", dev),
                                   _ptr(out, "out", dev), _ptr(status, "status", dev), _stream())
    _check(rc, "iq_quantize_noalloc")
    return out


def quantize_every_choice(fmt, w: torch.Tensor, grid: torch.Tensor, importance: torch.Tensor | None = None,
                          rows_per_expert: int | None = None, out: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Encode w under every choice: uint8 [num_choices, rows, cols/256, block_bytes],
    out[c] == quantize(fmt, w, grid, importance, choices=full(c))."""
    f, rows, cols, rpe, info = _encode_args(fmt, w, grid, importance, rows_per_expert)
    shape = (info["num_choices"], rows, cols // 256, info["block_bytes"])
    if out is not None:
        _need(out, "out", shape, torch.uint8)
    _status_ok(status)
    dev = _device_of(w)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=dev)
    ws, wp, wn = _workspace(quantize_workspace_size(f, rows, cols, rpe, importance is not None), dev, workspace)
    rc = lib().iq_quantize_every_choice(f, _ptr(w, "w", dev), DTYPE[w.dtype], rows, cols, rpe,
                                        _ptr(grid, "grid", dev), _ptr(importance, "importance", dev),
                                        _ptr(out, "out", dev), wp, wn, _ptr(status, "status", dev), _stream())
    _check(rc, "iq_quantize_every_choice")
    return out


def choice_search(fmt, w: torch.Tensor, grid: torch.Tensor, hess: torch.Tensor,
                  importance: torch.Tensor | None = None, rows_per_expert: int | None = None,
                  perc_damp: float = 0.3, out: torch.Tensor | None = None,
                  status: torch.Tensor | None = None, payload: torch.Tensor | bool | None = None,
                  workspace: torch.Tensor | None = None):
    """Local-Hessian choice search -> uint8 choices [rows, cols/256, choice_groups];
    hess: [rows / rows_per_expert, cols/256, 256, 256] f32 diagonal Hessian blocks.
    With `payload` (True, or a uint8 [rows, cols/256, block_bytes] tensor to fill)
    the payload under the picks is written as well and (choices, payload) returned."""
    f, rows, cols, rpe, info = _encode_args(fmt, w, grid, importance, rows_per_expert)
    nb = cols // 256
    _need(hess, "hess", (rows // rpe, nb, 256, 256), torch.float32)
    if out is not None:
        _need(out, "out", (rows, nb, info["choice_groups"]), torch.uint8)
    if isinstance(payload, torch.Tensor):
        _need(payload, "payload", (rows, nb, info["block_bytes"]), torch.uint8)
    _status_ok(status)
    dev = _device_of(w)
    if out is None:
        out = torch.empty((rows, nb, info["choice_groups"]), dtype=torch.uint8, device=dev)
    if payload is True:
        payload = torch.empty((rows, nb, info["block_bytes"]), dtype=torch.uint8, device=dev)
    elif payload is False:
        payload = None
    ws, wp, wn = _workspace(choice_search_workspace_size(f, rows, cols, rpe, importance is not None), dev,
                            workspace)
    rc = lib().iq_choice_search(f, _ptr(w, "w", dev), DTYPE[w.dtype], rows, cols, rpe, _ptr(grid, "grid", dev),
                                _ptr(importance, "importance", dev), _ptr(hess, "hess", dev), float(perc_damp),
                                _ptr(out, "out", dev), _ptr(payload, "payload", dev), wp, wn,
                                _ptr(status, "status", dev), _stream())
    _check(rc, "iq_choice_search")
    return out if payload is None else (out, payload)


def dequantize(fmt, packed: torch.Tensor, grid: torch.Tensor, dtype=torch.float32,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """Decode uint8 [rows, cols/256, block_bytes] -> [rows, cols]."""
    f = _fmt(fmt)
    info = format_info(f)
    _need(packed, "packed", (None, None, info["block_bytes"]), torch.uint8)
    _need(grid, "grid", (info["grid_size"], 8), torch.float32)
    rows, nb = packed.shape[0], packed.shape[1]
    cols = nb * 256
    if out is not None:
        _need(out, "out", (rows, cols), tuple(DTYPE))
    elif dtype not in DTYPE:
        raise IQError(f"unsupported output dtype {dtype}")
    dev = _device_of(packed)
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=dev)
    rc = lib().iq_dequantize(f, _ptr(packed, "packed", dev), rows, cols, _ptr(grid, "grid", dev),
                             _ptr(out, "out", dev), DTYPE[out.dtype], _stream())
    _check(rc, "iq_dequantize")
    return out


# --------------------------------------------------------------------------
# Tokens through encoded weights (include/iq_run.h).  These calls sit in serving
# loops, where a launch takes microseconds: the checks below compare whole
# shapes first and spell out what is wrong only when something is, and the
# answers of the (pure) size and format queries are kept.
# --------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _geometry(f: int):
    info = format_info(f)
    return info["grid_size"], info["block_bytes"]


@functools.lru_cache(maxsize=4096)
def _run_size(fn: str, *args) -> int:
    return _size_query(fn, *args)


def _is(t, name: str, shape, dtype):
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype is not dtype:
        _need(t, name, shape, dtype)


def _ends(t, name: str, shape, dtype):
    """As _need, for a shape whose last entry alone is fixed; the shape."""
    if not isinstance(t, torch.Tensor) or t.dim() != len(shape) or t.shape[-1] != shape[-1] or t.dtype is not dtype:
        _need(t, name, shape, dtype)
    return t.shape


def _home(t: torch.Tensor) -> int:
    """The index of the current device, on which t must be."""
    index = t.get_device()
    if index < 0 or index != torch._C._cuda_getDevice():
        _device_of(t)
    return index


def _addr(t, name: str, index: int):
    if t is None:
        return None
    if t.get_device() != index or not t.is_contiguous():
        _ptr(t, name, torch.device("cuda", index))
    return t.data_ptr()


def _no_grad(*tensors):
    """Encoded weights are frozen and the calls below record no derivatives (their backward passes are calls of their
    own): refused where one would be recorded, or carried along in forward mode (which torch.no_grad() does not
    stop)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise IQError("the call has no backward pass: tensors that require a gradient need torch.no_grad()")
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise IQError("the call has no forward-mode derivative: a tensor carries a tangent")


def _scratch(nbytes: int, x: torch.Tensor, workspace):
    if workspace is None and nbytes:
        workspace = x.new_empty(nbytes, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), nbytes
    return _workspace(nbytes, x.device, workspace)


def linear_workspace_size(fmt, rows: int, cols: int, dtype, T: int, rank: int = 0) -> int:
    if dtype not in DTYPE:
        raise IQError(f"unsupported dtype {dtype}")
    return _run_size("iq_linear_workspace_size", _fmt(fmt), int(rows), int(cols), DTYPE[dtype], int(T), int(rank))


def moe_workspace_size(fmt, hidden: int, inter: int, num_experts: int, dtype, T: int, top_k: int,
                       down_fmt=None) -> int:
    if dtype not in DTYPE:
        raise IQError(f"unsupported dtype {dtype}")
    f = _fmt(fmt)
    return _run_size("iq_moe_workspace_size", f, f if down_fmt is None else _fmt(down_fmt), int(hidden), int(inter),
                     int(num_experts), DTYPE[dtype], int(T), int(top_k))


def linear(fmt, packed: torch.Tensor, grid: torch.Tensor, x: torch.Tensor, lora_a: torch.Tensor | None = None,
           lora_b: torch.Tensor | None = None, lora_scale: torch.Tensor | None = None,
           lora_ids: torch.Tensor | None = None, out: torch.Tensor | None = None,
           status: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Tokens x [T, cols] through the encoded weight packed [rows, cols/256, block_bytes] -> [T, rows], of x's dtype.
    With lora_a [N, r, cols], lora_b [N, rows, r] (x's dtype) and lora_ids [T] int32 (-1: none), token t also gets
    lora_scale[a] * (x[t] A_a^T) B_a^T, a = lora_ids[t] (lora_scale [N] f32; None: ones).  linear_backward() is the
    backward pass."""
    f = _fmt(fmt)
    entries, nbytes = _geometry(f)
    rows, nb, _ = _ends(packed, "packed", (None, None, nbytes), torch.uint8)
    cols = nb * 256
    _is(grid, "grid", (entries, 8), torch.float32)
    if not isinstance(x, torch.Tensor) or x.dtype not in DTYPE:
        _need(x, "x", (None, cols), tuple(DTYPE))
    dtype = x.dtype
    T = _ends(x, "x", (None, cols), dtype)[0]
    N = rank = 0
    if lora_a is not None:
        N, rank, _ = _ends(lora_a, "lora_a", (None, None, cols), dtype)
        if N < 1 or rank < 1:
            raise IQError("lora_a holds no adapter")
        _is(lora_b, "lora_b", (N, rows, rank), dtype)
        if lora_scale is not None:
            _is(lora_scale, "lora_scale", (N,), torch.float32)
        _is(lora_ids, "lora_ids", (T,), torch.int32)
    elif lora_b is not None or lora_scale is not None or lora_ids is not None:
        raise IQError("lora_b, lora_scale and lora_ids need lora_a")
    if out is not None:
        _is(out, "out", (T, rows), dtype)
    if status is not None:
        _status_ok(status)
    _no_grad(grid, x, lora_a, lora_b, lora_scale, out)
    dev = _home(x)
    if out is None:
        out = x.new_empty((T, rows))
    dt = DTYPE[dtype]
    ws, wp, wn = _scratch(_run_size("iq_linear_workspace_size", f, rows, cols, dt, T, rank), x, workspace)
    rc = lib().iq_linear(f, _addr(packed, "packed", dev), rows, cols, _addr(grid, "grid", dev), _addr(x, "x", dev),
                         dt, T, _addr(lora_a, "lora_a", dev), _addr(lora_b, "lora_b", dev),
                         _addr(lora_scale, "lora_scale", dev), _addr(lora_ids, "lora_ids", dev), N, rank,
                         _addr(out, "out", dev), wp, wn, _addr(status, "status", dev),
                         torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "iq_linear")
    return out


def moe(fmt, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, grid: torch.Tensor, x: torch.Tensor,
        num_experts: int, router: torch.Tensor | None = None, top_k: int | None = None, renormalize: bool = True,
        ids: torch.Tensor | None = None, weights: torch.Tensor | None = None, down_fmt=None,
        down_grid: torch.Tensor | None = None, out: torch.Tensor | None = None,
        status: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """A mixture-of-experts layer on encoded experts: gate, up [E*inter, hidden/256, bytes], down
    [E*hidden, inter/256, bytes] (down_fmt and down_grid where they differ), x [T, hidden].
    With router [E, hidden] and top_k the layer routes its tokens (ids and weights, where given, are filled);
    without, ids [T, top_k] int32 and weights [T, top_k] f32 are the caller's.  Returns (y, ids, weights).
    No backward pass."""
    f = _fmt(fmt)
    fd = f if down_fmt is None else _fmt(down_fmt)
    (entries, nbytes), (dentries, dbytes) = _geometry(f), _geometry(fd)
    E = int(num_experts)
    if E < 1:
        raise IQError("num_experts must be at least 1")
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in DTYPE:
        _need(x, "x", (None, None), tuple(DTYPE))
    (T, hidden), dtype = x.shape, x.dtype
    if hidden % 256 or hidden == 0:
        raise IQError(f"x has {hidden} columns, not a multiple of 256")
    if not isinstance(gate, torch.Tensor) or gate.shape[1:] != (hidden // 256, nbytes) or gate.dtype is not torch.uint8:
        _need(gate, "gate", (None, hidden // 256, nbytes), torch.uint8)
    if gate.shape[0] % E or gate.shape[0] // E % 256 or gate.shape[0] == 0:
        raise IQError(f"gate has {gate.shape[0]} rows, not a multiple of 256 for each of {E} experts")
    inter = gate.shape[0] // E
    _is(up, "up", (E * inter, hidden // 256, nbytes), torch.uint8)
    _is(down, "down", (E * hidden, inter // 256, dbytes), torch.uint8)
    _is(grid, "grid", (entries, 8), torch.float32)
    if down_grid is None:
        if fd != f and dentries != entries:
            raise IQError("down_grid is needed where down_fmt has another codebook")
        down_grid = grid
    else:
        _is(down_grid, "down_grid", (dentries, 8), torch.float32)
    if router is not None:
        if not isinstance(router, torch.Tensor) or router.shape != (E, hidden) or router.dtype not in DTYPE:
            _need(router, "router", (E, hidden), tuple(DTYPE))
        if top_k is None or not 1 <= int(top_k) <= E:
            raise IQError("top_k must lie in 1 .. num_experts with a router")
    elif ids is None or weights is None:
        raise IQError("either router or ids and weights must be given")
    k = int(top_k) if top_k is not None else _need(ids, "ids", (T, None)).shape[1]
    if ids is not None:
        _is(ids, "ids", (T, k), torch.int32)
    if weights is not None:
        _is(weights, "weights", (T, k), torch.float32)
    if out is not None:
        _is(out, "out", (T, hidden), dtype)
    if status is not None:
        _status_ok(status)
    _no_grad(grid, down_grid, x, router, weights, out)
    dev = _home(x)
    if ids is None:
        ids = x.new_empty((T, k), dtype=torch.int32)
    if weights is None:
        weights = x.new_empty((T, k), dtype=torch.float32)
    if out is None:
        out = x.new_empty((T, hidden))
    dt = DTYPE[dtype]
    ws, wp, wn = _scratch(_run_size("iq_moe_workspace_size", f, fd, hidden, inter, E, dt, T, k), x, workspace)
    rc = lib().iq_moe(f, fd, _addr(gate, "gate", dev), _addr(up, "up", dev), _addr(down, "down", dev), hidden, inter,
                      E, _addr(grid, "grid", dev), _addr(down_grid, "down_grid", dev), _addr(x, "x", dev), dt, T,
                      _addr(router, "router", dev), 0 if router is None else DTYPE[router.dtype], k,
                      int(bool(renormalize)), _addr(ids, "ids", dev), _addr(weights, "weights", dev),
                      _addr(out, "out", dev), wp, wn, _addr(status, "status", dev),
                      torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "iq_moe")
    return out, ids, weights


# --------------------------------------------------------------------------
# Adapting a model whose weights stay encoded (include/iq_train.h)
# --------------------------------------------------------------------------
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def _activation(name) -> int:
    act = ACTIVATIONS.get(name) if isinstance(name, str) else None
    if act is None:
        raise IQError(f"unknown activation {name!r}")
    return act


def _tokens(x, name: str, cols):
    """Shape (T, cols) and dtype of a tensor of tokens; cols None: any."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in DTYPE or x.shape[1] != cols:
        _need(x, name, (None, cols), tuple(DTYPE))
    return x.shape[0], x.shape[1], x.dtype


def _kept(x, T: int, cols: int, dtype):
    """The data and exponents of tokens kept for the backward pass: a tensor [T, cols] of dtype, or the
    (codes, exponents) that checkpoint() returned for one."""
    if isinstance(x, (tuple, list)):
        if len(x) != 2:
            raise IQError("a checkpoint is a pair of codes and exponents")
        _is(x[0], "codes", (T, cols), torch.int8)
        _is(x[1], "exponents", (T, -(-cols // 32)), torch.uint8)
        return x[0], x[1]
    _is(x, "x", (T, cols), dtype)
    return x, None


def checkpoint(x: torch.Tensor, codes: torch.Tensor | None = None, exponents: torch.Tensor | None = None,
               status: torch.Tensor | None = None):
    """Activations x [T, cols] in 8 bits: (codes [T, cols] int8, exponents [T, ceil(cols/32)] uint8), a value being
    code * 2^(exponent - 133).  Code -128 stands for an infinity or NaN."""
    T, cols, dtype = _tokens(x, "x", None)
    if codes is not None:
        _is(codes, "codes", (T, cols), torch.int8)
    if exponents is not None:
        _is(exponents, "exponents", (T, -(-cols // 32)), torch.uint8)
    if status is not None:
        _status_ok(status)
    _no_grad(x)
    dev = _home(x)
    if codes is None:
        codes = x.new_empty((T, cols), dtype=torch.int8)
    if exponents is None:
        exponents = x.new_empty((T, -(-cols // 32)), dtype=torch.uint8)
    rc = lib().iq_checkpoint(_addr(x, "x", dev), DTYPE[dtype], T, cols, _addr(codes, "codes", dev),
                             _addr(exponents, "exponents", dev), _addr(status, "status", dev),
                             torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "iq_checkpoint")
    return codes, exponents


def restore(codes: torch.Tensor, exponents: torch.Tensor, dtype=torch.float32,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """The values of a checkpoint, [T, cols] of dtype (or of out's); exact in either."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2 or codes.dtype is not torch.int8:
        _need(codes, "codes", (None, None), torch.int8)
    T, cols = codes.shape
    _is(exponents, "exponents", (T, -(-cols // 32)), torch.uint8)
    if out is not None:
        _need(out, "out", (T, cols), tuple(DTYPE))
    elif dtype not in DTYPE:
        raise IQError(f"unsupported output dtype {dtype}")
    _no_grad(out)
    dev = _home(codes)
    if out is None:
        out = codes.new_empty((T, cols), dtype=dtype)
    rc = lib().iq_restore(_addr(codes, "codes", dev), _addr(exponents, "exponents", dev), T, cols,
                          _addr(out, "out", dev), DTYPE[out.dtype], torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "iq_restore")
    return out


def glu_workspace_size(fmt, inter: int, hidden: int, dtype, T: int) -> int:
    if dtype not in DTYPE:
        raise IQError(f"unsupported dtype {dtype}")
    return _run_size("iq_glu_workspace_size", _fmt(fmt), int(inter), int(hidden), DTYPE[dtype], int(T))


def glu_backward_workspace_size(fmt, inter: int, hidden: int, dtype, T: int) -> int:
    if dtype not in DTYPE:
        raise IQError(f"unsupported dtype {dtype}")
    return _run_size("iq_glu_backward_workspace_size", _fmt(fmt), int(inter), int(hidden), DTYPE[dtype], int(T))


def _glu_args(fmt, gate, up, grid, activation):
    f = _fmt(fmt)
    entries, nbytes = _geometry(f)
    inter, nb, _ = _ends(gate, "gate", (None, None, nbytes), torch.uint8)
    _is(up, "up", (inter, nb, nbytes), torch.uint8)
    _is(grid, "grid", (entries, 8), torch.float32)
    return f, inter, nb * 256, _activation(activation)


def glu(fmt, gate: torch.Tensor, up: torch.Tensor, grid: torch.Tensor, x: torch.Tensor, activation: str = "silu",
        out: torch.Tensor | None = None, status: torch.Tensor | None = None,
        workspace: torch.Tensor | None = None) -> torch.Tensor:
    """A gated feed-forward block's first half on encoded weights gate, up [inter, hidden/256, block_bytes]:
    act(x gate^T) * (x up^T) for tokens x [T, hidden] -> [T, inter], of x's dtype.  activation: "silu", "gelu" or
    "gelu_tanh".  linear() is the second half; glu_backward() the backward pass."""
    f, inter, hidden, act = _glu_args(fmt, gate, up, grid, activation)
    T, _, dtype = _tokens(x, "x", hidden)
    if out is not None:
        _is(out, "out", (T, inter), dtype)
    if status is not None:
        _status_ok(status)
    _no_grad(grid, x, out)
    dev = _home(x)
    if out is None:
        out = x.new_empty((T, inter))
    dt = DTYPE[dtype]
    ws, wp, wn = _scratch(_run_size("iq_glu_workspace_size", f, inter, hidden, dt, T), x, workspace)
    rc = lib().iq_glu(f, _addr(gate, "gate", dev), _addr(up, "up", dev), inter, hidden, _addr(grid, "grid", dev),
                      _addr(x, "x", dev), dt, T, act, _addr(out, "out", dev), wp, wn, _addr(status, "status", dev),
                      torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "iq_glu")
    return out


def glu_backward(fmt, gate: torch.Tensor, up: torch.Tensor, grid: torch.Tensor, x, dh: torch.Tensor,
                 activation: str = "silu", out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient [T, hidden] by glu()'s x, from dh [T, inter], the gradient by its result.  x: the tokens, or the
    (codes, exponents) that checkpoint() made of them."""
    f, inter, hidden, act = _glu_args(fmt, gate, up, grid, activation)
    T, _, dtype = _tokens(dh, "dh", inter)
    x, exponents = _kept(x, T, hidden, dtype)
    if out is not None:
        _is(out, "out", (T, hidden), dtype)
    if status is not None:
        _status_ok(status)
    _no_grad(grid, x, dh, out)
    dev = _home(dh)
    if out is None:
        out = dh.new_empty((T, hidden))
    dt = DTYPE[dtype]
    ws, wp, wn = _scratch(_run_size("iq_glu_backward_workspace_size", f, inter, hidden, dt, T), dh, workspace)
    rc = lib().iq_glu_backward(f, _addr(gate, "gate", dev), _addr(up, "up", dev), inter, hidden,
                               _addr(grid, "grid", dev), _addr(x, "x", dev), _addr(exponents, "exponents", dev),
                               _addr(dh, "dh", dev), dt, T, act, _addr(out, "out", dev), wp, wn,
                               _addr(status, "status", dev), torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "iq_glu_backward")
    return out


def linear_backward_workspace_size(fmt, rows: int, cols: int, dtype, T: int, num_adapters: int = 0,
                                   rank: int = 0) -> int:
    if dtype not in DTYPE:
        raise IQError(f"unsupported dtype {dtype}")
    return _run_size("iq_linear_backward_workspace_size", _fmt(fmt), int(rows), int(cols), DTYPE[dtype], int(T),
                     int(num_adapters), int(rank))


def linear_backward(fmt, packed: torch.Tensor, grid: torch.Tensor, dy: torch.Tensor, x=None,
                    lora_a: torch.Tensor | None = None, lora_b: torch.Tensor | None = None,
                    lora_scale: torch.Tensor | None = None, lora_ids: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, grad_a: torch.Tensor | None = None,
                    grad_b: torch.Tensor | None = None, need_dx: bool = True, status: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None):
    """The backward pass of linear(): from dy [T, rows], the gradient by its result, the gradient dx [T, cols] by its
    tokens; with adapters (as linear() takes them, and x, the tokens or the (codes, exponents) that checkpoint() made
    of them) the tuple (dx, gradient by lora_a, gradient by lora_b).  need_dx=False leaves dx out (None)."""
    f = _fmt(fmt)
    entries, nbytes = _geometry(f)
    rows, nb, _ = _ends(packed, "packed", (None, None, nbytes), torch.uint8)
    cols = nb * 256
    _is(grid, "grid", (entries, 8), torch.float32)
    T, _, dtype = _tokens(dy, "dy", rows)
    N = rank = 0
    exponents = None
    if lora_a is not None:
        N, rank, _ = _ends(lora_a, "lora_a", (None, None, cols), dtype)
        if N < 1 or rank < 1:
            raise IQError("lora_a holds no adapter")
        _is(lora_b, "lora_b", (N, rows, rank), dtype)
        if lora_scale is not None:
            _is(lora_scale, "lora_scale", (N,), torch.float32)
        _is(lora_ids, "lora_ids", (T,), torch.int32)
        x, exponents = _kept(x, T, cols, dtype)
        if grad_a is not None:
            _is(grad_a, "grad_a", (N, rank, cols), dtype)
        if grad_b is not None:
            _is(grad_b, "grad_b", (N, rows, rank), dtype)
    else:
        if any(t is not None for t in (lora_b, lora_scale, lora_ids, grad_a, grad_b)):
            raise IQError("lora_b, lora_scale, lora_ids, grad_a and grad_b need lora_a")
        x = None
    if out is not None:
        if not need_dx:
            raise IQError("out is given, but dx is not wanted")
        _is(out, "out", (T, cols), dtype)
    if status is not None:
        _status_ok(status)
    _no_grad(grid, dy, x, lora_a, lora_b, lora_scale, out, grad_a, grad_b)
    dev = _home(dy)
    if out is None and need_dx:
        out = dy.new_empty((T, cols))
    if N:
        if grad_a is None:
            grad_a = torch.empty_like(lora_a)
        if grad_b is None:
            grad_b = torch.empty_like(lora_b)
    dt = DTYPE[dtype]
    ws, wp, wn = _scratch(_run_size("iq_linear_backward_workspace_size", f, rows, cols, dt, T, N, rank), dy, workspace)
    rc = lib().iq_linear_backward(f, _addr(packed, "packed", dev), rows, cols, _addr(grid, "grid", dev),
                                  _addr(dy, "dy", dev), _addr(x, "x", dev), _addr(exponents, "exponents", dev), dt, T,
                                  _addr(lora_a, "lora_a", dev), _addr(lora_b, "lora_b", dev),
                                  _addr(lora_scale, "lora_scale", dev), _addr(lora_ids, "lora_ids", dev), N, rank,
                                  _addr(out, "out", dev), _addr(grad_a, "grad_a", dev), _addr(grad_b, "grad_b", dev),
                                  wp, wn, _addr(status, "status", dev), torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, "iq_linear_backward")
    return (out, grad_a, grad_b) if N else out
