"""Python binding of the GB300 SpMM library (``include/spmm.h``).

Argument marshalling only: every step of the product runs in the CUDA
kernels of ``libspmm_gb300.so``.  The functions keep the C names:

    h = spmm_bcsr_create(m, k, row_ptr, col_idx, vals, in_t, out_t, b_row=64, b_col=64)
    h = spmm_wcsr_create(m, k, row_ptr, col_idx, vals, in_t, out_t, window_h=16, col_pad=16)
    spmm_run(h, B_ptr, C_ptr, N, stream_ptr)
    spmm_destroy(h)

plus ``spmm_format_info``, ``spmm_export_format``, ``spmm_check``,
``spmm_set_max_ctas``, ``spmm_run_host``, the host-only converters
``spmm_bcsr_convert`` / ``spmm_wcsr_convert`` and
``spmm_selftest_wait_timeout``.  ``run_torch`` is a convenience that passes
torch tensors and the current stream; ``Adapters`` (low-rank adapters beside
the block-sparse linear layer) and ``route_sort`` / ``route_gather`` /
``route_combine`` / ``route_combine_grad`` (tokens sorted by expert and back)
do the same for the ``spmm_adapters_*`` and ``spmm_route_*`` calls.

There is no fallback: if the shared library cannot be loaded, importing a
function that needs it raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspmm_gb300.so")

SPMM_OK = 0
SPMM_ERR_INVALID_ARG = 1
SPMM_ERR_UNSUPPORTED = 2
SPMM_ERR_CUDA = 3
SPMM_ERR_OOM = 4
SPMM_ERR_TIMEOUT = 5
SPMM_ERR_DEVICE_CHECK = 6

SPMM_F16 = 0
SPMM_BF16 = 1
SPMM_F32 = 2
DTYPES = {"f16": SPMM_F16, "bf16": SPMM_BF16, "f32": SPMM_F32}

SPMM_FORMAT_BCSR = 0
SPMM_FORMAT_WCSR = 1

# Every symbol the header declares.
EXPORTS = (
    "spmm_bcsr_create", "spmm_wcsr_create", "spmm_run", "spmm_run_host", "spmm_destroy",
    "spmm_format_info", "spmm_export_format", "spmm_bcsr_convert", "spmm_wcsr_convert",
    "spmm_check", "spmm_set_max_ctas", "spmm_selftest_wait_timeout", "spmm_status_str",
    "spmm_last_error", "spmm_wcsr_run_noalloc", "spmm_run_linear", "spmm_set_schedule",
    "spmm_probe_l2_read", "spmm_wcsr_noalloc_check",
    "spmm_adapters_create", "spmm_adapters_destroy", "spmm_run_linear_adapters", "spmm_adapters_grad",
    "spmm_route_workspace_bytes", "spmm_route_sort", "spmm_route_gather", "spmm_route_combine",
    "spmm_route_combine_grad",
)


class SpmmError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {_status_name(status)}: {msg}")
        self.status = status


class spmm_info(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int32), ("b_row", ctypes.c_int32), ("b_col", ctypes.c_int32),
        ("m", ctypes.c_int64), ("k", ctypes.c_int64), ("nnz", ctypes.c_int64),
        ("n_groups", ctypes.c_int64), ("n_units", ctypes.c_int64), ("stored", ctypes.c_int64),
        ("padding", ctypes.c_int64), ("idx_bytes", ctypes.c_int64), ("val_bytes", ctypes.c_int64),
        ("n_tasks", ctypes.c_int64), ("n_split_windows", ctypes.c_int64), ("split_cols", ctypes.c_int64),
    ]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libspmm_gb300.so (raises OSError if it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} is missing; build it with sparse_dense_matrix_bcsr_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    I64 = ctypes.c_int64
    I32 = ctypes.c_int
    st = ctypes.c_int
    sig = {
        "spmm_bcsr_create": [ctypes.POINTER(P), I64, I64, P, P, P, I32, I32, I32, I32],
        "spmm_wcsr_create": [ctypes.POINTER(P), I64, I64, P, P, P, I32, I32, I32, I32],
        "spmm_run": [P, P, P, I64, P],
        "spmm_run_linear": [P, P, P, I64, P],
        "spmm_run_host": [P, P, P, I64, P],
        "spmm_destroy": [P],
        "spmm_format_info": [P, ctypes.POINTER(spmm_info)],
        "spmm_export_format": [P, P, P, P],
        "spmm_bcsr_convert": [I64, I64, P, P, P, I32, I32, ctypes.POINTER(I64), P, P, P],
        "spmm_wcsr_convert": [I64, I64, P, P, P, I32, I32, ctypes.POINTER(I64), P, P, P],
        "spmm_check": [P, P],
        "spmm_set_max_ctas": [P, ctypes.c_int32],
        "spmm_set_schedule": [P, ctypes.c_int32],
        "spmm_selftest_wait_timeout": [I64, P, ctypes.POINTER(ctypes.c_int32)],
        "spmm_probe_l2_read": [P, I64, I32, P, P],
        "spmm_wcsr_noalloc_check": [P],
        "spmm_wcsr_run_noalloc": [P, P, P, I64, I64, I64, I32, I32, P, P, I64, P],
        "spmm_adapters_create": [ctypes.POINTER(P), I64, I64, I32, I32, I32, I64, I64, I32],
        "spmm_adapters_destroy": [P],
        "spmm_run_linear_adapters": [P, P, P, P, I64, P, P, P, P, P, I64, P],
        "spmm_adapters_grad": [P, P, P, P, P, P, P, I64, P, P, P, P, P, I64, P],
        "spmm_route_sort": [P, I64, I32, I32, P, P, P, P, P],
        "spmm_route_gather": [P, P, P, P, I64, I32, I64, I32, P],
        "spmm_route_combine": [P, P, P, P, I64, I32, I64, I32, P],
        "spmm_route_combine_grad": [P, P, P, P, P, P, P, I64, I32, I64, I32, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = st
    lib.spmm_route_workspace_bytes.argtypes = [I64, I32, I32]
    lib.spmm_route_workspace_bytes.restype = I64
    lib.spmm_status_str.argtypes = [st]
    lib.spmm_status_str.restype = ctypes.c_char_p
    lib.spmm_last_error.argtypes = []
    lib.spmm_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _status_name(s: int) -> str:
    try:
        return load_library().spmm_status_str(s).decode()
    except OSError:
        return str(s)


def _check(status: int, where: str):
    if status != SPMM_OK:
        msg = load_library().spmm_last_error().decode()
        raise SpmmError(status, where, msg)


def _arr(a, dtype):
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def _dt(t) -> int:
    return DTYPES[t] if isinstance(t, str) else int(t)


def _csr_args(row_ptr, col_idx, vals):
    rp, prp = _arr(row_ptr, np.int64)
    ci, pci = _arr(col_idx if len(col_idx) else np.zeros(1, np.int32), np.int32)
    vv, pvv = _arr(vals if len(vals) else np.zeros(1, np.uint16), np.uint16)
    return (rp, ci, vv), prp, pci, pvv


def spmm_bcsr_create(m, k, row_ptr, col_idx, vals, in_t="bf16", out_t="f32", b_row=64, b_col=64) -> int:
    lib = load_library()
    keep, prp, pci, pvv = _csr_args(row_ptr, col_idx, vals)
    h = ctypes.c_void_p()
    _check(lib.spmm_bcsr_create(ctypes.byref(h), m, k, prp, pci, pvv, _dt(in_t), _dt(out_t), b_row, b_col),
           "spmm_bcsr_create")
    return h.value


def spmm_wcsr_create(m, k, row_ptr, col_idx, vals, in_t="bf16", out_t="f32", window_h=16, col_pad=16) -> int:
    lib = load_library()
    keep, prp, pci, pvv = _csr_args(row_ptr, col_idx, vals)
    h = ctypes.c_void_p()
    _check(lib.spmm_wcsr_create(ctypes.byref(h), m, k, prp, pci, pvv, _dt(in_t), _dt(out_t), window_h, col_pad),
           "spmm_wcsr_create")
    return h.value


def spmm_run(h: int, B_ptr: int, C_ptr: int, N: int, stream: int = 0) -> None:
    _check(load_library().spmm_run(h, B_ptr, C_ptr, N, stream or None), "spmm_run")


def spmm_run_linear(h: int, X_ptr: int, Y_ptr: int, N: int, stream: int = 0) -> None:
    """Y = X * A^T on the GPU (BCSR handle; X is N x k, Y is N x m, both row-major device pointers)."""
    _check(load_library().spmm_run_linear(h, X_ptr, Y_ptr, N, stream or None), "spmm_run_linear")


def spmm_run_status(h: int, B_ptr: int, C_ptr: int, N: int, stream: int = 0) -> int:
    """spmm_run returning the raw status instead of raising."""
    return load_library().spmm_run(h, B_ptr, C_ptr, N, stream or None)


def spmm_run_host(h: int, B_host: np.ndarray, C_host: np.ndarray, N: int, stream: int = 0) -> None:
    assert B_host.flags.c_contiguous and C_host.flags.c_contiguous
    _check(load_library().spmm_run_host(h, B_host.ctypes.data, C_host.ctypes.data, N, stream or None),
           "spmm_run_host")


def spmm_run_host_ptr(h: int, B_ptr: int, C_ptr: int, N: int, stream: int = 0) -> None:
    _check(load_library().spmm_run_host(h, B_ptr, C_ptr, N, stream or None), "spmm_run_host")


def spmm_destroy(h: int) -> None:
    _check(load_library().spmm_destroy(h), "spmm_destroy")


def spmm_format_info(h: int) -> dict:
    info = spmm_info()
    _check(load_library().spmm_format_info(h, ctypes.byref(info)), "spmm_format_info")
    return {name: getattr(info, name) for name, _ in spmm_info._fields_}


def spmm_export_format(h: int):
    """(ptr int64, idx int32, vals uint16) host copies of the device format arrays."""
    info = spmm_format_info(h)
    ptr = np.zeros(info["n_groups"] + 1, np.int64)
    idx = np.zeros(max(info["n_units"], 1), np.int32)
    vals = np.zeros(max(info["stored"], 1), np.uint16)
    _check(load_library().spmm_export_format(h, ptr.ctypes.data, idx.ctypes.data, vals.ctypes.data),
           "spmm_export_format")
    idx = idx[: info["n_units"]]
    vals = vals[: info["stored"]]
    if info["format"] == SPMM_FORMAT_BCSR:
        vals = vals.reshape(info["n_units"], info["b_row"], info["b_col"])
    else:
        vals = vals.reshape(info["b_row"], info["n_units"])
    return ptr, idx, vals


def spmm_check(h: int, stream: int = 0) -> int:
    """Status word of the handle's kernels (SPMM_OK, SPMM_ERR_TIMEOUT, ...); does not raise."""
    return load_library().spmm_check(h, stream or None)


def spmm_set_max_ctas(h: int, ctas: int) -> None:
    _check(load_library().spmm_set_max_ctas(h, ctas), "spmm_set_max_ctas")


SPMM_SCHEDULE_AUTO = 0
SPMM_SCHEDULE_TILES = 1
SPMM_SCHEDULE_SPLIT = 2
SPMM_SCHEDULE_DYNAMIC = 3


def spmm_set_schedule(h: int, schedule: int) -> None:
    """Work schedule: SPMM_SCHEDULE_AUTO, _TILES, _SPLIT (BCSR) or _DYNAMIC (WCSR, window height 16)."""
    _check(load_library().spmm_set_schedule(h, schedule), "spmm_set_schedule")


def spmm_selftest_wait_timeout(timeout_ns: int, stream: int = 0) -> int:
    out = ctypes.c_int32(-1)
    _check(load_library().spmm_selftest_wait_timeout(timeout_ns, stream or None, ctypes.byref(out)),
           "spmm_selftest_wait_timeout")
    return out.value


def spmm_wcsr_noalloc_check(stream: int = 0) -> int:
    """Status of the last spmm_wcsr_run_noalloc call on the current device
    (waits for `stream`): SPMM_OK, SPMM_ERR_DEVICE_CHECK or SPMM_ERR_TIMEOUT."""
    return load_library().spmm_wcsr_noalloc_check(stream or None)


def spmm_probe_l2_read(buf: int, nbytes: int, passes: int, sink: int, stream: int = 0) -> None:
    """Enqueue `passes` reads of nbytes at device pointer buf (measurement helper)."""
    _check(load_library().spmm_probe_l2_read(buf, nbytes, passes, sink, stream or None), "spmm_probe_l2_read")


def spmm_wcsr_run_noalloc(window_row_ptr: int, window_col_idx: int, values: int, m: int, k: int, p_total: int,
                          in_t, out_t, B_ptr: int, C_ptr: int, N: int, stream: int = 0) -> None:
    """WCSR product from caller-owned device arrays, allocating nothing (pointers are device addresses)."""
    _check(load_library().spmm_wcsr_run_noalloc(window_row_ptr, window_col_idx, values, m, k, p_total, _dt(in_t),
                                                _dt(out_t), B_ptr, C_ptr, N, stream or None), "spmm_wcsr_run_noalloc")


def spmm_bcsr_convert(m, k, row_ptr, col_idx, vals, b_row=64, b_col=64):
    """Host-only CSR -> BCSR with the library's converter: (block_row_ptr, block_col_idx, blocks)."""
    lib = load_library()
    keep, prp, pci, pvv = _csr_args(row_ptr, col_idx, vals)
    nb = ctypes.c_int64(0)
    _check(lib.spmm_bcsr_convert(m, k, prp, pci, pvv, b_row, b_col, ctypes.byref(nb), None, None, None),
           "spmm_bcsr_convert")
    n = nb.value
    ptr = np.zeros(-(-m // b_row) + 1, np.int64)
    idx = np.zeros(max(n, 1), np.int32)
    blocks = np.zeros(max(n, 1) * b_row * b_col, np.uint16)
    _check(lib.spmm_bcsr_convert(m, k, prp, pci, pvv, b_row, b_col, ctypes.byref(nb), ptr.ctypes.data,
                                 idx.ctypes.data, blocks.ctypes.data), "spmm_bcsr_convert")
    return ptr, idx[:n], blocks[: n * b_row * b_col].reshape(n, b_row, b_col)


def spmm_wcsr_convert(m, k, row_ptr, col_idx, vals, window_h=16, col_pad=16):
    """Host-only CSR -> WCSR with the library's converter: (window_row_ptr, window_col_idx, values[h, P])."""
    lib = load_library()
    keep, prp, pci, pvv = _csr_args(row_ptr, col_idx, vals)
    pt = ctypes.c_int64(0)
    _check(lib.spmm_wcsr_convert(m, k, prp, pci, pvv, window_h, col_pad, ctypes.byref(pt), None, None, None),
           "spmm_wcsr_convert")
    P = pt.value
    ptr = np.zeros(-(-m // window_h) + 1, np.int64)
    idx = np.zeros(max(P, 1), np.int32)
    values = np.zeros(max(P, 1) * window_h, np.uint16)
    _check(lib.spmm_wcsr_convert(m, k, prp, pci, pvv, window_h, col_pad, ctypes.byref(pt), ptr.ctypes.data,
                                 idx.ctypes.data, values.ctypes.data), "spmm_wcsr_convert")
    return ptr, idx[:P], values[: P * window_h].reshape(window_h, P)


def spmm_adapters_create(m, k, n_adapters, rank, in_t="bf16", max_rows=0, max_segments=0, grad=False) -> int:
    a = ctypes.c_void_p()
    _check(load_library().spmm_adapters_create(ctypes.byref(a), m, k, n_adapters, rank, _dt(in_t), max_rows,
                                               max_segments, int(grad)), "spmm_adapters_create")
    return a.value


def spmm_adapters_destroy(a: int) -> None:
    _check(load_library().spmm_adapters_destroy(a), "spmm_adapters_destroy")


def spmm_run_linear_adapters(h: int, a: int, X: int, Y: int, N: int, down: int, up: int, scale: int, seg_ptr: int,
                             seg_adapter: int, n_seg: int, stream: int = 0) -> None:
    """Y = X * A^T plus each row's low-rank adapter (device pointers; see include/spmm.h)."""
    _check(load_library().spmm_run_linear_adapters(h, a, X, Y, N, down, up, scale, seg_ptr, seg_adapter, n_seg,
                                                   stream or None), "spmm_run_linear_adapters")


def spmm_adapters_grad(h_t: int, a: int, X: int, dY: int, dX: int, d_down: int, d_up: int, N: int, down: int, up: int,
                       scale: int, seg_ptr: int, seg_adapter: int, n_seg: int, stream: int = 0) -> None:
    """Gradients of spmm_run_linear_adapters (h_t: handle of A^T; dX may be None)."""
    _check(load_library().spmm_adapters_grad(h_t, a, X, dY, dX, d_down, d_up, N, down, up, scale, seg_ptr, seg_adapter,
                                             n_seg, stream or None), "spmm_adapters_grad")


def spmm_route_workspace_bytes(T: int, topk: int, n_experts: int) -> int:
    return load_library().spmm_route_workspace_bytes(T, topk, n_experts)


def spmm_route_sort(ids: int, T: int, topk: int, n_experts: int, offsets: int, order: int, position: int,
                    workspace: int, stream: int = 0) -> None:
    """Stable sort of T x topk expert ids: offsets, order and position (device pointers)."""
    _check(load_library().spmm_route_sort(ids, T, topk, n_experts, offsets, order, position, workspace, stream or None),
           "spmm_route_sort")


def spmm_route_gather(x: int, position: int, n_kept: int, out: int, T: int, topk: int, d: int, dtype, stream: int = 0) -> None:
    _check(load_library().spmm_route_gather(x, position, n_kept, out, T, topk, d, _dt(dtype), stream or None),
           "spmm_route_gather")


def spmm_route_combine(y: int, position: int, weights: int, out: int, T: int, topk: int, d: int, dtype,
                       stream: int = 0) -> None:
    _check(load_library().spmm_route_combine(y, position, weights, out, T, topk, d, _dt(dtype), stream or None),
           "spmm_route_combine")


def spmm_route_combine_grad(dout: int, y: int, position: int, weights: int, n_kept: int, dy: int, dweights: int, T: int,
                            topk: int, d: int, dtype, stream: int = 0) -> None:
    _check(load_library().spmm_route_combine_grad(dout, y, position, weights, n_kept, dy, dweights, T, topk, d, _dt(dtype),
                                                  stream or None), "spmm_route_combine_grad")


# ---------------------------------------------------------------- torch glue
def _torch_stream_ptr():
    import torch
    return torch.cuda.current_stream().cuda_stream


def run_torch(h: int, B, C, stream=None) -> None:
    """spmm_run on torch CUDA tensors B (k x N) and C (m x N), on the current stream."""
    assert B.is_cuda and C.is_cuda and B.is_contiguous() and C.is_contiguous()
    N = B.shape[1]
    assert C.shape[1] == N
    s = stream.cuda_stream if stream is not None else _torch_stream_ptr()
    spmm_run(h, B.data_ptr(), C.data_ptr(), N, s)


class SpMM:
    """Owning wrapper of one handle (destroyed with the object)."""

    def __init__(self, fmt: str, m: int, k: int, row_ptr, col_idx, vals, in_t="bf16", out_t="f32",
                 b_row=None, b_col=None):
        self.fmt = fmt
        self.m, self.k = m, k
        self.in_t, self.out_t = in_t, out_t
        if fmt == "bcsr":
            self.h = spmm_bcsr_create(m, k, row_ptr, col_idx, vals, in_t, out_t, b_row or 64, b_col or 64)
        elif fmt == "wcsr":
            self.h = spmm_wcsr_create(m, k, row_ptr, col_idx, vals, in_t, out_t, b_row or 16, b_col or 16)
        else:
            raise ValueError(fmt)

    def info(self) -> dict:
        return spmm_format_info(self.h)

    def __call__(self, B, C, stream=None):
        run_torch(self.h, B, C, stream)
        return C

    def check(self, stream: int = 0) -> int:
        return spmm_check(self.h, stream)

    def close(self):
        if getattr(self, "h", None):
            spmm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# What the calls below need of torch, looked up once at their first use: a
# decoding step makes several of them, each a few microseconds of host time.
_torch = None
_raw_stream = None
_current_device = None
_ROW_DTYPES = {}


def _load_torch():
    global _torch, _raw_stream, _current_device
    import torch
    _ROW_DTYPES.update({torch.float16: SPMM_F16, torch.bfloat16: SPMM_BF16, torch.float32: SPMM_F32})
    # the current stream's handle without building a Stream object around it (3 us)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    load_library()
    _torch = torch
    return torch


def _refuse(what, t, dtype, shape):
    raise ValueError(f"{what}: expected a contiguous tensor {dtype} {tuple(shape)} on the CUDA device of the others, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _tensor(t, what, dtype, shape, device):
    """Address of t; raises ValueError unless it is a contiguous tensor of this dtype and shape on CUDA device `device`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or device < 0 or not t.is_contiguous():
        _refuse(what, t, dtype, shape)
    return t.data_ptr()


def _stream(device, stream=None):
    """The stream's handle; raises ValueError unless `device`, where the tensors are, is the current device: the library
    launches there, whatever its arguments point to."""
    if device < 0:
        raise ValueError("the tensors are not on a CUDA device")
    if device != _current_device():
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{_current_device()}: call it under "
                         "torch.cuda.device")
    return (stream.cuda_stream if stream is not None else _raw_stream(device)) or None


class Adapters:
    """Low-rank adapters of many requests beside one block-sparse linear layer.

    Holds the shapes and the workspace for batches of up to `max_rows` rows in
    up to `max_segments` segments; the adapters' weights are the caller's:
    down [n_adapters, rank, k], up [n_adapters, m, rank], scale [n_adapters]
    (fp32).  Rows [seg_ptr[s], seg_ptr[s + 1]) use adapter seg_adapter[s], -1 for
    none (int64 / int32 CUDA tensors, read on the device only)."""

    def __init__(self, m: int, k: int, n_adapters: int, rank: int, in_t="bf16", max_rows: int = 0,
                 max_segments: int = 0, grad: bool = True):
        torch = _torch or _load_torch()
        self.m, self.k, self.n_adapters, self.rank = m, k, n_adapters, rank
        self._dtype = {SPMM_F16: torch.float16, SPMM_BF16: torch.bfloat16}.get(_dt(in_t))
        self._down, self._up, self._scale = (n_adapters, rank, k), (n_adapters, m, rank), (n_adapters,)
        self.a = spmm_adapters_create(m, k, n_adapters, rank, in_t, max_rows, max_segments, grad)
        self.device = _current_device()

    def _out(self, layer):
        return _torch.bfloat16 if _dt(layer.out_t) == SPMM_BF16 else _torch.float32

    def _batch(self, device, down, up, scale, seg_ptr, seg_adapter):
        n_seg, dtype = seg_adapter.shape[0], self._dtype
        if device != self.device:
            raise ValueError(f"the tensors are on device {device}, the adapters' workspace on cuda:{self.device}")
        return (_tensor(down, "down", dtype, self._down, device), _tensor(up, "up", dtype, self._up, device),
                _tensor(scale, "scale", _torch.float32, self._scale, device),
                _tensor(seg_ptr, "seg_ptr", _torch.int64, (n_seg + 1,), device),
                _tensor(seg_adapter, "seg_adapter", _torch.int32, (n_seg,), device), n_seg)

    def linear(self, layer: SpMM, X, Y, down, up, scale, seg_ptr, seg_adapter, stream=None):
        """Y = X * A^T plus each row's adapter, for a BCSR layer A (m x k); returns Y."""
        N, device = X.shape[0], X.get_device()
        status = _lib.spmm_run_linear_adapters(
            layer.h, self.a, _tensor(X, "X", self._dtype, (N, self.k), device),
            _tensor(Y, "Y", self._out(layer), (N, self.m), device), N,
            *self._batch(device, down, up, scale, seg_ptr, seg_adapter),
            _stream(device, stream))
        if status:
            _check(status, "spmm_run_linear_adapters")
        return Y

    def grad(self, layer_t: SpMM, X, dY, dX, d_down, d_up, down, up, scale, seg_ptr, seg_adapter, stream=None):
        """Gradients of `linear` into dX (None to leave it out), d_down and d_up; layer_t holds A^T (k x m)."""
        N, device, dtype = X.shape[0], X.get_device(), self._dtype
        status = _lib.spmm_adapters_grad(
            layer_t.h, self.a, _tensor(X, "X", dtype, (N, self.k), device), _tensor(dY, "dY", dtype, (N, self.m), device),
            None if dX is None else _tensor(dX, "dX", self._out(layer_t), (N, self.k), device),
            _tensor(d_down, "d_down", dtype, self._down, device), _tensor(d_up, "d_up", dtype, self._up, device), N,
            *self._batch(device, down, up, scale, seg_ptr, seg_adapter),
            _stream(device, stream))
        if status:
            _check(status, "spmm_adapters_grad")

    def close(self):
        if getattr(self, "a", None):
            spmm_adapters_destroy(self.a)
            self.a = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _row_dtype(t):
    dt = _ROW_DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"rows must be float16, bfloat16 or float32, got {t.dtype}")
    return dt


def route_sort(ids, n_experts: int):
    """(offsets [n_experts + 1] int64, order [T * topk] int32, position [T, topk] int32) of expert ids [T, topk]
    (int32; ids outside [0, n_experts) are dropped), on the current stream."""
    torch = _torch or _load_torch()
    T, topk = shape = ids.shape
    n, at, where = T * topk, ids.get_device(), ids.device
    p, stream = _tensor(ids, "ids", torch.int32, shape, at), _stream(at)
    offsets = torch.empty(n_experts + 1, dtype=torch.int64, device=where)
    order = torch.empty(n, dtype=torch.int32, device=where)
    position = torch.empty_like(ids)
    size = _lib.spmm_route_workspace_bytes(T, topk, n_experts) if n > 4096 else 0  # short lists need none
    work = torch.empty(size, dtype=torch.uint8, device=where) if size else None
    status = _lib.spmm_route_sort(p, T, topk, n_experts, offsets.data_ptr(), order.data_ptr(), position.data_ptr(),
                                  work.data_ptr() if size else None, stream)
    if status:
        _check(status, "spmm_route_sort")
    return offsets, order, position


def route_gather(x, position, offsets):
    """Rows of x [T, d] in slot order [T * topk, d]; slots that no entry takes are 0.  Current stream."""
    torch = _torch or _load_torch()
    T, topk = shape = position.shape
    d, dtype, at, last = x.shape[1], x.dtype, x.get_device(), offsets.shape[0] - 1
    stream = _stream(at)
    out = torch.empty((T * topk, d), dtype=dtype, device=x.device)
    status = _lib.spmm_route_gather(
        _tensor(x, "x", dtype, (T, d), at), _tensor(position, "position", torch.int32, shape, at),
        _tensor(offsets, "offsets", torch.int64, (last + 1,), at) + 8 * last, out.data_ptr(), T, topk, d, _row_dtype(x),
        stream)
    if status:
        _check(status, "spmm_route_gather")
    return out


def route_combine(y, position, weights=None):
    """out[t] = sum_j weights[t, j] * y[position[t, j]] (weights None: ones), fp32 sums.  Current stream."""
    torch = _torch or _load_torch()
    T, topk = shape = position.shape
    d, dtype, at = y.shape[1], y.dtype, y.get_device()
    stream = _stream(at)
    out = torch.empty((T, d), dtype=dtype, device=y.device)
    status = _lib.spmm_route_combine(
        _tensor(y, "y", dtype, (T * topk, d), at), _tensor(position, "position", torch.int32, shape, at),
        None if weights is None else _tensor(weights, "weights", torch.float32, shape, at), out.data_ptr(), T, topk, d,
        _row_dtype(y), stream)
    if status:
        _check(status, "spmm_route_combine")
    return out


def route_combine_grad(dout, y, position, weights, offsets):
    """(dy [T * topk, d], dweights [T, topk] fp32) of route_combine.  Current stream."""
    torch = _torch or _load_torch()
    T, topk = shape = position.shape
    d, dtype, at, last = y.shape[1], y.dtype, y.get_device(), offsets.shape[0] - 1
    stream = _stream(at)
    dy = torch.empty_like(y)
    dw = torch.empty(shape, dtype=torch.float32, device=y.device)
    status = _lib.spmm_route_combine_grad(
        _tensor(dout, "dout", dtype, (T, d), at), _tensor(y, "y", dtype, (T * topk, d), at),
        _tensor(position, "position", torch.int32, shape, at),
        None if weights is None else _tensor(weights, "weights", torch.float32, shape, at),
        _tensor(offsets, "offsets", torch.int64, (last + 1,), at) + 8 * last, dy.data_ptr(), dw.data_ptr(), T, topk, d,
        _row_dtype(y), stream)
    if status:
        _check(status, "spmm_route_combine_grad")
    return dy, dw
