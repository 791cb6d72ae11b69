"""ctypes binding of libqz.so -- argument marshalling only.

Every byte of quantization work happens in the CUDA kernels behind the C ABI
(include/qz.h).  This module packs expert tables into device memory, passes
pointers, sizes and the current CUDA stream, and turns status codes into
exceptions.  There is no fallback: if libqz.so is missing or a call fails, it
raises.  PyTorch supplies device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading
from dataclasses import dataclass
from typing import Iterable, NamedTuple, Optional, Sequence

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqz.so")

# enums of include/qz.h
QZ_OK, QZ_ERR_INVALID_ARG, QZ_ERR_ALIGNMENT, QZ_ERR_UNSUPPORTED, QZ_ERR_CUDA = range(5)
SF_LINEAR, SF_SWIZZLED = 0, 1
FMT_MXFP8, FMT_NVFP4, FMT_FP8_BLOCK128 = 0, 1, 2
NVFP4_PER_TENSOR_GIVEN, NVFP4_PER_TENSOR_COMPUTE, NVFP4_PER_ROW = 0, 1, 2
AMAX_NONE, AMAX_PER_TENSOR, AMAX_PER_ROW = 0, 1, 2
DERR_SHAPE, DERR_NULL, DERR_ALIGN, DERR_TOO_LARGE = 0x1, 0x2, 0x4, 0x8
DERR_TIMEOUT, DERR_CUT = 0x10, 0x20
TEST_WITHHOLD_ARRIVALS = 0x1
OPT_INDEPENDENT = 0x1
MAX_EXPERTS = 4096
MAX_HIDDEN = 16384
MAX_RANKS = 8
TYPE_BF16, TYPE_F32 = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
MAX_ROUTE_EXPERTS, MAX_TOP_K, MAX_GROUPS = 1024, 32, 32

EXPORTED = (
    "qz_sf_bytes",
    "qz_quantize_grouped_mxfp8",
    "qz_quantize_grouped_nvfp4",
    "qz_rmsnorm_quantize",
    "qz_swizzle_scales",
    "qz_status_string",
    "qz_version",
    "qz_workspace_bytes",
    "qz_quantize_grouped_nvfp4_compute_noalloc",
    "qz_dequantize_grouped",
    "qz_attention_merge_quantize",
    "qz_quantize_grouped_colwise",
    "qz_split_fused_experts",
    "qz_allreduce_rmsnorm_quantize",
    "qz_ipc_export",
    "qz_ipc_import",
    "qz_ipc_close",
    "qz_route_experts",
    "qz_route_experts_grad",
    "qz_plan_slots",
    "qz_plan_bytes",
    "qz_plan_experts",
    "qz_expert_product",
    "qz_product_bytes",
    "qz_expert_weight_grad",
    "qz_expert_activation_grad",
    "qz_activation_grad_bytes",
    "qz_dispatch_experts",
    "qz_combine_experts",
)
STATIC_WS_MAX_EXPERTS = 1024


class QzError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class _Expert(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("q", ctypes.c_void_p), ("sf", ctypes.c_void_p),
                ("amax", ctypes.c_void_p)]


class _DqExpert(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64)]


class _SfPair(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("kv", ctypes.c_int64)]


class _FusedSplit(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("cut", ctypes.c_int64),
                ("q_out", ctypes.c_void_p * 2), ("sf_out", ctypes.c_void_p * 2), ("amax_out", ctypes.c_void_p * 2)]


class IpcHandle(ctypes.Structure):
    """struct qz_ipc_handle: a CUDA IPC handle of an allocation and the offset
    of the exported pointer in it."""
    _fields_ = [("handle", ctypes.c_ubyte * 64), ("offset", ctypes.c_uint64), ("alloc_bytes", ctypes.c_uint64),
                ("device", ctypes.c_int), ("reserved", ctypes.c_int)]


class _Router(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("top_k", ctypes.c_int), ("n_groups", ctypes.c_int),
                ("top_groups", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


class _Product(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("activation", ctypes.c_int), ("n_experts", ctypes.c_int),
                ("x_amax_per_row", ctypes.c_int), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("x_rows", ctypes.c_int64), ("slots", ctypes.c_int64), ("x_q", ctypes.c_void_p),
                ("x_sf", ctypes.c_void_p), ("x_amax", ctypes.c_void_p), ("d_rows", ctypes.c_void_p),
                ("d_offsets", ctypes.c_void_p), ("d_counts", ctypes.c_void_p), ("w_q", ctypes.c_void_p),
                ("w_sf", ctypes.c_void_p), ("w_amax", ctypes.c_void_p), ("up_q", ctypes.c_void_p),
                ("up_sf", ctypes.c_void_p), ("up_amax", ctypes.c_void_p), ("w_stride", ctypes.c_int64),
                ("w_sf_stride", ctypes.c_int64), ("bias", ctypes.c_void_p), ("up_bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("ld_out", ctypes.c_int64), ("pre", ctypes.c_void_p), ("ld_pre", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("sf", ctypes.c_void_p)]


# struct qz_product as bytes: packing them is several times faster than filling the ctypes mirror above
_PRODUCT = struct.Struct("=4i4q12Q2q3QqQqQq2Q")


class _WeightGrad(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("n_experts", ctypes.c_int), ("out_type", ctypes.c_int),
                ("accumulate", ctypes.c_int), ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("slots", ctypes.c_int64),
                ("dz_q", ctypes.c_void_p), ("dz_sf", ctypes.c_void_p), ("dz_amax", ctypes.c_void_p),
                ("x_q", ctypes.c_void_p), ("x_sf", ctypes.c_void_p), ("x_amax", ctypes.c_void_p),
                ("d_offsets", ctypes.c_void_p), ("d_counts", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class _Opts(ctypes.Structure):
    _fields_ = [("d_err", ctypes.c_void_p), ("max_ctas", ctypes.c_int), ("d_workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("elems_hint", ctypes.c_int64),
                ("wait_limit_ns", ctypes.c_int64), ("test_flags", ctypes.c_uint), ("launch_flags", ctypes.c_uint)]


assert ctypes.sizeof(_Expert) == 56 and ctypes.sizeof(_SfPair) == 32 and ctypes.sizeof(_DqExpert) == 56
assert ctypes.sizeof(_FusedSplit) == 96 and ctypes.sizeof(IpcHandle) == 88
assert ctypes.sizeof(_Product) == _PRODUCT.size

_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libqz.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m nvfp4_quantization_moe_b200.build` (nvcc, sm_100a)")
        lib = ctypes.CDLL(path)
        P, I, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        lib.qz_sf_bytes.restype = ctypes.c_size_t
        lib.qz_sf_bytes.argtypes = [i64, i64, I, I]
        lib.qz_quantize_grouped_mxfp8.restype = I
        lib.qz_quantize_grouped_mxfp8.argtypes = [P, I, I, P, P]
        lib.qz_quantize_grouped_nvfp4.restype = I
        lib.qz_quantize_grouped_nvfp4.argtypes = [P, I, I, I, P, P]
        lib.qz_rmsnorm_quantize.restype = I
        lib.qz_rmsnorm_quantize.argtypes = [P, P, P, ctypes.c_float, i64, i64, P, P, I, P, P, I, P, P]
        lib.qz_swizzle_scales.restype = I
        lib.qz_swizzle_scales.argtypes = [P, I, P, P]
        lib.qz_status_string.restype = ctypes.c_char_p
        lib.qz_status_string.argtypes = [I]
        lib.qz_version.restype = I
        lib.qz_version.argtypes = []
        lib.qz_workspace_bytes.restype = ctypes.c_size_t
        lib.qz_workspace_bytes.argtypes = [I]
        lib.qz_quantize_grouped_nvfp4_compute_noalloc.restype = I
        lib.qz_quantize_grouped_nvfp4_compute_noalloc.argtypes = [P, I, I, P, P]
        lib.qz_dequantize_grouped.restype = I
        lib.qz_dequantize_grouped.argtypes = [P, I, I, I, I, P, P]
        lib.qz_quantize_grouped_colwise.restype = I
        lib.qz_quantize_grouped_colwise.argtypes = [P, I, I, I, P, P]
        lib.qz_attention_merge_quantize.restype = I
        lib.qz_attention_merge_quantize.argtypes = [P, P, I, i64, i64, P, P, P, I, P]
        lib.qz_split_fused_experts.restype = I
        lib.qz_split_fused_experts.argtypes = [P, I, I, I, I, I, P, P]
        lib.qz_ipc_export.restype = I
        lib.qz_ipc_export.argtypes = [P, P]
        lib.qz_ipc_import.restype = I
        lib.qz_ipc_import.argtypes = [P, P]
        lib.qz_ipc_close.restype = I
        lib.qz_ipc_close.argtypes = [P, P]
        lib.qz_allreduce_rmsnorm_quantize.restype = I
        lib.qz_allreduce_rmsnorm_quantize.argtypes = [P, I, P, P, ctypes.c_float, i64, i64, i64, i64, P, I, I, I,
                                                      P, P]
        lib.qz_route_experts.restype = I
        lib.qz_route_experts.argtypes = [P, I, i64, I, i64, P, P, P, P, P]
        lib.qz_route_experts_grad.restype = I
        lib.qz_route_experts_grad.argtypes = [P, I, i64, I, i64, P, P, P, P, i64, P]
        lib.qz_plan_slots.restype = i64
        lib.qz_plan_slots.argtypes = [i64, I, I, I]
        lib.qz_plan_bytes.restype = ctypes.c_size_t
        lib.qz_plan_bytes.argtypes = [i64, I, I]
        lib.qz_plan_experts.restype = I
        lib.qz_plan_experts.argtypes = [P, i64, I, I, I, P, P, P, P, P, ctypes.c_size_t, P]
        lib.qz_expert_product.restype = I
        lib.qz_expert_product.argtypes = [P, P, P]
        lib.qz_product_bytes.restype = ctypes.c_size_t
        lib.qz_product_bytes.argtypes = [P]
        lib.qz_expert_weight_grad.restype = I
        lib.qz_expert_weight_grad.argtypes = [P, P, P]
        lib.qz_activation_grad_bytes.restype = ctypes.c_size_t
        lib.qz_activation_grad_bytes.argtypes = [i64, i64, I, I]
        lib.qz_expert_activation_grad.restype = I
        lib.qz_expert_activation_grad.argtypes = [P, i64, P, i64, i64, i64, I, I, P, P, I, P, i64, P, P, P]
        lib.qz_dispatch_experts.restype = I
        lib.qz_dispatch_experts.argtypes = [P, i64, P, P, i64, I, i64, i64, P, P, i64, P, i64, P, P]
        lib.qz_combine_experts.restype = I
        lib.qz_combine_experts.argtypes = [P, i64, P, i64, I, i64, i64, P, P, i64, P, i64, P]
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().qz_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != QZ_OK:
        raise QzError(status, where)


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _opts(err: Optional[torch.Tensor], max_ctas: int, workspace: Optional[torch.Tensor] = None, elems_hint: int = 0,
          wait_limit_ns: int = 0, test_flags: int = 0, launch_flags: int = 0):
    if (err is None and not max_ctas and workspace is None and not elems_hint and not wait_limit_ns and not test_flags
            and not launch_flags):
        return None
    if err is not None:
        assert err.dtype in (torch.int32, torch.uint32) and err.is_cuda and err.numel() >= 1
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return ctypes.byref(_Opts(ctypes.c_void_p(err.data_ptr() if err is not None else 0), int(max_ctas),
                              ctypes.c_void_p(ws_ptr), ctypes.c_size_t(ws_bytes), ctypes.c_int64(int(elems_hint)),
                              ctypes.c_int64(int(wait_limit_ns)), ctypes.c_uint(int(test_flags)),
                              ctypes.c_uint(int(launch_flags))))


def workspace_bytes(n_experts: int) -> int:
    """Device scratch for the single-launch computed-amax NVFP4 path."""
    return int(load().qz_workspace_bytes(int(n_experts)))


def alloc_workspace(n_experts: int, device=None) -> torch.Tensor:
    return torch.empty(max(workspace_bytes(n_experts), 4), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else int(t.data_ptr())


def sf_bytes(rows: int, cols: int, fmt: int, layout: int) -> int:
    return int(load().qz_sf_bytes(int(rows), int(cols), int(fmt), int(layout)))


# ---------------------------------------------------------------------------
# device tables
# ---------------------------------------------------------------------------

@dataclass
class Entry:
    """One expert: a bf16 [rows, cols] view (row stride in elements may exceed
    cols), its payload, SF region and (NVFP4) amax storage."""
    x: torch.Tensor
    q: torch.Tensor
    sf: torch.Tensor
    amax: Optional[torch.Tensor] = None


class ExpertTable:
    """A device-resident array of qz_expert entries.  Keeps references to the
    tensors it points into, so they outlive the table."""

    def __init__(self, entries: Sequence[Entry], device=None):
        self.entries = list(entries)
        n = len(self.entries)
        arr = (_Expert * max(n, 1))()
        for i, e in enumerate(self.entries):
            x = e.x
            assert x.dtype == torch.bfloat16 and x.dim() == 2
            rows, cols = x.shape
            ld = x.stride(0) if rows > 1 else max(cols, x.stride(0))
            assert rows == 0 or x.stride(1) == 1, "rows must be contiguous"
            arr[i] = _Expert(x.data_ptr() if rows else 0, rows, cols, ld, _ptr(e.q) if rows else 0,
                             _ptr(e.sf) if rows else 0, _ptr(e.amax))
        host = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
        dev = device if device is not None else (self.entries[0].x.device if n else torch.device("cuda"))
        self.dev = host.to(dev)
        self.n = n
        self.elems = sum(int(e.x.shape[0]) * int(e.x.shape[1]) for e in self.entries)

    @property
    def ptr(self) -> int:
        return int(self.dev.data_ptr()) if self.n else 0

    @classmethod
    def from_raw(cls, raw: Iterable[tuple], device) -> "ExpertTable":
        """Entries from raw (x_ptr, rows, cols, ld, q_ptr, sf_ptr, amax_ptr) tuples
        (tests use this to build deliberately invalid entries)."""
        self = cls.__new__(cls)
        raw = list(raw)
        arr = (_Expert * max(len(raw), 1))(*[_Expert(*r) for r in raw])
        self.entries = []
        self.n = len(raw)
        self.elems = 0
        self.dev = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(device)
        return self


@dataclass
class DqEntry:
    """One quantized expert to decode: payload q ([rows, cols] e4m3 or
    [rows, cols/2] packed e2m1), its SF region, its amax (NVFP4) and the bf16
    output y [rows, cols] (row stride may exceed cols)."""
    q: torch.Tensor
    sf: torch.Tensor
    y: torch.Tensor
    amax: Optional[torch.Tensor] = None


class DqTable:
    """A device-resident array of qz_dq_expert entries (keeps its tensors alive)."""

    def __init__(self, entries: Sequence[DqEntry], device=None):
        self.entries = list(entries)
        n = len(self.entries)
        arr = (_DqExpert * max(n, 1))()
        for i, e in enumerate(self.entries):
            y = e.y
            assert y.dtype == torch.bfloat16 and y.dim() == 2
            rows, cols = y.shape
            ldy = y.stride(0) if rows > 1 else max(cols, y.stride(0))
            assert rows == 0 or y.stride(1) == 1, "rows must be contiguous"
            arr[i] = _DqExpert(_ptr(e.q) if rows else 0, _ptr(e.sf) if rows else 0, _ptr(e.amax), rows, cols,
                               y.data_ptr() if rows else 0, ldy)
        host = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
        dev = device if device is not None else (self.entries[0].y.device if n else torch.device("cuda"))
        self.dev = host.to(dev)
        self.n = n
        self.elems = sum(int(e.y.shape[0]) * int(e.y.shape[1]) for e in self.entries)

    @property
    def ptr(self) -> int:
        return int(self.dev.data_ptr()) if self.n else 0

    @classmethod
    def from_raw(cls, raw: Iterable[tuple], device) -> "DqTable":
        """Entries from raw (q_ptr, sf_ptr, amax_ptr, rows, cols, y_ptr, ldy) tuples."""
        self = cls.__new__(cls)
        raw = list(raw)
        arr = (_DqExpert * max(len(raw), 1))(*[_DqExpert(*r) for r in raw])
        self.entries = []
        self.n = len(raw)
        self.elems = 0
        self.dev = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(device)
        return self


@dataclass
class SplitEntry:
    """One folded fused expert to cut at row ``cut``: its payload q (rows
    [rows, row_bytes]), scales sf, amax, and each part's outputs.  q_out[p] may
    be None (that part's payload is not copied)."""
    q: torch.Tensor
    sf: torch.Tensor
    rows: int
    cols: int
    cut: int
    sf_out: tuple
    q_out: tuple = (None, None)
    amax: Optional[torch.Tensor] = None
    amax_out: tuple = (None, None)


class SplitTable:
    """A device-resident array of qz_fused_split entries (keeps its tensors alive)."""

    def __init__(self, entries: Sequence[SplitEntry], device=None):
        self.entries = list(entries)
        n = len(self.entries)
        arr = (_FusedSplit * max(n, 1))()
        P2 = ctypes.c_void_p * 2
        for i, e in enumerate(self.entries):
            arr[i] = _FusedSplit(_ptr(e.q), _ptr(e.sf), _ptr(e.amax), int(e.rows), int(e.cols), int(e.cut),
                                 P2(*[_ptr(t) for t in e.q_out]), P2(*[_ptr(t) for t in e.sf_out]),
                                 P2(*[_ptr(t) for t in e.amax_out]))
        host = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8)
        dev = device if device is not None else (self.entries[0].q.device if n else torch.device("cuda"))
        self.dev = host.to(dev)
        self.n = n

    @property
    def ptr(self) -> int:
        return int(self.dev.data_ptr()) if self.n else 0

    @classmethod
    def from_raw(cls, raw: Iterable[tuple], device) -> "SplitTable":
        """Entries from raw (q, sf, amax, rows, cols, cut, (q0, q1), (sf0, sf1), (a0, a1)) tuples of
        integers (tests use this to build deliberately invalid entries)."""
        self = cls.__new__(cls)
        raw = list(raw)
        P2 = ctypes.c_void_p * 2
        arr = (_FusedSplit * max(len(raw), 1))(*[_FusedSplit(*r[:6], P2(*r[6]), P2(*r[7]), P2(*r[8])) for r in raw])
        self.entries = []
        self.n = len(raw)
        self.dev = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(device)
        return self


class SfPairTable:
    def __init__(self, pairs: Sequence[tuple], device):
        """pairs: (src linear uint8 tensor, dst swizzled uint8 tensor, rows, kv)."""
        self.pairs = list(pairs)
        arr = (_SfPair * max(len(self.pairs), 1))()
        for i, (src, dst, rows, kv) in enumerate(self.pairs):
            arr[i] = _SfPair(_ptr(src), _ptr(dst), int(rows), int(kv))
        self.dev = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(device)
        self.n = len(self.pairs)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def quantize_grouped_mxfp8(table: ExpertTable, layout: int, stream=None, err=None, max_ctas: int = 0,
                           independent: bool = False):
    """MXFP8 over the table; the table's element count goes along as the
    grid-size hint.  ``independent`` sets QZ_OPT_INDEPENDENT (the call touches
    nothing that work still running on the stream touches)."""
    _check(load().qz_quantize_grouped_mxfp8(ctypes.c_void_p(table.ptr), table.n, int(layout),
                                            _stream_ptr(stream),
                                            _opts(err, max_ctas, elems_hint=getattr(table, "elems", 0),
                                                  launch_flags=OPT_INDEPENDENT if independent else 0)),
           "qz_quantize_grouped_mxfp8")


def quantize_grouped_nvfp4(table: ExpertTable, mode: int, layout: int, stream=None, err=None, max_ctas: int = 0,
                           workspace: Optional[torch.Tensor] = None, wait_limit_ns: int = 0, test_flags: int = 0,
                           independent: bool = False):
    _check(load().qz_quantize_grouped_nvfp4(ctypes.c_void_p(table.ptr), table.n, int(mode), int(layout),
                                            _stream_ptr(stream),
                                            _opts(err, max_ctas, workspace, wait_limit_ns=wait_limit_ns,
                                                  test_flags=test_flags,
                                                  launch_flags=OPT_INDEPENDENT if independent else 0)),
           "qz_quantize_grouped_nvfp4")


def quantize_grouped_nvfp4_compute_noalloc(table: ExpertTable, layout: int, stream=None, err=None, max_ctas: int = 0,
                                           wait_limit_ns: int = 0):
    """NVFP4 with computed per-tensor amax, scratch inside the library (no
    device allocation by anyone; see qz_quantize_grouped_nvfp4_compute_noalloc)."""
    _check(load().qz_quantize_grouped_nvfp4_compute_noalloc(ctypes.c_void_p(table.ptr), table.n, int(layout),
                                                            _stream_ptr(stream),
                                                            _opts(err, max_ctas, wait_limit_ns=wait_limit_ns)),
           "qz_quantize_grouped_nvfp4_compute_noalloc")


def rmsnorm_quantize(x, residual, gamma, eps: float, norm_out, residual_out, fmt: int, q, sf, layout: int,
                     global_amax=None, stream=None):
    T, H = x.shape
    _check(load().qz_rmsnorm_quantize(ctypes.c_void_p(_ptr(x)), ctypes.c_void_p(_ptr(residual)),
                                      ctypes.c_void_p(_ptr(gamma)), ctypes.c_float(eps), int(T), int(H),
                                      ctypes.c_void_p(_ptr(norm_out)), ctypes.c_void_p(_ptr(residual_out)),
                                      int(fmt), ctypes.c_void_p(_ptr(q)), ctypes.c_void_p(_ptr(sf)), int(layout),
                                      ctypes.c_void_p(_ptr(global_amax)), _stream_ptr(stream)),
           "qz_rmsnorm_quantize")


class NormDest(ctypes.Structure):
    """One destination of the AllReduce epilogue (struct qz_norm_dest)."""
    _fields_ = [("norm_out", ctypes.c_void_p), ("residual_out", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("sf", ctypes.c_void_p)]


def _addr(t) -> int:
    """A tensor's device address, or an address given as an int (a peer mapping)."""
    return int(t) if isinstance(t, int) else _ptr(t)


def allreduce_rmsnorm_quantize(rank_x, residual, gamma, eps: float, dests, fmt: int, layout: int, T: int, H: int,
                               rows=None, global_amax=None, stream=None):
    """AllReduce of the rank inputs + residual add + RMSNorm + quantize
    (qz_allreduce_rmsnorm_quantize).  ``rank_x``: bf16 [T, H] tensors or device
    addresses (peer mappings), summed in this order; ``dests``: tuples
    (norm_out, residual_out or None, q, sf) of tensors or addresses, each
    written with the rows ``rows`` = (row_begin, row_end), default all T.
    Every pointer argument takes a tensor, an int address or None."""
    row_begin, row_end = (0, T) if rows is None else rows
    xs = (ctypes.c_void_p * len(rank_x))(*[_addr(x) for x in rank_x])
    ds = (NormDest * len(dests))(*[NormDest(*[_addr(p) for p in d]) for d in dests])
    _check(load().qz_allreduce_rmsnorm_quantize(
        ctypes.cast(xs, ctypes.c_void_p), len(rank_x), ctypes.c_void_p(_addr(residual)),
        ctypes.c_void_p(_addr(gamma)), ctypes.c_float(eps), int(T), int(H), int(row_begin), int(row_end),
        ctypes.cast(ds, ctypes.c_void_p), len(dests), int(fmt), int(layout), ctypes.c_void_p(_addr(global_amax)),
        _stream_ptr(stream)),
        "qz_allreduce_rmsnorm_quantize")


def ipc_export(ptr: int) -> bytes:
    """qz_ipc_export: the IPC handle (88 bytes) of the device allocation holding ``ptr``."""
    h = IpcHandle()
    _check(load().qz_ipc_export(ctypes.c_void_p(int(ptr)), ctypes.byref(h)), "qz_ipc_export")
    return bytes(h)


def ipc_import(handle: bytes) -> int:
    """qz_ipc_import: map a peer process's exported allocation; returns the
    peer's pointer as an address in this process."""
    h = IpcHandle.from_buffer_copy(handle)
    out = ctypes.c_void_p()
    _check(load().qz_ipc_import(ctypes.byref(h), ctypes.byref(out)), "qz_ipc_import")
    return int(out.value)


def ipc_close(ptr: int, handle: bytes) -> None:
    """qz_ipc_close: unmap a pointer returned by ipc_import for ``handle``."""
    h = IpcHandle.from_buffer_copy(handle)
    _check(load().qz_ipc_close(ctypes.c_void_p(int(ptr)), ctypes.byref(h)), "qz_ipc_close")


def dequantize_grouped(table: DqTable, fmt: int, per_row: bool, layout: int, stream=None, err=None,
                       max_ctas: int = 0):
    _check(load().qz_dequantize_grouped(ctypes.c_void_p(table.ptr), table.n, int(fmt), 1 if per_row else 0,
                                        int(layout), _stream_ptr(stream),
                                        _opts(err, max_ctas, elems_hint=getattr(table, "elems", 0))),
           "qz_dequantize_grouped")


def quantize_grouped_colwise(table: ExpertTable, fmt: int, layout: int, stream=None, err=None, max_ctas: int = 0):
    """Column-wise quantization: each entry's q / sf receive x^T quantized
    row-wise (q [cols, rows] or [cols, rows/2]); NVFP4 uses the given amax."""
    _check(load().qz_quantize_grouped_colwise(ctypes.c_void_p(table.ptr), table.n, int(fmt), int(layout),
                                              _stream_ptr(stream), _opts(err, max_ctas)),
           "qz_quantize_grouped_colwise")


def attention_merge_quantize(partial, lse, out, q=None, sf=None, layout: int = SF_SWIZZLED, stream=None):
    """Merge float partial outputs [S, T, H] by their log-sum-exps [S, T] into
    bf16 out [T, H] and (q given) its MXFP8 form q [T, H] + SF region sf."""
    S, T, H = partial.shape
    _check(load().qz_attention_merge_quantize(ctypes.c_void_p(_ptr(partial)), ctypes.c_void_p(_ptr(lse)), int(S),
                                              int(T), int(H), ctypes.c_void_p(_ptr(out)), ctypes.c_void_p(_ptr(q)),
                                              ctypes.c_void_p(_ptr(sf)), int(layout), _stream_ptr(stream)),
           "qz_attention_merge_quantize")


def split_fused_experts(table: SplitTable, fmt: int, amax_kind: int, src_layout: int, dst_layout: int, stream=None,
                        err=None, max_ctas: int = 0):
    """Cut folded fused experts into gate (rows [0, cut)) and up (rows [cut, rows)):
    payload rows, scales re-laid per part in dst_layout, amax shared or cut."""
    _check(load().qz_split_fused_experts(ctypes.c_void_p(table.ptr), table.n, int(fmt), int(amax_kind),
                                         int(src_layout), int(dst_layout), _stream_ptr(stream), _opts(err, max_ctas)),
           "qz_split_fused_experts")


def swizzle_scales(table: SfPairTable, stream=None, err=None, max_ctas: int = 0):
    _check(load().qz_swizzle_scales(ctypes.c_void_p(int(table.dev.data_ptr()) if table.n else 0), table.n,
                                    _stream_ptr(stream), _opts(err, max_ctas)),
           "qz_swizzle_scales")


# ---------------------------------------------------------------------------
# the mixture-of-experts layer: routing, the experts' products, the moves
# between token order and expert order
# ---------------------------------------------------------------------------

# A decode step makes these calls once per layer and is bound by the host, so
# the checks below read each property once and format a message only to raise it.
# What a call allocates, outputs and scratch, belongs to the stream it runs on.

def _require(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _raw_stream(stream, dev: int) -> int:
    """The stream to launch on; refuses a call whose tensors (all on device
    ``dev``) are not on the current CUDA device, where the launch goes."""
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current CUDA device, not " + (f"cuda:{dev}" if dev >= 0 else "cpu"))
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _tensor(t, name: str, dtype, dev: int, shape=None, optional: bool = False) -> int:
    """Address of a contiguous CUDA tensor of the given type (and shape), 0 for an absent optional one."""
    if t is None:
        if not optional:
            raise ValueError(f"{name} is required")
        return 0
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device: {t.device}")
    return t.data_ptr()


def _matrix(t, name: str, dtype, dev: int, shape, optional: bool = False):
    """(address, row stride) of a CUDA matrix whose rows are contiguous; (0, 0) for an absent optional one."""
    if t is None:
        if not optional:
            raise ValueError(f"{name} is required")
        return 0, 0
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    ld, one = t.stride()
    if one != 1 and shape[1] != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device: {t.device}")
    return t.data_ptr(), ld if shape[0] > 1 else shape[1]


def _codes(t, name: str, cols: int, fmt: int, dev: int) -> int:
    """Payloads come as uint8 bytes (or, for MXFP8, as torch.float8_e4m3fn): [..., cols] or [..., cols / 2]."""
    if t.dtype is not torch.uint8 and (fmt != FMT_MXFP8 or t.dtype is not torch.float8_e4m3fn):
        raise ValueError(f"{name} must be a quantized payload, not {t.dtype}")
    if t.shape[-1] != (cols if fmt == FMT_MXFP8 else cols // 2):
        raise ValueError(f"the last axis of {name} does not match")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device: {t.device}")
    return t.data_ptr()


def _torch_stream(stream):
    """The torch stream of a stream argument (a torch stream, an object with cuda_stream, or a handle)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.ExternalStream(raw) if raw else torch.cuda.default_stream()


def _on(stream):
    """A context in which torch allocates, copies and frees on the call's stream
    (a table of pointers too is scratch of the launch that reads it)."""
    return torch.cuda.stream(None if stream is None else _torch_stream(stream))


def _empty(like: torch.Tensor, shape, dtype, stream):
    """A buffer that a call writes, from the pool of the call's stream: a block of
    the current stream's pool may still be in use there by what it was freed from,
    and the call does not wait for that."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on(stream):
        return like.new_empty(shape, dtype=dtype)


def _scratch(nbytes: int, like: torch.Tensor, stream):
    """Device scratch of one call from torch's allocator, None for none.  Freed
    after the launch, it goes to the next user on the same stream."""
    return _empty(like, nbytes, torch.uint8, stream) if nbytes else None


def _parts(x, name: str):
    n = len(x) if isinstance(x, (tuple, list)) else 0
    if n == 3:
        return x
    if n != 2:
        raise ValueError(f"{name} must be (payload, scales) or (payload, scales, amax)")
    return x[0], x[1], None


@functools.lru_cache(maxsize=64)
def _router(top_k, score, n_groups, top_groups, renormalize, scale):
    """struct qz_router of these values (only ever read)."""
    return ctypes.byref(_Router(int(score), int(top_k), int(n_groups), int(top_groups), 1 if renormalize else 0,
                                float(scale)))


def _float_type(t, name: str) -> int:
    if t.dtype is torch.bfloat16:
        return TYPE_BF16
    if t.dtype is not torch.float32:
        raise ValueError(f"{name} must be bfloat16 or float32, not {t.dtype}")
    return TYPE_F32


def route_experts(logits: torch.Tensor, top_k: int, *, score: int = SCORE_SOFTMAX, bias=None, n_groups: int = 1,
                  top_groups: Optional[int] = None, renormalize: bool = True, scale: float = 1.0, ids=None,
                  weights=None, stream=None):
    """Router (qz_route_experts): bf16 or fp32 logits [T, E] to the top_k experts
    of each token.  Returns (ids int32 [T, top_k], weights fp32 [T, top_k]),
    written into ``ids`` and ``weights`` when given.  ``bias`` (fp32 [E]) steers
    the choice only; ``top_groups`` (default all) of ``n_groups`` groups of
    consecutive experts stay in the choice."""
    _require(logits.dim() == 2, "logits must be [T, E]")
    kind = _float_type(logits, "logits")
    dev = logits.get_device()
    T, E = logits.shape
    x, ld = _matrix(logits, "logits", logits.dtype, dev, (T, E))
    b = _tensor(bias, "bias", torch.float32, dev, (E,), optional=True)
    _require(top_k >= 1, "top_k must be at least 1")
    if ids is None:
        ids = _empty(logits, (T, top_k), torch.int32, stream)
        i = ids.data_ptr()
    else:
        i = _tensor(ids, "ids", torch.int32, dev, (T, top_k))
    if weights is None:
        weights = _empty(logits, (T, top_k), torch.float32, stream)
        w = weights.data_ptr()
    else:
        w = _tensor(weights, "weights", torch.float32, dev, (T, top_k))
    _check(load().qz_route_experts(x, kind, T, E, ld, b,
                                   _router(top_k, score, n_groups, n_groups if top_groups is None else top_groups,
                                           renormalize, scale), i, w, _raw_stream(stream, dev)), "qz_route_experts")
    return ids, weights


def route_experts_grad(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor, *, score: int = SCORE_SOFTMAX,
                       renormalize: bool = True, scale: float = 1.0, dlogits=None, stream=None):
    """Gradient of the router's weights with respect to the logits, for the
    choices ``ids`` (qz_route_experts_grad); returns dlogits [T, E] of the
    logits' type."""
    _require(logits.dim() == 2 and ids.dim() == 2, "logits must be [T, E] and ids [T, top_k]")
    kind = _float_type(logits, "logits")
    dev = logits.get_device()
    T, E = logits.shape
    k = ids.shape[1]
    x, ld = _matrix(logits, "logits", logits.dtype, dev, (T, E))
    i = _tensor(ids, "ids", torch.int32, dev, (T, k))
    g = _tensor(dweights, "dweights", torch.float32, dev, (T, k))
    if dlogits is None:
        dlogits = _empty(logits, (T, E), logits.dtype, stream)
        d, ldd = dlogits.data_ptr(), E
    else:
        d, ldd = _matrix(dlogits, "dlogits", logits.dtype, dev, (T, E))
    _check(load().qz_route_experts_grad(x, kind, T, E, ld, _router(k, score, 1, 1, renormalize, scale), i, g, d, ldd,
                                        _raw_stream(stream, dev)), "qz_route_experts_grad")
    return dlogits


def plan_slots(T: int, top_k: int, n_experts: int, align: int = 1) -> int:
    """Slots a plan of T tokens can need (qz_plan_slots)."""
    return int(load().qz_plan_slots(int(T), int(top_k), int(n_experts), int(align)))


class ExpertPlan(NamedTuple):
    """Expert order of a router's choices: expert e has the slots [offsets[e],
    offsets[e] + counts[e]); rows gives each slot's token (-1: unused), slots
    each (token, choice) pair's slot (-1: none).  All int32 on the device."""
    offsets: torch.Tensor
    counts: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


@functools.lru_cache(maxsize=256)
def _plan_sizes(T: int, k: int, n_experts: int, align: int):
    return load().qz_plan_slots(T, k, n_experts, align), load().qz_plan_bytes(T, k, n_experts)


@functools.lru_cache(maxsize=256)
def _region(N: int, K: int, fmt: int) -> int:
    return load().qz_sf_bytes(N, K, fmt, SF_SWIZZLED)


def plan_experts(ids: torch.Tensor, n_experts: int, *, align: int = 1, plan: Optional[ExpertPlan] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> ExpertPlan:
    """Sort the choices ``ids`` [T, top_k] by expert (qz_plan_experts), each
    expert's slots starting at a multiple of ``align``.  The outputs (and, for
    many pairs, the scratch) are allocated unless given."""
    _require(ids.dim() == 2, "ids must be [T, top_k]")
    T, k = ids.shape
    dev = ids.get_device()
    i = _tensor(ids, "ids", torch.int32, dev)
    lib = load()
    n, need = _plan_sizes(T, k, n_experts, align)
    if plan is None:
        _require(n_experts >= 1, "n_experts must be at least 1")
        buf = _empty(ids, 2 * n_experts + 1 + n + T * k, torch.int32, stream)
        offsets, counts, rows, slots = buf.split_with_sizes((n_experts + 1, n_experts, n, T * k))
        plan = ExpertPlan(offsets, counts, rows, slots.view(T, k))
        at = buf.data_ptr()
        parts = (at, at + 4 * (n_experts + 1), at + 4 * (2 * n_experts + 1), at + 4 * (2 * n_experts + 1 + n))
    else:
        parts = (_tensor(plan.offsets, "offsets", torch.int32, dev, (n_experts + 1,)),
                 _tensor(plan.counts, "counts", torch.int32, dev, (n_experts,)),
                 _tensor(plan.rows, "rows", torch.int32, dev, (n,)),
                 _tensor(plan.slots, "slots", torch.int32, dev, (T, k)))
    ws = 0
    if workspace is not None:
        ws = _tensor(workspace, "workspace", torch.uint8, dev)
    elif need:
        workspace = _scratch(need, ids, stream)
        ws = workspace.data_ptr()
    _check(lib.qz_plan_experts(i, T, k, n_experts, align, *parts, ws, 0 if workspace is None else workspace.numel(),
                               _raw_stream(stream, dev)), "qz_plan_experts")
    return plan


def _expert_lists(offsets, counts, n_experts: int, dev: int):
    """Addresses of offsets ([n_experts] or [n_experts + 1]) and counts."""
    _require(offsets.dim() == 1 and offsets.numel() in (n_experts, n_experts + 1), "offsets must be [n_experts + 1]")
    return _tensor(offsets, "offsets", torch.int32, dev), _tensor(counts, "counts", torch.int32, dev, (n_experts,))


def _stacked(part, name: str, fmt: int, E: int, N: int, K: int, region: int, dev: int):
    """(payload, scales, amax, payload stride, scale stride) of stacked expert weights."""
    q, sf, amax = part
    if q.dim() != 3 or q.shape[0] != E or q.shape[1] != N:
        raise ValueError(f"{name} must be [E, N, K]")
    apart, row, one = q.stride()
    cols = q.shape[2]
    if one != 1 or (N > 1 and row != cols):
        raise ValueError(f"{name}: an expert's rows must be dense")
    if (sf.dim() != 2 or sf.shape[0] != E or sf.dtype is not torch.uint8 or sf.stride(1) != 1 or sf.shape[1] < region
            or sf.get_device() != dev):
        raise ValueError(f"{name}: scales must be [E, region] bytes on the weights' device")
    return (_codes(q, name, K, fmt, dev), sf.data_ptr(),
            _tensor(amax, "a weight's amax", torch.float32, dev, (E,)) if fmt == FMT_NVFP4 else 0,
            apart if E > 1 else N * cols, sf.stride(0) if E > 1 else (sf.shape[1] + 15) // 16 * 16)


def expert_product(fmt: int, x, w, offsets: torch.Tensor, counts: torch.Tensor, out: torch.Tensor, *, rows=None,
                   up=None, bias=None, up_bias=None, activation: int = ACT_NONE, residual=None, pre=None, q=None,
                   sf=None, workspace=None, stream=None, err=None, max_ctas: int = 0):
    """The experts' matrix products with bias, activation, gate and residual in
    the epilogue (qz_expert_product).

    x:  (payload [R, K], linear scales [R, K/block], NVFP4: amax [R] or [1])
    w:  (payload [E, N, K], swizzled scales [E, region], NVFP4: amax [E]); an
        expert's payload rows and region are dense, experts may be further
        apart (a view of the gate or up half of fused weights)
    up: a second weight like w (same strides): out = act(x w) * (x up)
    out: bf16 [slots, N]; rows: int32 [slots] row of x of each slot (None: the
    slot's own number); bias, up_bias: bf16 [E, N]; residual: bf16 [slots, N];
    pre: bf16 [slots, N or 2N] receives the pre-activations; q [slots, N] and
    sf [slots, N/32] receive the MXFP8 form of out.  A large call with rows
    uses a workspace (allocated unless given) to put them in order first."""
    xq, xsf, xa = _parts(x, "x")
    wq, wsf, wa = _parts(w, "w")
    if xq.dim() != 2 or wq.dim() != 3 or out.dim() != 2:
        raise ValueError("x must be [R, K], w [E, N, K], out [slots, N]")
    if fmt != FMT_MXFP8 and fmt != FMT_NVFP4:
        raise ValueError("fmt must be FMT_MXFP8 or FMT_NVFP4")
    if not xq.is_contiguous():
        raise ValueError("x must be contiguous")
    fp4 = fmt == FMT_NVFP4
    dev = out.get_device()
    E, N, _ = wq.shape
    R, K = xq.shape
    S = out.shape[0]
    if fp4:
        K *= 2
    kv = K // (16 if fp4 else 32)

    region = _region(N, K, fmt)
    wp = _stacked((wq, wsf, wa), "w", fmt, E, N, K, region, dev)
    upp = (0, 0, 0)
    if up is not None:
        upp = _stacked(_parts(up, "up"), "up", fmt, E, N, K, region, dev)
        if upp[3:] != wp[3:]:
            raise ValueError("w and up must have the same strides")
    offs, cnts = _expert_lists(offsets, counts, E, dev)
    o, ldo = _matrix(out, "out", torch.bfloat16, dev, (S, N))
    r, ldr = _matrix(residual, "residual", torch.bfloat16, dev, (S, N), optional=True)
    z, ldz = _matrix(pre, "pre", torch.bfloat16, dev, (S, N if up is None else 2 * N), optional=True)
    if (q is None) != (sf is None):
        raise ValueError("q and sf come together")
    qp = sfp = amax = 0
    if q is not None:
        if not q.is_contiguous() or q.shape != (S, N):
            raise ValueError("q must be a contiguous [slots, N]")
        qp, sfp = _codes(q, "q", N, FMT_MXFP8, dev), _tensor(sf, "sf", torch.uint8, dev, (S, N // 32))
    if fp4:
        if xa is None or xa.numel() not in (1, R):
            raise ValueError("x's amax must be [R] or [1]")
        amax = _tensor(xa, "x's amax", torch.float32, dev)
    p = _PRODUCT.pack(fmt, activation, E, 1 if fp4 and xa.numel() == R and R > 1 else 0, N, K, R, S,
                 _codes(xq, "x", K, fmt, dev), _tensor(xsf, "x's scales", torch.uint8, dev, (R, kv)), amax,
                 _tensor(rows, "rows", torch.int32, dev, (S,), optional=True), offs, cnts, wp[0], wp[1], wp[2], upp[0],
                 upp[1], upp[2], wp[3], wp[4], _tensor(bias, "bias", torch.bfloat16, dev, (E, N), optional=True),
                 _tensor(up_bias, "up_bias", torch.bfloat16, dev, (E, N), optional=True), r, ldr, o, ldo, z, ldz,
                 qp, sfp)
    lib, s = load(), _raw_stream(stream, dev)
    if workspace is not None:
        _tensor(workspace, "workspace", torch.uint8, dev)
    elif rows is not None:
        workspace = _scratch(lib.qz_product_bytes(p), out, stream)
    _check(lib.qz_expert_product(p, s, _opts(err, max_ctas, workspace)), "qz_expert_product")
    return out


def expert_weight_grad(fmt: int, dz, x, offsets: torch.Tensor, counts: torch.Tensor, out: torch.Tensor, *,
                       accumulate: bool = False, stream=None, err=None, max_ctas: int = 0):
    """The experts' weight gradients out[e] (+)= dZ_e^T X_e (qz_expert_weight_grad).

    dz, x: column-wise quantized over all slots: (payload [N, slots] / [K,
    slots] (packed: slots / 2), swizzled scales of that matrix, NVFP4: amax
    [1]); out: [E, N, K] fp32 or bf16.  offsets must be multiples of 128 (a
    plan with align=128) and unused slots must hold zeros."""
    zq, zsf, za = _parts(dz, "dz")
    xq, xsf, xa = _parts(x, "x")
    _require(zq.dim() == 2 and xq.dim() == 2 and out.dim() == 3, "dz must be [N, slots], x [K, slots], out [E, N, K]")
    _require(fmt in (FMT_MXFP8, FMT_NVFP4), "fmt must be FMT_MXFP8 or FMT_NVFP4")
    fp4 = fmt == FMT_NVFP4
    dev = out.get_device()
    E, N, K = out.shape
    S = zq.shape[1] * (2 if fp4 else 1)
    _require(zq.shape[0] == N and xq.shape[0] == K, "dz, x and out do not match")
    _require(zq.is_contiguous() and xq.is_contiguous(), "dz and x must be contiguous")
    _require(zsf.numel() >= sf_bytes(N, S, fmt, SF_SWIZZLED) and xsf.numel() >= sf_bytes(K, S, fmt, SF_SWIZZLED),
             "the scales are smaller than the swizzled region")
    offs, cnts = _expert_lists(offsets, counts, E, dev)
    p = _WeightGrad(fmt, E, _float_type(out, "out"), 1 if accumulate else 0, N, K, S, _codes(zq, "dz", S, fmt, dev),
                    _tensor(zsf, "dz's scales", torch.uint8, dev),
                    _tensor(za, "dz's amax", torch.float32, dev, (1,)) if fp4 else 0, _codes(xq, "x", S, fmt, dev),
                    _tensor(xsf, "x's scales", torch.uint8, dev),
                    _tensor(xa, "x's amax", torch.float32, dev, (1,)) if fp4 else 0, offs, cnts,
                    _tensor(out, "out", out.dtype, dev))
    _check(load().qz_expert_weight_grad(ctypes.byref(p), _raw_stream(stream, dev), _opts(err, max_ctas)),
           "qz_expert_weight_grad")
    return out


def expert_activation_grad(dout: torch.Tensor, pre: torch.Tensor, offsets: torch.Tensor, counts: torch.Tensor,
                           dpre: torch.Tensor, *, activation: int, gated: bool = False, dbias=None, workspace=None,
                           stream=None, err=None):
    """Gradient of expert_product's activation from its saved pre-activations,
    with the bias gradients (qz_expert_activation_grad): dout [slots, N], pre
    and dpre bf16 [slots, N or 2N], dbias fp32 [E, N or 2N] or None.  offsets
    must be [E + 1] or [E], as the plan writes them; rows of dpre that are no
    live slot become zeros.  dbias needs a workspace (allocated unless given)."""
    _require(dout.dim() == 2, "dout must be [slots, N]")
    dev = dout.get_device()
    S, N = dout.shape
    width = 2 * N if gated else N
    E = counts.numel()
    offs, cnts = _expert_lists(offsets, counts, E, dev)
    d, ldd = _matrix(dout, "dout", torch.bfloat16, dev, (S, N))
    z, ldz = _matrix(pre, "pre", torch.bfloat16, dev, (S, width))
    g, ldg = _matrix(dpre, "dpre", torch.bfloat16, dev, (S, width))
    lib, b, st = load(), _tensor(dbias, "dbias", torch.float32, dev, (E, width), optional=True), _raw_stream(stream, dev)
    if workspace is not None:
        _tensor(workspace, "workspace", torch.uint8, dev)
    elif b:
        workspace = _scratch(lib.qz_activation_grad_bytes(S, N, 1 if gated else 0, E), dout, stream)
    _check(lib.qz_expert_activation_grad(d, ldd, z, ldz, S, N, int(activation), 1 if gated else 0, offs, cnts, E, g, ldg,
                                         b, st, _opts(err, 0, workspace)), "qz_expert_activation_grad")
    return dpre


def dispatch_experts(x: torch.Tensor, slots: torch.Tensor, rows: torch.Tensor, y: torch.Tensor, *, weights=None,
                     other=None, dots=None, stream=None):
    """Token order to expert order (qz_dispatch_experts): y[slots[t, j]] =
    weights[t, j] * x[t], zeros in unused slots; with ``other`` [slots, H] also
    dots[t, j] = <x[t], other[slots[t, j]]>.  The gradient of combine_experts."""
    _require(x.dim() == 2 and slots.dim() == 2 and y.dim() == 2, "x must be [T, H], slots [T, top_k], y [slots, H]")
    dev = x.get_device()
    T, H = x.shape
    k, S = slots.shape[1], y.shape[0]
    a, lda = _matrix(x, "x", torch.bfloat16, dev, (T, H))
    b, ldb = _matrix(y, "y", torch.bfloat16, dev, (S, H))
    o, ldo = _matrix(other, "other", torch.bfloat16, dev, (S, H), optional=True)
    _check(load().qz_dispatch_experts(a, lda, _tensor(slots, "slots", torch.int32, dev, (T, k)),
                                      _tensor(rows, "rows", torch.int32, dev, (S,)), T, k, S, H,
                                      _tensor(weights, "weights", torch.float32, dev, (T, k), optional=True), b, ldb, o,
                                      ldo, _tensor(dots, "dots", torch.float32, dev, (T, k), optional=True),
                                      _raw_stream(stream, dev)), "qz_dispatch_experts")
    return y


def combine_experts(y: torch.Tensor, slots: torch.Tensor, out: torch.Tensor, *, weights=None, residual=None,
                    stream=None):
    """Expert order to token order (qz_combine_experts): out[t] = residual[t] +
    sum_j weights[t, j] * y[slots[t, j]] (a missing weight counts 1).  The
    gradient of dispatch_experts."""
    _require(y.dim() == 2 and slots.dim() == 2 and out.dim() == 2, "y must be [slots, H], slots [T, top_k], out [T, H]")
    dev = out.get_device()
    T, H = out.shape
    S, k = y.shape[0], slots.shape[1]
    a, lda = _matrix(y, "y", torch.bfloat16, dev, (S, H))
    o, ldo = _matrix(out, "out", torch.bfloat16, dev, (T, H))
    r, ldr = _matrix(residual, "residual", torch.bfloat16, dev, (T, H), optional=True)
    _check(load().qz_combine_experts(a, lda, _tensor(slots, "slots", torch.int32, dev, (T, k)), T, k, S, H,
                                     _tensor(weights, "weights", torch.float32, dev, (T, k), optional=True), r, ldr, o, ldo,
                                     _raw_stream(stream, dev)), "qz_combine_experts")
    return out


# ---------------------------------------------------------------------------
# conveniences that allocate outputs with torch and call the entry points
# ---------------------------------------------------------------------------

def alloc_outputs(xs: Sequence[torch.Tensor], fmt: int, layout: int, mode: int = NVFP4_PER_ROW):
    """Payload, SF and amax buffers for a list of bf16 [rows, cols] experts."""
    entries = []
    for x in xs:
        rows, cols = x.shape
        qcols = cols if fmt == FMT_MXFP8 else cols // 2
        q = torch.empty((rows, qcols), dtype=torch.uint8, device=x.device)
        sf = torch.empty(max(sf_bytes(rows, cols, fmt, layout), 16), dtype=torch.uint8, device=x.device)
        amax = None
        if fmt == FMT_NVFP4:
            amax = torch.zeros(max(rows, 1) if mode == NVFP4_PER_ROW else 1, dtype=torch.float32, device=x.device)
        entries.append(Entry(x, q, sf, amax))
    return entries


def quantize_experts(xs: Sequence[torch.Tensor], fmt: int, layout: int, mode: int = NVFP4_PER_ROW,
                     amax_in: Optional[Sequence[float]] = None, stream=None, workspace: Optional[torch.Tensor] = None):
    """Quantize a list of bf16 experts in one launch; returns the entries with
    q, sf (trimmed to the region size) and amax filled."""
    entries = alloc_outputs(xs, fmt, layout, mode)
    if fmt == FMT_NVFP4 and mode == NVFP4_PER_TENSOR_GIVEN:
        for e, a in zip(entries, amax_in):
            e.amax.fill_(float(a))
    table = ExpertTable(entries)
    if fmt == FMT_MXFP8:
        quantize_grouped_mxfp8(table, layout, stream)
    else:
        quantize_grouped_nvfp4(table, mode, layout, stream, workspace=workspace)
    for e in entries:
        rows, cols = e.x.shape
        e.sf = e.sf[: sf_bytes(rows, cols, fmt, layout)]
    return entries


def quantize_expert_weights(w: torch.Tensor, fmt: int, stream=None):
    """Quantize stacked bf16 expert weights [E, N, K] in one launch into the
    form expert_product takes: (payload [E, N, K or K/2], swizzled scales
    [E, region], NVFP4: amax [E], computed).  The outputs are allocated on the
    stream; not for a captured stream (the table comes from the host)."""
    _require(w.dim() == 3, "w must be [E, N, K]")
    E, N, K = w.shape
    with _on(stream):
        q = torch.empty((E, N, K if fmt == FMT_MXFP8 else K // 2), dtype=torch.uint8, device=w.device)
        sf = torch.empty((E, sf_bytes(N, K, fmt, SF_SWIZZLED)), dtype=torch.uint8, device=w.device)
        amax = torch.empty(E, dtype=torch.float32, device=w.device) if fmt == FMT_NVFP4 else None
        table = ExpertTable([Entry(w[e], q[e], sf[e], None if amax is None else amax[e:e + 1]) for e in range(E)],
                            device=w.device)
        if fmt == FMT_MXFP8:
            quantize_grouped_mxfp8(table, SF_SWIZZLED)
        else:
            quantize_grouped_nvfp4(table, NVFP4_PER_TENSOR_COMPUTE, SF_SWIZZLED)
        del table
    return q, sf, amax


def quantize_tokens(x: torch.Tensor, fmt: int, stream=None):
    """Quantize bf16 rows [R, K] into the form expert_product takes as x:
    (payload, linear scales [R, K/block], NVFP4: amax [R], one per row); streams
    as in quantize_expert_weights."""
    _require(x.dim() == 2, "x must be [R, K]")
    with _on(stream):
        (e,) = quantize_experts([x], fmt, SF_LINEAR, NVFP4_PER_ROW)
    R, K = x.shape
    return e.q, e.sf.view(R, K // (32 if fmt == FMT_MXFP8 else 16)), (None if e.amax is None else e.amax[:R])


def quantize_slots_colwise(x: torch.Tensor, fmt: int, amax: Optional[torch.Tensor] = None, stream=None):
    """Quantize bf16 [slots, n] down its columns into the form
    expert_weight_grad takes: (payload [n, slots or slots/2], swizzled scales,
    NVFP4: amax [1], max |x| unless given); streams as in
    quantize_expert_weights."""
    _require(x.dim() == 2, "x must be [slots, n]")
    S, n = x.shape
    with _on(stream):
        q = torch.empty((n, S if fmt == FMT_MXFP8 else S // 2), dtype=torch.uint8, device=x.device)
        sf = torch.empty(max(sf_bytes(n, S, fmt, SF_SWIZZLED), 16), dtype=torch.uint8, device=x.device)
        if fmt == FMT_NVFP4 and amax is None:
            amax = (x.abs().amax().to(torch.float32).reshape(1) if x.numel() else
                    torch.zeros(1, dtype=torch.float32, device=x.device))
        quantize_grouped_colwise(ExpertTable([Entry(x, q, sf, amax)]), fmt, SF_SWIZZLED)
    return q, sf, amax
