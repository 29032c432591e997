"""Thin ctypes binding of libep_mi355x.so (include/ep.h) for torch tensors.

Argument marshalling only: every step of dispatch and combine runs in the HIP
kernels behind the C ABI; torch provides device memory and the current
stream.  The functions allocate their outputs with ``torch.empty`` unless
``out``-style arguments are passed (the benchmark passes them so that nothing
is allocated in its timed loop).  If the library is not built the first call
raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep_mi355x.so")

EP_OK = 0
EP_DTYPE_BF16 = 0
EP_DTYPE_FP8_E4M3 = 1
EP_DTYPE_FP32 = 2
SCORES = {"softmax": 0, "sigmoid": 1}
MAX_EXPERTS = 1024
MAX_TOPK = 64
LL_MAX_SLOTS = 8192
MAX_EXPERT_ALIGNMENT = 1024
MAX_ROUTE_GROUPS = 64


class EpError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s" % (what, status_string(status)))


_lib = None
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f32 = ctypes.c_float

SIGNATURES = {
    "ep_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "ep_get_dispatch_layout": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                              _vp, _vp, _sz, _vp]),
    "ep_dispatch": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _i32, _i32, ctypes.c_int, _vp,
                                   _vp, _vp, _vp, _vp, _sz, _vp]),
    "ep_combine": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _vp]),
    "ep_combine_cu": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp]),
    "ep_layout_dispatch_cu": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _i32, _i32, ctypes.c_int,
                                             _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                             _sz, _i32, _vp]),
    "ep_layout_dispatch": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _i32, _i32, ctypes.c_int,
                                          _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                          _vp]),
    "ep_layout_dispatch_static": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _i32, _i32,
                                                 ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                 _vp, _vp, _vp]),
    "ep_aligned_rows": (_i64, [_i32, _i32, _i32, _i32]),
    "ep_layout_dispatch_aligned": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _i32, _i32, _i32,
                                                  ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                  _vp, _vp, _vp, _sz, _vp]),
    "ep_dispatch_dedup": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _i32, _i32, ctypes.c_int,
                                         _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _sz, _vp]),
    "ep_low_latency_dispatch": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _i32, _i32,
                                               ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "ep_combine_backward": (ctypes.c_int, [_vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _vp,
                                           _vp]),
    "ep_dispatch_backward": (ctypes.c_int, [_vp, _i64, _vp, _i32, _i32, _i32, _vp, _vp]),
    "ep_route": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i32, _i32, _i32, ctypes.c_int, _i32,
                                _i32, _i32, _f32, _vp, _vp, _vp]),
    "ep_route_backward": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _i32, _i32, _i32,
                                         ctypes.c_int, _i32, _f32, _vp, _vp]),
    "ep_expert_linear_w4": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _vp, _vp, _i32, _i32,
                                           _i32, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp]),
    "ep_expert_linear": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _i64, _vp, _vp, _i32, _i32, _i32,
                                        _i32, _vp, _vp, _i32, _vp, _vp]),
    "ep_expert_linear_backward": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32,
                                                 _i32, _vp, _vp, ctypes.c_int, _i32, _vp]),
    "ep_expert_swiglu": (ctypes.c_int, [_vp, _i64, _vp, _vp, _i32, _i32, _i32, ctypes.c_int, _vp,
                                        _vp, _vp]),
    "ep_expert_swiglu_backward": (ctypes.c_int, [_vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _vp,
                                                 _vp]),
    "ep_rms_norm": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _i32, _i32, _f32, _vp, _vp, _vp,
                                   _vp, _vp, _vp]),
    "ep_rms_norm_backward_workspace_bytes": (_sz, [_i32, _i32]),
    "ep_rms_norm_backward": (ctypes.c_int, [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _i32,
                                            _vp, _vp, _vp, _sz, _vp]),
    "ep_get_device_error": (ctypes.c_int, [_vp, _sz, ctypes.POINTER(_i64), _vp]),
    "ep_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ep_convert_e4m3": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp]),
    "ep_convert_bf16": (ctypes.c_int, [_vp, _vp, _i64, _vp]),
    "ep_copy": (ctypes.c_int, [_vp, _vp, _sz, _vp]),
}


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libep_mi355x.so is not built: run `python -m combine_ep_get_dispatch_amd.build`"
                " (or __graft_entry__.build()) first")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().ep_status_string(status).decode()


def _check(status: int, what: str):
    if status != EP_OK:
        raise EpError(status, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(t: torch.Tensor):
    """torch's current stream on t's device, as a hipStream_t."""
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(t.device.index))
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _is_gpu(t: torch.Tensor) -> bool:
    return t.device.type == "cuda"


def _need(t: torch.Tensor, dtype, name: str, shape=None, device=None):
    # the usual case in one expression; what it does not pass is looked at below
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape) and (device is None or t.device == device)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not _is_gpu(t):
        raise ValueError("%s must be a GPU tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


# ---------------------------------------------------------------------------
# layout
# ---------------------------------------------------------------------------

def workspace_bytes(num_tokens: int, num_topk: int, num_experts: int, num_partitions: int) -> int:
    n = lib().ep_workspace_bytes(num_tokens, num_topk, num_experts, num_partitions)
    if n == 0:
        raise ValueError("invalid shape T=%d K=%d E=%d P=%d" % (
            num_tokens, num_topk, num_experts, num_partitions))
    return int(n)


def new_workspace(num_tokens, num_topk, num_experts, num_partitions, device="cuda"):
    """A workspace for this shape.  It needs no initialisation (every layout
    call writes all that later calls read from it); it is zero-filled only so
    that its contents are defined before the first call."""
    return torch.zeros(workspace_bytes(num_tokens, num_topk, num_experts, num_partitions),
                       dtype=torch.uint8, device=device)


@dataclass
class Layout:
    num_tokens_per_expert: torch.Tensor     # [E] int32
    num_tokens_per_partition: torch.Tensor  # [P] int32
    is_token_in_partition: torch.Tensor     # [T, P] uint8
    expert_offsets: torch.Tensor            # [E+1] int32
    partition_offsets: torch.Tensor         # [P+1] int32
    workspace: torch.Tensor                 # uint8, consumed by dispatch


def get_dispatch_layout(topk_idx: torch.Tensor, num_experts: int, num_partitions: int,
                        workspace: torch.Tensor | None = None,
                        out: Layout | None = None) -> Layout:
    """ep_get_dispatch_layout on ``topk_idx`` [T, K] int64."""
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    T, K = topk_idx.shape
    dev = topk_idx.device
    _need(topk_idx, torch.int64, "topk_idx", device=dev)
    E, P = int(num_experts), int(num_partitions)
    if workspace is None:
        workspace = new_workspace(T, K, E, P, dev)
    _need(workspace, torch.uint8, "workspace", device=dev)
    if out is None:
        out = Layout(torch.empty(E, dtype=torch.int32, device=dev),
                     torch.empty(P, dtype=torch.int32, device=dev),
                     torch.empty((T, P), dtype=torch.uint8, device=dev),
                     torch.empty(E + 1, dtype=torch.int32, device=dev),
                     torch.empty(P + 1, dtype=torch.int32, device=dev), workspace)
    else:
        out.workspace = workspace
    _need(out.num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=dev)
    _need(out.num_tokens_per_partition, torch.int32, "num_tokens_per_partition", (P,), device=dev)
    _need(out.is_token_in_partition, torch.uint8, "is_token_in_partition", (T, P), device=dev)
    _need(out.expert_offsets, torch.int32, "expert_offsets", (E + 1,), device=dev)
    _need(out.partition_offsets, torch.int32, "partition_offsets", (P + 1,), device=dev)
    _check(lib().ep_get_dispatch_layout(
        _ptr(topk_idx), T, K, E, P, _ptr(out.num_tokens_per_expert),
        _ptr(out.num_tokens_per_partition), _ptr(out.is_token_in_partition),
        _ptr(out.expert_offsets), _ptr(out.partition_offsets), _ptr(workspace),
        workspace.numel(), _stream(topk_idx)), "ep_get_dispatch_layout")
    return out


def get_device_error(workspace: torch.Tensor) -> int:
    """Invalid topk_idx entries met by the last layout call (synchronises)."""
    n = _i64(0)
    _check(lib().ep_get_device_error(_ptr(workspace), workspace.numel(), ctypes.byref(n),
                                     _stream(workspace)), "ep_get_device_error")
    return int(n.value)


# ---------------------------------------------------------------------------
# dispatch / combine
# ---------------------------------------------------------------------------

@dataclass
class Dispatched:
    recv_x: torch.Tensor                 # [T*K, H] bf16, or uint8 E4M3 codes
    recv_scales: torch.Tensor | None     # [T*K, H/128] float32 (FP8 only)
    recv_src_token: torch.Tensor         # [T*K] int32
    dst_row: torch.Tensor                # [T, K] int32


def dispatch(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int, num_partitions: int,
             workspace: torch.Tensor, fp8: bool = False,
             out: Dispatched | None = None) -> Dispatched:
    """ep_dispatch: x [T, H] bf16 -> receive rows grouped by expert."""
    if x.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H] and topk_idx [T, K]")
    T, H = x.shape
    K = topk_idx.shape[1]
    dev = x.device
    _need(x, torch.bfloat16, "x", device=dev)
    _need(topk_idx, torch.int64, "topk_idx", (T, K), device=dev)
    _need(workspace, torch.uint8, "workspace", device=dev)
    R = T * K
    if out is None:
        out = Dispatched(
            torch.empty((R, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev),
            torch.empty((R, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((T, K), dtype=torch.int32, device=dev))
    _need(out.recv_x, torch.uint8 if fp8 else torch.bfloat16, "recv_x", (R, H), device=dev)
    if fp8:
        _need(out.recv_scales, torch.float32, "recv_scales", (R, H // 128), device=dev)
    _need(out.recv_src_token, torch.int32, "recv_src_token", (R,), device=dev)
    _need(out.dst_row, torch.int32, "dst_row", (T, K), device=dev)
    _check(lib().ep_dispatch(
        _ptr(x), T, H, _ptr(topk_idx), K, int(num_experts), int(num_partitions),
        EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16, _ptr(out.recv_x),
        _ptr(out.recv_scales) if fp8 else None, _ptr(out.recv_src_token), _ptr(out.dst_row),
        _ptr(workspace), workspace.numel(), _stream(x)), "ep_dispatch")
    return out


def layout_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int,
                    num_partitions: int, workspace: torch.Tensor | None = None,
                    fp8: bool = False, out_layout: Layout | None = None,
                    out: Dispatched | None = None, num_cus: int = 0):
    """ep_layout_dispatch: the outputs of get_dispatch_layout + dispatch from
    one call (one kernel launch fewer).  num_cus > 0 confines the dispatch
    launch to that many CUs (ep_layout_dispatch_cu).  Returns (Layout,
    Dispatched)."""
    if x.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H] and topk_idx [T, K]")
    T, H = x.shape
    K = topk_idx.shape[1]
    E, P = int(num_experts), int(num_partitions)
    dev = x.device
    _need(x, torch.bfloat16, "x", device=dev)
    _need(topk_idx, torch.int64, "topk_idx", (T, K), device=dev)
    if workspace is None:
        workspace = new_workspace(T, K, E, P, dev)
    _need(workspace, torch.uint8, "workspace", device=dev)
    if out_layout is None:
        out_layout = Layout(torch.empty(E, dtype=torch.int32, device=dev),
                            torch.empty(P, dtype=torch.int32, device=dev),
                            torch.empty((T, P), dtype=torch.uint8, device=dev),
                            torch.empty(E + 1, dtype=torch.int32, device=dev),
                            torch.empty(P + 1, dtype=torch.int32, device=dev), workspace)
    else:
        out_layout.workspace = workspace
    R = T * K
    if out is None:
        out = Dispatched(
            torch.empty((R, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev),
            torch.empty((R, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((T, K), dtype=torch.int32, device=dev))
    lo = out_layout
    _need(lo.num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=dev)
    _need(lo.num_tokens_per_partition, torch.int32, "num_tokens_per_partition", (P,), device=dev)
    _need(lo.is_token_in_partition, torch.uint8, "is_token_in_partition", (T, P), device=dev)
    _need(lo.expert_offsets, torch.int32, "expert_offsets", (E + 1,), device=dev)
    _need(lo.partition_offsets, torch.int32, "partition_offsets", (P + 1,), device=dev)
    _need(out.recv_x, torch.uint8 if fp8 else torch.bfloat16, "recv_x", (R, H), device=dev)
    if fp8:
        _need(out.recv_scales, torch.float32, "recv_scales", (R, H // 128), device=dev)
    _need(out.recv_src_token, torch.int32, "recv_src_token", (R,), device=dev)
    _need(out.dst_row, torch.int32, "dst_row", (T, K), device=dev)
    _check(lib().ep_layout_dispatch_cu(
        _ptr(x), T, H, _ptr(topk_idx), K, E, P, EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
        _ptr(lo.num_tokens_per_expert), _ptr(lo.num_tokens_per_partition),
        _ptr(lo.is_token_in_partition), _ptr(lo.expert_offsets), _ptr(lo.partition_offsets),
        _ptr(out.recv_x), _ptr(out.recv_scales) if fp8 else None, _ptr(out.recv_src_token),
        _ptr(out.dst_row), _ptr(workspace), workspace.numel(), int(num_cus), _stream(x)),
        "ep_layout_dispatch_cu")
    return out_layout, out


def layout_dispatch_static(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int,
                           num_partitions: int, fp8: bool = False,
                           out_layout: Layout | None = None, out: Dispatched | None = None):
    """ep_layout_dispatch_static: the outputs of layout_dispatch, with the
    library's static per-GPU scratch as the workspace (the C call allocates
    nothing; outputs not given are allocated here).  The Layout's workspace
    is None: the invalid-id count is not reported.  Returns (Layout,
    Dispatched)."""
    if x.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H] and topk_idx [T, K]")
    T, H = x.shape
    K = topk_idx.shape[1]
    E, P = int(num_experts), int(num_partitions)
    dev = x.device
    _need(x, torch.bfloat16, "x", device=dev)
    _need(topk_idx, torch.int64, "topk_idx", (T, K), device=dev)
    if out_layout is None:
        out_layout = Layout(torch.empty(E, dtype=torch.int32, device=dev),
                            torch.empty(P, dtype=torch.int32, device=dev),
                            torch.empty((T, P), dtype=torch.uint8, device=dev),
                            torch.empty(E + 1, dtype=torch.int32, device=dev),
                            torch.empty(P + 1, dtype=torch.int32, device=dev), None)
    R = T * K
    if out is None:
        out = Dispatched(
            torch.empty((R, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev),
            torch.empty((R, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((T, K), dtype=torch.int32, device=dev))
    lo = out_layout
    _need(lo.num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=dev)
    _need(lo.num_tokens_per_partition, torch.int32, "num_tokens_per_partition", (P,), device=dev)
    _need(lo.is_token_in_partition, torch.uint8, "is_token_in_partition", (T, P), device=dev)
    _need(lo.expert_offsets, torch.int32, "expert_offsets", (E + 1,), device=dev)
    _need(lo.partition_offsets, torch.int32, "partition_offsets", (P + 1,), device=dev)
    _need(out.recv_x, torch.uint8 if fp8 else torch.bfloat16, "recv_x", (R, H), device=dev)
    if fp8:
        _need(out.recv_scales, torch.float32, "recv_scales", (R, H // 128), device=dev)
    _need(out.recv_src_token, torch.int32, "recv_src_token", (R,), device=dev)
    _need(out.dst_row, torch.int32, "dst_row", (T, K), device=dev)
    _check(lib().ep_layout_dispatch_static(
        _ptr(x), T, H, _ptr(topk_idx), K, E, P, EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
        _ptr(lo.num_tokens_per_expert), _ptr(lo.num_tokens_per_partition),
        _ptr(lo.is_token_in_partition), _ptr(lo.expert_offsets), _ptr(lo.partition_offsets),
        _ptr(out.recv_x), _ptr(out.recv_scales) if fp8 else None, _ptr(out.recv_src_token),
        _ptr(out.dst_row), _stream(x)), "ep_layout_dispatch_static")
    return out_layout, out


def aligned_rows(num_tokens: int, num_topk: int, num_experts: int, expert_alignment: int) -> int:
    """ep_aligned_rows: receive rows of layout_dispatch_aligned (0 if rejected)."""
    return int(lib().ep_aligned_rows(num_tokens, num_topk, num_experts, expert_alignment))


def layout_dispatch_aligned(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int,
                            num_partitions: int, expert_alignment: int,
                            workspace: torch.Tensor | None = None, fp8: bool = False,
                            out_layout: Layout | None = None, out: Dispatched | None = None):
    """ep_layout_dispatch_aligned: layout and dispatch with every expert's run
    of receive rows padded to a multiple of expert_alignment rows (recv_x,
    recv_scales and recv_src_token have aligned_rows(...) rows).  Returns
    (Layout, Dispatched)."""
    if x.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H] and topk_idx [T, K]")
    T, H = x.shape
    K = topk_idx.shape[1]
    E, P, A = int(num_experts), int(num_partitions), int(expert_alignment)
    dev = x.device
    _need(x, torch.bfloat16, "x", device=dev)
    _need(topk_idx, torch.int64, "topk_idx", (T, K), device=dev)
    R = aligned_rows(T, K, E, A)
    if R == 0 and T > 0:
        raise ValueError("expert_alignment %d rejected for T=%d K=%d E=%d" % (A, T, K, E))
    if workspace is None:
        workspace = new_workspace(T, K, E, P, dev)
    _need(workspace, torch.uint8, "workspace", device=dev)
    if out_layout is None:
        out_layout = Layout(torch.empty(E, dtype=torch.int32, device=dev),
                            torch.empty(P, dtype=torch.int32, device=dev),
                            torch.empty((T, P), dtype=torch.uint8, device=dev),
                            torch.empty(E + 1, dtype=torch.int32, device=dev),
                            torch.empty(P + 1, dtype=torch.int32, device=dev), workspace)
    else:
        out_layout.workspace = workspace
    if out is None:
        out = Dispatched(
            torch.empty((R, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev),
            torch.empty((R, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((T, K), dtype=torch.int32, device=dev))
    lo = out_layout
    _need(lo.num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=dev)
    _need(lo.num_tokens_per_partition, torch.int32, "num_tokens_per_partition", (P,), device=dev)
    _need(lo.is_token_in_partition, torch.uint8, "is_token_in_partition", (T, P), device=dev)
    _need(lo.expert_offsets, torch.int32, "expert_offsets", (E + 1,), device=dev)
    _need(lo.partition_offsets, torch.int32, "partition_offsets", (P + 1,), device=dev)
    _need(out.recv_x, torch.uint8 if fp8 else torch.bfloat16, "recv_x", (R, H), device=dev)
    if fp8:
        _need(out.recv_scales, torch.float32, "recv_scales", (R, H // 128), device=dev)
    _need(out.recv_src_token, torch.int32, "recv_src_token", (R,), device=dev)
    _need(out.dst_row, torch.int32, "dst_row", (T, K), device=dev)
    _check(lib().ep_layout_dispatch_aligned(
        _ptr(x), T, H, _ptr(topk_idx), K, E, P, A, EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
        _ptr(lo.num_tokens_per_expert), _ptr(lo.num_tokens_per_partition),
        _ptr(lo.is_token_in_partition), _ptr(lo.expert_offsets), _ptr(lo.partition_offsets),
        _ptr(out.recv_x), _ptr(out.recv_scales) if fp8 else None, _ptr(out.recv_src_token),
        _ptr(out.dst_row), _ptr(workspace), workspace.numel(), _stream(x)),
        "ep_layout_dispatch_aligned")
    return out_layout, out


@dataclass
class DedupDispatched:
    partition_token_offsets: torch.Tensor  # [P+1] int32
    recv_x: torch.Tensor                   # [T*Kp, H] bf16, or uint8 E4M3 codes
    recv_scales: torch.Tensor | None       # [T*Kp, H/128] float32 (FP8 only)
    recv_src_token: torch.Tensor           # [T*Kp] int32, -1 past the rows used
    recv_topk_idx: torch.Tensor            # [T*Kp, K] int32 local expert ids or -1
    slot_src_row: torch.Tensor             # [T*K] int32
    dst_row: torch.Tensor                  # [T, K] int32


def dispatch_dedup(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int,
                   num_partitions: int, workspace: torch.Tensor | None = None,
                   fp8: bool = False, out_layout: Layout | None = None,
                   out: DedupDispatched | None = None):
    """ep_dispatch_dedup: one copy of each token per partition it reaches.
    Returns (Layout, DedupDispatched)."""
    if x.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H] and topk_idx [T, K]")
    T, H = x.shape
    K = topk_idx.shape[1]
    E, P = int(num_experts), int(num_partitions)
    Kp = min(K, P)
    RD = T * Kp
    dev = x.device
    _need(x, torch.bfloat16, "x", device=dev)
    _need(topk_idx, torch.int64, "topk_idx", (T, K), device=dev)
    if workspace is None:
        workspace = new_workspace(T, K, E, P, dev)
    _need(workspace, torch.uint8, "workspace", device=dev)
    if out_layout is None:
        out_layout = Layout(torch.empty(E, dtype=torch.int32, device=dev),
                            torch.empty(P, dtype=torch.int32, device=dev),
                            torch.empty((T, P), dtype=torch.uint8, device=dev),
                            torch.empty(E + 1, dtype=torch.int32, device=dev),
                            torch.empty(P + 1, dtype=torch.int32, device=dev), workspace)
    else:
        out_layout.workspace = workspace
    if out is None:
        out = DedupDispatched(
            torch.empty(P + 1, dtype=torch.int32, device=dev),
            torch.empty((RD, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev),
            torch.empty((RD, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
            torch.empty(RD, dtype=torch.int32, device=dev),
            torch.empty((RD, K), dtype=torch.int32, device=dev),
            torch.empty(T * K, dtype=torch.int32, device=dev),
            torch.empty((T, K), dtype=torch.int32, device=dev))
    lo = out_layout
    _need(lo.num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=dev)
    _need(lo.num_tokens_per_partition, torch.int32, "num_tokens_per_partition", (P,), device=dev)
    _need(lo.is_token_in_partition, torch.uint8, "is_token_in_partition", (T, P), device=dev)
    _need(lo.expert_offsets, torch.int32, "expert_offsets", (E + 1,), device=dev)
    _need(lo.partition_offsets, torch.int32, "partition_offsets", (P + 1,), device=dev)
    _need(out.partition_token_offsets, torch.int32, "partition_token_offsets", (P + 1,), device=dev)
    _need(out.recv_x, torch.uint8 if fp8 else torch.bfloat16, "recv_x", (RD, H), device=dev)
    if fp8:
        _need(out.recv_scales, torch.float32, "recv_scales", (RD, H // 128), device=dev)
    _need(out.recv_src_token, torch.int32, "recv_src_token", (RD,), device=dev)
    _need(out.recv_topk_idx, torch.int32, "recv_topk_idx", (RD, K), device=dev)
    _need(out.slot_src_row, torch.int32, "slot_src_row", (T * K,), device=dev)
    _need(out.dst_row, torch.int32, "dst_row", (T, K), device=dev)
    _check(lib().ep_dispatch_dedup(
        _ptr(x), T, H, _ptr(topk_idx), K, E, P, EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
        _ptr(lo.num_tokens_per_expert), _ptr(lo.num_tokens_per_partition),
        _ptr(lo.is_token_in_partition), _ptr(lo.expert_offsets), _ptr(lo.partition_offsets),
        _ptr(out.partition_token_offsets), _ptr(out.recv_x),
        _ptr(out.recv_scales) if fp8 else None, _ptr(out.recv_src_token),
        _ptr(out.recv_topk_idx), _ptr(out.slot_src_row), _ptr(out.dst_row), _ptr(workspace),
        workspace.numel(), _stream(x)), "ep_dispatch_dedup")
    return out_layout, out


@dataclass
class LowLatencyDispatched:
    num_tokens_per_expert: torch.Tensor  # [E] int32 (dropped slots included)
    recv_x: torch.Tensor                 # [E*C, H] bf16, or uint8 E4M3 codes
    recv_scales: torch.Tensor | None     # [E*C, H/128] float32 (FP8 only)
    recv_src_token: torch.Tensor         # [E*C] int32, -1 for unfilled rows
    dst_row: torch.Tensor                # [T, K] int32
    num_invalid: torch.Tensor            # [1] int64


def low_latency_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, num_experts: int,
                         capacity: int, fp8: bool = False,
                         out: LowLatencyDispatched | None = None) -> LowLatencyDispatched:
    """ep_low_latency_dispatch: x [T, H] bf16 -> fixed-capacity rows, expert
    e owning rows [e*C, (e+1)*C), in one launch."""
    if x.dim() != 2 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H] and topk_idx [T, K]")
    T, H = x.shape
    K = topk_idx.shape[1]
    E, C = int(num_experts), int(capacity)
    dev = x.device
    _need(x, torch.bfloat16, "x", device=dev)
    _need(topk_idx, torch.int64, "topk_idx", (T, K), device=dev)
    R = E * C
    if out is None:
        out = LowLatencyDispatched(
            torch.empty(E, dtype=torch.int32, device=dev),
            torch.empty((R, H), dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev),
            torch.empty((R, H // 128), dtype=torch.float32, device=dev) if fp8 else None,
            torch.empty(R, dtype=torch.int32, device=dev),
            torch.empty((T, K), dtype=torch.int32, device=dev),
            torch.empty(1, dtype=torch.int64, device=dev))
    _need(out.num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=dev)
    _need(out.recv_x, torch.uint8 if fp8 else torch.bfloat16, "recv_x", (R, H), device=dev)
    if fp8:
        _need(out.recv_scales, torch.float32, "recv_scales", (R, H // 128), device=dev)
    _need(out.recv_src_token, torch.int32, "recv_src_token", (R,), device=dev)
    _need(out.dst_row, torch.int32, "dst_row", (T, K), device=dev)
    _need(out.num_invalid, torch.int64, "num_invalid", (1,), device=dev)
    _check(lib().ep_low_latency_dispatch(
        _ptr(x), T, H, _ptr(topk_idx), K, E, C, EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
        _ptr(out.num_tokens_per_expert), _ptr(out.recv_x),
        _ptr(out.recv_scales) if fp8 else None, _ptr(out.recv_src_token), _ptr(out.dst_row),
        _ptr(out.num_invalid), _stream(x)), "ep_low_latency_dispatch")
    return out


def combine(y: torch.Tensor, dst_row: torch.Tensor, topk_weights: torch.Tensor,
            out: torch.Tensor | None = None, num_cus: int = 0) -> torch.Tensor:
    """ep_combine: y [R, H] bf16 expert outputs -> out [T, H] bf16.  num_cus >
    0 confines it to that many CUs (ep_combine_cu)."""
    if y.dim() != 2 or dst_row.dim() != 2:
        raise ValueError("y must be [R, H] and dst_row [T, K]")
    T, K = dst_row.shape
    H = y.shape[1]
    dev = y.device
    _need(y, torch.bfloat16, "y", device=dev)
    _need(dst_row, torch.int32, "dst_row", device=dev)
    _need(topk_weights, torch.float32, "topk_weights", (T, K), device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _need(out, torch.bfloat16, "out", (T, H), device=dev)
    _check(lib().ep_combine_cu(_ptr(y), y.shape[0], _ptr(dst_row), _ptr(topk_weights), T, K, H,
                               _ptr(out), int(num_cus), _stream(y)), "ep_combine_cu")
    return out


# ---------------------------------------------------------------------------
# gradients of dispatch and combine
# ---------------------------------------------------------------------------

def _sizes(bits: int):
    """Refuse sizes (joined by |) that the library's 32-bit arguments would cut."""
    if bits >> 31 not in (0, -1):
        raise ValueError("sizes must be below 2^31")


def _launch(name: str, t: torch.Tensor, *args):
    """Call ``name`` with ``args`` and torch's current stream on t's device,
    with that device current."""
    fn = getattr(_lib or lib(), name)
    index = t.get_device()
    if _get_device is None or index != _get_device():
        with torch.cuda.device(t.device):
            status = fn(*args, _stream(t))
    else:
        status = fn(*args, _raw_stream(index) if _raw_stream is not None else _stream(t))
    if status != EP_OK:
        raise EpError(status, name)


def combine_backward(grad_out: torch.Tensor, y: torch.Tensor | None, dst_row: torch.Tensor,
                     topk_weights: torch.Tensor | None, out=None, num_rows: int | None = None):
    """ep_combine_backward: from grad_out [T, H] bf16 the gradients of
    combine(y, dst_row, topk_weights): (grad_y [R, H] bf16, grad_weights
    [T, K] float32), or the ones given in ``out``.  Rows of grad_y that no slot
    names are left as they are (a grad_y not given is allocated
    uninitialised).  Without ``topk_weights`` only grad_weights is computed,
    without ``y`` only grad_y (with ``num_rows`` rows if it is allocated here);
    the other one is None."""
    if grad_out.dim() != 2 or dst_row.dim() != 2 or (y is not None and y.dim() != 2):
        raise ValueError("grad_out must be [T, H], y [R, H] and dst_row [T, K]")
    T, K = dst_row.shape
    H = grad_out.shape[1]
    _sizes(T | K | H)
    dev = grad_out.device
    _need(grad_out, torch.bfloat16, "grad_out", (T, H), device=dev)
    _need(dst_row, torch.int32, "dst_row", device=dev)
    grad_y, grad_weights = (None, None) if out is None else out
    if y is None and topk_weights is None:
        raise ValueError("combine_backward needs y or topk_weights")
    if y is not None:
        num_rows = y.shape[0]
    elif grad_y is not None:
        num_rows = grad_y.shape[0]
    elif num_rows is None:
        raise ValueError("combine_backward without y needs num_rows or a grad_y in out")
    R = int(num_rows)
    if y is not None:
        _need(y, torch.bfloat16, "y", (R, H), device=dev)
        if grad_weights is None:
            grad_weights = torch.empty((T, K), dtype=torch.float32, device=dev)
        _need(grad_weights, torch.float32, "grad_weights", (T, K), device=dev)
    elif grad_weights is not None:
        raise ValueError("grad_weights needs y")
    if topk_weights is not None:
        _need(topk_weights, torch.float32, "topk_weights", (T, K), device=dev)
        if grad_y is None:
            grad_y = torch.empty((R, H), dtype=torch.bfloat16, device=dev)
        _need(grad_y, torch.bfloat16, "grad_y", (R, H), device=dev)
    elif grad_y is not None:
        raise ValueError("grad_y needs topk_weights")
    _launch("ep_combine_backward", grad_out, _addr(grad_out), _addr(y), R, _addr(dst_row),
            _addr(topk_weights), T, K, H, _addr(grad_y), _addr(grad_weights))
    return grad_y, grad_weights


def dispatch_backward(grad_recv_x: torch.Tensor, dst_row: torch.Tensor,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """ep_dispatch_backward: from grad_recv_x [R, H] bf16, laid out like the
    receive rows, the gradient of dispatch's x: grad_x [T, H] bf16."""
    if grad_recv_x.dim() != 2 or dst_row.dim() != 2:
        raise ValueError("grad_recv_x must be [R, H] and dst_row [T, K]")
    T, K = dst_row.shape
    R, H = grad_recv_x.shape
    _sizes(T | K | H)
    dev = grad_recv_x.device
    _need(grad_recv_x, torch.bfloat16, "grad_recv_x", device=dev)
    _need(dst_row, torch.int32, "dst_row", device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", (T, H), device=dev)
    _launch("ep_dispatch_backward", grad_recv_x, _addr(grad_recv_x), R, _addr(dst_row), T, K, H,
            _addr(out))
    return out


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

def _logits_dtype(logits: torch.Tensor) -> int:
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be float32 or bfloat16, got %s" % logits.dtype)
    _need(logits, logits.dtype, "logits", device=logits.device)
    return EP_DTYPE_FP32 if logits.dtype == torch.float32 else EP_DTYPE_BF16


def _score(score: str) -> int:
    if score not in SCORES:
        raise ValueError("score must be one of %s, got %r" % (sorted(SCORES), score))
    return SCORES[score]


def route(logits: torch.Tensor, num_topk: int, expert_bias: torch.Tensor | None = None,
          score: str = "softmax", num_groups: int = 1, topk_groups: int = 1,
          normalize: bool = False, scale: float = 1.0, out=None):
    """ep_route: logits [T, E] float32 or bf16 -> (topk_idx [T, K] int64,
    topk_weights [T, K] float32), the arguments of the dispatch calls and of
    combine.  ``out`` = (topk_idx, topk_weights) may be given."""
    dt = _logits_dtype(logits)
    T, E = logits.shape
    K, NG, TG = int(num_topk), int(num_groups), int(topk_groups)
    _sizes(T | E | K | NG | TG)
    dev = logits.device
    if expert_bias is not None:
        _need(expert_bias, torch.float32, "expert_bias", (E,), device=dev)
    if out is None:
        out = (torch.empty((T, K), dtype=torch.int64, device=dev),
               torch.empty((T, K), dtype=torch.float32, device=dev))
    idx, w = out
    _need(idx, torch.int64, "topk_idx", (T, K), device=dev)
    _need(w, torch.float32, "topk_weights", (T, K), device=dev)
    _launch("ep_route", logits, _addr(logits), dt, _addr(expert_bias), T, E, K, _score(score),
            NG, TG, int(bool(normalize)), float(scale), _addr(idx), _addr(w))
    return idx, w


def route_backward(logits: torch.Tensor, topk_idx: torch.Tensor, grad_weights: torch.Tensor,
                   score: str = "softmax", normalize: bool = False, scale: float = 1.0,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """ep_route_backward: the gradient of route's topk_weights with respect to
    its logits, [T, E] in their type."""
    dt = _logits_dtype(logits)
    T, E = logits.shape
    dev = logits.device
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    K = topk_idx.shape[1]
    _sizes(T | E | K)
    _need(topk_idx, torch.int64, "topk_idx", (T, K), device=dev)
    _need(grad_weights, torch.float32, "grad_weights", (T, K), device=dev)
    if out is None:
        out = torch.empty_like(logits)
    _need(out, logits.dtype, "out", (T, E), device=dev)
    _launch("ep_route_backward", logits, _addr(logits), dt, _addr(topk_idx), _addr(grad_weights), T,
            E, K, _score(score), int(bool(normalize)), float(scale), _addr(out))
    return out


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def expert_linear_w4(x: torch.Tensor, weight: torch.Tensor, scales: torch.Tensor,
                     num_tokens_per_expert: torch.Tensor,
                     expert_offsets: torch.Tensor | None = None, capacity: int = 0,
                     x_scales: torch.Tensor | None = None, zeros: torch.Tensor | None = None,
                     swiglu: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """ep_expert_linear_w4: the experts' products over the rows of a dispatch.

    x is [R, I] bf16, or uint8 E4M3 codes with x_scales [R, I/128]; weight
    uint8 [E, W, I/2], scales bf16 [E, I/G, W], zeros uint8 [E, I/G, W] or
    None, W = N, or 2N with swiglu.  The rows are those of a dispatch with
    offsets (expert_offsets [E+1] and the counts of its Layout) or of a
    low_latency_dispatch (its counts and ``capacity``).  Returns y [R, N]
    bf16; rows that hold no token are left as they are (an ``out`` not given
    is allocated uninitialised)."""
    if x.dim() != 2 or weight.dim() != 3 or scales.dim() != 3:
        raise ValueError("x must be [R, I], weight [E, W, I/2] and scales [E, I/G, W]")
    R, I = x.shape
    E, W = weight.shape[0], weight.shape[1]
    NG = scales.shape[1]
    C = int(capacity)
    _sizes(E | I | W | C)
    dev = x.device
    if swiglu and W % 2 != 0:
        raise ValueError("swiglu needs an even number of weight channels, got %d" % W)
    N = W // 2 if swiglu else W
    if I % 2 != 0 or NG == 0 or I % NG != 0:
        raise ValueError("scales must hold I/G groups: I = %d, groups = %d" % (I, NG))
    fp8 = x.dtype == torch.uint8
    _need(x, torch.uint8 if fp8 else torch.bfloat16, "x", device=dev)
    if fp8:
        if x_scales is None:
            raise ValueError("E4M3 codes need x_scales")
        _need(x_scales, torch.float32, "x_scales", (R, I // 128), device=dev)
    elif x_scales is not None:
        raise ValueError("x_scales belong to E4M3 codes (uint8 x)")
    _need(weight, torch.uint8, "weight", (E, W, I // 2), device=dev)
    _need(scales, torch.bfloat16, "scales", (E, NG, W), device=dev)
    if zeros is not None:
        _need(zeros, torch.uint8, "zeros", (E, NG, W), device=dev)
    _need(num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=dev)
    if expert_offsets is not None:
        if C:
            raise ValueError("give expert_offsets or capacity, not both")
        _need(expert_offsets, torch.int32, "expert_offsets", (E + 1,), device=dev)
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", (R, N), device=dev)
    _launch("ep_expert_linear_w4", x, _addr(x), _addr(x_scales),
            EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16, R, _addr(expert_offsets),
            _addr(num_tokens_per_expert), C, E, I, N, I // NG, _addr(weight),
            _addr(scales), _addr(zeros), int(bool(swiglu)), _addr(out))
    return out


def _runs(num_tokens_per_expert: torch.Tensor, expert_offsets: torch.Tensor | None, capacity: int,
          E: int, device):
    """Check the tensors that say which rows an expert has."""
    _need(num_tokens_per_expert, torch.int32, "num_tokens_per_expert", (E,), device=device)
    if expert_offsets is not None:
        if capacity:
            raise ValueError("give expert_offsets or capacity, not both")
        _need(expert_offsets, torch.int32, "expert_offsets", (E + 1,), device=device)


def expert_linear(x: torch.Tensor, weight: torch.Tensor, num_tokens_per_expert: torch.Tensor,
                  expert_offsets: torch.Tensor | None = None, capacity: int = 0,
                  x_scales: torch.Tensor | None = None,
                  weight_scales: torch.Tensor | None = None, swiglu: bool = False,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """ep_expert_linear: the experts' products over the rows of a dispatch.

    x [R, I] and weight [E, W, I] are both bf16, or both uint8 E4M3 codes with
    x_scales [R, I/128] and weight_scales [E, S, I/128] float32, one scale per
    128 x 128 block; W = N and S = ceil(N/128), or both doubled with swiglu
    (gate half first).  The rows are those of a dispatch with offsets
    (expert_offsets [E+1] and the counts of its Layout) or of a
    low_latency_dispatch (its counts and ``capacity``).  Returns y [R, N] bf16;
    rows that hold no token are left as they are (an ``out`` not given is
    allocated uninitialised)."""
    if x.dim() != 2 or weight.dim() != 3:
        raise ValueError("x must be [R, I] and weight [E, W, I]")
    R, I = x.shape
    E, W = weight.shape[0], weight.shape[1]
    C = int(capacity)
    _sizes(E | I | W | C)
    dev = x.device
    if swiglu and W % 2 != 0:
        raise ValueError("swiglu needs an even number of weight channels, got %d" % W)
    N = W // 2 if swiglu else W
    fp8 = x.dtype == torch.uint8
    dt = torch.uint8 if fp8 else torch.bfloat16
    _need(x, dt, "x", device=dev)
    _need(weight, dt, "weight", (E, W, I), device=dev)
    if fp8:
        if x_scales is None or weight_scales is None:
            raise ValueError("E4M3 codes need x_scales and weight_scales")
        _need(x_scales, torch.float32, "x_scales", (R, I // 128), device=dev)
        S = (N + 127) // 128 * (2 if swiglu else 1)
        _need(weight_scales, torch.float32, "weight_scales", (E, S, I // 128), device=dev)
    elif x_scales is not None or weight_scales is not None:
        raise ValueError("x_scales and weight_scales belong to E4M3 codes (uint8)")
    _runs(num_tokens_per_expert, expert_offsets, C, E, dev)
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", (R, N), device=dev)
    _launch("ep_expert_linear", x, _addr(x), _addr(x_scales),
            EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16, R, _addr(expert_offsets),
            _addr(num_tokens_per_expert), C, E, I, N, _addr(weight), _addr(weight_scales),
            int(bool(swiglu)), _addr(out))
    return out


def expert_linear_backward(grad_y: torch.Tensor, x: torch.Tensor | None,
                           weight: torch.Tensor | None, num_tokens_per_expert: torch.Tensor,
                           expert_offsets: torch.Tensor | None = None, capacity: int = 0,
                           grad_weight_dtype: torch.dtype = torch.bfloat16,
                           accumulate: bool = False, out=None):
    """ep_expert_linear_backward: from grad_y [R, N] bf16 the gradients of
    expert_linear(x, weight, ...) in bf16 without swiglu: (grad_x [R, I] bf16,
    grad_weight [E, N, I] bf16 or float32), or the ones given in ``out``.
    Without ``weight`` only grad_weight is computed, without ``x`` only grad_x;
    the other one is None.  ``accumulate`` adds to a float32 grad_weight given
    in ``out``.  Rows of grad_x that hold no token are left as they are (a
    grad_x not given is allocated uninitialised)."""
    if x is None and weight is None:
        raise ValueError("expert_linear_backward needs x or weight")
    if (grad_y.dim() != 2 or (x is not None and x.dim() != 2)
            or (weight is not None and weight.dim() != 3)):
        raise ValueError("grad_y must be [R, N], x [R, I] and weight [E, N, I]")
    R, N = grad_y.shape
    E = num_tokens_per_expert.numel() if weight is None else weight.shape[0]
    I = x.shape[1] if weight is None else weight.shape[2]
    C = int(capacity)
    _sizes(E | I | N | C)
    dev = grad_y.device
    _need(grad_y, torch.bfloat16, "grad_y", device=dev)
    grad_x, grad_weight = (None, None) if out is None else out
    if weight is not None:
        _need(weight, torch.bfloat16, "weight", (E, N, I), device=dev)
        if grad_x is None:
            grad_x = torch.empty((R, I), dtype=torch.bfloat16, device=dev)
        _need(grad_x, torch.bfloat16, "grad_x", (R, I), device=dev)
    elif grad_x is not None:
        raise ValueError("grad_x needs weight")
    if x is not None:
        _need(x, torch.bfloat16, "x", (R, I), device=dev)
        if grad_weight is None:
            if accumulate:
                raise ValueError("accumulate needs a grad_weight in out")
            grad_weight = torch.empty((E, N, I), dtype=grad_weight_dtype, device=dev)
        dt = grad_weight.dtype
        if dt != torch.float32 and (dt != torch.bfloat16 or accumulate):
            raise TypeError("grad_weight must be float32%s, got %s"
                            % (" to accumulate" if accumulate else " or bfloat16", dt))
        _need(grad_weight, dt, "grad_weight", (E, N, I), device=dev)
    elif grad_weight is not None:
        raise ValueError("grad_weight needs x")
    _runs(num_tokens_per_expert, expert_offsets, C, E, dev)
    f32 = grad_weight is not None and grad_weight.dtype == torch.float32
    _launch("ep_expert_linear_backward", grad_y, _addr(grad_y), _addr(x), _addr(weight), R,
            _addr(expert_offsets), _addr(num_tokens_per_expert), C, E, I, N, _addr(grad_x),
            _addr(grad_weight), EP_DTYPE_FP32 if f32 else EP_DTYPE_BF16, int(bool(accumulate)))
    return grad_x, grad_weight


def expert_swiglu(gate_up: torch.Tensor, num_tokens_per_expert: torch.Tensor | None = None,
                  expert_offsets: torch.Tensor | None = None, capacity: int = 0,
                  fp8: bool = False, out=None):
    """ep_expert_swiglu: gate_up [R, 2N] bf16 -> silu(gate) * up, y [R, N] bf16,
    or with ``fp8`` (codes [R, N] uint8, scales [R, N/128] float32).  The rows
    are the experts', as expert_linear takes them, or all of them without
    ``num_tokens_per_expert``; the others are left as they are (an ``out`` not
    given is allocated uninitialised)."""
    R, N = _gate_shape(gate_up)
    dev = gate_up.device
    E, C = _gate_runs(num_tokens_per_expert, expert_offsets, capacity, N, dev)
    _need(gate_up, torch.bfloat16, "gate_up", device=dev)
    if fp8:
        if out is None:
            out = (torch.empty((R, N), dtype=torch.uint8, device=dev),
                   torch.empty((R, N // 128), dtype=torch.float32, device=dev))
        y, scales = out
        _need(y, torch.uint8, "codes", (R, N), device=dev)
        _need(scales, torch.float32, "scales", (R, N // 128), device=dev)
    else:
        if out is None:
            out = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
        y, scales = out, None
        _need(y, torch.bfloat16, "out", (R, N), device=dev)
    _launch("ep_expert_swiglu", gate_up, _addr(gate_up), R, _addr(expert_offsets),
            _addr(num_tokens_per_expert), C, E, N, EP_DTYPE_FP8_E4M3 if fp8 else EP_DTYPE_BF16,
            _addr(y), _addr(scales))
    return out


def expert_swiglu_backward(grad_y: torch.Tensor, gate_up: torch.Tensor,
                           num_tokens_per_expert: torch.Tensor | None = None,
                           expert_offsets: torch.Tensor | None = None, capacity: int = 0,
                           out: torch.Tensor | None = None) -> torch.Tensor:
    """ep_expert_swiglu_backward: from grad_y [R, N] bf16 the gradient of
    expert_swiglu's gate_up, [R, 2N] bf16."""
    R, N = _gate_shape(gate_up)
    dev = gate_up.device
    E, C = _gate_runs(num_tokens_per_expert, expert_offsets, capacity, N, dev)
    _need(gate_up, torch.bfloat16, "gate_up", device=dev)
    _need(grad_y, torch.bfloat16, "grad_y", (R, N), device=dev)
    if out is None:
        out = torch.empty((R, 2 * N), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", (R, 2 * N), device=dev)
    _launch("ep_expert_swiglu_backward", gate_up, _addr(grad_y), _addr(gate_up), R,
            _addr(expert_offsets), _addr(num_tokens_per_expert), C, E, N, _addr(out))
    return out


def _gate_shape(gate_up: torch.Tensor):
    if gate_up.dim() != 2 or gate_up.shape[1] % 2 != 0:
        raise ValueError("gate_up must be [R, 2N]")
    return gate_up.shape[0], gate_up.shape[1] // 2


def _gate_runs(num_tokens_per_expert, expert_offsets, capacity, N, device):
    C = int(capacity)
    if num_tokens_per_expert is None:
        if expert_offsets is not None or C:
            raise ValueError("expert_offsets and capacity need num_tokens_per_expert")
        _sizes(N)
        return 0, 0
    E = num_tokens_per_expert.numel()
    _sizes(E | N | C)
    _runs(num_tokens_per_expert, expert_offsets, C, E, device)
    return E, C


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

@dataclass
class RmsNormed:
    y: torch.Tensor | None               # [T, H] bf16
    codes: torch.Tensor | None           # [T, H] uint8 E4M3 codes of y
    scales: torch.Tensor | None          # [T, H/128] float32
    residual: torch.Tensor | None        # [T, H] bf16: x + residual
    inv_rms: torch.Tensor                # [T] float32


def _norm_weight(weight: torch.Tensor, H: int, device) -> int:
    if weight.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("weight must be float32 or bfloat16, got %s" % weight.dtype)
    _need(weight, weight.dtype, "weight", (H,), device=device)
    return EP_DTYPE_FP32 if weight.dtype == torch.float32 else EP_DTYPE_BF16


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, bf16: bool = True, fp8: bool = False,
             out: RmsNormed | None = None) -> RmsNormed:
    """ep_rms_norm: h / rms(h) * weight of h = x [T, H] bf16, or of h = x +
    residual, which is then the next residual: in bf16 (``bf16``), in E4M3 with a
    scale per 128 channels (``fp8``), or both."""
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    _sizes(T | H)
    dev = x.device
    if not bf16 and not fp8:
        raise ValueError("rms_norm needs bf16 or fp8")
    _need(x, torch.bfloat16, "x", device=dev)
    wdt = _norm_weight(weight, H, dev)
    if residual is not None:
        _need(residual, torch.bfloat16, "residual", (T, H), device=dev)
    if out is None:
        f32 = torch.float32
        out = RmsNormed(
            torch.empty_like(x) if bf16 else None,
            torch.empty_like(x, dtype=torch.uint8) if fp8 else None,
            x.new_empty((T, H // 128), dtype=f32) if fp8 else None,
            torch.empty_like(x) if residual is not None else None,
            x.new_empty(T, dtype=f32))
    else:
        if bf16:
            _need(out.y, torch.bfloat16, "y", (T, H), device=dev)
        if fp8:
            _need(out.codes, torch.uint8, "codes", (T, H), device=dev)
            _need(out.scales, torch.float32, "scales", (T, H // 128), device=dev)
        if residual is not None:
            _need(out.residual, torch.bfloat16, "out.residual", (T, H), device=dev)
        _need(out.inv_rms, torch.float32, "inv_rms", (T,), device=dev)
    _launch("ep_rms_norm", x, _addr(x), _addr(residual), _addr(weight), wdt, T, H, float(eps),
            _addr(out.y) if bf16 else None, _addr(out.codes) if fp8 else None,
            _addr(out.scales) if fp8 else None,
            _addr(out.residual) if residual is not None else None, _addr(out.inv_rms))
    return out


def rms_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                      inv_rms: torch.Tensor, grad_residual: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, out=None):
    """ep_rms_norm_backward: from grad_y [T, H] bf16 the gradients of rms_norm:
    (grad_x [T, H] bf16, of x and residual alike, grad_weight [H] float32).
    ``x`` is what was normed, with a residual the call's ``residual`` output, whose
    own gradient ``grad_residual`` is added.  ``workspace``: uint8, at least
    rms_norm_backward_workspace_bytes; allocated if not given."""
    if grad_y.dim() != 2:
        raise ValueError("grad_y must be [T, H]")
    T, H = grad_y.shape
    _sizes(T | H)
    dev = grad_y.device
    _need(grad_y, torch.bfloat16, "grad_y", device=dev)
    _need(x, torch.bfloat16, "x", (T, H), device=dev)
    wdt = _norm_weight(weight, H, dev)
    _need(inv_rms, torch.float32, "inv_rms", (T,), device=dev)
    if grad_residual is not None:
        _need(grad_residual, torch.bfloat16, "grad_residual", (T, H), device=dev)
    if out is None:
        grad_x, grad_weight = torch.empty_like(grad_y), grad_y.new_empty(H, dtype=torch.float32)
    else:
        grad_x, grad_weight = out
        _need(grad_x, torch.bfloat16, "grad_x", (T, H), device=dev)
        _need(grad_weight, torch.float32, "grad_weight", (H,), device=dev)
    if workspace is None:
        workspace = grad_y.new_empty(rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8)
    else:
        _need(workspace, torch.uint8, "workspace", device=dev)
    _launch("ep_rms_norm_backward", grad_y, _addr(grad_y), _addr(x), _addr(weight), wdt,
            _addr(inv_rms), _addr(grad_residual), T, H, _addr(grad_x), _addr(grad_weight),
            _addr(workspace), workspace.numel())
    return grad_x, grad_weight


def rms_norm_backward_workspace_bytes(num_tokens: int, hidden: int) -> int:
    """Bytes of rms_norm_backward's workspace (0 for an invalid shape)."""
    _sizes(num_tokens | hidden)
    return (_lib or lib()).ep_rms_norm_backward_workspace_bytes(num_tokens, hidden)


# ---------------------------------------------------------------------------
# diagnostics
# ---------------------------------------------------------------------------

def convert_e4m3(v: torch.Tensor, mode: int = 0) -> torch.Tensor:
    """E4M3 codes of fp32 ``v`` with the dispatch kernel's conversion (mode 0)
    or the software conversion (mode 1)."""
    _need(v, torch.float32, "v")
    out = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check(lib().ep_convert_e4m3(_ptr(v), _ptr(out), v.numel(), mode, _stream(v)),
           "ep_convert_e4m3")
    return out


def convert_bf16(v: torch.Tensor) -> torch.Tensor:
    """bf16 bits (as int16) of fp32 ``v`` with the combine kernel's rounding."""
    _need(v, torch.float32, "v")
    out = torch.empty(v.shape, dtype=torch.int16, device=v.device)
    _check(lib().ep_convert_bf16(_ptr(v), _ptr(out), v.numel(), _stream(v)), "ep_convert_bf16")
    return out


def copy(src: torch.Tensor, dst: torch.Tensor):
    """ep_copy of all of ``src``'s bytes into ``dst``."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst too small")
    _check(lib().ep_copy(_ptr(src), _ptr(dst), nbytes, _stream(src)), "ep_copy")
