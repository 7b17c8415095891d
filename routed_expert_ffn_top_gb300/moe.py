"""Thin ctypes binding of the C ABI in ``include/moe.h`` (argument marshalling only).

Every function here has the name of the C entry point it calls and does no arithmetic of
its own: it checks dtypes/devices/contiguity of torch tensors, allocates outputs the
caller did not pass, hands raw device pointers and the current CUDA stream to the library,
and raises :class:`MoeError` on a non-zero status.  The library must have been built
(``python -m routed_expert_ffn_top_gb300.build`` or ``__graft_entry__.build()``); there is
no fallback of any kind when it is missing.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import build as _build

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_DEVICE = 5

MOE_DEV_INVALID_EXPERT = 0x1
MOE_DEV_WAIT_TIMEOUT = 0x2
MOE_DEV_BAD_ALIGNMENT = 0x4

MOE_W_DENSE_BF16 = 0
MOE_W_VQ_GATEUP = 1
MOE_W_VQLR_GATEUP = 2

MOE_DT_BF16 = 0
MOE_DT_F16 = 1
MOE_DT_F32 = 2
MOE_MICROSCALE_STATUS_BYTES = 256

# Every symbol include/moe.h declares (checked against the header by the tests).
EXPORTS = (
    "moe_status_string", "moe_route_topk", "moe_align_capacity", "moe_align_block_size",
    "moe_workspace_bytes", "moe_expert_ffn", "moe_decode_block", "moe_decode_block_host",
    "moe_read_device_status", "moe_set_trace_events", "moe_decode_block_noalloc",
    "moe_selftest_wait_timeout", "moe_reader_build", "moe_reader_workspace_bytes",
    "moe_reader_ffn", "moe_library_block_size", "moe_workspace_layout",
    "moe_token_plan", "moe_token_sort", "moe_token_sort_grad", "moe_token_unsort",
    "moe_token_unsort_grad", "moe_microscale_pitch", "moe_microscale_quantize",
    "moe_microscale_dequantize", "moe_microscale_product", "moe_microscale_gated_product",
    "moe_microscale_workspace_bytes", "moe_microscale_ffn",
)


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, moe_status_string(status), status))


class ExpertWeights(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
        ("j_gate", ctypes.c_void_p), ("j_up", ctypes.c_void_p),
        ("cb_gate", ctypes.c_void_p), ("cb_up", ctypes.c_void_p),
        ("d", ctypes.c_int32), ("K", ctypes.c_int32),
        ("w_down", ctypes.c_void_p),
        ("d_gate", ctypes.c_void_p), ("d_up", ctypes.c_void_p),
        ("c_gate", ctypes.c_void_p), ("c_up", ctypes.c_void_p),
        ("r", ctypes.c_int32),
        ("vq_form", ctypes.c_int32),
    ]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [
        ("b", ctypes.c_int32), ("kn", ctypes.c_int32), ("cap", ctypes.c_int64),
        ("status", ctypes.c_size_t), ("sorted_route_ids", ctypes.c_size_t),
        ("expert_block_ids", ctypes.c_size_t), ("num_padded", ctypes.c_size_t),
        ("y", ctypes.c_size_t), ("p_tiles", ctypes.c_size_t),
        ("tpb", ctypes.c_int32), ("zero_bytes", ctypes.c_int32),
        ("launches", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("p_rows", ctypes.c_size_t),
    ]


class ReaderStruct(ctypes.Structure):
    _fields_ = [
        ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
        ("rank", ctypes.c_int32),
        ("signs", ctypes.c_void_p), ("g_rows", ctypes.c_void_p), ("v_rows", ctypes.c_void_p),
        ("w_down", ctypes.c_void_p), ("g_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("g_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("dnorm", ctypes.c_void_p),
        ("U", ctypes.c_void_p), ("coef", ctypes.c_void_p),
    ]


class MicroscaleWeights(ctypes.Structure):
    _fields_ = [
        ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("gate_up_codes", ctypes.c_void_p), ("gate_up_scales", ctypes.c_void_p),
        ("down_codes", ctypes.c_void_p), ("down_scales", ctypes.c_void_p),
    ]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """The loaded CDLL (raises if the library has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    "CUDA library %s is missing: build it with "
                    "`python -m routed_expert_ffn_top_gb300.build`" % path)
            L = ctypes.CDLL(path)
            vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            wp = ctypes.POINTER(ExpertWeights)
            L.moe_status_string.argtypes = [ci]
            L.moe_status_string.restype = ctypes.c_char_p
            L.moe_route_topk.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, vp, vp, vp]
            L.moe_align_capacity.argtypes = [ci, ci, ci, ci]
            L.moe_align_capacity.restype = sz
            L.moe_align_block_size.argtypes = [vp, ci, ci, ci, ci, vp, vp, vp, sz, vp]
            L.moe_workspace_bytes.argtypes = [wp, ci, ci, ci]
            L.moe_workspace_bytes.restype = sz
            L.moe_library_block_size.argtypes = [wp, ci, ci, ci]
            L.moe_library_block_size.restype = ci
            L.moe_workspace_layout.argtypes = [wp, ci, ci, ci, ctypes.POINTER(WorkspaceLayout)]
            L.moe_expert_ffn.argtypes = [vp, wp, ci, ci, vp, vp, vp, vp, vp, ci, vp, vp, vp, sz, vp]
            L.moe_decode_block.argtypes = [vp, vp, vp, wp, ci, ci, ci, vp, vp, vp, vp, vp, sz, vp]
            L.moe_decode_block_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, wp, ci, ci, ci,
                                                vp, vp, vp, sz, vp]
            L.moe_read_device_status.argtypes = [vp, vp, vp]
            L.moe_set_trace_events.argtypes = [vp, ci]
            L.moe_decode_block_noalloc.argtypes = [vp, vp, vp, wp, ci, ci, ci, vp, vp, vp, vp, vp]
            L.moe_selftest_wait_timeout.argtypes = [vp, sz, vp]
            rp = ctypes.POINTER(ReaderStruct)
            L.moe_reader_build.argtypes = [wp, rp, vp]
            L.moe_reader_workspace_bytes.argtypes = [rp, ci, ci, ci]
            L.moe_reader_workspace_bytes.restype = sz
            L.moe_reader_ffn.argtypes = [vp, rp, ci, ci, vp, vp, ci, ci, vp, vp, vp, vp, vp, sz, vp]
            i64 = ctypes.c_int64
            mp = ctypes.POINTER(MicroscaleWeights)
            L.moe_token_plan.argtypes = [vp, ci, ci, ci, vp, vp, vp, vp]
            L.moe_token_sort.argtypes = [vp, i64, ci, ci, ci, ci, vp, vp, i64, vp]
            L.moe_token_sort_grad.argtypes = [vp, i64, ci, ci, ci, ci, vp, vp, i64, vp]
            L.moe_token_unsort.argtypes = [vp, i64, ci, ci, ci, ci, vp, vp, vp, i64, vp, i64, vp]
            L.moe_token_unsort_grad.argtypes = [vp, i64, vp, i64, ci, ci, ci, ci, vp, vp, vp, i64,
                                                vp, vp]
            L.moe_microscale_pitch.argtypes = [ci]
            L.moe_microscale_quantize.argtypes = [vp, i64, ci, i64, ci, vp, ci, vp, vp, vp]
            L.moe_microscale_dequantize.argtypes = [vp, vp, i64, ci, vp, i64, ci, vp]
            L.moe_microscale_product.argtypes = [vp, vp, i64, vp, vp, vp, ci, ci, ci, ci, vp, i64,
                                                 vp, sz, vp]
            L.moe_microscale_gated_product.argtypes = [vp, vp, i64, vp, vp, vp, ci, ci, ci, vp, vp,
                                                       vp, sz, vp]
            L.moe_microscale_workspace_bytes.argtypes = [mp, ci, ci]
            L.moe_microscale_workspace_bytes.restype = sz
            L.moe_microscale_ffn.argtypes = [vp, mp, ci, ci, vp, vp, vp, vp, vp, sz, vp]
            for f in ("moe_token_plan", "moe_token_sort", "moe_token_sort_grad",
                      "moe_token_unsort", "moe_token_unsort_grad", "moe_microscale_pitch",
                      "moe_microscale_quantize", "moe_microscale_dequantize",
                      "moe_microscale_product", "moe_microscale_gated_product",
                      "moe_microscale_ffn"):
                getattr(L, f).restype = ci
            for f in ("moe_route_topk", "moe_align_block_size", "moe_expert_ffn",
                      "moe_decode_block", "moe_decode_block_host", "moe_read_device_status",
                      "moe_set_trace_events", "moe_decode_block_noalloc",
                      "moe_selftest_wait_timeout", "moe_reader_build", "moe_reader_ffn"):
                getattr(L, f).restype = ci
            _lib = L
    return _lib


# ----------------------------------------------------------------------------- marshalling
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current device, and the handle of its current stream without a Stream object, by torch's own
# short calls where it has them (the public ones take a microsecond each of calls that take 5).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        return ctypes.c_void_p(_current_stream(torch.cuda.current_device()))
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


def _need(t, dtype, name, device=None):
    if t is None:
        raise ValueError("%s is required" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    return t


def _need_cuda(device):
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device, got %s" % device)


def _workspace(t, device):
    """Checks a workspace: contiguous bytes on the device.  Returns (address, bytes)."""
    if not (t.dtype is torch.uint8 and t.device == device and t.is_contiguous()):
        _need(t, torch.uint8, "workspace", device)
    return t.data_ptr(), t.numel()


def _one_device(device, layer):
    """A layer's tensors (one device's, as its descriptor checks) are on the GPU of the rows."""
    _need_cuda(device)
    if layer["w_down"].device != device:
        raise ValueError("the layer must be on %s, got %s" % (device, layer["w_down"].device))


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def expert_weights(layer: dict) -> ExpertWeights:
    """C weight descriptor for a layer dict (as made by :mod:`.synthetic`).

    The descriptor holds raw pointers; the caller keeps ``layer``'s tensors alive.
    """
    w = ExpertWeights()
    w.kind = int(layer.get("kind", MOE_W_DENSE_BF16))
    w.H, w.I, w.E = int(layer["H"]), int(layer["I"]), int(layer["E"])
    w.d, w.K = int(layer.get("d", 0) or 0), int(layer.get("K", 0) or 0)
    w.vq_form = int(layer.get("vq_form", 0) or 0)
    dev = layer["w_down"].device
    _need(layer["w_down"], torch.bfloat16, "w_down", dev)
    w.w_down = layer["w_down"].data_ptr()
    if w.kind == MOE_W_DENSE_BF16:
        w.w_gate = _need(layer["w_gate"], torch.bfloat16, "w_gate", dev).data_ptr()
        w.w_up = _need(layer["w_up"], torch.bfloat16, "w_up", dev).data_ptr()
    else:
        w.j_gate = _need(layer["j_gate"], torch.uint8, "j_gate", dev).data_ptr()
        w.j_up = _need(layer["j_up"], torch.uint8, "j_up", dev).data_ptr()
        w.cb_gate = _need(layer["cb_gate"], torch.bfloat16, "cb_gate", dev).data_ptr()
        w.cb_up = _need(layer["cb_up"], torch.bfloat16, "cb_up", dev).data_ptr()
    if w.kind == MOE_W_VQLR_GATEUP:
        w.r = int(layer["r"])
        w.d_gate = _need(layer["d_gate"], torch.bfloat16, "d_gate", dev).data_ptr()
        w.d_up = _need(layer["d_up"], torch.bfloat16, "d_up", dev).data_ptr()
        w.c_gate = _need(layer["c_gate"], torch.bfloat16, "c_gate", dev).data_ptr()
        w.c_up = _need(layer["c_up"], torch.bfloat16, "c_up", dev).data_ptr()
    return w


# ------------------------------------------------------------------------------ entry points
def moe_route_topk(h, w_router, bias, k, renormalize=True, topk_ids=None, topk_weights=None,
                   stream=None):
    dev = h.device
    _need_cuda(dev)
    _need(h, torch.bfloat16, "h", dev)
    _need(w_router, torch.bfloat16, "w_router", dev)
    if bias is not None:
        _need(bias, torch.float32, "bias", dev)
    M, H = h.shape
    E = w_router.shape[1]
    if topk_ids is None:
        topk_ids = torch.empty((M, k), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty((M, k), dtype=torch.float32, device=dev)
    _need(topk_ids, torch.int32, "topk_ids", dev)
    _need(topk_weights, torch.float32, "topk_weights", dev)
    _check(lib().moe_route_topk(_ptr(h), _ptr(w_router), _ptr(bias), M, H, E, k,
                                int(bool(renormalize)), _ptr(topk_ids), _ptr(topk_weights),
                                _stream(stream)), "moe_route_topk")
    return topk_ids, topk_weights


def moe_align_capacity(M, k, E, b) -> int:
    return int(lib().moe_align_capacity(M, k, E, b))


def moe_align_block_size(topk_ids, E, b, sorted_route_ids=None, expert_block_ids=None,
                         num_padded=None, stream=None):
    dev = topk_ids.device
    _need_cuda(dev)
    _need(topk_ids, torch.int32, "topk_ids", dev)
    M, k = topk_ids.shape
    cap = moe_align_capacity(M, k, E, b)
    if sorted_route_ids is None:
        sorted_route_ids = torch.empty((cap,), dtype=torch.int32, device=dev)
    if expert_block_ids is None:
        expert_block_ids = torch.empty((max(cap // b, 1),), dtype=torch.int32, device=dev)
    if num_padded is None:
        num_padded = torch.empty((1,), dtype=torch.int32, device=dev)
    _need(sorted_route_ids, torch.int32, "sorted_route_ids", dev)
    _need(expert_block_ids, torch.int32, "expert_block_ids", dev)
    _need(num_padded, torch.int32, "num_padded", dev)
    if expert_block_ids.numel() < sorted_route_ids.numel() // b:
        raise ValueError("expert_block_ids must hold cap // b entries")
    _check(lib().moe_align_block_size(_ptr(topk_ids), M, k, E, b, _ptr(sorted_route_ids),
                                      _ptr(expert_block_ids), _ptr(num_padded),
                                      sorted_route_ids.numel(), _stream(stream)),
           "moe_align_block_size")
    return sorted_route_ids, expert_block_ids, num_padded


def moe_workspace_bytes(layer: dict, M, k, b) -> int:
    w = expert_weights(layer)
    return int(lib().moe_workspace_bytes(ctypes.byref(w), M, k, b))


def moe_library_block_size(layer: dict, M, k, b) -> int:
    """The block size moe_decode_block aligns with for these weights and sizes."""
    w = expert_weights(layer)
    return int(lib().moe_library_block_size(ctypes.byref(w), M, k, b))


def moe_workspace_layout(layer: dict, M, k, b) -> dict:
    """Block size, capacity and byte offsets of the alignment inside the workspace of
    moe_decode_block / moe_expert_ffn (library alignment) for these sizes."""
    w = expert_weights(layer)
    out = WorkspaceLayout()
    _check(lib().moe_workspace_layout(ctypes.byref(w), M, k, b, ctypes.byref(out)),
           "moe_workspace_layout")
    return {f: int(getattr(out, f)) for f, _ in WorkspaceLayout._fields_ if f != "reserved"}


def workspace_alignment(workspace: torch.Tensor, layout: dict):
    """Views (sorted_route_ids, expert_block_ids, num_padded) of the alignment a call left in
    `workspace`, at the offsets of `layout` (moe_workspace_layout)."""
    cap, b = layout["cap"], layout["b"]

    def view(off, n):
        return workspace[off:off + 4 * n].view(torch.int32)

    return (view(layout["sorted_route_ids"], cap), view(layout["expert_block_ids"], cap // b),
            view(layout["num_padded"], 1))


def alloc_workspace(layer: dict, M, k, b, device=None) -> torch.Tensor:
    """A zero-filled workspace of the size the library asks for (256-byte aligned)."""
    n = moe_workspace_bytes(layer, M, k, b)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_workspace_bytes")
    device = layer["w_down"].device if device is None else device
    return torch.zeros((n,), dtype=torch.uint8, device=device)


def moe_expert_ffn(h, layer, topk_ids, topk_weights, b, alignment=None, residual=None,
                   out=None, workspace=None, stream=None):
    dev = h.device
    _need(h, torch.bfloat16, "h", dev)
    _need(topk_ids, torch.int32, "topk_ids", dev)
    _need(topk_weights, torch.float32, "topk_weights", dev)
    M, k = topk_ids.shape
    w = expert_weights(layer)
    _one_device(dev, layer)
    if residual is not None:
        _need(residual, torch.bfloat16, "residual", dev)
    if out is None:
        out = torch.empty((M, w.H), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out", dev)
    if workspace is None:
        workspace = alloc_workspace(layer, M, k, b, dev)
    srt = blk = npad = None
    if alignment is not None:
        srt, blk, npad = alignment
    _check(lib().moe_expert_ffn(_ptr(h), ctypes.byref(w), M, k, _ptr(topk_ids),
                                _ptr(topk_weights), _ptr(srt), _ptr(blk), _ptr(npad), b,
                                _ptr(residual), _ptr(out), *_workspace(workspace, dev),
                                _stream(stream)), "moe_expert_ffn")
    return out


def moe_decode_block(h, layer, k, b, residual=None, out=None, topk_ids=None, topk_weights=None,
                     workspace=None, stream=None):
    dev = h.device
    _need(h, torch.bfloat16, "h", dev)
    M = h.shape[0]
    w = expert_weights(layer)
    _one_device(dev, layer)
    w_router = _need(layer["w_router"], torch.bfloat16, "w_router", dev)
    bias = layer.get("bias")
    if bias is not None:
        _need(bias, torch.float32, "bias", dev)
    if residual is not None:
        _need(residual, torch.bfloat16, "residual", dev)
    if out is None:
        out = torch.empty((M, w.H), dtype=torch.bfloat16, device=dev)
    if topk_ids is None:
        topk_ids = torch.empty((M, k), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty((M, k), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(layer, M, k, b, dev)
    _need(out, torch.bfloat16, "out", dev)
    _need(topk_ids, torch.int32, "topk_ids", dev)
    _need(topk_weights, torch.float32, "topk_weights", dev)
    _check(lib().moe_decode_block(_ptr(h), _ptr(w_router), _ptr(bias), ctypes.byref(w), M, k, b,
                                  _ptr(residual), _ptr(out), _ptr(topk_ids), _ptr(topk_weights),
                                  *_workspace(workspace, dev), _stream(stream)),
           "moe_decode_block")
    return out, topk_ids, topk_weights


def moe_decode_block_noalloc(h, layer, k, b, residual=None, out=None, topk_ids=None,
                             topk_weights=None, stream=None):
    """moe_decode_block without a workspace: for callers that cannot allocate device memory,
    the library runs the block on its own fixed scratch array (see include/moe.h).  Outputs
    the caller does not pass are allocated here by torch, as for the other wrappers."""
    dev = h.device
    _need(h, torch.bfloat16, "h", dev)
    M = h.shape[0]
    w = expert_weights(layer)
    _one_device(dev, layer)
    w_router = _need(layer["w_router"], torch.bfloat16, "w_router", dev)
    bias = layer.get("bias")
    if bias is not None:
        _need(bias, torch.float32, "bias", dev)
    if residual is not None:
        _need(residual, torch.bfloat16, "residual", dev)
    if out is None:
        out = torch.empty((M, w.H), dtype=torch.bfloat16, device=dev)
    if topk_ids is None:
        topk_ids = torch.empty((M, k), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty((M, k), dtype=torch.float32, device=dev)
    _need(out, torch.bfloat16, "out", dev)
    _need(topk_ids, torch.int32, "topk_ids", dev)
    _need(topk_weights, torch.float32, "topk_weights", dev)
    _check(lib().moe_decode_block_noalloc(_ptr(h), _ptr(w_router), _ptr(bias), ctypes.byref(w),
                                          M, k, b, _ptr(residual), _ptr(out), _ptr(topk_ids),
                                          _ptr(topk_weights), _stream(stream)),
           "moe_decode_block_noalloc")
    return out, topk_ids, topk_weights


def moe_decode_block_host(h_host, layer, k, b, h_dev, out_dev, out_host, topk_ids, topk_weights,
                          workspace, residual_host=None, residual_dev=None, stream=None):
    """Host in, host out: the library copies h to the device and the result back, and
    synchronises the stream before returning."""
    w = expert_weights(layer)
    bias = layer.get("bias")
    M = h_host.shape[0]
    _check(lib().moe_decode_block_host(_ptr(h_host), _ptr(residual_host), _ptr(out_host),
                                       _ptr(h_dev), _ptr(residual_dev), _ptr(out_dev),
                                       _ptr(layer["w_router"]), _ptr(bias), ctypes.byref(w), M, k,
                                       b, _ptr(topk_ids), _ptr(topk_weights), _ptr(workspace),
                                       workspace.numel(), _stream(stream)),
           "moe_decode_block_host")
    return out_host


def moe_read_device_status(workspace, stream=None) -> int:
    """Synchronises the stream, returns the device status bits and clears them."""
    out = ctypes.c_int32(0)
    rc = lib().moe_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(out))
    if rc not in (MOE_OK, MOE_ERR_DEVICE):
        raise MoeError(rc, "moe_read_device_status")
    return int(out.value)


def moe_selftest_wait_timeout(workspace, stream=None):
    """Enqueue the failure-detection self-test (include/moe.h): one CTA whose bounded wait
    runs out after about a second and sets MOE_DEV_WAIT_TIMEOUT in the workspace's status."""
    _check(lib().moe_selftest_wait_timeout(_ptr(workspace), workspace.numel(), _stream(stream)),
           "moe_selftest_wait_timeout")


def moe_set_trace_events(events=None):
    """Record the given six torch.cuda.Event objects around the block's kernels on every
    later call from this thread (see include/moe.h); ``None`` stops tracing."""
    if events is None:
        _check(lib().moe_set_trace_events(None, 0), "moe_set_trace_events")
        return
    events = list(events)
    for e in events:  # torch creates the CUDA event lazily, on first record
        if e.cuda_event == 0:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().moe_set_trace_events(arr, len(events)), "moe_set_trace_events")


# ------------------------------------------------------------------------------ CUDA graphs
def capture_graph(fn, stream: Optional[torch.cuda.Stream] = None) -> torch.cuda.CUDAGraph:
    """Capture ``fn(stream)`` -- one or more calls of the entry points above on ``stream`` --
    into a CUDA graph, after one eager run of it on the same stream.

    Decoding repeats the same block shapes step after step.  Replaying the captured
    launches (programmatic dependent launches included) skips the per-call host work:
    argument checks, marshalling, tensor-map encoding and one launch per kernel.  At small
    M that host work takes longer than the block's GPU time.  The graph keeps the raw
    pointers of the tensors ``fn`` used: a replay reads the inputs that are in those same
    tensors at that time and writes the same outputs.  Its workspace must not be shared
    with calls that run at the same time.
    """
    if stream is None:
        stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fn(stream)  # eager run: one-time kernel attributes are set outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        fn(stream)
    torch.cuda.current_stream().wait_stream(stream)
    return graph


# ------------------------------------------------------------------------ channel reader
def _reader_struct(rd: dict) -> ReaderStruct:
    s = ReaderStruct()
    s.H, s.I, s.E, s.rank = rd["H"], rd["I"], rd["E"], rd["rank"]
    for name in ("signs", "g_rows", "v_rows", "w_down", "g_codes", "v_codes", "g_scales",
                 "v_scales", "dnorm", "U", "coef"):
        setattr(s, name, rd[name].data_ptr())
    return s


def reader_build(layer: dict, signs: torch.Tensor, U: torch.Tensor, stream=None) -> dict:
    """Allocate and build the reader's data for a dense layer (see include/moe.h)."""
    E, H, I = layer["E"], layer["H"], layer["I"]
    rank = U.shape[1]
    dev = layer["w_down"].device
    nb = H // 128
    rd = {"H": H, "I": I, "E": E, "rank": rank, "signs": signs.contiguous(),
          "U": U.to(torch.float32).contiguous(), "w_down": layer["w_down"],
          "g_rows": torch.empty((E, I, H), dtype=torch.bfloat16, device=dev),
          "v_rows": torch.empty((E, I, H), dtype=torch.bfloat16, device=dev),
          "g_codes": torch.empty((E, I, nb, 8), dtype=torch.int32, device=dev),
          "v_codes": torch.empty((E, I, nb, 8), dtype=torch.int32, device=dev),
          "g_scales": torch.empty((E, I, nb), dtype=torch.float32, device=dev),
          "v_scales": torch.empty((E, I, nb), dtype=torch.float32, device=dev),
          "dnorm": torch.empty((E, I), dtype=torch.float32, device=dev),
          "coef": torch.empty((E, I, rank), dtype=torch.bfloat16, device=dev)}
    w = expert_weights(layer)
    s = _reader_struct(rd)
    _check(lib().moe_reader_build(ctypes.byref(w), ctypes.byref(s), _stream(stream)),
           "moe_reader_build")
    return rd


def reader_workspace(rd: dict, M: int, k: int, K: int, device=None) -> torch.Tensor:
    s = _reader_struct(rd)
    n = lib().moe_reader_workspace_bytes(ctypes.byref(s), M, k, K)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_reader_workspace_bytes")
    return torch.zeros((n,), dtype=torch.uint8, device=rd["w_down"].device if device is None else device)


def moe_reader_ffn(h, rd: dict, topk_ids, topk_weights, K: int, nscan: int = 80, residual=None,
                   out=None, workspace=None, want_decisions=False, stream=None):
    """The reader's decode (include/moe.h).  Returns out, or (out, selected [M,K] int32,
    xr [M,H] fp32) with ``want_decisions``."""
    _one_device(h.device, rd)
    M, k = topk_ids.shape
    if out is None:
        out = torch.empty_like(h)
    if workspace is None:
        workspace = reader_workspace(rd, M, k, K)
    sel = xr = None
    if want_decisions:
        sel = torch.empty((M, max(K, 1)), dtype=torch.int32, device=h.device)
        xr = torch.empty((M, rd["H"]), dtype=torch.float32, device=h.device)
    s = _reader_struct(rd)
    _check(lib().moe_reader_ffn(_ptr(h), ctypes.byref(s), M, k, _ptr(topk_ids), _ptr(topk_weights),
                                K, nscan, _ptr(residual), _ptr(out), _ptr(sel), _ptr(xr),
                                *_workspace(workspace, h.device), _stream(stream)),
           "moe_reader_ffn")
    if want_decisions:
        return out, sel[:, :K], xr
    return out


# ---------------------------------------------------------- tokens sorted by expert and back
# These calls are short (2 to 5 us of GPU time for a few tokens), so their argument checks
# test the usual case -- right type, shape and device, contiguous -- in one expression.
_ROW_DTYPES = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16, torch.float32: MOE_DT_F32}


def _launch_stream(stream, device):
    """Makes a given stream (an object or a handle) the current one.  The calls below run whole
    under it, so that the outputs and temporaries they allocate are that stream's: memory of
    another stream may still be in use there, and a temporary would be given away there while
    the launches use it."""
    _need_cuda(device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)  # 0 and 1 name the default stream
        stream = (torch.cuda.ExternalStream(handle, device) if handle > 1 else
                  torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


def _raw_stream(device):
    """Handle of the current stream.  The library launches on the current device, which has to be
    the tensors'."""
    index = device.index
    if index is None:
        _need_cuda(device)
    if index != _current_device():
        raise ValueError("tensors on %s, but the current device is cuda:%d" % (device, _current_device()))
    return _current_stream(index)


def _rows(t, name, device, dtype, shape):
    """Checks a matrix with contiguous columns (any row pitch); returns its pitch in elements."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return shape[1]
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    rows, cols = shape
    sr, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError("%s must have contiguous columns" % name)
    if rows > 1 and sr < cols:
        raise ValueError("%s must not have overlapping rows" % name)
    return sr if rows > 1 else cols


def _row_dtype(t, name):
    """MOE_DT_* of a matrix."""
    code = _ROW_DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be bfloat16, float16 or float32, got %s" % (name, t.dtype))
    if t.dim() != 2:
        _not_a_matrix(t, name)
    return code


def _vector(t, name, dtype, device, shape):
    """Checks a contiguous tensor; returns its address."""
    if not (t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()):
        _need(t, dtype, name, device)
        if tuple(t.shape) != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    return t.data_ptr()


def _not_a_matrix(t, name):
    raise ValueError("%s must be a matrix, got shape %s" % (name, tuple(t.shape)))


def _routes(t, device):
    """Checks route_row [M,k]; returns (address, M, k)."""
    if t.dim() != 2:
        _not_a_matrix(t, "route_row")
    M, k = t.shape
    return _vector(t, "route_row", torch.int32, device, (M, k)), M, k


def moe_token_plan(topk_ids, E, offsets=None, row_route=None, route_row=None, stream=None):
    """(offsets [E+1], row_route [M*k], route_row [M,k]) of topk_ids [M,k] (include/moe.h)."""
    if stream is not None:
        with _launch_stream(stream, topk_ids.device):
            return moe_token_plan(topk_ids, E, offsets, row_route, route_row)
    dev = topk_ids.device
    i32 = torch.int32
    if topk_ids.dim() != 2:
        _not_a_matrix(topk_ids, "topk_ids")
    M, k = topk_ids.shape
    ids = _vector(topk_ids, "topk_ids", i32, dev, (M, k))
    if offsets is None:
        offsets = torch.empty(E + 1, dtype=i32, device=dev)
    else:
        _vector(offsets, "offsets", i32, dev, (E + 1,))
    if row_route is None:
        row_route = torch.empty(M * k, dtype=i32, device=dev)
    else:
        _vector(row_route, "row_route", i32, dev, (M * k,))
    if route_row is None:
        route_row = torch.empty((M, k), dtype=i32, device=dev)
    else:
        _vector(route_row, "route_row", i32, dev, (M, k))
    rc = lib().moe_token_plan(ids, M, k, E, offsets.data_ptr(), row_route.data_ptr(),
                              route_row.data_ptr(), _raw_stream(dev))
    _check(rc, "moe_token_plan")
    return offsets, row_route, route_row


def moe_token_sort(x, route_row, rows=None, stream=None):
    """The token rows x [M,H] in sorted order: rows [M*k,H]."""
    if stream is not None:
        with _launch_stream(stream, x.device):
            return moe_token_sort(x, route_row, rows)
    dev, dt = x.device, x.dtype
    code = _row_dtype(x, "x")
    rr, M, k = _routes(route_row, dev)
    H = x.shape[1]
    ldx = _rows(x, "x", dev, dt, (M, H))
    if rows is None:
        rows, ldr = torch.empty((M * k, H), dtype=dt, device=dev), H
    else:
        ldr = _rows(rows, "rows", dev, dt, (M * k, H))
    _check(lib().moe_token_sort(x.data_ptr(), ldx, code, M, k, H, rr, rows.data_ptr(), ldr,
                                _raw_stream(dev)), "moe_token_sort")
    return rows


def moe_token_sort_grad(grad_rows, route_row, grad_x=None, stream=None):
    """Gradient of moe_token_sort: grad_x [M,H] of grad_rows [M*k,H]."""
    if stream is not None:
        with _launch_stream(stream, grad_rows.device):
            return moe_token_sort_grad(grad_rows, route_row, grad_x)
    dev, dt = grad_rows.device, grad_rows.dtype
    code = _row_dtype(grad_rows, "grad_rows")
    rr, M, k = _routes(route_row, dev)
    H = grad_rows.shape[1]
    ldr = _rows(grad_rows, "grad_rows", dev, dt, (M * k, H))
    if grad_x is None:
        grad_x, ldx = torch.empty((M, H), dtype=dt, device=dev), H
    else:
        ldx = _rows(grad_x, "grad_x", dev, dt, (M, H))
    _check(lib().moe_token_sort_grad(grad_rows.data_ptr(), ldr, code, M, k, H, rr,
                                     grad_x.data_ptr(), ldx, _raw_stream(dev)),
           "moe_token_sort_grad")
    return grad_x


def moe_token_unsort(rows, route_row, topk_weights=None, residual=None, out=None, stream=None):
    """out [M,H] = residual + the weighted sum of each token's rows (include/moe.h)."""
    if stream is not None:
        with _launch_stream(stream, rows.device):
            return moe_token_unsort(rows, route_row, topk_weights, residual, out)
    dev, dt = rows.device, rows.dtype
    code = _row_dtype(rows, "rows")
    rr, M, k = _routes(route_row, dev)
    H = rows.shape[1]
    ldr = _rows(rows, "rows", dev, dt, (M * k, H))
    w = res = None
    ldres = 0
    if topk_weights is not None:
        w = _vector(topk_weights, "topk_weights", torch.float32, dev, (M, k))
    if residual is not None:
        ldres = _rows(residual, "residual", dev, dt, (M, H))
        res = residual.data_ptr()
    if out is None:
        out, ldo = torch.empty((M, H), dtype=dt, device=dev), H
    else:
        ldo = _rows(out, "out", dev, dt, (M, H))
    _check(lib().moe_token_unsort(rows.data_ptr(), ldr, code, M, k, H, rr, w, res, ldres,
                                  out.data_ptr(), ldo, _raw_stream(dev)),
           "moe_token_unsort")
    return out


def moe_token_unsort_grad(grad_out, rows, route_row, topk_weights=None, grad_rows=None,
                          grad_weights=None, stream=None):
    """Gradients of moe_token_unsort: (grad_rows [M*k,H], grad_weights [M,k] fp32)."""
    if stream is not None:
        with _launch_stream(stream, rows.device):
            return moe_token_unsort_grad(grad_out, rows, route_row, topk_weights, grad_rows,
                                         grad_weights)
    dev, dt = rows.device, rows.dtype
    code = _row_dtype(rows, "rows")
    rr, M, k = _routes(route_row, dev)
    H = rows.shape[1]
    ldr = _rows(rows, "rows", dev, dt, (M * k, H))
    ldo = _rows(grad_out, "grad_out", dev, dt, (M, H))
    w = None
    if topk_weights is not None:
        w = _vector(topk_weights, "topk_weights", torch.float32, dev, (M, k))
    if grad_rows is None:
        grad_rows, ldg = torch.empty((M * k, H), dtype=dt, device=dev), H
    else:
        ldg = _rows(grad_rows, "grad_rows", dev, dt, (M * k, H))
    if grad_weights is None:
        grad_weights = torch.empty((M, k), dtype=torch.float32, device=dev)
    else:
        _vector(grad_weights, "grad_weights", torch.float32, dev, (M, k))
    _check(lib().moe_token_unsort_grad(grad_out.data_ptr(), ldo, rows.data_ptr(), ldr, code, M, k,
                                       H, rr, w, grad_rows.data_ptr(), ldg, grad_weights.data_ptr(),
                                       _raw_stream(dev)), "moe_token_unsort_grad")
    return grad_rows, grad_weights


# ------------------------------------------------------------- 4-bit block floating point
def moe_microscale_pitch(cols) -> int:
    return int(lib().moe_microscale_pitch(cols))


def _pitch(cols):
    return -(-cols // 512) * 16


def _microscaled(codes, scales, device, name):
    """Checks a pair of codes [..., cols/2] and scales [..., pitch]; returns cols."""
    u8 = torch.uint8
    cs = codes.shape
    cols = 2 * cs[-1]
    ss = cs[:-1] + (_pitch(cols),)
    if not (codes.dtype is u8 and scales.dtype is u8 and codes.device == device
            and scales.device == device and codes.is_contiguous() and scales.is_contiguous()
            and scales.shape == ss):
        _need(codes, u8, name + "_codes", device)
        _need(scales, u8, name + "_scales", device)
        raise ValueError("%s_scales must have shape %s, got %s" % (name, tuple(ss), tuple(scales.shape)))
    return cols


def _quantised_outputs(codes, scales, rows, cols, dev):
    """Codes and scales of a [rows, cols] result, allocated where the caller gave none."""
    if codes is None and scales is None:
        return (torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev),
                torch.empty((rows, _pitch(cols)), dtype=torch.uint8, device=dev))
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((rows, _pitch(cols)), dtype=torch.uint8, device=dev)
    if codes.shape != (rows, cols // 2):
        raise ValueError("codes must have shape %s, got %s" % ((rows, cols // 2), tuple(codes.shape)))
    _microscaled(codes, scales, dev, "out")
    return codes, scales


def moe_microscale_quantize(x, route_row=None, codes=None, scales=None, stream=None):
    """x [rows,cols] as 4-bit codes and scales; with route_row [rows,k] (a token plan's) in
    sorted order, rows * k of them."""
    if stream is not None:
        with _launch_stream(stream, x.device):
            return moe_microscale_quantize(x, route_row, codes, scales)
    dev = x.device
    code = _row_dtype(x, "x")
    rows, cols = x.shape
    ldx = _rows(x, "x", dev, x.dtype, (rows, cols))
    if cols % 32:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_microscale_quantize")
    rr, k = None, 1
    if route_row is not None:
        if route_row.dim() != 2:
            _not_a_matrix(route_row, "route_row")
        k = route_row.shape[1]
        rr = _vector(route_row, "route_row", torch.int32, dev, (rows, k))
    codes, scales = _quantised_outputs(codes, scales, rows * k, cols, dev)
    _check(lib().moe_microscale_quantize(x.data_ptr(), ldx, code, rows, cols, rr, k,
                                         codes.data_ptr(), scales.data_ptr(),
                                         _raw_stream(dev)), "moe_microscale_quantize")
    return codes, scales


def moe_microscale_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values [rows,cols] of codes [rows,cols/2] and scales."""
    if stream is not None:
        with _launch_stream(stream, codes.device):
            return moe_microscale_dequantize(codes, scales, dtype, out)
    dev = codes.device
    cols = _microscaled(codes, scales, dev, "x")
    if codes.dim() != 2:
        _not_a_matrix(codes, "codes")
    rows = codes.shape[0]
    if out is None:
        out, ldx = torch.empty((rows, cols), dtype=dtype, device=dev), cols
    else:
        ldx = _rows(out, "out", dev, out.dtype, (rows, cols))
    code = _row_dtype(out, "out")
    _check(lib().moe_microscale_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols,
                                           out.data_ptr(), ldx, code, _raw_stream(dev)),
           "moe_microscale_dequantize")
    return out


def _own_status(workspace, where):
    """After a call that made its own workspace, whose status word has no other reader: waits for
    the result and raises if a device wait ran out.  (A call that a graph captures cannot wait.)"""
    if not torch.cuda.is_current_stream_capturing():
        status = ctypes.c_int32(0)
        _check(lib().moe_read_device_status(workspace.data_ptr(), _raw_stream(workspace.device),
                                            ctypes.byref(status)), where)


def _product_args(x_codes, x_scales, w_codes, w_scales, offsets, workspace):
    """Checks of the grouped products; returns (rows, E, N, K, offsets' address, the workspace
    made here or None, (the workspace's address, its bytes))."""
    dev = x_codes.device
    if x_codes.dim() != 2:
        _not_a_matrix(x_codes, "x_codes")
    K = _microscaled(x_codes, x_scales, dev, "x")
    if _microscaled(w_codes, w_scales, dev, "w") != K:
        raise ValueError("x and w must have the same number of columns")
    ws = w_codes.shape
    if len(ws) != 2 and len(ws) != 3:
        raise ValueError("w_codes must have shape [N,K/2] or [E,N,K/2], got %s" % (tuple(ws),))
    E, N = (1, ws[0]) if len(ws) == 2 else (ws[0], ws[1])
    off = None
    if offsets is not None:
        off = _vector(offsets, "offsets", torch.int32, dev, (E + 1,))
    own = None
    if workspace is None:
        workspace = own = torch.zeros(MOE_MICROSCALE_STATUS_BYTES, dtype=torch.uint8, device=dev)
    return x_codes.shape[0], E, N, K, off, own, _workspace(workspace, dev)


def moe_microscale_product(x_codes, x_scales, w_codes, w_scales, offsets=None,
                           dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """y [rows,N] of 4-bit rows and 4-bit weights [E,N,K] (or [N,K]), rows grouped by offsets
    [E+1]; rows past the last group are zero.  The workspace holds the status word; without one
    the call makes its own, waits for the result and raises what the device found."""
    if stream is not None:
        with _launch_stream(stream, x_codes.device):
            return moe_microscale_product(x_codes, x_scales, w_codes, w_scales, offsets, dtype,
                                          out, workspace)
    rows, E, N, K, off, own, ws = _product_args(x_codes, x_scales, w_codes, w_scales, offsets,
                                                workspace)
    dev = x_codes.device
    if out is None:
        out, ldy = torch.empty((rows, N), dtype=dtype, device=dev), N
    else:
        ldy = _rows(out, "out", dev, out.dtype, (rows, N))
    code = _row_dtype(out, "out")
    _check(lib().moe_microscale_product(x_codes.data_ptr(), x_scales.data_ptr(), rows, off,
                                        w_codes.data_ptr(), w_scales.data_ptr(), E, N, K, code,
                                        out.data_ptr(), ldy, *ws, _raw_stream(dev)),
           "moe_microscale_product")
    if own is not None:
        _own_status(own, "moe_microscale_product")
    return out


def moe_microscale_gated_product(x_codes, x_scales, w_codes, w_scales, offsets=None, codes=None,
                                 scales=None, workspace=None, stream=None):
    """SiLU(g) * u of the gate and up halves of w [E,N,K], quantised: (codes, scales) of
    [rows,N/2].  Workspace as for moe_microscale_product."""
    if stream is not None:
        with _launch_stream(stream, x_codes.device):
            return moe_microscale_gated_product(x_codes, x_scales, w_codes, w_scales, offsets,
                                                codes, scales, workspace)
    rows, E, N, K, off, own, ws = _product_args(x_codes, x_scales, w_codes, w_scales, offsets,
                                                workspace)
    if N % 64:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_microscale_gated_product")
    dev = x_codes.device
    codes, scales = _quantised_outputs(codes, scales, rows, N // 2, dev)
    _check(lib().moe_microscale_gated_product(x_codes.data_ptr(), x_scales.data_ptr(), rows, off,
                                              w_codes.data_ptr(), w_scales.data_ptr(), E, N, K,
                                              codes.data_ptr(), scales.data_ptr(), *ws,
                                              _raw_stream(dev)),
           "moe_microscale_gated_product")
    if own is not None:
        _own_status(own, "moe_microscale_gated_product")
    return codes, scales


def microscale_weights(layer: dict, device=None) -> MicroscaleWeights:
    """C descriptor of a layer's 4-bit weights: H, I, E and gate_up_codes [E,2I,H/2],
    gate_up_scales, down_codes [E,H,I/2], down_scales (the caller keeps the tensors alive), all
    on one device, `device` if given; y_dtype, torch.bfloat16 if it has none, is the type of the
    down product's results before their sum (torch.float32 keeps them unrounded)."""
    H, I, E = layer["H"], layer["I"], layer["E"]
    gc, gs, dc, ds = (layer["gate_up_codes"], layer["gate_up_scales"], layer["down_codes"],
                      layer["down_scales"])
    dev = dc.device if device is None else device
    if gc.shape != (E, 2 * I, H // 2) or _microscaled(gc, gs, dev, "gate_up") != H:
        raise ValueError("gate_up_codes must have shape %s" % ((E, 2 * I, H // 2),))
    if dc.shape != (E, H, I // 2) or _microscaled(dc, ds, dev, "down") != I:
        raise ValueError("down_codes must have shape %s" % ((E, H, I // 2),))
    y = layer.get("y_dtype", torch.bfloat16)
    if y is not torch.bfloat16 and y is not torch.float32:
        raise TypeError("y_dtype must be bfloat16 or float32, got %s" % (y,))
    return MicroscaleWeights(H, I, E, _ROW_DTYPES[y], gc.data_ptr(), gs.data_ptr(), dc.data_ptr(),
                             ds.data_ptr())


def microscale_layer(layer: dict, stream=None, y_dtype=torch.bfloat16) -> dict:
    """4-bit weights of a dense layer (w_gate, w_up [E,H,I], w_down [E,I,H] bf16): each
    projection's output channels become rows, quantised along the summed dimension.  y_dtype as
    microscale_weights takes it."""
    if stream is not None:
        with _launch_stream(stream, layer["w_down"].device):
            return microscale_layer(layer, y_dtype=y_dtype)
    H, I, E = layer["H"], layer["I"], layer["E"]
    dev = layer["w_down"].device
    if H % 32 or I % 32:
        raise MoeError(MOE_ERR_UNSUPPORTED, "microscale_layer")
    out = {"H": H, "I": I, "E": E, "y_dtype": y_dtype}
    for name, n, cols in (("gate_up", 2 * I, H), ("down", H, I)):
        out[name + "_codes"] = torch.empty((E, n, cols // 2), dtype=torch.uint8, device=dev)
        out[name + "_scales"] = torch.empty((E, n, _pitch(cols)), dtype=torch.uint8, device=dev)
    for e in range(E):
        for name, w, at in (("gate_up", layer["w_gate"][e], 0), ("gate_up", layer["w_up"][e], I),
                            ("down", layer["w_down"][e], 0)):
            rows = w.t().contiguous()
            moe_microscale_quantize(rows, codes=out[name + "_codes"][e, at:at + len(rows)],
                                    scales=out[name + "_scales"][e, at:at + len(rows)])
    return out


def moe_microscale_workspace_bytes(layer: dict, M, k) -> int:
    return int(lib().moe_microscale_workspace_bytes(ctypes.byref(microscale_weights(layer)), M, k))


def microscale_workspace(layer: dict, M, k) -> torch.Tensor:
    """A workspace of moe_microscale_ffn, its status word zero."""
    n = moe_microscale_workspace_bytes(layer, M, k)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_microscale_workspace_bytes")
    work = torch.empty((n,), dtype=torch.uint8, device=layer["down_codes"].device)
    work[:MOE_MICROSCALE_STATUS_BYTES].zero_()
    return work


def moe_microscale_ffn(h, layer, topk_ids, topk_weights, residual=None, out=None, workspace=None,
                       stream=None):
    """The 4-bit expert step (include/moe.h) for given routes; `layer` as microscale_weights
    takes it.  Without a workspace (microscale_workspace) the call makes its own, waits for the
    result and raises what the device found."""
    if stream is not None:
        with _launch_stream(stream, h.device):
            return moe_microscale_ffn(h, layer, topk_ids, topk_weights, residual, out, workspace)
    dev = h.device
    w = microscale_weights(layer, dev)
    if topk_ids.dim() != 2:
        _not_a_matrix(topk_ids, "topk_ids")
    M, k = topk_ids.shape
    H = w.H
    bf16 = torch.bfloat16
    ph = _vector(h, "h", bf16, dev, (M, H))
    ids = _vector(topk_ids, "topk_ids", torch.int32, dev, (M, k))
    pw = _vector(topk_weights, "topk_weights", torch.float32, dev, (M, k))
    res = None if residual is None else _vector(residual, "residual", bf16, dev, (M, H))
    if out is None:
        out = torch.empty((M, H), dtype=bf16, device=dev)
    else:
        _vector(out, "out", bf16, dev, (M, H))
    own = workspace is None
    if own:
        workspace = microscale_workspace(layer, M, k)
    _check(lib().moe_microscale_ffn(ph, ctypes.byref(w), M, k, ids, pw, res, out.data_ptr(),
                                    *_workspace(workspace, dev), _raw_stream(dev)),
           "moe_microscale_ffn")
    if own:
        _own_status(workspace, "moe_microscale_ffn")
    return out
