"""ctypes binding of the experts' block (include/moe_experts.h).

Argument marshalling as in _lib, and what the library cannot see in a
pointer: the sizes (of weights, of what forward saved) are compared with the
tensors given, since a short one would be read or written past its end, and
the kernels run on the stream's device (the current one's where no stream is
given), so every tensor must lie there.  A tensor that is not contiguous, of
another element size or shape, of a floating type other than bfloat16, in host
memory or on another device is refused with E_INVALID_ARG like the library's
own refusals.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import Dims, E_INVALID_ARG, MoeShuffleError, Plan, _check, _cur_device, _stream

ACT_SILU, ACT_GELU_TANH = 0, 1
GROUP8 = 32  # MOE_EXPERTS_GROUP8

# Every function moe_experts.h declares.
EXPERTS_EXPORTS = ("moe_experts_ffn_workspace_size", "moe_experts_ffn_forward", "moe_experts_ffn_backward",
                   "moe_experts_ffn_w4_forward", "moe_experts_w4_quantize", "moe_experts_pack8",
                   "moe_experts_unpack8")

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_SIGNATURES = {
    "moe_experts_ffn_workspace_size": [ctypes.POINTER(Dims), _i32, _i32, ctypes.POINTER(_sz)],
    "moe_experts_ffn_forward": [_vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_experts_ffn_backward": [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_experts_ffn_w4_forward": [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _sz, _vp],
    "moe_experts_w4_quantize": [_vp, _i64, _i32, _i32, _vp, _vp, _vp],
    "moe_experts_pack8": [_vp, _i64, _i32, _vp, _vp, _vp],
    "moe_experts_unpack8": [_vp, _vp, _i64, _i32, _vp, _vp],
}

_ready = None


def _load():
    global _ready
    if _ready is None:
        lib = _lib.load()
        for name, args in _SIGNATURES.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = ctypes.c_int, args
        _ready = lib
    return _ready


def _refuse(func: str, what: str):
    raise MoeShuffleError(func, E_INVALID_ARG, f"invalid argument: {what}")


def _at(func: str, name: str, t, shape, width: int):
    """The address of a contiguous tensor of this shape and element size (None stays None).  Any type of that size
    stands for its bits (int16 for bf16, uint8 for int8), but another floating type means other values."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape) or t.element_size() != width or not t.is_contiguous():
        _refuse(func, f"{name} must be contiguous {list(shape)} of {width}-byte elements, "
                      f"not {list(t.shape)} of {t.element_size()}")
    if t.is_floating_point() and t.dtype != torch.bfloat16:
        _refuse(func, f"{name} must not be {t.dtype}")
    return t.data_ptr()


def _on_gpu(func: str, stream, **tensors):
    """Every tensor given lies on the device that the kernels run on."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            _refuse(func, f"{name} must be on the GPU, not on {t.device}")
    device = getattr(stream, "device_index", None)
    if device is None:
        device = _cur_device() if _cur_device is not None else torch.cuda.current_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != device:
            _refuse(func, f"{name} must be on GPU {device}, not on {t.device}")


def _block(func: str, plan: Plan, w, half: int, name: str):
    """(rows, H, E, width between the projections) from the plan and the down projection's last axis."""
    if plan.handle is None:
        _refuse(func, "the plan was destroyed")
    if w is None or w.dim() != 3:
        _refuse(func, f"{name} must have three axes")
    d = plan.dims
    return d.num_tokens * d.top_k, d.hidden, d.num_experts, w.shape[2] * half


def _workspace(func: str, w):
    if w is None or not w.is_contiguous():
        _refuse(func, "workspace must be contiguous")
    return w.data_ptr(), w.numel() * w.element_size()


def _saved(func: str, saved, scale, rows: int, inter: int):
    if scale is not None and saved is None:
        _refuse(func, "saved_scale without saved")
    return (_at(func, "saved", saved, (rows, 2 * inter), 2 if scale is None else 1),
            _at(func, "saved_scale", scale, (rows, 2, -(-inter // GROUP8)), 2))


def moe_experts_ffn_workspace_size(dims: Dims, inter: int, backward: bool = False) -> int:
    n = _sz(0)
    _check("moe_experts_ffn_workspace_size",
           _load().moe_experts_ffn_workspace_size(ctypes.byref(dims), int(inter), int(bool(backward)),
                                                  ctypes.byref(n)))
    return n.value


def moe_experts_ffn_forward(plan: Plan, xe, w_gate_up, w_down, ye, workspace, saved=None, saved_scale=None,
                            act: int = ACT_SILU, stream=None):
    """ye = the gated block of each expert on its rows of xe.  `saved` (bf16, or int8 with `saved_scale`) receives
    the pre-activations that moe_experts_ffn_backward needs."""
    f = "moe_experts_ffn_forward"
    P, H, E, inter = _block(f, plan, w_down, 1, "w_down")
    ws, ws_bytes = _workspace(f, workspace)
    held, scale = _saved(f, saved, saved_scale, P, inter)
    args = (_at(f, "xe", xe, (P, H), 2), _at(f, "w_gate_up", w_gate_up, (E, 2 * inter, H), 2),
            _at(f, "w_down", w_down, (E, H, inter), 2), inter, int(act), _at(f, "ye", ye, (P, H), 2), held, scale, ws,
            ws_bytes)
    _on_gpu(f, stream, xe=xe, w_gate_up=w_gate_up, w_down=w_down, ye=ye, saved=saved, saved_scale=saved_scale,
            workspace=workspace, plan=plan.workspace)
    _check(f, _load().moe_experts_ffn_forward(plan.handle, *args, _stream(stream)))


def moe_experts_ffn_backward(plan: Plan, grad_ye, xe, w_gate_up, w_down, saved, grad_xe, grad_w_gate_up,
                             grad_w_down, workspace, saved_scale=None, act: int = ACT_SILU, stream=None):
    """The gradients of the block; each of grad_xe, grad_w_gate_up and grad_w_down may be None."""
    f = "moe_experts_ffn_backward"
    P, H, E, inter = _block(f, plan, w_down, 1, "w_down")
    ws, ws_bytes = _workspace(f, workspace)
    held, scale = _saved(f, saved, saved_scale, P, inter)
    up, down = (E, 2 * inter, H), (E, H, inter)
    args = (_at(f, "grad_ye", grad_ye, (P, H), 2), _at(f, "xe", xe, (P, H), 2), _at(f, "w_gate_up", w_gate_up, up, 2),
            _at(f, "w_down", w_down, down, 2), inter, int(act), held, scale, _at(f, "grad_xe", grad_xe, (P, H), 2),
            _at(f, "grad_w_gate_up", grad_w_gate_up, up, 2), _at(f, "grad_w_down", grad_w_down, down, 2), ws, ws_bytes)
    _on_gpu(f, stream, grad_ye=grad_ye, xe=xe, w_gate_up=w_gate_up, w_down=w_down, saved=saved,
            saved_scale=saved_scale, grad_xe=grad_xe, grad_w_gate_up=grad_w_gate_up, grad_w_down=grad_w_down,
            workspace=workspace, plan=plan.workspace)
    _check(f, _load().moe_experts_ffn_backward(plan.handle, *args, _stream(stream)))


def moe_experts_ffn_w4_forward(plan: Plan, xe, q_gate_up, s_gate_up, q_down, s_down, ye, workspace, group: int = 128,
                               act: int = ACT_SILU, stream=None):
    """The gated block with 4-bit weights (two a byte) and a bf16 scale for every `group` columns."""
    f = "moe_experts_ffn_w4_forward"
    P, H, E, inter = _block(f, plan, q_down, 2, "q_down")
    if group <= 0:
        _refuse(f, "group must be 32, 64 or 128")
    ws, ws_bytes = _workspace(f, workspace)
    args = (_at(f, "xe", xe, (P, H), 2), _at(f, "q_gate_up", q_gate_up, (E, 2 * inter, H // 2), 1),
            _at(f, "s_gate_up", s_gate_up, (E, 2 * inter, H // group), 2),
            _at(f, "q_down", q_down, (E, H, inter // 2), 1), _at(f, "s_down", s_down, (E, H, inter // group), 2), inter,
            int(group), int(act), _at(f, "ye", ye, (P, H), 2), ws, ws_bytes)
    _on_gpu(f, stream, xe=xe, q_gate_up=q_gate_up, s_gate_up=s_gate_up, q_down=q_down, s_down=s_down, ye=ye,
            workspace=workspace, plan=plan.workspace)
    _check(f, _load().moe_experts_ffn_w4_forward(plan.handle, *args, _stream(stream)))


def moe_experts_w4_quantize(w, q, scale, group: int = 128, stream=None):
    """4-bit values and scales of bf16 weights, along the last axis."""
    f = "moe_experts_w4_quantize"
    if group <= 0:
        _refuse(f, "group must be 32, 64 or 128")
    lead, cols = tuple(w.shape[:-1]), w.shape[-1]
    args = (_at(f, "w", w, w.shape, 2), w.numel() // max(cols, 1), cols, int(group),
            _at(f, "q", q, lead + (cols // 2,), 1), _at(f, "scale", scale, lead + (cols // group,), 2))
    _on_gpu(f, stream, w=w, q=q, scale=scale)
    _check(f, _load().moe_experts_w4_quantize(*args, _stream(stream)))


def moe_experts_pack8(x, q, scale, stream=None):
    """Rows of x (bf16) to int8 with a bf16 scale for every 32 elements along the last axis."""
    f = "moe_experts_pack8"
    lead, cols = tuple(x.shape[:-1]), x.shape[-1]
    args = (_at(f, "x", x, x.shape, 2), x.numel() // max(cols, 1), cols, _at(f, "q", q, x.shape, 1),
            _at(f, "scale", scale, lead + (-(-cols // GROUP8),), 2))
    _on_gpu(f, stream, x=x, q=q, scale=scale)
    _check(f, _load().moe_experts_pack8(*args, _stream(stream)))


def moe_experts_unpack8(q, scale, x, stream=None):
    """The bf16 values that packed rows hold."""
    f = "moe_experts_unpack8"
    lead, cols = tuple(x.shape[:-1]), x.shape[-1]
    args = (_at(f, "q", q, x.shape, 1), _at(f, "scale", scale, lead + (-(-cols // GROUP8),), 2),
            x.numel() // max(cols, 1), cols, _at(f, "x", x, x.shape, 2))
    _on_gpu(f, stream, q=q, scale=scale, x=x)
    _check(f, _load().moe_experts_unpack8(*args, _stream(stream)))
