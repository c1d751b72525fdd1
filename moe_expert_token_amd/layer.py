"""ctypes binding of the router and of the layer for few tokens
(include/moe_layer.h).  Tensors are checked as those of the experts' block are:
shape, element size, contiguous, on the device that the kernels run on.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import Dims, _check, _stream
from .experts import ACT_SILU, _at, _on_gpu, _refuse, _workspace

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
LAYER_MAX_TOKENS, LAYER_MAX_PAIRS = 64, 512

# Every function moe_layer.h declares.
LAYER_EXPORTS = ("moe_router_workspace_size", "moe_router_forward", "moe_router_backward", "moe_layer_workspace_size",
                 "moe_layer_forward", "moe_layer_w4_forward")

_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t


class _Rule(ctypes.Structure):
    _fields_ = [("scoring", _i32), ("normalize", _i32), ("scale", ctypes.c_float), ("reserved", _i32), ("bias", _vp)]


_SIGNATURES = {
    "moe_router_workspace_size": [ctypes.POINTER(Dims), _i32, ctypes.POINTER(_sz)],
    "moe_router_forward": [ctypes.POINTER(Dims), ctypes.POINTER(_Rule), _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "moe_router_backward": [ctypes.POINTER(Dims), ctypes.POINTER(_Rule)] + [_vp] * 10 + [_sz, _vp],
    "moe_layer_workspace_size": [ctypes.POINTER(Dims), _i32, ctypes.POINTER(_sz)],
    "moe_layer_forward": [ctypes.POINTER(Dims), ctypes.POINTER(_Rule), _vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp,
                          _vp, _vp, _sz, _vp],
    "moe_layer_w4_forward": [ctypes.POINTER(Dims), ctypes.POINTER(_Rule), _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                             _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
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


class RouterRule:
    """How logits become gates: the scores, whether the chosen ones are normalized, their scale, and (sigmoid scores
    only) a bias fp32 [E] that the choice goes by and the gates do not.  `bias` may be written to or set to another
    tensor between calls: each call takes the one that is there."""

    def __init__(self, scoring: int = SCORE_SOFTMAX, normalize: bool = True, scale: float = 1.0, bias=None):
        if bias is not None and (bias.dtype != torch.float32 or bias.dim() != 1):
            _refuse("RouterRule", "bias must be float32 [E]")
        self.bias = bias
        self._fixed = int(scoring), int(bool(normalize)), float(scale), 0

    @property
    def struct(self):
        return _Rule(*self._fixed, None if self.bias is None else self.bias.data_ptr())


def _f32(func: str, name: str, t, shape):
    if t is not None and t.dtype != torch.float32:
        _refuse(func, f"{name} must be float32, not {t.dtype}")
    if t is not None and (tuple(t.shape) != shape or not t.is_contiguous()):
        _refuse(func, f"{name} must be contiguous {list(shape)}, not {list(t.shape)}")
    return None if t is None else t.data_ptr()


def _ids(func: str, t, shape):
    if t is not None and t.dtype != torch.int32:
        _refuse(func, f"topk_idx must be int32, not {t.dtype}")
    if t is not None and (tuple(t.shape) != shape or not t.is_contiguous()):
        _refuse(func, f"topk_idx must be contiguous {list(shape)}, not {list(t.shape)}")
    return None if t is None else t.data_ptr()


def _bias(func: str, rule: RouterRule, E: int):
    b = rule.bias
    if b is not None and (b.dtype != torch.float32 or tuple(b.shape) != (E,) or not b.is_contiguous()):
        _refuse(func, f"the rule's bias must be contiguous float32 [{E}], not {list(b.shape)} of {b.dtype}")


def moe_router_workspace_size(dims: Dims, backward: bool = False) -> int:
    n = _sz(0)
    _check("moe_router_workspace_size",
           _load().moe_router_workspace_size(ctypes.byref(dims), int(bool(backward)), ctypes.byref(n)))
    return n.value


def moe_router_forward(dims: Dims, rule: RouterRule, x, w_router, topk_idx, topk_w, workspace, logits=None, stream=None):
    """Ids and gates of the rows x by the rule; `logits` (fp32 [T, E]) receives what moe_router_backward needs."""
    f = "moe_router_forward"
    T, H, E, k = dims.num_tokens, dims.hidden, dims.num_experts, dims.top_k
    _bias(f, rule, E)
    ws, ws_bytes = _workspace(f, workspace)
    args = (_at(f, "x", x, (T, H), 2), _at(f, "w_router", w_router, (E, H), 2), _ids(f, topk_idx, (T, k)),
            _f32(f, "topk_w", topk_w, (T, k)), _f32(f, "logits", logits, (T, E)))
    _on_gpu(f, stream, x=x, w_router=w_router, topk_idx=topk_idx, topk_w=topk_w, logits=logits, workspace=workspace,
            bias=rule.bias)
    _check(f, _load().moe_router_forward(ctypes.byref(dims), ctypes.byref(rule.struct), *args, ws, ws_bytes,
                                         _stream(stream)))


def moe_router_backward(dims: Dims, rule: RouterRule, grad_topk_w, logits, topk_idx, x, w_router, grad_x,
                        grad_w_router, workspace, grad_x_in=None, grad_logits=None, stream=None):
    """Gradients of rows and router's weights from the gates' (and, with grad_logits, the logits' own); grad_x_in, which
    may be grad_x, is added to grad_x.  Each of grad_x and grad_w_router may be None."""
    f = "moe_router_backward"
    T, H, E, k = dims.num_tokens, dims.hidden, dims.num_experts, dims.top_k
    ws, ws_bytes = _workspace(f, workspace)
    args = (_f32(f, "grad_topk_w", grad_topk_w, (T, k)), _f32(f, "logits", logits, (T, E)), _ids(f, topk_idx, (T, k)),
            _at(f, "x", x, (T, H), 2), _at(f, "w_router", w_router, (E, H), 2),
            _f32(f, "grad_logits", grad_logits, (T, E)), _at(f, "grad_x_in", grad_x_in, (T, H), 2),
            _at(f, "grad_x", grad_x, (T, H), 2), _at(f, "grad_w_router", grad_w_router, (E, H), 2))
    _on_gpu(f, stream, grad_topk_w=grad_topk_w, logits=logits, topk_idx=topk_idx, x=x, w_router=w_router,
            grad_logits=grad_logits, grad_x_in=grad_x_in, grad_x=grad_x, grad_w_router=grad_w_router,
            workspace=workspace)
    _check(f, _load().moe_router_backward(ctypes.byref(dims), ctypes.byref(rule.struct), *args, ws, ws_bytes,
                                          _stream(stream)))


def moe_layer_workspace_size(dims: Dims, inter: int) -> int:
    n = _sz(0)
    _check("moe_layer_workspace_size",
           _load().moe_layer_workspace_size(ctypes.byref(dims), int(inter), ctypes.byref(n)))
    return n.value


def _rows(f, dims, rule, x, w_router, residual, out, topk_idx, topk_w):
    T, H, E, k = dims.num_tokens, dims.hidden, dims.num_experts, dims.top_k
    _bias(f, rule, E)
    return (_at(f, "x", x, (T, H), 2), _at(f, "w_router", w_router, (E, H), 2),
            _at(f, "residual", residual, (T, H), 2), _at(f, "out", out, (T, H), 2), _ids(f, topk_idx, (T, k)),
            _f32(f, "topk_w", topk_w, (T, k)))


def moe_layer_forward(dims: Dims, rule: RouterRule, x, w_router, w_gate_up, w_down, out, workspace, residual=None,
                      topk_idx=None, topk_w=None, act: int = ACT_SILU, stream=None):
    """out = residual + the layer of the rows x: router, experts (bf16 weights) and combine, for at most 64 tokens."""
    f = "moe_layer_forward"
    if w_down is None or w_down.dim() != 3:
        _refuse(f, "w_down must have three axes")
    H, E, inter = dims.hidden, dims.num_experts, w_down.shape[2]
    ws, ws_bytes = _workspace(f, workspace)
    px, pr, pres, pout, pidx, pw = _rows(f, dims, rule, x, w_router, residual, out, topk_idx, topk_w)
    up, down = _at(f, "w_gate_up", w_gate_up, (E, 2 * inter, H), 2), _at(f, "w_down", w_down, (E, H, inter), 2)
    _on_gpu(f, stream, x=x, w_router=w_router, w_gate_up=w_gate_up, w_down=w_down, residual=residual, out=out,
            topk_idx=topk_idx, topk_w=topk_w, workspace=workspace, bias=rule.bias)
    _check(f, _load().moe_layer_forward(ctypes.byref(dims), ctypes.byref(rule.struct), px, pr, up, down, inter, int(act),
                                        pres, pout, pidx, pw, ws, ws_bytes, _stream(stream)))


def moe_layer_w4_forward(dims: Dims, rule: RouterRule, x, w_router, q_gate_up, s_gate_up, q_down, s_down, out,
                         workspace, group: int = 128, residual=None, topk_idx=None, topk_w=None, act: int = ACT_SILU,
                         stream=None):
    """The layer with 4-bit experts (two values a byte, a bf16 scale for every `group` columns)."""
    f = "moe_layer_w4_forward"
    if q_down is None or q_down.dim() != 3:
        _refuse(f, "q_down must have three axes")
    if group <= 0:
        _refuse(f, "group must be 32, 64 or 128")
    H, E, inter = dims.hidden, dims.num_experts, q_down.shape[2] * 2
    ws, ws_bytes = _workspace(f, workspace)
    px, pr, pres, pout, pidx, pw = _rows(f, dims, rule, x, w_router, residual, out, topk_idx, topk_w)
    args = (_at(f, "q_gate_up", q_gate_up, (E, 2 * inter, H // 2), 1),
            _at(f, "s_gate_up", s_gate_up, (E, 2 * inter, H // group), 2),
            _at(f, "q_down", q_down, (E, H, inter // 2), 1), _at(f, "s_down", s_down, (E, H, inter // group), 2))
    _on_gpu(f, stream, x=x, w_router=w_router, q_gate_up=q_gate_up, s_gate_up=s_gate_up, q_down=q_down, s_down=s_down,
            residual=residual, out=out, topk_idx=topk_idx, topk_w=topk_w, workspace=workspace, bias=rule.bias)
    _check(f, _load().moe_layer_w4_forward(ctypes.byref(dims), ctypes.byref(rule.struct), px, pr, *args, inter,
                                           int(group), int(act), pres, pout, pidx, pw, ws, ws_bytes, _stream(stream)))
