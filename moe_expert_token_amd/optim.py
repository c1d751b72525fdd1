"""ctypes binding of the optimizer's step (include/moe_optim.h).

A list of tensors is checked once, when AdamwTensors is made of it, and kept by
the caller from step to step: types, sizes, one device, and that no output
overlaps anything else of the list.  The calls then only pass it on.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import E_INVALID_ARG, MoeShuffleError, _check, _cur_device, _stream

GROUP_STATE = 128  # MOE_ADAMW_GROUP

# Every function moe_optim.h declares.
OPTIM_EXPORTS = ("moe_adamw_step", "moe_adamw_pack", "moe_adamw_unpack")

_F32, _BF16, _8BIT = 0, 1, 2
_vp, _i32, _i64, _f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class _Tensor(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("p", "copy", "g", "m", "v", "m_scale", "v_scale", "m_out", "v_out")] + [("n", _i64)]


class _Params(ctypes.Structure):
    _fields_ = [("param", _i32), ("grad", _i32), ("state", _i32), ("reserved", _i32), ("lr", _f64), ("beta1", _f64),
                ("beta2", _f64), ("eps", _f64), ("weight_decay", _f64), ("step", _i64), ("lr_device", _vp),
                ("step_device", _vp), ("grad_scale", _vp)]


_ready = None


def _load():
    global _ready
    if _ready is None:
        lib = _lib.load()
        signatures = {
            "moe_adamw_step": [_vp, _i32, ctypes.POINTER(_Params), _vp],
            "moe_adamw_pack": [_vp, _i32, _vp],
            "moe_adamw_unpack": [_vp, _i32, _i32, _vp],
        }
        for name, args in signatures.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = ctypes.c_int, args
        _ready = lib
    return _ready


def _refuse(func: str, what: str):
    raise MoeShuffleError(func, E_INVALID_ARG, f"invalid argument: {what}")


_KINDS = {
    "p": {torch.float32: _F32, torch.bfloat16: _BF16},
    "copy": {torch.bfloat16: _BF16},
    "g": {torch.float32: _F32, torch.bfloat16: _BF16},
    "m": {torch.float32: _F32, torch.uint8: _8BIT, torch.float8_e4m3fn: _8BIT},
    "v": {torch.float32: _F32, torch.uint8: _8BIT},
    "m_scale": {torch.float32: _F32},
    "v_scale": {torch.float32: _F32},
    "m_out": {torch.float32: _F32, torch.bfloat16: _BF16},
    "v_out": {torch.float32: _F32, torch.bfloat16: _BF16},
}


class AdamwTensors:
    """The tensors of a step, a dict each:

      p        fp32 or bf16 parameters;  copy  bf16, with fp32 parameters only (may be left out)
      g        fp32 or bf16 gradients
      m, v     fp32 states, or 8-bit ones (uint8; m may be float8_e4m3fn) with m_scale, v_scale
               (fp32, one for every 128 elements)
      m_out, v_out  values of 8-bit states, for moe_adamw_pack and moe_adamw_unpack

    Shapes are free: a tensor is its elements in memory order, and they must be contiguous.  All tensors of a kind
    have one type.  The list holds its tensors; a program keeps it as long as their memory stays the same.  Making it
    takes the host 6 to 10 us a tensor, which a program whose gradients are new tensors in each step pays each time.
    """

    def __init__(self, tensors):
        self.tensors = [dict(t) for t in tensors]
        self.kinds = {}
        self.device = None
        self.array = (_Tensor * max(1, len(self.tensors)))()
        spans = []
        for i, t in enumerate(self.tensors):
            self._add(i, t, spans)
        # in memory order: nothing may begin before the end of an output, nor an output before the end of anything
        spans.sort(key=lambda s: s[0])
        ends = {True: (-1, ""), False: (-1, "")}  # the furthest end so far, of outputs and of inputs
        for lo, hi, out, at in spans:
            for kind in (True, False) if out else (True,):
                if lo < ends[kind][0]:
                    _refuse("AdamwTensors", f"{at} overlaps {ends[kind][1]}")
            if hi > ends[out][0]:
                ends[out] = (hi, at)
        self.count = len(self.tensors)
        # names that every tensor with an element has
        self.full = {name for name in _KINDS if all(t.get(name) is not None for t, entry
                                                    in zip(self.tensors, self.array) if entry.n)}

    def _add(self, i, t, spans):
        who = "AdamwTensors"
        n = None
        for name, value in t.items():
            if value is None:
                continue
            at = f"{name} of tensor {i}"
            if name not in _KINDS:
                _refuse(who, f"{at}: no such tensor")
            if not value.is_cuda:
                _refuse(who, f"{at} must be on the GPU, not on {value.device}")
            kind = _KINDS[name].get(value.dtype)
            if kind is None:
                _refuse(who, f"{at} must not be {value.dtype}")
            if self.kinds.setdefault(name, kind) != kind:
                _refuse(who, f"{at} has another type than those before")
            if self.device is None:
                self.device = value.get_device()
            if value.get_device() != self.device:
                _refuse(who, f"{at} must be on GPU {self.device}, not on {value.device}")
            if not value.is_contiguous():
                _refuse(who, f"{at} must be contiguous")
            if not name.endswith("_scale"):
                if n is None:
                    n = value.numel()
                if value.numel() != n:
                    _refuse(who, f"{at} has {value.numel()} elements, and others {n}")
        n = n or 0
        for name in ("m_scale", "v_scale"):
            value = t.get(name)
            if value is not None and value.numel() != -(-n // GROUP_STATE):
                _refuse(who, f"{name} of tensor {i} must have {-(-n // GROUP_STATE)} elements, not {value.numel()}")
        if self.kinds.get("m") != self.kinds.get("v"):
            _refuse(who, f"m and v of tensor {i} must both be fp32 or both 8-bit")
        entry = self.array[i]
        entry.n = n
        for name, value in t.items():
            if value is not None and value.numel():
                address = value.data_ptr()
                setattr(entry, name, address)
                # which of m_out and m is written depends on the call: both count as outputs
                spans.append((address, address + value.numel() * value.element_size(), name != "g",
                              f"{name} of tensor {i}"))

    def _need(self, func: str, names, stream):
        for name in names:
            if name not in self.full:
                _refuse(func, f"a tensor has no {name}")
        if self.device is not None:
            _on_device(func, self.device, stream, "the tensors")


def _on_device(func, device, stream, what):
    """The kernels run on the stream's device (the current one's where no stream is given)."""
    at = getattr(stream, "device_index", None)
    if at is None:
        at = _cur_device() if _cur_device is not None else torch.cuda.current_device()
    if at != device:
        _refuse(func, f"{what} must be on GPU {at}, not on GPU {device}")


def _scalar(func: str, name: str, t, dtype, device, stream):
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != 1 or not t.is_cuda:
        _refuse(func, f"{name} must be one {dtype} on the GPU")
    _on_device(func, t.get_device(), stream, name)
    return t.data_ptr()


def moe_adamw_step(tensors: AdamwTensors, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, weight_decay: float = 0.01, lr_device=None, step_device=None, grad_scale=None,
                   stream=None):
    """One AdamW step on all tensors, in place.  lr_device (fp32), step_device (int64) and grad_scale (fp32) are
    one-element tensors that the kernels read, so that a captured graph follows them."""
    f = "moe_adamw_step"
    kinds = tensors.kinds
    eight = kinds.get("m") == _8BIT
    tensors._need(f, ("p", "g", "m", "v") + (("m_scale", "v_scale") if eight else ()), stream)
    params = _Params(kinds.get("p", _F32), kinds.get("g", _F32), kinds.get("m", _F32), 0, lr, beta1, beta2, eps,
                     weight_decay, int(step), _scalar(f, "lr_device", lr_device, torch.float32, tensors.device, stream),
                     _scalar(f, "step_device", step_device, torch.int64, tensors.device, stream),
                     _scalar(f, "grad_scale", grad_scale, torch.float32, tensors.device, stream))
    _check(f, _load().moe_adamw_step(tensors.array, tensors.count, ctypes.byref(params), _stream(stream)))


def _states(func, tensors, stream):
    tensors._need(func, ("m", "v", "m_scale", "v_scale", "m_out", "v_out"), stream)
    if tensors.kinds.get("m", _8BIT) != _8BIT:
        _refuse(func, "the states must be 8-bit")
    if tensors.kinds.get("m_out") != tensors.kinds.get("v_out"):
        _refuse(func, "m_out and v_out must have one type")


def moe_adamw_pack(tensors: AdamwTensors, stream=None):
    """8-bit states (m, v and their scales) of the fp32 values m_out and v_out."""
    f = "moe_adamw_pack"
    _states(f, tensors, stream)
    if tensors.kinds.get("m_out", _F32) != _F32:
        _refuse(f, "m_out and v_out must be fp32")
    _check(f, _load().moe_adamw_pack(tensors.array, tensors.count, _stream(stream)))


def moe_adamw_unpack(tensors: AdamwTensors, stream=None):
    """The values of 8-bit states into m_out and v_out (fp32 or bf16)."""
    f = "moe_adamw_unpack"
    _states(f, tensors, stream)
    _check(f, _load().moe_adamw_unpack(tensors.array, tensors.count, tensors.kinds.get("m_out", _F32),
                                       _stream(stream)))
