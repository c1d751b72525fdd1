"""The optimizer's step on the CPU: what the library and its binding refuse
before anything is launched, and the header's functions."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40  # addresses that no refused call touches


def _ms():
    import moe_expert_token_amd as ms
    from moe_expert_token_amd import optim
    return ms, optim, optim._load()


def test_every_declared_symbol_is_exported():
    ms, optim, lib = _ms()
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_optim.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_adamw_\w+)\s*\(", text)))
    assert names == sorted(ms.OPTIM_EXPORTS)
    for n in names:
        assert getattr(lib, n) is not None


def tensor(optim, n=1000, **change):
    at = {name: BASE + (i << 30) for i, name in
          enumerate(("p", "copy", "g", "m", "v", "m_scale", "v_scale", "m_out", "v_out"))}
    at.update(change)
    return optim._Tensor(n=n, **at)


def params(optim, **change):
    p = dict(param=0, grad=1, state=0, reserved=0, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
    p.update(change)
    return optim._Params(**p)


def step(t, p, count=1):
    ms, optim, lib = _ms()
    return lib.moe_adamw_step(ctypes.byref(t) if t is not None else None, count,
                              ctypes.byref(p) if p is not None else None, None)


def test_what_a_step_refuses():
    ms, optim, lib = _ms()
    t, p = tensor(optim), params(optim)
    bad, align, over = ms.E_INVALID_ARG, ms.E_ALIGN, ms.E_OVERFLOW
    assert step(t, None) == bad
    assert step(None, p) == bad
    assert step(t, p, -1) == bad
    assert step(t, p, 0) == ms.OK
    assert step(tensor(optim, 0, p=0, g=0, m=0, v=0), p) == ms.OK
    for change in (dict(param=2), dict(grad=2), dict(state=1), dict(reserved=1), dict(lr=-1.0), dict(lr=float("nan")),
                   dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
                   dict(eps=-1e-9), dict(weight_decay=-1.0), dict(step=0), dict(step=-5)):
        assert step(t, params(optim, **change)) == bad, change
    for name in ("lr_device", "step_device", "grad_scale"):
        assert step(t, params(optim, **{name: BASE + 2})) == align, name
    assert step(tensor(optim, -1), p) == bad
    assert step(tensor(optim, 1 << 40), p) == over
    assert step(tensor(optim, (1 << 40) - 1, p=8), p) == align
    for name in ("p", "g", "m", "v"):
        assert step(tensor(optim, **{name: 0}), p) == bad, name
        assert step(tensor(optim, **{name: BASE + (20 << 30) + 8}), p) == align, name
    assert step(tensor(optim, copy=BASE + (20 << 30) + 8), p) == align
    assert step(t, params(optim, param=1)) == bad  # a copy of bf16 parameters
    eight = params(optim, state=2)
    for name in ("m_scale", "v_scale"):
        assert step(tensor(optim, **{name: 0}), eight) == bad, name
        assert step(tensor(optim, **{name: BASE + (20 << 30) + 2}), eight) == align, name
    # overlaps: an output's last bytes and another's first
    for name, size in (("copy", 4000), ("g", 4000), ("m", 4000), ("v", 4000)):
        assert step(tensor(optim, **{name: BASE + size - 16}), p) == bad, name
    assert step(tensor(optim, m_scale=BASE + (3 << 30) + 992), eight) == bad  # the last codes of m
    assert step(tensor(optim, v_scale=BASE + (5 << 30) + 28), eight) == bad   # m_scale's last


def test_what_pack_and_unpack_refuse():
    ms, optim, lib = _ms()
    calls = {"pack": lambda t, count=1: lib.moe_adamw_pack(ctypes.byref(t), count, None),
             "unpack": lambda t, count=1: lib.moe_adamw_unpack(ctypes.byref(t), count, 0, None)}
    for name, call in calls.items():
        assert call(tensor(optim), 0) == ms.OK
        assert call(tensor(optim), -1) == ms.E_INVALID_ARG
        assert call(tensor(optim, 0)) == ms.OK
        assert call(tensor(optim, -1)) == ms.E_INVALID_ARG
        for field in ("m", "v", "m_scale", "v_scale", "m_out", "v_out"):
            assert call(tensor(optim, **{field: 0})) == ms.E_INVALID_ARG, (name, field)
        for field in ("m", "v", "m_out", "v_out"):
            assert call(tensor(optim, **{field: BASE + (20 << 30) + 4})) == ms.E_ALIGN, (name, field)
        assert call(tensor(optim, m_out=BASE + (3 << 30) + 992)) == ms.E_INVALID_ARG, name
    assert lib.moe_adamw_unpack(ctypes.byref(tensor(optim)), 1, 2, None) == ms.E_INVALID_ARG


class Fake:
    """What a tensor on a GPU says of itself, without one."""

    def __init__(self, n, dtype=torch.float32, at=BASE, device=0, contiguous=True):
        self.n, self.dtype, self.at, self.index, self.whole = n, dtype, at, device, contiguous
        self.is_cuda, self.device = True, f"cuda:{device}"

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.whole

    def numel(self):
        return self.n

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        return self.at


class Stream:
    device_index, cuda_stream = 0, 0


def fakes(n=256, **change):
    t = {"p": Fake(n, at=BASE), "g": Fake(n, torch.bfloat16, at=BASE + (1 << 20)), "m": Fake(n, at=BASE + (2 << 20)),
         "v": Fake(n, at=BASE + (3 << 20))}
    t.update(change)
    return t


def test_lists_that_are_refused():
    ms, _, _ = _ms()

    def refused(*tensors):
        with pytest.raises(ms.MoeShuffleError) as e:
            ms.AdamwTensors(tensors)
        assert e.value.code == ms.E_INVALID_ARG
        return str(e.value)

    ms.AdamwTensors([fakes()])
    ms.AdamwTensors([])
    assert "on the GPU" in refused(fakes(p=torch.empty(256)))
    assert "float16" in refused(fakes(g=Fake(256, torch.float16, BASE + (1 << 20))))
    assert "another type" in refused(fakes(), {k: Fake(8, v.dtype if k != "g" else torch.float32, v.at + (9 << 20))
                                               for k, v in fakes().items()})
    assert "GPU 0" in refused(fakes(v=Fake(256, at=BASE + (3 << 20), device=1)))
    assert "contiguous" in refused(fakes(m=Fake(256, at=BASE + (2 << 20), contiguous=False)))
    assert "elements" in refused(fakes(m=Fake(255, at=BASE + (2 << 20))))
    assert "no such" in refused(fakes(q=Fake(256, at=BASE + (9 << 20))))
    assert "both" in refused(fakes(m=Fake(256, torch.uint8, BASE + (2 << 20))))
    eight = fakes(m=Fake(256, torch.uint8, BASE + (2 << 20)), v=Fake(256, torch.uint8, BASE + (3 << 20)))
    assert "2 elements" in refused(dict(eight, m_scale=Fake(3, at=BASE + (9 << 20))))
    # the same parameters twice, a gradient inside them, states that run into each other
    assert "overlaps" in refused(fakes(), fakes())
    assert "overlaps" in refused(fakes(g=Fake(256, torch.bfloat16, BASE + 1008)))
    assert "overlaps" in refused(fakes(v=Fake(256, at=BASE + (2 << 20) + 1020)))
    # two tensors may share a gradient
    ms.AdamwTensors([fakes(), {k: v if k == "g" else Fake(256, v.dtype, v.at + (9 << 20)) for k, v in fakes().items()}])


def test_calls_that_are_refused():
    ms, _, _ = _ms()

    def refused(call, *args, **kw):
        with pytest.raises(ms.MoeShuffleError) as e:
            call(*args, stream=Stream(), **kw)
        assert e.value.code == ms.E_INVALID_ARG
        return str(e.value)

    t = fakes()
    del t["g"]
    assert "no g" in refused(ms.moe_adamw_step, ms.AdamwTensors([t]), 1, 1e-3)
    whole = ms.AdamwTensors([fakes()])
    assert "grad_scale" in refused(ms.moe_adamw_step, whole, 1, 1e-3, grad_scale=torch.ones(1))
    assert "step_device" in refused(ms.moe_adamw_step, whole, 1, 1e-3, step_device=Fake(1, torch.int32))
    assert "on GPU 0" in refused(ms.moe_adamw_step, whole, 1, 1e-3, lr_device=Fake(1, torch.float32, device=1))
    far = ms.AdamwTensors([{k: Fake(256, v.dtype, v.at, device=1) for k, v in fakes().items()}])
    assert "on GPU 0" in refused(ms.moe_adamw_step, far, 1, 1e-3)
    assert "m_scale" in refused(ms.moe_adamw_unpack, whole)
    wide = fakes(m_scale=Fake(2, at=BASE + (4 << 20)), v_scale=Fake(2, at=BASE + (5 << 20)),
                 m_out=Fake(256, at=BASE + (6 << 20)), v_out=Fake(256, torch.bfloat16, at=BASE + (7 << 20)))
    assert "8-bit" in refused(ms.moe_adamw_unpack, ms.AdamwTensors([wide]))
    eight = dict(wide, m=Fake(256, torch.uint8, BASE + (2 << 20)), v=Fake(256, torch.uint8, BASE + (3 << 20)))
    assert "one type" in refused(ms.moe_adamw_unpack, ms.AdamwTensors([eight]))
    half = dict(eight, m_out=Fake(256, torch.bfloat16, BASE + (6 << 20)))
    assert "fp32" in refused(ms.moe_adamw_pack, ms.AdamwTensors([half]))
