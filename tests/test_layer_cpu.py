"""The router and the layer on the CPU: what the library and its binding refuse
before anything is launched, the header's functions, and the tests' own
definition of the router's gradient against differences and torch."""

import ctypes
import os
import re

import pytest
import torch

import layer_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40  # addresses that no refused call touches
GIB = 1 << 30


def _ms():
    import moe_expert_token_amd as ms
    from moe_expert_token_amd import layer
    return ms, layer, layer._load()


def test_every_declared_symbol_is_exported():
    ms, layer, lib = _ms()
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_layer.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_(?:router|layer)_\w+)\s*\(", text)))
    assert names == sorted(ms.LAYER_EXPORTS)
    for n in names:
        assert getattr(lib, n) is not None


class Call:
    """A call with arguments that are fine, by name, so that a test changes one."""

    def __init__(self, which, T=5, H=64, E=8, k=2, R=4, I=64, group=32):
        self.which = which
        self.dims = dict(T=T, H=H, E=E, k=k, R=R)
        self.args = dict(I=I, group=group, act=0, ws_bytes=1 << 40)
        self.rule = dict(scoring=1, normalize=1, scale=1.0, reserved=0, bias=BASE + 40 * GIB)
        names = {"router": ("x", "w_router", "topk_idx", "topk_w", "logits", "ws"),
                 "back": ("grad", "logits", "topk_idx", "x", "w_router", "grad_logits", "grad_x_in", "grad_x", "grad_w", "ws"),
                 "layer": ("x", "w_router", "up", "down", "residual", "out", "topk_idx", "topk_w", "ws"),
                 "w4": ("x", "w_router", "up", "up_s", "down", "down_s", "residual", "out", "topk_idx", "topk_w", "ws")}
        self.names = names[which]
        self.at = {n: BASE + i * GIB for i, n in enumerate(self.names)}

    def go(self, **change):
        ms, layer, lib = _ms()
        d = dict(self.dims, **{k: v for k, v in change.items() if k in self.dims})
        a = dict(self.args, **{k: v for k, v in change.items() if k in self.args})
        r = dict(self.rule, **{k: v for k, v in change.items() if k in self.rule})
        p = dict(self.at, **{k: v for k, v in change.items() if k in self.at})
        unknown = set(change) - set(self.dims) - set(self.args) - set(self.rule) - set(self.at)
        assert not unknown, unknown
        dims = ctypes.byref(ms.dims_of(d["T"], d["H"], d["E"], d["k"], d["R"]))
        rule = ctypes.byref(layer._Rule(r["scoring"], r["normalize"], r["scale"], r["reserved"], r["bias"] or None))
        v = [p[n] or None for n in self.names]
        if self.which == "router":
            return lib.moe_router_forward(dims, rule, *v, a["ws_bytes"], None)
        if self.which == "back":
            return lib.moe_router_backward(dims, rule, *v, a["ws_bytes"], None)
        if self.which == "layer":
            return lib.moe_layer_forward(dims, rule, *v[:4], a["I"], a["act"], *v[4:], a["ws_bytes"], None)
        return lib.moe_layer_w4_forward(dims, rule, *v[:6], a["I"], a["group"], a["act"], *v[6:], a["ws_bytes"], None)


CALLS = ("router", "back", "layer", "w4")


@pytest.mark.parametrize("which", CALLS)
def test_dims_and_rules_that_are_refused(which):
    ms, _, _ = _ms()
    c = Call(which)
    bad = ms.E_INVALID_ARG
    for change in (dict(T=-1), dict(H=0), dict(E=0), dict(k=0), dict(k=9), dict(R=3), dict(scoring=2), dict(scoring=-1),
                   dict(reserved=1), dict(scale=float("nan")), dict(scale=float("inf")), dict(scoring=0)):
        assert c.go(**change) == bad, change  # the last: a bias with softmax
    assert c.go(H=60) == ms.E_ALIGN
    assert c.go(bias=BASE + 2) == ms.E_ALIGN
    assert c.go(H=1 << 20) == ms.E_OVERFLOW
    assert c.go(E=1024, R=4) == ms.E_OVERFLOW
    assert c.go(T=0, scoring=0, bias=0, **({"grad_w": 0} if which == "back" else {})) == ms.OK


@pytest.mark.parametrize("which", CALLS)
def test_pointers_that_are_refused(which):
    ms, _, _ = _ms()
    c = Call(which)
    may_be_null = {"logits": which == "router", "grad_logits": True, "residual": True, "topk_idx": which in ("layer", "w4"),
                   "topk_w": which in ("layer", "w4"), "grad_x_in": True, "grad_w": True}
    for n in c.names:
        if not may_be_null.get(n, n == "grad_x"):
            assert c.go(**{n: 0}) == ms.E_INVALID_ARG, n
        wide = n not in ("topk_idx", "topk_w", "logits", "grad", "grad_logits")
        assert c.go(**{n: c.at[n] + (8 if wide else 2)}) == ms.E_ALIGN, n
    assert c.go(ws=c.at["ws"] + 128) == ms.E_ALIGN
    assert c.go(ws_bytes=16) == ms.E_WORKSPACE
    if which == "back":
        assert c.go(grad_x=0) == ms.E_INVALID_ARG            # something to add, and nowhere to
        assert c.go(grad_x=0, grad_x_in=0, grad_w=0) == ms.OK  # nothing is asked for


@pytest.mark.parametrize("which", CALLS)
def test_overlaps_that_are_refused(which):
    ms, layer, lib = _ms()
    c = Call(which)
    outs = {"router": ("topk_idx", "topk_w", "logits", "ws"), "back": ("grad_x", "grad_w", "ws"),
            "layer": ("out", "topk_idx", "topk_w", "ws"), "w4": ("out", "topk_idx", "topk_w", "ws")}[which]
    for o in outs:
        for n in c.names:
            if n == o or (n == "grad_x_in" and o == "grad_x") or (n == "residual" and o == "out"):
                continue
            assert c.go(**{o: c.at[n]}) == ms.E_INVALID_ARG, (o, n)
        assert c.go(bias=c.at[o]) == ms.E_INVALID_ARG or which == "back", o
    # what is added may be the output itself, but not a part of it
    if which == "back":
        assert c.go(grad_x_in=c.at["grad_x"] + 16) == ms.E_INVALID_ARG
    elif which != "router":
        assert c.go(residual=c.at["out"] + 16) == ms.E_INVALID_ARG


def test_limits_of_the_layer():
    ms, _, _ = _ms()
    for which in ("layer", "w4"):
        c = Call(which)
        assert c.go(T=65) == ms.E_OVERFLOW
        assert c.go(T=64, k=8, E=64, ws_bytes=0) == ms.E_WORKSPACE
        assert c.go(T=57, k=9, E=64) == ms.E_OVERFLOW
        assert c.go(I=0) == ms.E_INVALID_ARG and c.go(I=1 << 20) == ms.E_OVERFLOW
        assert c.go(act=2) == ms.E_INVALID_ARG
    assert Call("layer").go(I=60) == ms.E_ALIGN
    for change in (dict(group=16), dict(group=0), dict(group=256)):
        assert Call("w4").go(**change) == ms.E_INVALID_ARG
    assert Call("w4").go(I=72) == ms.E_ALIGN
    assert Call("w4").go(group=128, I=128) == ms.E_ALIGN  # H = 64
    # huge sizes come back with a code, not with a wrapped product
    assert Call("layer").go(T=64, H=(1 << 20) - 8, E=1000, k=8, R=1, I=(1 << 20) - 8, ws_bytes=0) == ms.E_WORKSPACE


def test_limits_of_the_router():
    ms, _, _ = _ms()
    assert Call("router").go(T=1 << 30, E=512, R=1, k=1, H=8, ws_bytes=0) == ms.E_WORKSPACE
    assert Call("router").go(T=(1 << 31) - 1, E=513, R=1, k=1, H=8) == ms.E_OVERFLOW
    assert Call("back").go(T=1 << 30, E=8, R=1, k=1, H=8) == ms.E_OVERFLOW


def test_workspace_sizes_grow_with_the_dims():
    ms, _, _ = _ms()
    size = ms.moe_router_workspace_size
    assert size(ms.dims_of(0, 64, 8, 2, 1)) > 0
    for T in (1, 100, 8192, 100000):
        d = ms.dims_of(T, 7168, 256, 8, 1)
        assert size(d, True) >= size(d) >= T * 256 * 4
        assert size(d, True) >= T * 256 * 2 + 256 * 7168 * 4
    n = ms.moe_layer_workspace_size(ms.dims_of(48, 7168, 256, 8, 1), 2048)
    assert n >= 48 * 8 * (2048 * 2 + 7168 * 4) + 48 * 256 * 12


class Stream:
    device_index, cuda_stream = 0, 0


def bf(*s):
    return torch.empty(s, dtype=torch.bfloat16)


def binding_calls(ms):
    T, H, E, k, I, G = 5, 64, 8, 2, 32, 32
    dims = ms.dims_of(T, H, E, k, 1)
    rule = ms.RouterRule()
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    ids, gates, table = torch.empty(T, k, dtype=torch.int32), torch.empty(T, k), torch.empty(T, E)
    rows = dict(dims=dims, rule=rule, x=bf(T, H), w_router=bf(E, H), workspace=ws)
    outs = dict(out=bf(T, H), residual=bf(T, H), topk_idx=ids, topk_w=gates)
    byte = lambda *s: torch.empty(s, dtype=torch.uint8)  # noqa: E731
    return {
        "router": (ms.moe_router_forward, dict(rows, topk_idx=ids, topk_w=gates, logits=table)),
        "back": (ms.moe_router_backward,
                 dict(rows, grad_topk_w=gates, logits=table, topk_idx=ids, grad_x=bf(T, H), grad_w_router=bf(E, H),
                      grad_x_in=bf(T, H), grad_logits=table)),
        "layer": (ms.moe_layer_forward, dict(rows, **outs, w_gate_up=bf(E, 2 * I, H), w_down=bf(E, H, I))),
        "w4": (ms.moe_layer_w4_forward,
               dict(rows, **outs, q_gate_up=byte(E, 2 * I, H // 2), s_gate_up=bf(E, 2 * I, H // G), q_down=byte(E, H, I // 2),
                    s_down=bf(E, H, I // G), group=G)),
    }


@pytest.mark.parametrize("which", CALLS)
def test_tensors_that_the_binding_refuses(which):
    """Host memory, other types, other shapes, strides: each named, before the library is called."""
    ms, _, _ = _ms()
    call, args = binding_calls(ms)[which]

    def refused(**change):
        with pytest.raises(ms.MoeShuffleError) as e:
            call(**dict(args, **change), stream=Stream())
        assert e.value.code == ms.E_INVALID_ARG
        return str(e.value)

    assert "on the GPU" in refused()
    for name, t in args.items():
        if not torch.is_tensor(t) or name == "workspace":
            continue
        assert name in refused(**{name: t[:-1]}), name
        assert name in refused(**{name: torch.empty(t.shape + (2,), dtype=t.dtype)[..., 0]}), name
        other = {torch.bfloat16: torch.float16, torch.float32: torch.int32, torch.int32: torch.float32,
                 torch.uint8: torch.int16}[t.dtype]
        assert name in refused(**{name: torch.empty(t.shape, dtype=other)}), name
    if which != "back":  # the backward pass does not look at it
        assert "bias" in refused(rule=ms.RouterRule(ms.SCORE_SIGMOID, bias=torch.zeros(7)))
    assert "workspace" in refused(workspace=None)


def test_rules_that_are_refused():
    ms, _, _ = _ms()
    for bias in (torch.zeros(8, dtype=torch.float64), torch.zeros(8, 1)):
        with pytest.raises(ms.MoeShuffleError):
            ms.RouterRule(ms.SCORE_SIGMOID, bias=bias)


@pytest.mark.parametrize("which", CALLS)
def test_the_rules_bias_is_that_of_the_call(which, monkeypatch):
    """A bias set anew, or one whose memory moved, after the rule was made: the library is given the new address."""
    ms, layer, _ = _ms()
    call, args = binding_calls(ms)[which]
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda dims, rule, *rest: seen.append(rule._obj.bias) or 0

    monkeypatch.setattr(layer, "_load", Library)
    monkeypatch.setattr(layer, "_on_gpu", lambda *a, **k: None)
    rule = ms.RouterRule(ms.SCORE_SIGMOID, bias=torch.zeros(8))
    first, other = rule.bias, torch.ones(8)
    call(**dict(args, rule=rule), stream=Stream())
    rule.bias = other
    call(**dict(args, rule=rule), stream=Stream())
    moved = torch.ones(8)
    other.data = moved
    call(**dict(args, rule=rule), stream=Stream())
    rule.bias = None
    call(**dict(args, rule=rule), stream=Stream())
    assert seen == [first.data_ptr(), seen[1], moved.data_ptr(), None] and seen[1] not in (seen[0], seen[2])
    if which != "back":
        for bias in (torch.zeros(8, dtype=torch.float64), torch.zeros(8, 1), torch.zeros(9)):
            rule.bias = bias
            with pytest.raises(ms.MoeShuffleError):
                call(**dict(args, rule=rule), stream=Stream())


# ---- the tests' own definition ----

@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_the_gradients_formula_against_differences_and_autograd(sigmoid, normalize):
    gen = torch.Generator().manual_seed(3)
    T, E, k, scale = 6, 9, 3, 1.7
    l = torch.randn(T, E, dtype=torch.float64, generator=gen)
    idx = ref.choose(l, k, sigmoid)
    grad = torch.randn(T, k, dtype=torch.float64, generator=gen)
    dl, bound = ref.score_gradient(l, idx, grad, sigmoid, normalize, scale)
    step = 1e-6
    for e in range(E):
        up, down = l.clone(), l.clone()
        up[:, e] += step
        down[:, e] -= step
        a, _ = ref.gates(up, idx, sigmoid, normalize, scale)
        b, _ = ref.gates(down, idx, sigmoid, normalize, scale)
        diff = ((a - b) * grad).sum(1) / (2 * step)
        assert float((diff - dl[:, e]).abs().max()) < 1e-8
    leaf = l.clone().requires_grad_(True)
    w, _ = ref.gates(leaf, idx, sigmoid, normalize, scale)
    (want,) = torch.autograd.grad(w, leaf, grad)
    assert float((want - dl).abs().max()) < 1e-14
    # the bound is of fp32's size, and holds the same formula computed in fp32
    s32 = ref.scores(l.float().double(), sigmoid)
    assert float(bound.max()) < 1e-3 * float(s32.max()) * 40


def test_a_planted_mistake_exceeds_the_bounds():
    """Gates of the next slot, gradients without the normalization's term, an expert's weights of its neighbour."""
    gen = torch.Generator().manual_seed(4)
    T, H, E, k, I = 5, 64, 8, 3, 32
    x, w = torch.randn(T, H, generator=gen).to(torch.bfloat16), torch.randn(E, H, generator=gen).to(torch.bfloat16) / 8
    l = ref.logits(x, w)
    idx = ref.choose(l, k, True)
    gates, rel = ref.gates(l, idx, True, True, 1.0)
    assert bool(((gates.roll(1, 1) - gates).abs() > rel * gates).all())
    grad = torch.randn(T, k, generator=gen)
    dl, err = ref.score_gradient(l, idx, grad, True, True, 1.0)
    wrong, _ = ref.score_gradient(l, idx, grad, True, False, 1.0)
    chosen = dl != 0
    assert bool(((wrong - dl).abs() > err)[chosen].all())
    import experts_bounds as bounds
    w1 = (torch.randn(E, 2 * I, H, generator=gen) / 8).to(torch.bfloat16)
    w2 = (torch.randn(E, H, I, generator=gen) / 6).to(torch.bfloat16)
    args = [lambda e: bounds.bf16_weights(w1[e]), lambda e: bounds.bf16_weights(w2[e])]
    out, bound = ref.layer(x, idx, gates, rel.expand_as(gates), *args, 0)
    other, _ = ref.layer(x, idx, gates, rel.expand_as(gates), args[0], lambda e: bounds.bf16_weights(w2[(e + 1) % E]), 0)
    assert float(((out - other).abs() > bound).double().mean()) > 0.9
    dropped = gates.clone()
    dropped[:, -1] = 0
    less, _ = ref.layer(x, idx, dropped, rel.expand_as(gates), *args, 0)
    assert float(((out - less).abs() > bound).double().mean()) > 0.8


@pytest.mark.parametrize("T,H", [(300, 7168), (8192, 7168), (64, 1544)])
def test_a_lost_product_exceeds_the_bound_of_a_logit(T, H):
    """Four products in five are more than a logit may be off (at H = 7168 it may by 0.06 of their usual size, which the product of
    two normal numbers is under once in six); sums in fp32, element after element and split alike, are not."""
    gen = torch.Generator().manual_seed(5)
    x, w = torch.randn(5, H, generator=gen).to(torch.bfloat16), (torch.randn(3, H, generator=gen) / H ** 0.5).to(torch.bfloat16)
    bound = ref.logit_bound(x, w, T)
    products = x.double()[:, None] * w.double()
    assert float((products.abs() > bound[..., None]).double().mean()) > 0.8
    in32 = torch.zeros(5, 3)
    for i in range(H):
        in32 = in32 + products[..., i].float()
    assert bool(((in32.double() - products.sum(2)).abs() < bound * 4).all())
