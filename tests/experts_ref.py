"""The experts' block in 64 bits, and how far a result computed in fp32 with
bf16 operands may be from it (CPU or GPU tensors; test infrastructure).

Bounds.  U = 2^-8 is half a bf16 step relative to the value.  A sum of n fp32
products is off by at most GAMMA(n) times the sum of magnitudes.  The gate's
sigmoid(a) is computed from exp2 and a reciprocal: relative error at most
(4 + 2 |a|) 2^-23 (the argument's rounding is worth |a| 2^-24 twice, the two
instructions 2^-23 each, the sum 2^-24).
"""

from __future__ import annotations

import math

import torch

U = 2.0 ** -8
TINY = 2.0 ** -120  # far below every value the tests use; underflow stays under it
GROUP8 = 32


def GAMMA(n: int) -> float:
    return (n + 8) * 2.0 ** -24


def slope(act: int):
    c = 2 * math.sqrt(2 / math.pi)
    return (1.0, 0.0) if act == 0 else (c, c * 0.044715)


def gate(g, act: int):
    """act(g), act'(g), and bounds of the errors of both for an exact g."""
    c0, c1 = slope(act)
    a = c0 * g + c1 * g ** 3
    s = torch.sigmoid(a)
    t = g * (1 - s) * (c0 + 3 * c1 * g * g)
    rel = (6 + 2 * a.abs()) * 2.0 ** -23
    # 1 - s is off by s * rel; the products by a few roundings
    return g * s, s * (1 + t), (g * s).abs() * rel, s * rel * (1 + t.abs() + (g * s * (c0 + 3 * c1 * g * g)).abs()) + \
        8 * 2.0 ** -24 * s * (1 + t.abs())


def expert_norm(w):
    return float(torch.linalg.matrix_norm(w, 2)) if min(w.shape) else 0.0


def step8(top):
    """max(top / 127, 2^-126) rounded up to bf16, of float32 tops."""
    s = (top / 127).clamp(min=2.0 ** -126)
    return ((s.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)


def pack8(x):
    """(int8 values, bf16 steps) of fp32 rows, by the definition."""
    cols = x.shape[-1]
    t = torch.nn.functional.pad(x, (0, -cols % GROUP8)).unflatten(-1, (-1, GROUP8))
    top = t.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(t).all(-1, keepdim=True)
    step = torch.where(fine, step8(torch.where(fine, top, 0.0)), float("nan"))
    q = torch.round(t * (1 / step)).clamp(-127, 127)
    q = torch.where(fine, q, 0.0).flatten(-2)[..., :cols]
    return q.to(torch.int8), step.squeeze(-1).to(torch.bfloat16)


def unpack8(q, step):
    """The exact values, in 64 bits."""
    cols = q.shape[-1]
    return q.double() * step.double().repeat_interleave(GROUP8, -1)[..., :cols]


def four_bit(q, scale, group):
    """4-bit weights as 64-bit values."""
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).double() - 8
    return v * scale.double().repeat_interleave(group, -1)


def forward(x, w_gate_up, w_down, act, up_terms=None, down_terms=None):
    """One expert, 64-bit operands.  dict of h, y, g, u and the bounds e_h, e_y, e_g, e_u; ny bounds the 2-norm of
    each row's error in y."""
    inter = w_down.shape[1]
    wg, wu = w_gate_up[:inter], w_gate_up[inter:]
    g, u = x @ wg.T, x @ wu.T
    n = up_terms or x.shape[1]
    eg, eu = GAMMA(n) * (x.abs() @ wg.abs().T), GAMMA(n) * (x.abs() @ wu.abs().T)
    a, _, ea, _ = gate(g, act)
    ea = ea + 1.2 * eg  # |act'| < 1.2
    h = a * u
    eh = ea * u.abs() + (a.abs() + ea) * eu + 4 * 2.0 ** -24 * h.abs() + TINY
    eh = eh + U * (h.abs() + eh)
    y = h @ w_down.T
    m = GAMMA(down_terms or inter) * ((h.abs() + eh) @ w_down.abs().T)
    ey = eh @ w_down.abs().T + m
    ey = ey + U * (y.abs() + ey) + TINY
    spread = expert_norm(w_down) * eh.norm(dim=1) + m.norm(dim=1)
    ny = spread + U * (y.norm(dim=1) + spread) + TINY
    return dict(g=g, u=u, e_g=eg, e_u=eu, h=h, e_h=eh, y=y, e_y=ey, n_y=ny)


def backward(gy, x, w_gate_up, w_down, g, u, act):
    """One expert, 64-bit operands; g and u as saved.  Gradients and their bounds: by element (e_*), and by
    2-norm (n_*) of a row of grad_xe or of a whole weight gradient."""
    inter = w_down.shape[1]
    wg, wu = w_gate_up[:inter], w_gate_up[inter:]
    dh = gy @ w_down
    edh = GAMMA(gy.shape[1]) * (gy.abs() @ w_down.abs())
    a, da, ea, eda = gate(g, act)
    h = a * u
    eh = ea * u.abs() + 4 * 2.0 ** -24 * h.abs() + TINY
    eh = eh + U * (h.abs() + eh)
    dg, du = dh * u * da, dh * a
    edg = edh * (u * da).abs() + (dh.abs() + edh) * u.abs() * eda + 8 * 2.0 ** -24 * dg.abs() + TINY
    edu = edh * a.abs() + (dh.abs() + edh) * ea + 8 * 2.0 ** -24 * du.abs() + TINY
    edg, edu = edg + U * (dg.abs() + edg), edu + U * (du.abs() + edu)
    d, ed, w = torch.cat((dg, du), 1), torch.cat((edg, edu), 1), torch.cat((wg, wu), 0)
    out = {}

    def product(name, left, e_left, right, rows):
        v = left @ right
        m = GAMMA(left.shape[1]) * ((left.abs() + e_left) @ right.abs())
        e = e_left @ right.abs() + m
        out[name], out["e_" + name] = v, e + U * (v.abs() + e) + TINY
        s = expert_norm(right)
        norm = (lambda t: t.norm(dim=1)) if rows else (lambda t: t.norm())
        spread = s * norm(e_left) + norm(m)
        out["n_" + name] = spread + U * (norm(v) + spread) + TINY

    product("grad_xe", d, ed, w, True)
    product("grad_w_gate_up", d.T, ed.T, x, False)
    # grad_ye^T h: the error is in the right operand
    v, m = gy.T @ h, GAMMA(x.shape[0]) * (gy.abs().T @ (h.abs() + eh))
    e = gy.abs().T @ eh + m
    spread = expert_norm(gy) * eh.norm() + m.norm()
    out["grad_w_down"], out["e_grad_w_down"] = v, e + U * (v.abs() + e) + TINY
    out["n_grad_w_down"] = spread + U * (v.norm() + spread) + TINY
    return out
