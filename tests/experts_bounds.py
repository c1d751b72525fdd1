"""Bounds of the experts' block's results that a wrong result exceeds (CPU or
GPU tensors; test infrastructure).  They follow the arithmetic: every place
that rounds is counted once, and the gate's error goes to zero where its
sigmoid is saturated.

U = 2^-8 is half a bf16 step relative to the value; a sum of n fp32 terms is
off by at most GAMMA(n) times the sum of their magnitudes.

Weights are pairs (value, error): `error` is a matrix M such that |x| M^T
bounds the error of x value^T.  For bf16 weights M = GAMMA(k) |w|.  A group of
G 4-bit weights is summed as sum q x - 8 sum x, 2 G terms of magnitude
(q + 8) |x| at most, times its scale; the groups' sums are added in fp32, as
many again of a product's waves.
"""

from __future__ import annotations

import math

import torch

from experts_ref import GAMMA, TINY, U, four_bit, slope

STEP = 2.0 ** -24  # half an fp32 step, relative
WAYS = 8           # waves that share a sum, at most


def bf16_weights(w):
    w = w.double()
    return w, GAMMA(w.shape[-1] + WAYS) * w.abs()


def w4_weights(q, scale, group):
    w = four_bit(q, scale, group)
    nibble = torch.stack((q & 15, q >> 4), -1).flatten(-2).double()
    wide = scale.double().abs().repeat_interleave(group, -1)
    return w, GAMMA(2 * group) * (nibble + 8) * wide + GAMMA(w.shape[-1] // group + WAYS) * w.abs()


def norm_bound(w):
    """An upper bound of the 2-norm, at most n^(1/32) above it: the Frobenius norm of (w w^T)^8."""
    if 0 in w.shape:
        return 0.0
    a = w @ w.T if w.shape[0] <= w.shape[1] else w.T @ w
    top, power = float(a.norm()), 1.0
    if top == 0:
        return 0.0
    log = math.log(top)  # of the bound of a's norm
    a = a / top
    for _ in range(3):
        a = a @ a
        power *= 2
        n = float(a.norm())
        if n == 0:
            return math.exp(log / 2)
        log += math.log(n) / power
        a = a / n
    return math.exp(log / 2)


def gate(g, act: int):
    """act(g), act'(g) and bounds of their computed values' errors for an exact g.

    s = 1 / (1 + E), E = exp(-a).  The argument's roundings (eight of them, the constants' included) are worth
    8 |a| STEP of E, the exponential 2 STEP; of that (1 - s) reaches s.  The sum and the reciprocal are worth 4 STEP;
    where E is lost beside 1, s is 1 and off by 1 - s.  A sigmoid below 2^-126 may come out as 0."""
    c0, c1 = slope(act)
    a = c0 * g + c1 * g ** 3
    s = torch.sigmoid(a)
    rest = torch.sigmoid(-a)  # 1 - s without cancellation
    es = s * (rest * (8 * a.abs() + 2) * STEP + torch.where(rest >= 2.0 ** -26, 4 * STEP, rest)) + 2.0 ** -126
    out = g * s
    e_out = g.abs() * es + 2 * STEP * out.abs()
    # past +-64 the slope is taken at the clamped g; there s or 1 - s is 0 and removes it
    inside = (g.abs() <= 64).double()
    t = inside * (c0 + 3 * c1 * g * g) + (1 - inside) * (c0 + 3 * c1 * 64.0 ** 2)
    d = s + out * rest * t
    saturated = ((a > 40) | (a < -104)).double()  # 1 - s, or s, is exactly 0
    e_prod = t * (out.abs() * es + rest * e_out) * (1 - saturated) + 8 * STEP * t * out.abs() * rest
    return out, d, e_out, es + e_prod + 2 * STEP * d.abs()


def steepest(g, eg, act: int):
    """The largest |act'| between g - eg and g + eg: under 1.2 anywhere, and falling below -4."""
    near = g + eg
    return torch.where(near < -4, gate(near, act)[1].abs(), torch.full_like(g, 1.2))


def forward(x, up, down, act):
    """One expert's rows (64 bits), weights as pairs.  Values, element bounds e_*, and n_y of each row of y."""
    (wu, mu), (wd, md) = up, down
    inter = wd.shape[1]
    pre, err = x @ wu.T, x.abs() @ mu.T
    g, u, eg, eu = pre[:, :inter], pre[:, inter:], err[:, :inter], err[:, inter:]
    a, _, ea, _ = gate(g, act)
    ea = ea + steepest(g, eg, act) * eg
    h = a * u
    eh = ea * u.abs() + (a.abs() + ea) * eu + 2 * STEP * h.abs() + TINY
    eh = eh + U * (h.abs() + eh)
    y = h @ wd.T
    m = (h.abs() + eh) @ md.T
    ey = eh @ wd.abs().T + m
    ey = ey + U * (y.abs() + ey) + TINY
    spread = norm_bound(wd) * eh.norm(dim=1) + m.norm(dim=1)
    ny = spread + U * (y.norm(dim=1) + spread) + TINY
    return dict(g=g, u=u, e_g=eg, e_u=eu, h=h, e_h=eh, y=y, e_y=ey, n_y=ny)


def backward(gy, x, w_gate_up, w_down, g, u, act):
    """One expert, bf16 weights (64-bit values); g and u as saved.  Gradients, element bounds e_*, norm bounds n_* (of
    a row of grad_xe, of a whole weight gradient)."""
    dh = gy @ w_down
    edh = GAMMA(gy.shape[1]) * (gy.abs() @ w_down.abs())
    a, da, ea, eda = gate(g, act)
    h = a * u
    eh = ea * u.abs() + 2 * STEP * h.abs() + TINY
    eh = eh + U * (h.abs() + eh)
    dg, du = dh * u * da, dh * a
    edg = edh * (u * da).abs() + (dh.abs() + edh) * u.abs() * eda + 4 * STEP * dg.abs() + TINY
    edu = edh * a.abs() + (dh.abs() + edh) * ea + 4 * STEP * du.abs() + TINY
    edg, edu = edg + U * (dg.abs() + edg), edu + U * (du.abs() + edu)
    d, ed = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    out = {}

    def product(name, left, e_left, right, e_right, rows):
        v = left @ right
        m = GAMMA(left.shape[1]) * ((left.abs() + e_left) @ (right.abs() + e_right))
        e = e_left @ right.abs() + left.abs() @ e_right + e_left @ e_right + m
        out[name], out["e_" + name] = v, e + U * (v.abs() + e) + TINY
        size = (lambda t: t.norm(dim=1)) if rows else (lambda t: t.norm())
        spread = norm_bound(right) * size(e_left) + norm_bound(left) * e_right.norm() + size(e_left @ e_right) + size(m)
        out["n_" + name] = spread + U * (size(v) + spread) + TINY

    none = torch.zeros_like
    product("grad_xe", d, ed, w_gate_up, none(w_gate_up), True)
    product("grad_w_gate_up", d.T, ed.T, x, none(x), False)
    product("grad_w_down", gy.T, none(gy.T), h, eh, False)
    return out


def excess(got, want, bound):
    """The largest error in units of its bound (infinite where got is not finite)."""
    if not bool(torch.isfinite(got).all()):
        return math.inf
    return float(((got.double() - want).abs() / bound).max()) if got.numel() else 0.0


def row_excess(got, want, bound):
    return float(((got.double() - want).norm(dim=1) / bound).max()) if got.numel() else 0.0
