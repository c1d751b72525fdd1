"""The routing rule and the layer in 64 bits, with bounds of each result (CPU
or GPU tensors; test infrastructure)."""

from __future__ import annotations

import torch

import experts_bounds as bounds
from experts_ref import TINY, U

STEP = 2.0 ** -24  # half an fp32 step, relative


def logits(x, w):
    return x.double() @ w.double().T


def logit_bound(x, w, T=None):
    """How far the router's fp32 logits may be off, of each row and expert: 4 2^-23 sqrt(sum c_i x_i^2) sqrt(sum c_i w_i^2),
    with c_i the tiles of 64 k from i on in its part of H and (8 + parts) / 4 more.  The parts are those of a batch of T rows
    (x's own where not given): as many, a power of two up to 16, as fill the card with blocks and leave four tiles each."""
    (rows, H), E = x.shape, w.shape[0]
    T = rows if T is None else T
    tokens, blocks = (128, 256) if T >= 2048 else (64, 512)
    tiles, parts = -(-T // tokens) * -(-E // 256), 1
    while parts < 16 and tiles * parts * 2 <= blocks and H >= parts * 2 * 4 * 64:
        parts *= 2
    each = -(-(-(-H // parts)) // 64) * 64
    parts = -(-H // each)
    i = torch.arange(H, device=x.device)
    k0 = i // each * each
    c = (-(-(H - k0).clamp(max=each) // 64) - (i - k0) // 64).double() + (8 + parts) / 4
    norm = lambda v: (c * v.double() ** 2).sum(1).sqrt()  # noqa: E731
    return 4 * 2.0 ** -23 * norm(x)[:, None] * norm(w)[None, :]


def scores(l, sigmoid: bool):
    if sigmoid:
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def choose(l, k: int, sigmoid: bool, bias=None):
    """Ids by falling key, ties to the lowest index, NaN as minus infinity."""
    key = l if bias is None else scores(l, True) + bias.double()
    key = torch.where(key.isnan(), -torch.inf, key)
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]


def gates(l, idx, sigmoid: bool, normalize: bool, scale: float):
    """Gates of chosen experts, and a bound of the fp32 ones' relative error: a logit rounds once (worth |l| STEP of its
    exponential, and the largest's as much), the difference once more, the exponential 2 STEP, a sum over E and one
    over k (their terms' errors, and a step for each addition in a tree of the wave), and six more roundings."""
    s = scores(l, sigmoid).gather(1, idx)
    w = s / (s.sum(1, keepdim=True) + 1e-20) if normalize else s
    most = l.abs().amax(1, keepdim=True).clamp(max=1e4)
    return scale * w, (8 * most + 2 * (6 + l.shape[1] / 64) + 24) * STEP


def layer(x, idx, w, rel, up, down, act, residual=None):
    """The layer's output and element bounds.  up(e), down(e): an expert's weights as pairs (value, error matrix) of
    experts_bounds; idx, w, rel: ids, gates and their relative error."""
    T, k = idx.shape
    H = x.shape[1]
    y = torch.zeros((T, k, H), dtype=torch.float64, device=x.device)
    ey = torch.zeros_like(y)
    for e in sorted(set(idx.flatten().tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        r = bounds.forward(x[t].double(), up(e), down(e), act)
        y[t, j] = r["y"]
        # the bound there counts y's rounding to bf16, which is left out here
        ey[t, j] = ((r["e_y"] - TINY) - U * r["y"].abs()) / (1 + U) + TINY
    terms = w[:, :, None] * y
    out = terms.sum(1)
    err = (w.abs()[:, :, None] * (1 + rel[:, :, None]) * ey).sum(1) + (rel[:, :, None] * terms.abs()).sum(1)
    size = terms.abs().sum(1)
    if residual is not None:
        out = out + residual.double()
        size = size + residual.double().abs()
    err = err + (k + 1) * STEP * (size + err)
    return out, err + U * (out.abs() + err) + TINY


def score_gradient(l, idx, grad, sigmoid: bool, normalize: bool, scale: float):
    """dl, and a bound of the error of one computed in fp32 from the same logits.

    A score's relative error: the logit's difference to the largest rounds (|l| STEP each), the exponential, the sum over
    E and the division a few steps more; D and the sum over the k chosen have as much again, and each further product
    or difference rounds its terms once."""
    s = scores(l, sigmoid)
    at, g = s.gather(1, idx), scale * grad.double()
    size = g.abs()
    if normalize:
        total = at.sum(1, keepdim=True) + 1e-20
        size = (g.abs() + (g.abs() * at).sum(1, keepdim=True) / total) / total
        g = (g - (g * at).sum(1, keepdim=True) / total) / total
    wide, wide_size = torch.zeros_like(s).scatter_(1, idx, g), torch.zeros_like(s).scatter_(1, idx, size)
    rel = (16 * l.abs().amax(1, keepdim=True).clamp(max=1e4) + 4 * (6 + l.shape[1] / 64) + 64) * STEP
    if sigmoid:
        # 1 - s loses what s rounds
        return wide * s * (1 - s), rel * wide_size * s
    mean, mean_size = (g * at).sum(1, keepdim=True), (size * at).sum(1, keepdim=True)
    return s * (wide - mean), rel * s * (wide_size + mean_size)


def router_backward(x, w, dl, e_dl, grad_x_in=None):
    """grad_x and grad_w_router of a dl held as two bf16 numbers (U of what U leaves is lost), with element bounds; the
    products are twice as many terms."""
    from experts_ref import GAMMA
    x, w = x.double(), w.double()
    err = e_dl + U * U * (dl.abs() + e_dl) + TINY
    size = dl.abs() + err
    gx, ex = dl @ w, err @ w.abs() + GAMMA(2 * w.shape[0]) * (size @ w.abs())
    if grad_x_in is not None:
        gx = gx + grad_x_in.double()
        ex = ex + 2 * STEP * (gx.abs() + ex)
    gw, ew = dl.T @ x, err.T @ x.abs() + GAMMA(2 * x.shape[0] + 32) * (size.T @ x.abs())
    return gx, ex + U * (gx.abs() + ex) + TINY, gw, ew + U * (gw.abs() + ew) + TINY
