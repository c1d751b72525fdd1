"""Inputs for the experts' kernels, made alike on the CPU (where planted
mistakes show what the bounds catch) and on the GPU (test infrastructure).

Two kinds.  `dense`: random rows and weights; a row's error norm is held.
`sparse`: few elements of a row, and of each feature's weights, are not zero, so
that a result has few terms and each of its elements shows a term that is
missing or wrong, at any length of the sum.
"""

from __future__ import annotations

import numpy as np
import torch

import experts_bounds as eb

CHUNK = 128

# rows of each expert: 7.4 on average (a full and a second row tile among them), and 26
FEW, MANY = [1, 3, 0, 16, 17], [70, 0, 33, 1]

# H, I of the bf16 streams: sums of whole chunks below and from 4096 on, either way round, and of broken ones
BF16_FORMS = [(512, 256), (4096, 4224), (4096, 256), (512, 4096), (4104, 136), (136, 4104)]

# group, rows, length of the sum: two waves a sum or eight (from 4096 on, or past what two ways' scales take in LDS),
# whole chunks or not, and lengths past what any scales in LDS allow
W4_FORMS = [(32, n, k) for n, ks in (("few", (512, 544, 4096, 4128, 16416)), ("many", (512, 544, 8320, 8224, 32800)))
            for k in ks] + \
           [(64, n, k) for n, ks in (("few", (512, 576, 4096, 4160, 32832)), ("many", (512, 576, 8320, 8256, 32832)))
            for k in ks] + \
           [(128, n, k) for n, ks in (("few", (512, 4096, 65664)), ("many", (512, 16512, 65664))) for k in ks]


def ids(counts):
    """Top-1 ids that give expert e counts[e] rows, the tokens shuffled."""
    v = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    np.random.default_rng(len(v)).shuffle(v)
    return v.reshape(-1, 1)


def _kept(H, I, device):
    """[2I, H]: where the sparse kind's projections are not zero, one feature a column or the other way round."""
    d = min(H, I)
    n = torch.arange(I, device=device) % d
    return (n[:, None] == torch.arange(H, device=device)[None, :] % d).repeat(2, 1)


def rows(kind, P, H, I, gen, device):
    if kind == "dense":
        return torch.empty((P, H), dtype=torch.bfloat16, device=device).normal_(0, 1, generator=gen)
    many = 16 if H >= I else 1
    at = (torch.arange(P * many, device=device) * (CHUNK + 3)) % H  # 131 (prime) further: the next chunk
    v = torch.rand(P * many, generator=gen, device=device) + 0.5
    v = torch.where(torch.rand(P * many, generator=gen, device=device) < 0.5, -v, v).to(torch.bfloat16)
    x = torch.zeros((P, H), dtype=torch.bfloat16, device=device)
    x[torch.arange(P * many, device=device) // many, at] = v
    return x


def bf16(kind, E, H, I, gen, device):
    """w_gate_up, w_down."""
    w1 = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=device)
    w2 = torch.empty((E, H, I), dtype=torch.bfloat16, device=device)
    w1.normal_(0, 1 if kind == "sparse" else H ** -0.5, generator=gen)
    w2.normal_(0, I ** -0.5, generator=gen)
    if kind == "sparse":
        w1 *= _kept(H, I, device)
    return w1, w2


def w4(kind, E, H, I, group, gen, device):
    """q_gate_up, s_gate_up, q_down, s_down."""
    q1 = torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, device=device, generator=gen)
    q2 = torch.randint(0, 256, (E, H, I // 2), dtype=torch.uint8, device=device, generator=gen)
    if kind == "sparse":  # 8 stands for zero
        keep = _kept(H, I, device)
        q1 = torch.where(keep[:, 0::2], q1 & 15, 8) | (torch.where(keep[:, 1::2], q1 >> 4, 8) << 4)
        del keep

    def scales(n, k, size):
        s = (torch.rand((E, n, k // group), device=device, generator=gen) + 0.5) * size
        return torch.where(torch.rand(s.shape, device=device, generator=gen) < 0.1, -s, s).to(torch.bfloat16)

    return q1, scales(2 * I, H, 0.25 if kind == "sparse" else 0.22 * H ** -0.5), q2, scales(H, I, 0.22 * I ** -0.5)


def mistakes(x, up, down, act):
    """name -> what y becomes when a kernel makes that mistake (weights as pairs)."""
    (wu, _), (wd, _) = up, down
    out = {}

    def run(name, a, b):
        out[name] = eb.forward(x, (a, a), (b, b), act)["y"]

    def dropped(w, c):
        w = w.clone()
        w[:, CHUNK * c:CHUNK * (c + 1)] = 0
        return w

    def swapped(w):
        return w.unflatten(1, (-1, 2)).flip(2).flatten(1)

    out["zero"] = torch.zeros((x.shape[0], wd.shape[0]), dtype=torch.float64, device=x.device)
    for side, w in (("up", wu), ("down", wd)):
        n = -(-w.shape[1] // CHUNK)
        for c in sorted({0, n // 2, n - 1}):
            run(f"{side}: chunk {c} of {n} dropped", *((dropped(wu, c), wd) if side == "up" else (wu, dropped(wd, c))))
        run(f"{side}: neighbouring columns swapped", *((swapped(wu), wd) if side == "up" else (wu, swapped(wd))))
    half = wu.shape[0] // 2
    run("gate and up features swapped", torch.cat((wu[half:], wu[:half])), wd)
    return out


def caught(y, r):
    """Whether a result y lies outside the bounds of r."""
    return eb.excess(y, r["y"], r["e_y"]) > 1 or eb.row_excess(y, r["y"], r["n_y"]) > 1
