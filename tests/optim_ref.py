"""AdamW in 64 bits, with bounds of each result (CPU or GPU tensors; test
infrastructure).  Every place that rounds is counted once."""

import math

import torch

GROUP = 128
STEP = 2.0 ** -24  # half an fp32 step, relative
U = 2.0 ** -8      # half a bf16 step, relative
TINY = 2.0 ** -126


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, scale=1.0):
    """New p, m, v (64-bit values of 64-bit inputs) and bounds of the fp32 results' errors.

    d = scale g rounds once.  m: its value may come from a code (once), the constant, the product and the sum round: under
    5 STEP of each term.  v: the root from a code (once), its square (3 by then), constant, product and sum: under 8
    STEP of each term.  The quotient: sqrt, the constants, two products, a sum, a division."""
    d = g * scale
    terms_m, terms_v = (beta1 * m).abs() + ((1 - beta1) * d).abs(), beta2 * v + (1 - beta2) * d * d
    m1, v1 = beta1 * m + (1 - beta1) * d, terms_v
    em, ev = 5 * STEP * terms_m + TINY, 8 * STEP * terms_v + TINY
    root = 1 / math.sqrt(1 - beta2 ** step)
    gain = lr / (1 - beta1 ** step)
    den = v1.sqrt() * root + eps
    # sqrt(v + ev) - sqrt(v) is at most ev / (2 sqrt(v)) and at most sqrt(ev)
    es = torch.minimum(ev.sqrt(), ev / (2 * v1.sqrt()).clamp_min(1e-300)) * root
    t = gain * m1 / den
    et = (t.abs() * (es / den + 10 * STEP) + gain * em / den) * (1 + es / (den - es).clamp_min(den * 1e-3))
    p1 = p * (1 - lr * decay) - t
    ep = 3 * STEP * p.abs() + et + STEP * t.abs() + TINY
    return p1, m1, v1, ep, em, ev


def groups(t):
    """[groups, GROUP], zeros behind the last element."""
    return torch.nn.functional.pad(t, (0, -t.numel() % GROUP)).view(-1, GROUP)


def wide(step, n):
    return step.double().repeat_interleave(GROUP)[:n]


def m_value(code, step):
    return code.view(torch.float8_e4m3fn).double() * wide(step, code.numel())


def s_value(code, step):
    c = code.long()
    return torch.where(c > 0, (32 + c % 32) * 2.0 ** (c // 32).double(), 0.0) * wide(step, code.numel())


def scales(values, top):
    """The exact steps of groups of 64-bit values."""
    return (groups(values).abs().amax(1) / top).clamp_min(TINY)


def m_slack(m, step):
    """How far the nearest code of m may be off: half a step of e4m3, relative or at its smallest exponent; three fp32
    roundings of the step, its reciprocal and the product move the border."""
    return (2.0 ** -4 * m.abs()).clamp_min(2.0 ** -10 * wide(step, m.numel())) * (1 + 2.0 ** -18) + 8 * STEP * m.abs()


def s_slack(s, step):
    """As m_slack; what lies under the code 1 (33 steps) comes back as that."""
    w = wide(step, s.numel())
    near = 2.0 ** -6 * s * (1 + 2.0 ** -18) + 8 * STEP * s
    return torch.where(s == 0, 0.0, torch.where(s < 33 * w, 33 * w - s + near, near))
