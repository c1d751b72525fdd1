"""The bounds of the experts' block catch mistakes (CPU): results of zero,
chunks of a sum left out, scales of other groups, neighbours swapped, gates
without saturation.  Each planted mistake is one of the definition's copies,
never of a kernel."""

import pytest
import torch

import experts_bounds as eb
import experts_inputs as inputs
import experts_ref as ref

# (H, I, group): each has the long sum of its side in parts that the GPU tests' longer ones repeat
SIZES = [(512, 256, 0), (4096, 256, 0), (256, 4096, 0), (136, 1096, 0), (512, 128, 32), (544, 128, 32), (128, 544, 32),
         (4224, 1920, 128), (1056, 544, 32), (4096, 128, 64), (512, 4160, 64), (256, 384, 128)]


def case(kind, H, I, group, act, P=37):
    gen = torch.Generator().manual_seed(H + I + group)
    x = inputs.rows(kind, P, H, I, gen, "cpu").double()
    if not group:
        w1, w2 = inputs.bf16(kind, 1, H, I, gen, "cpu")
        return x, eb.bf16_weights(w1[0]), eb.bf16_weights(w2[0])
    q1, s1, q2, s2 = inputs.w4(kind, 1, H, I, group, gen, "cpu")
    return x, (q1[0], s1[0]), (q2[0], s2[0])


@pytest.mark.parametrize("H,I,group", SIZES)
def test_mistakes_in_the_sums_exceed_the_bounds(H, I, group):
    left = None
    for kind in ("dense", "sparse"):
        x, up, down = case(kind, H, I, group, 0)
        if group:
            raw = up, down
            up, down = (eb.w4_weights(*t, group) for t in raw)
        r = eb.forward(x, up, down, 0)
        # what the definition gives, rounded as a kernel may, is inside: h and y to bf16
        h = r["h"].to(torch.bfloat16).double()
        good = (h @ down[0].T).to(torch.bfloat16)
        assert not inputs.caught(good, r)
        wrong = inputs.mistakes(x, up, down, 0)
        if group:
            for i, side in enumerate(("up", "down")):
                q, s = raw[i]
                if s.shape[1] > 1:
                    other = ref.four_bit(q, s.roll(1, 1), group)
                    both = [up[0], down[0]]
                    both[i] = other
                    wrong[f"{side}: scales of the group before"] = \
                        eb.forward(x, (both[0], both[0]), (both[1], both[1]), 0)["y"]
        missed = {n for n, y in wrong.items() if not inputs.caught(y, r)}
        assert "zero" not in missed, kind
        left = missed if left is None else left & missed
    assert not left, left


def far(act, gen):
    """Rows and weights whose gates lie far from zero on either side."""
    n, H, I = 40, 64, 32
    x = torch.randn((n, H), generator=gen, dtype=torch.float64) * 1e4
    w1 = torch.randn((2 * I, H), generator=gen, dtype=torch.float64) * 125
    w2 = torch.randn((H, I), generator=gen, dtype=torch.float64) / 6
    gy = torch.randn((n, H), generator=gen, dtype=torch.float64)
    return tuple(t.to(torch.bfloat16).double() for t in (x, w1, w2, gy))


@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
def test_mistakes_far_from_zero_exceed_the_bounds(act):
    x, w1, w2, gy = far(act, torch.Generator().manual_seed(act))
    up, down = eb.bf16_weights(w1), eb.bf16_weights(w2)
    r = eb.forward(x, up, down, act)
    assert not inputs.caught((r["h"].to(torch.bfloat16).double() @ w2.T).to(torch.bfloat16), r)
    assert inputs.caught(torch.zeros_like(r["y"]), r)
    # a gate that is zero for large g, and one that does not close for far negative ones
    assert inputs.caught((r["h"] * (r["g"].abs() < 64)) @ w2.T, r)
    assert inputs.caught((r["g"] * r["u"]) @ w2.T, r)
    g, u = r["g"], r["u"]
    b = eb.backward(gy, x, w1, w2, g, u, act)
    for n in ("grad_xe", "grad_w_gate_up", "grad_w_down"):
        assert eb.excess(torch.zeros_like(b[n]), b[n], b["e_" + n]) > 1, n
    # a derivative lost in saturation: dg = 0
    lost = eb.backward(gy, x, w1, w2, g, u, act)["grad_w_gate_up"].clone()
    lost[:w2.shape[1]] = 0
    assert eb.excess(lost, b["grad_w_gate_up"], b["e_grad_w_gate_up"]) > 1


@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
def test_gate_bounds_hold_for_32_bits(act):
    """The gate computed in fp32 with torch's exp stays inside its bounds, far out too, and they are narrow there."""
    g = torch.cat((torch.linspace(-130, 130, 20001), torch.logspace(1, 30, 200), -torch.logspace(1, 30, 200))).float()
    a, d, ea, ed = eb.gate(g.double(), act)
    c0, c1 = ref.slope(act)
    t = g.clamp(-64, 64)
    s = 1 / (1 + torch.exp(-(c0 * g + c1 * t * t * t)))
    assert bool(((g * s).double() - a).abs().le(ea).all())
    mine = s + g * s * (1 - s) * (c0 + 3 * c1 * t * t)
    assert bool((mine.double() - d).abs().le(ed).all())
    out = g.abs() > 200
    assert bool((ea[out] <= a[out].abs() * 2.0 ** -22 + g[out].double().abs() * 2.0 ** -125).all())
    assert bool((ed[out] <= 2.0 ** -21).all())


def test_norm_bound():
    gen = torch.Generator().manual_seed(1)
    for shape in ((5, 9), (200, 40), (64, 300), (1, 7)):
        w = torch.randn(shape, generator=gen, dtype=torch.float64) * 1e-3
        n = float(torch.linalg.matrix_norm(w, 2))
        assert n * (1 - 1e-12) <= eb.norm_bound(w) <= n * min(shape) ** (1 / 32) * (1 + 1e-12)
    assert eb.norm_bound(torch.zeros((3, 4), dtype=torch.float64)) == 0
    assert eb.norm_bound(torch.zeros((0, 4), dtype=torch.float64)) == 0
