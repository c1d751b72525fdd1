"""Every form of the experts' kernels that the library chooses by size, against
64 bits under bounds that a wrong result exceeds (test_experts_bounds.py shows
what they catch), and values at the ends of their ranges: 4-bit sums beside one
large element, gates far from zero, subnormal rows, offsets past 2^31."""

import numpy as np
import pytest
import torch

import experts_bounds as eb
import experts_inputs as inputs
import experts_ref as ref
from test_gpu_experts import SENTINEL, W4_SHAPES, Case, routed, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_token_amd as ms
    ms.load()


class Block:
    """A plan with rows and weights given; calls that return whole outputs."""

    def __init__(self, counts, H, I, seed):
        import moe_expert_token_amd as ms
        self.ms, self.counts, self.P, self.H, self.I, self.E = ms, counts, sum(counts), H, I, len(counts)
        idx = inputs.ids(counts)
        self.dims = ms.dims_of(self.P, H, self.E, 1, 1)
        self.plan_ws = torch.empty(ms.moe_shuffle_workspace_size(self.dims), dtype=torch.uint8, device="cuda")
        self.plan = ms.moe_shuffle_plan(self.dims, torch.from_numpy(idx).cuda(), self.plan_ws)
        self.offset = np.concatenate([[0], np.cumsum(counts)])
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ws = torch.empty(ms.moe_experts_ffn_workspace_size(self.dims, I, True), dtype=torch.uint8, device="cuda")

    def segments(self):
        return [(e, int(self.offset[e]), int(self.offset[e + 1])) for e in range(self.E) if self.counts[e]]

    def out(self):
        return torch.full((self.P + 1, self.H), SENTINEL, dtype=torch.bfloat16, device="cuda")

    def forward(self, x, w1, w2, act=0, saved=None, scale=None):
        ye = self.out()
        self.ms.moe_experts_ffn_forward(self.plan, x, w1, w2, ye[:self.P], self.ws, saved=saved, saved_scale=scale,
                                        act=act)
        return ye

    def w4(self, x, weights, group, act=0):
        ye = self.out()
        self.ms.moe_experts_ffn_w4_forward(self.plan, x, *weights, ye[:self.P], self.ws, group=group, act=act)
        return ye


def inside(what, ye, lo, hi, r, worst):
    a, b = eb.excess(ye[lo:hi], r["y"], r["e_y"]), eb.row_excess(ye[lo:hi], r["y"], r["n_y"])
    assert a <= 1, f"{what}: an element's error is {a:.3g} of its bound"
    assert b <= 1, f"{what}: a row's error norm is {b:.3g} of its bound"
    worst[0], worst[1] = max(worst[0], a), max(worst[1], b)


def check_saved(what, c, saved, scale, lo, hi, r):
    for which, (v, d) in enumerate(((r["g"], r["e_g"]), (r["u"], r["e_u"]))):
        held = saved[lo:hi, which * c.I:(which + 1) * c.I]
        if scale is None:
            assert eb.excess(held, v, d + ref.U * (v.abs() + d) + ref.TINY) <= 1, f"{what}: saved"
            continue
        step = scale[lo:hi, which].double()
        wide = step.repeat_interleave(32, -1)[:, :c.I]
        # the nearest of the 8-bit values; the reciprocal's and the product's roundings move 127 by 2^-23 each
        assert eb.excess(ref.unpack8(held, scale[lo:hi, which]), v, d + wide * (0.5 + 127 * 2.0 ** -22) + ref.TINY) <= 1, \
            f"{what}: 8 bits"
        pad = torch.nn.functional.pad
        top = pad(v.abs(), (0, -c.I % 32)).unflatten(-1, (-1, 32)).amax(-1)
        dt = pad(d, (0, -c.I % 32)).unflatten(-1, (-1, 32)).amax(-1)
        # the step is the largest / 127 rounded up to bf16: never under it, less than a bf16 step (2^-7) over it
        assert bool((step * 127 >= (top - dt) * (1 - 2.0 ** -23)).all()), what
        assert bool((step * 127 <= (top + dt) * (1 + 2.0 ** -7 + 2.0 ** -22) + 2.0 ** -118).all()), what


@pytest.mark.parametrize("kind", ["dense", "sparse"])
@pytest.mark.parametrize("H,I", inputs.BF16_FORMS)
def test_bf16_streams(H, I, kind):
    act = (H > I) * 1
    say(f"[experts] bf16 streams {H} x {I} {kind}")
    c = Block(inputs.FEW, H, I, H + I)
    x = inputs.rows(kind, c.P, H, I, c.gen, "cuda")
    w1, w2 = inputs.bf16(kind, c.E, H, I, c.gen, "cuda")
    ye = c.forward(x, w1, w2, act)
    held = [(torch.empty((c.P, 2 * I), dtype=torch.bfloat16, device="cuda"), None),
            (torch.empty((c.P, 2 * I), dtype=torch.int8, device="cuda"),
             torch.empty((c.P, 2, -(-I // 32)), dtype=torch.bfloat16, device="cuda"))]
    for saved, scale in held:
        assert torch.equal(c.forward(x, w1, w2, act, saved, scale), ye), "what is saved does not change ye"
    assert bool((ye[c.P:] == SENTINEL).all())
    worst = [0.0, 0.0]
    for e, lo, hi in c.segments():
        r = eb.forward(x[lo:hi].double(), eb.bf16_weights(w1[e]), eb.bf16_weights(w2[e]), act)
        inside(f"expert {e}", ye, lo, hi, r, worst)
        for saved, scale in held:
            check_saved(f"expert {e}", c, saved, scale, lo, hi, r)
    say(f"[experts] bf16 streams {H} x {I} {kind}: of the bounds {worst}")


@pytest.mark.parametrize("kind", ["dense", "sparse"])
@pytest.mark.parametrize("group,rows,k", inputs.W4_FORMS)
def test_w4_forms(group, rows, k, kind):
    counts = inputs.FEW if rows == "few" else inputs.MANY
    for H, I in ((k, 128), (512, k)):
        act = (H > I) * 1
        say(f"[experts] w4 group {group} {rows} rows {H} x {I} {kind}")
        c = Block(counts, H, I, H + I + group)
        x = inputs.rows(kind, c.P, H, I, c.gen, "cuda")
        q1, s1, q2, s2 = inputs.w4(kind, c.E, H, I, group, c.gen, "cuda")
        ye = c.w4(x, (q1, s1, q2, s2), group, act)
        assert bool((ye[c.P:] == SENTINEL).all())
        worst = [0.0, 0.0]
        for e, lo, hi in c.segments():
            r = eb.forward(x[lo:hi].double(), eb.w4_weights(q1[e], s1[e], group), eb.w4_weights(q2[e], s2[e], group), act)
            inside(f"expert {e}", ye, lo, hi, r, worst)
        say(f"[experts] w4 group {group} {rows} rows {H} x {I} {kind}: of the bounds {worst}")


@pytest.mark.parametrize("name,idx,H,I,E,R,group", W4_SHAPES, ids=[s[0].replace(" ", "-") for s in W4_SHAPES])
def test_w4_shapes_under_narrow_bounds(name, idx, H, I, E, R, group):
    """The shapes of test_w4_forward; the bounds count what a group's sum rounds, not 64 terms for each of k."""
    say(f"[experts] w4 narrow {name}")
    c = Case(idx, H, I, E, R, seed=len(name) + 8)
    q1, s1, q2, s2 = inputs.w4("dense", E, H, I, group, c.gen, "cuda")
    whole, ye = c.out(c.P, H)
    act = len(name) % 2
    c.ms.moe_experts_ffn_w4_forward(c.plan, c.xe, q1, s1, q2, s2, ye, c.ws, group=group, act=act)
    worst = [0.0, 0.0]
    for e, lo, hi in c.segments():
        if lo < hi:
            r = eb.forward(c.xe[lo:hi].double(), eb.w4_weights(q1[e], s1[e], group), eb.w4_weights(q2[e], s2[e], group),
                           act)
            inside(f"expert {e}", whole, lo, hi, r, worst)
    say(f"[experts] w4 narrow {name}: of the bounds {worst}")


# ---- 4-bit sums beside a large element ----

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts", [[5, 9], [40, 30]], ids=["few", "many"])
def test_w4_sum_beside_a_large_element(counts, group):
    """One element is 2^18, its weights are all zero (q = 8), the others are odd integers up to 7.  Every product and
    every partial sum, in any order, is an integer below 15 * 2^18 + 128 * 15 * 7 < 2^22, which fp32 holds: a group's
    sum is exact, and the result is that of the other elements alone, within the roundings of scale, h and y."""
    H, I = group, 128
    c = Block(counts, H, I, group)
    q1, s1, q2, s2 = inputs.w4("dense", c.E, H, I, group, c.gen, "cuda")
    at = 2 * (H // 4) + 1  # an odd column: the high four bits
    q1[:, :, at // 2] = (q1[:, :, at // 2] & 15) | 0x80
    x = (torch.randint(-4, 4, (c.P, H), generator=c.gen, device="cuda") * 2 + 1).to(torch.bfloat16)
    small = c.w4(x, (q1, s1, q2, s2), group)
    x[:, at] = 2.0 ** 18
    ye = c.w4(x, (q1, s1, q2, s2), group)
    assert torch.equal(ye[:c.P], c.w4(x, (q1, s1, q2, s2), group)[:c.P])
    for e, lo, hi in c.segments():
        w, _ = eb.w4_weights(q1[e], s1[e], group)
        # one group: its exact sum times the scale, rounded once; eight waves' sums, seven of them zero, are added
        r = eb.forward(x[lo:hi].double(), (w, 2 * eb.STEP * w.abs()), eb.w4_weights(q2[e], s2[e], group), 0)
        exact = x[lo:hi].double() @ w.T
        r_row = (ye[lo:hi].double() - r["y"]).norm(dim=1) / r["n_y"]
        say(f"[experts] w4 beside a large element, group {group}, expert {e}: {float(r_row.max()):.3g} of the row bound, "
            f"sums up to {float(exact.abs().max()):.3g}")
        assert bool((r_row <= 1).all())
    # the large element has no weight: the result is what it is without it (its place held an odd integer of no weight)
    assert torch.equal(ye[:c.P], small[:c.P])


@pytest.mark.parametrize("top", [122, 124])
@pytest.mark.parametrize("counts", [[5, 9], [40, 30]], ids=["few", "many"])
def test_w4_of_large_finite_rows(counts, top):
    """Elements of 2^top with weights of 1 to 7 steps of 2^-(top + 2) (q 9 to 15): g and u are of order 1, and 15 * 2^top
    is inside fp32, for 124 just so (2^128 / 15 is 1.07 * 2^124)."""
    H, I, group = 256, 128, 64
    c = Block(counts, H, I, 3)
    q1, s1, q2, s2 = inputs.w4("dense", c.E, H, I, group, c.gen, "cuda")
    q1 |= 0x88
    q1 = torch.where((q1 & 15) == 8, q1 + 1, q1)
    q1 = torch.where((q1 >> 4) == 8, q1 + 16, q1)
    s1 = torch.full_like(s1, 2.0 ** -(top + 2))
    x = torch.zeros((c.P, H), dtype=torch.bfloat16, device="cuda")
    # one element a group; the fourth group has none
    for i in range(3):
        x[torch.arange(c.P, device="cuda"), 64 * i + (torch.arange(c.P, device="cuda") * 7 + 3 * i) % 64] = 2.0 ** top
    ye = c.w4(x, (q1, s1, q2, s2), group)
    worst = [0.0, 0.0]
    for e, lo, hi in c.segments():
        r = eb.forward(x[lo:hi].double(), eb.w4_weights(q1[e], s1[e], group), eb.w4_weights(q2[e], s2[e], group), 0)
        inside(f"expert {e}", ye, lo, hi, r, worst)
    say(f"[experts] w4 of large rows: of the bounds {worst}")


# ---- gates far from zero ----

@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("rows", [3, 40, 90], ids=["streams", "small-tiles", "tiles"])
def test_far_gates(rows, act):
    """Gates of about +-1e7: act(g) is g or 0, its derivative 1 or 0, in every form of the block."""
    H, I = 64, 32
    c = Case(inputs.ids([rows, rows]), H, I, 2, 1, seed=rows + act)
    c.xe *= 1e4
    c.w1 *= 1e3
    ye, saved, scale = c.forward(act, "bf16")
    got = c.backward(saved, scale, act)
    for e, lo, hi in c.segments():
        x, w1, w2, gy = (t.double() for t in (c.xe[lo:hi], c.w1[e], c.w2[e], c.gy[lo:hi]))
        r = eb.forward(x, eb.bf16_weights(w1), eb.bf16_weights(w2), act)
        inside(f"expert {e}", ye, lo, hi, r, [0.0, 0.0])
        check_saved(f"expert {e}", c, saved, None, lo, hi, r)
        g, u = saved[lo:hi, :I].double(), saved[lo:hi, I:].double()
        b = eb.backward(gy, x, w1, w2, g, u, act)
        for n in ("grad_xe", "grad_w_gate_up", "grad_w_down"):
            mine = got[n][lo:hi] if n == "grad_xe" else got[n][e]
            a = eb.excess(mine, b[n], b["e_" + n])
            d = mine.double() - b[n]
            size = float(((d.norm(dim=1) if n == "grad_xe" else d.norm()) / b["n_" + n]).max())
            assert a <= 1 and size <= 1, (e, n, a, size)


@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("rows", [40, 90], ids=["small-tiles", "tiles"])
def test_closed_gates_stop_large_gradients(rows, act):
    """dh and u are 2^70 each, so dh u passes fp32's range; where the gate is closed (g = -200, act' = 0) dg is 0 all
    the same, and where it is open (g = 200) and u is 2^-70, dg = dh u is 1."""
    H, I = 64, 32
    c = Case(inputs.ids([rows]), H, I, 1, 1, seed=rows)
    g = torch.where(torch.rand((rows, I), device="cuda", generator=c.gen) < 0.5, -200.0, 200.0)
    u = torch.where(g < 0, 2.0 ** 70, 2.0 ** -70)
    saved = torch.cat((g, u), 1).to(torch.bfloat16)
    c.gy.zero_()
    c.gy[:, :I] = 1.0
    c.w2.zero_()
    c.w2[0, :I] = torch.eye(I, device="cuda").to(torch.bfloat16) * 2.0 ** 70  # dh = gy Wd = 2^70
    c.xe.zero_()
    c.xe[torch.arange(rows), torch.arange(rows) % H] = 1.0
    got = c.backward(saved, None, act, want=("grad_w_gate_up",))["grad_w_gate_up"][0]
    want = torch.zeros((I, H), dtype=torch.float64, device="cuda")
    want.index_add_(1, torch.arange(rows, device="cuda") % H, (g > 0).double().T)
    assert torch.equal(got[:I].double(), want)  # small whole numbers: exact


# ---- subnormal rows ----

def test_pack8_of_subnormals_that_round_to_one_step():
    """Magnitudes between 2^-127 and 2^-126 with the least step, 2^-126: q is +-1, or 0 at 2^-127 itself (a tie)."""
    import moe_expert_token_amd as ms
    k = torch.arange(64, 128, device="cuda").repeat(3, 2)[:, :96]  # x = k 2^-133
    sign = torch.where(torch.arange(96, device="cuda") % 3 == 0, -1.0, 1.0)
    x = (k.double() * 2.0 ** -133 * sign).to(torch.bfloat16)
    assert bool(((x.double() * 2.0 ** 133).abs() == k).all())
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty((3, 3), dtype=torch.bfloat16, device="cuda")
    back = torch.empty_like(x)
    ms.moe_experts_pack8(x, q, s)
    ms.moe_experts_unpack8(q, s, back)
    assert bool((s.double() == 2.0 ** -126).all())
    want = torch.where(k > 64, sign.expand(3, -1), 0.0)
    assert torch.equal(q.double(), want.double())
    assert torch.equal(back.double(), want.double() * 2.0 ** -126)


@pytest.mark.parametrize("rows", [3, 40, 90], ids=["streams", "small-tiles", "tiles"])
def test_subnormal_rows_through_the_block(rows):
    """Rows of k 2^-133 with weights of order 2^124: g and u are of order 1 and a little above."""
    H, I = 128, 64
    c = Case(inputs.ids([rows, rows]), H, I, 2, 1, seed=rows)
    k = torch.randint(-127, 128, (c.P, H), device="cuda", generator=c.gen)
    c.xe = (k.double() * 2.0 ** -133).to(torch.bfloat16)
    assert bool((c.xe.double() * 2.0 ** 133 == k).all())
    c.w1 = (c.w1.float() * 2.0 ** 127).to(torch.bfloat16)
    ye, _, _ = c.forward(0)
    for e, lo, hi in c.segments():
        r = eb.forward(c.xe[lo:hi].double(), eb.bf16_weights(c.w1[e]), eb.bf16_weights(c.w2[e]), 0)
        assert float(r["g"].abs().mean()) > 0.1
        inside(f"expert {e}", ye, lo, hi, r, [0.0, 0.0])


@pytest.mark.parametrize("counts", [[5, 9], [40, 30]], ids=["few", "many"])
def test_subnormal_rows_with_4_bit_weights(counts):
    H, I, group = 128, 128, 32
    c = Block(counts, H, I, 9)
    q1, s1, q2, s2 = inputs.w4("dense", c.E, H, I, group, c.gen, "cuda")
    s1 = (s1.float() * 2.0 ** 127).to(torch.bfloat16)
    k = torch.randint(-127, 128, (c.P, H), device="cuda", generator=c.gen)
    x = (k.double() * 2.0 ** -133).to(torch.bfloat16)
    ye = c.w4(x, (q1, s1, q2, s2), group)
    for e, lo, hi in c.segments():
        w1, m1 = eb.w4_weights(q1[e], s1[e], group)
        # a group's sum is a multiple of 2^-133 far below 2^-119: fp32 holds it without rounding (24 bits from 2^-149)
        r = eb.forward(x[lo:hi].double(), (w1, m1), eb.w4_weights(q2[e], s2[e], group), 0)
        assert float(r["g"].abs().mean()) > 0.1
        inside(f"expert {e}", ye, lo, hi, r, [0.0, 0.0])


# ---- a row's own result ----

@pytest.mark.parametrize("T", [8, 120, 400], ids=["streams", "small-tiles", "tiles"])
def test_a_row_depends_on_itself_and_its_experts_weights(T):
    """The same row as expert 0's only one, as one in the middle and as its last of T: the same bits in ye, in what is
    saved, in grad_xe and with 4-bit weights (the number of tokens and experts is the same, so is the form)."""
    H, I, E = 328, 200, 4
    row = grad = weights = None
    seen = []
    for counts in ([1, T - 3, 1, 1], [T // 2 + 1, 0, T - T // 2 - 1, 0], [T, 0, 0, 0]):
        c = Case(inputs.ids(counts), H, I, E, 2, seed=sum(counts[:2]))
        if row is None:
            row, grad, weights = c.xe[0].clone(), c.gy[0].clone(), (c.w1, c.w2)
        at = {1: 0, T: T - 1}.get(counts[0], T // 4)
        c.xe[at], c.gy[at], (c.w1, c.w2) = row, grad, weights
        ye, saved, scale = c.forward(1, "int8")
        got = c.backward(saved, scale, 1, want=("grad_xe",))["grad_xe"]
        seen.append([t[at].clone() for t in (ye, saved, scale, got)])
    for other in seen[1:]:
        for a, b in zip(seen[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [8, 120], ids=["few", "many"])
def test_a_row_with_4_bit_weights_depends_on_itself(T):
    H, I, group = 544, 256, 32
    row = weights = None
    seen = []
    for counts in ([1, T - 3, 1, 1], [T // 2 + 1, 0, T - T // 2 - 1, 0], [T, 0, 0, 0]):
        c = Block(counts, H, I, 4)
        x = inputs.rows("dense", T, H, I, c.gen, "cuda")
        if row is None:
            row, weights = x[0].clone(), inputs.w4("dense", 4, H, I, group, c.gen, "cuda")
        at = {1: 0, T: T - 1}.get(counts[0], T // 4)
        x[at] = row
        seen.append(c.w4(x, weights, group)[at].clone())
    assert torch.equal(seen[0], seen[1]) and torch.equal(seen[0], seen[2])


# ---- offsets past 2^31 bytes ----

@pytest.mark.parametrize("rows", [3, 20, 70], ids=["streams", "small-tiles", "tiles"])
def test_weights_past_two_gigabytes(rows):
    """136 experts of 4096 x 2048: the last ones' weights lie past 2^31 (down) and 2^32 bytes (up)."""
    H, I, E = 4096, 2048, 136
    say(f"[experts] {rows} rows an expert, 4.6 GB of weights")
    c = Case(inputs.ids([rows] * E), H, I, E, 1, seed=rows)
    assert c.w2[-1].data_ptr() - c.w2.data_ptr() > 1 << 31 and c.w1[-1].data_ptr() - c.w1.data_ptr() > 1 << 32
    ye, saved, scale = c.forward(0, "bf16")
    got = c.backward(saved, scale) if rows > 3 else None
    for e in (0, E // 2, E - 1):
        lo, hi = int(c.offset[e]), int(c.offset[e + 1])
        x, w1, w2, gy = (t.double() for t in (c.xe[lo:hi], c.w1[e], c.w2[e], c.gy[lo:hi]))
        r = eb.forward(x, eb.bf16_weights(w1), eb.bf16_weights(w2), 0)
        inside(f"expert {e}", ye, lo, hi, r, [0.0, 0.0])
        if got is None:
            continue
        b = eb.backward(gy, x, w1, w2, saved[lo:hi, :I].double(), saved[lo:hi, I:].double(), 0)
        for n in got:
            mine = got[n][lo:hi] if n == "grad_xe" else got[n][e]
            a = eb.excess(mine, b[n], b["e_" + n])
            d = mine.double() - b[n]
            size = float(((d.norm(dim=1) if n == "grad_xe" else d.norm()) / b["n_" + n]).max())
            assert a <= 1 and size <= 1, (e, n, a, size)


def test_4_bit_weights_past_two_gigabytes():
    H, I, E, group = 4096, 4096, 144, 128
    say("[experts] 3.6 GB of 4-bit weights")
    c = Block([2] * E, H, I, 5)
    q1, s1, q2, s2 = inputs.w4("dense", E, H, I, group, c.gen, "cuda")
    assert q1[-1].data_ptr() - q1.data_ptr() > 1 << 31
    x = inputs.rows("dense", c.P, H, I, c.gen, "cuda")
    ye = c.w4(x, (q1, s1, q2, s2), group)
    for e in (0, E // 2, E - 1):
        lo, hi = int(c.offset[e]), int(c.offset[e + 1])
        r = eb.forward(x[lo:hi].double(), eb.w4_weights(q1[e], s1[e], group), eb.w4_weights(q2[e], s2[e], group), 0)
        inside(f"expert {e}", ye, lo, hi, r, [0.0, 0.0])


def test_rows_past_two_gigabytes():
    """300000 rows of 4096: xe, ye and grad_xe pass 2^31 bytes; and of what is saved, 2I = 4096."""
    H, I, E = 4096, 2048, 4
    T = 300000
    c = Case(routed(T, E, 1, seed=2), H, I, E, 1, seed=6)
    say("[experts] 300000 rows")
    ye, saved, scale = c.forward(0, "bf16")
    got = c.backward(saved, scale, want=("grad_xe",))["grad_xe"]
    assert bool((ye[T:] == SENTINEL).all()) and bool((got[T:] == SENTINEL).all())
    for lo in (0, T // 2, T - 40):
        for i in (lo, lo + 39):
            e = int(np.searchsorted(c.offset, i, side="right")) - 1
            x, w1, w2, gy = (t.double() for t in (c.xe[i:i + 1], c.w1[e], c.w2[e], c.gy[i:i + 1]))
            r = eb.forward(x, eb.bf16_weights(w1), eb.bf16_weights(w2), 0)
            inside(f"row {i}", ye, i, i + 1, r, [0.0, 0.0])
            b = eb.backward(gy, x, w1, w2, saved[i:i + 1, :I].double(), saved[i:i + 1, I:].double(), 0)
            assert eb.excess(got[i:i + 1], b["grad_xe"], b["e_grad_xe"]) <= 1
            assert eb.row_excess(got[i:i + 1], b["grad_xe"], b["n_grad_xe"]) <= 1
