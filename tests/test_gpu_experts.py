"""The experts' block on the MI355X against its 64-bit reference: every
product at ragged shapes, single rows, empty and crowded experts, rows that
hold NaN, 8-bit checkpoints, 4-bit weights, streams, graphs and refusals."""

import numpy as np
import pytest
import torch

import experts_ref as ref
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_token_amd as ms
    ms.load()


SENTINEL = -12345.0  # exact in bf16; no output of these tests comes near it


def say(*a):
    print(*a, flush=True)


def bf16(gen, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=gen)


class Case:
    """A plan on given ids, with rows and weights of its own seed."""

    def __init__(self, idx, H, I, E, R, seed=0):
        import moe_expert_token_amd as ms
        self.ms = ms
        self.T, self.k = idx.shape
        self.P, self.H, self.I, self.E = idx.size, H, I, E
        self.dims = ms.dims_of(self.T, H, E, self.k, R)
        self.plan_ws = torch.empty(ms.moe_shuffle_workspace_size(self.dims), dtype=torch.uint8, device="cuda")
        self.idx = torch.from_numpy(np.ascontiguousarray(idx)).cuda()
        self.plan = ms.moe_shuffle_plan(self.dims, self.idx, self.plan_ws)
        self.offset = np.concatenate([[0], np.cumsum(np.bincount(idx.ravel(), minlength=E))])
        gen = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.xe = bf16(gen, self.P, H)
        self.gy = bf16(gen, self.P, H)
        self.w1 = bf16(gen, E, 2 * I, H, std=H ** -0.5)
        self.w2 = bf16(gen, E, H, I, std=I ** -0.5)
        self.ws = torch.empty(ms.moe_experts_ffn_workspace_size(self.dims, I, True), dtype=torch.uint8, device="cuda")

    def out(self, *shape, dtype=torch.bfloat16):
        """An output with a row more than is written, all of a value that no call writes."""
        t = torch.full((shape[0] + 1,) + shape[1:], SENTINEL if dtype == torch.bfloat16 else 77, dtype=dtype,
                       device="cuda")
        return t, t[:shape[0]]

    def held(self, kind):
        if kind is None:
            return None, None
        if kind == "bf16":
            return torch.empty((self.P, 2 * self.I), dtype=torch.bfloat16, device="cuda"), None
        return (torch.empty((self.P, 2 * self.I), dtype=torch.int8, device="cuda"),
                torch.empty((self.P, 2, -(-self.I // 32)), dtype=torch.bfloat16, device="cuda"))

    def forward(self, act=0, kind=None, **kw):
        saved, scale = self.held(kind)
        whole, ye = self.out(self.P, self.H)
        self.ms.moe_experts_ffn_forward(self.plan, self.xe, self.w1, self.w2, ye, self.ws, saved=saved,
                                        saved_scale=scale, act=act, **kw)
        return whole, saved, scale

    def backward(self, saved, scale, act=0, want=("grad_xe", "grad_w_gate_up", "grad_w_down"), **kw):
        pair = {"grad_xe": self.out(self.P, self.H), "grad_w_gate_up": self.out(self.E, 2 * self.I, self.H),
                "grad_w_down": self.out(self.E, self.H, self.I)}
        arg = {n: pair[n][1] if n in want else None for n in pair}
        self.ms.moe_experts_ffn_backward(self.plan, self.gy, self.xe, self.w1, self.w2, saved, arg["grad_xe"],
                                         arg["grad_w_gate_up"], arg["grad_w_down"], self.ws, saved_scale=scale,
                                         act=act, **kw)
        return {n: pair[n][0] for n in want}

    def segments(self):
        return [(e, int(self.offset[e]), int(self.offset[e + 1])) for e in range(self.E)]


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.3g} of the bound"
    return worst


def check_forward(c, ye, act, saved=None, scale=None, w1=None, w2=None, terms=(None, None)):
    w1, w2 = c.w1 if w1 is None else w1, c.w2 if w2 is None else w2
    assert bool((ye[c.P:] == SENTINEL).all()), "a row past the last was written"
    worst = [0.0, 0.0]
    for e, lo, hi in c.segments():
        if lo == hi:
            continue
        r = ref.forward(c.xe[lo:hi].double(), w1[e].double(), w2[e].double(), act, *terms)
        worst[0] = max(worst[0], within(ye[lo:hi], r["y"], r["e_y"], f"expert {e} y"))
        norm = (ye[lo:hi].double() - r["y"]).norm(dim=1)
        worst[1] = max(worst[1], float((norm / r["n_y"]).max()))
        assert worst[1] <= 1, f"expert {e}: a row's error norm is {worst[1]:.3g} of its bound"
        if saved is None:
            continue
        pre, err = torch.cat((r["g"], r["u"]), 1), torch.cat((r["e_g"], r["e_u"]), 1)
        if scale is None:
            within(saved[lo:hi], pre, err + ref.U * (pre.abs() + err) + ref.TINY, f"expert {e} saved")
            continue
        for which in range(2):
            v, d = pre[:, which * c.I:(which + 1) * c.I], err[:, which * c.I:(which + 1) * c.I]
            q, step = saved[lo:hi, which * c.I:(which + 1) * c.I], scale[lo:hi, which]
            wide = step.double().repeat_interleave(32, -1)[:, :c.I]
            # the nearest of the 8-bit values, with the roundings of the reciprocal and the product
            within(ref.unpack8(q, step), v, d + wide * (0.5 + 127 * 2.0 ** -23), f"expert {e} 8-bit")
            pad = -c.I % 32
            top = torch.nn.functional.pad(v.abs(), (0, pad)).unflatten(-1, (-1, 32)).amax(-1)
            dt = torch.nn.functional.pad(d, (0, pad)).unflatten(-1, (-1, 32)).amax(-1)
            # a step is at least its group's largest / 127 and less than a bf16 step above it
            assert bool((step.double() * 127 >= (top - dt) * (1 - 2.0 ** -23)).all())
            assert bool((step.double() * 127 <= (top + dt) * (1 + 2.0 ** -7 + 2.0 ** -23) + 2.0 ** -118).all())
    return worst


def check_backward(c, got, saved, scale, act):
    want_names = list(got)
    for n, rows in (("grad_xe", c.P), ("grad_w_gate_up", c.E), ("grad_w_down", c.E)):
        if n in got:
            assert bool((got[n][rows:] == SENTINEL).all()), f"{n}: written past its end"
    worst = {}
    for e, lo, hi in c.segments():
        if lo == hi:
            for n in want_names:
                if n != "grad_xe":
                    assert bool((got[n][e] == 0).all()), f"expert {e} has no rows: {n} must be zero"
            continue
        if scale is None:
            pre = saved[lo:hi].double()
        else:
            pre = torch.cat([ref.unpack8(saved[lo:hi, i * c.I:(i + 1) * c.I], scale[lo:hi, i]) for i in range(2)], 1)
        r = ref.backward(c.gy[lo:hi].double(), c.xe[lo:hi].double(), c.w1[e].double(), c.w2[e].double(),
                         pre[:, :c.I], pre[:, c.I:], act)
        for n in want_names:
            mine = got[n][lo:hi] if n == "grad_xe" else got[n][e]
            a = within(mine, r[n], r["e_" + n], f"expert {e} {n}")
            d = mine.double() - r[n]
            b = float(((d.norm(dim=1) if n == "grad_xe" else d.norm()) / r["n_" + n]).max())
            assert b <= 1, f"expert {e} {n}: error norm {b:.3g} of its bound"
            worst[n] = max(worst.get(n, 0.0), a, b)
    return worst


def crowd(counts, k=1):
    """Ids that give expert e counts[e] rows (top-1), the tokens shuffled."""
    ids = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    np.random.default_rng(len(ids)).shuffle(ids)
    return ids.reshape(-1, k)


def routed(T, E, k, seed=0):
    return synth.random_routing(np.random.default_rng(seed), T, E, k)[0]


# name, ids, H, I, E, R
SHAPES = [
    ("one row", crowd([0, 1, 0, 0]), 64, 32, 4, 2),
    ("smallest widths", routed(9, 4, 2), 8, 8, 4, 2),
    ("one wide chunk more", routed(40, 4, 2), 72, 40, 4, 2),
    ("odd widths", routed(100, 6, 3), 200, 104, 6, 3),
    ("one expert", routed(300, 1, 1), 128, 96, 1, 1),
    ("all on the last", crowd([0, 0, 0, 333]), 136, 72, 4, 4),
    ("tile edges", crowd([255, 256, 257, 1, 0, 511, 513, 15, 16, 17]), 264, 136, 10, 5),
    ("small tile edges", crowd([63, 64, 65, 127, 128, 129, 31, 32, 33, 95, 97, 191, 193]), 512, 256, 13, 13),
    ("few rows each", crowd([1, 2, 3, 0, 5, 8, 13, 16, 17, 20]), 1032, 520, 10, 2),
    ("top-8 of 64", routed(150, 64, 8), 256, 264, 64, 8),
    ("long sums", routed(70, 4, 2), 2304, 1288, 4, 2),
    ("many rows", routed(2100, 4, 2), 320, 192, 4, 2),
    ("wide experts", routed(600, 3, 1), 1024, 776, 3, 3),
    # tile heights other than 256 and 64 are taken where they make the rounds of blocks come out better
    ("shorter tiles", routed(1500, 16, 4), 136, 1000, 16, 4),
    ("shorter tiles of rows", routed(4096, 8, 2), 4096, 72, 8, 8),
]
IDS = [s[0].replace(" ", "-") for s in SHAPES]


@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("name,idx,H,I,E,R", SHAPES, ids=IDS)
def test_forward(name, idx, H, I, E, R, act):
    say(f"[experts] forward {name}")
    c = Case(idx, H, I, E, R, seed=len(name))
    ye, _, _ = c.forward(act)
    say(f"[experts] forward {name}: of the bounds {check_forward(c, ye, act)}")
    for kind in ("bf16", "int8"):
        again, saved, scale = c.forward(act, kind)
        assert torch.equal(again, ye), "what is saved does not change ye"
        check_forward(c, again, act, saved, scale)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("name,idx,H,I,E,R", SHAPES, ids=IDS)
def test_backward(name, idx, H, I, E, R, kind):
    act = len(name) % 2
    say(f"[experts] backward {name} {kind}")
    c = Case(idx, H, I, E, R, seed=len(name) + 100)
    _, saved, scale = c.forward(act, kind)
    got = c.backward(saved, scale, act)
    say(f"[experts] backward {name} {kind}: of the bounds {check_backward(c, got, saved, scale, act)}")
    # each gradient alone is the same gradient
    for n in got:
        alone = c.backward(saved, scale, act, want=(n,))
        assert torch.equal(alone[n], got[n]), n


def test_backward_matches_differences_of_forward():
    """The directional derivative that the gradients give against central differences of the 64-bit forward pass."""
    c = Case(routed(60, 4, 2), 96, 64, 4, 2, seed=5)
    _, saved, scale = c.forward(0, "bf16")
    got = c.backward(saved, scale)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for e, lo, hi in c.segments():
        x, w1, w2, gy = (t.double() for t in (c.xe[lo:hi], c.w1[e], c.w2[e], c.gy[lo:hi]))
        for n, t, mine in (("x", x, got["grad_xe"][lo:hi]), ("w1", w1, got["grad_w_gate_up"][e]),
                           ("w2", w2, got["grad_w_down"][e])):
            v = torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)
            eps, loss = 1e-5, []
            for sign in (1, -1):
                m = {k: a + sign * eps * v if k == n else a for k, a in (("x", x), ("w1", w1), ("w2", w2))}
                loss.append(float((ref.forward(m["x"], m["w1"], m["w2"], 0)["y"] * gy).sum()))
            want, have = (loss[0] - loss[1]) / (2 * eps), float((mine.double() * v).sum())
            # Roundings to bf16 (g and u as saved, then dg, du or h, then the gradient), each at most 2^-8 of its
            # value: a relative error of the gradient of under 4 * 2^-8 of the norms, taken along v whose
            # entries are N(0, 1): |<err, v>| <= 6 |err| but for 2e-9 of the draws.
            f = ref.backward(gy, x, w1, w2, ref.forward(x, w1, w2, 0)["g"], ref.forward(x, w1, w2, 0)["u"], 0)
            size = {"x": f["n_grad_xe"].norm(), "w1": f["n_grad_w_gate_up"], "w2": f["n_grad_w_down"]}[n]
            assert abs(want - have) <= 6 * 2 * float(size), (e, n, want, have)


def test_no_tokens_writes_zero_weight_gradients_only():
    c = Case(np.zeros((0, 2), np.int32), 64, 32, 4, 2)
    ye, saved, scale = c.forward(0, "int8")
    assert bool((ye == SENTINEL).all())
    got = c.backward(saved, scale)
    for n in ("grad_w_gate_up", "grad_w_down"):
        assert bool((got[n][:4] == 0).all()) and bool((got[n][4:] == SENTINEL).all())
    assert bool((got["grad_xe"] == SENTINEL).all())


def test_bad_ids_write_nothing():
    idx = routed(50, 8, 2)
    good = Case(idx, 64, 32, 8, 4)
    idx = idx.copy()
    idx[7, 1] = 8
    c = Case(routed(50, 8, 2), 64, 32, 8, 4)
    c.plan = c.ms.moe_shuffle_plan(c.dims, torch.from_numpy(idx).cuda(), c.plan_ws)
    saved, scale = torch.full((100, 64), 5, dtype=torch.int8, device="cuda"), good.held("int8")[1]
    whole, ye = c.out(c.P, c.H)
    c.ms.moe_experts_ffn_forward(c.plan, c.xe, c.w1, c.w2, ye, c.ws, saved=saved, saved_scale=scale)
    assert bool((whole == SENTINEL).all()) and bool((saved == 5).all())
    for t in c.backward(saved, scale).values():
        assert bool((t == SENTINEL).all())
    q1, s1, q2, s2 = four_bit_weights(c, 32)
    c.ms.moe_experts_ffn_w4_forward(c.plan, c.xe, q1, s1, q2, s2, ye, c.ws, group=32)
    assert bool((whole == SENTINEL).all())


@pytest.mark.parametrize("counts", [[3, 2, 4], [70, 65, 300]], ids=["few", "many"])
def test_rows_and_experts_do_not_reach_each_other(counts):
    """NaN and infinite rows of one expert, and its NaN weights, leave every other expert's results as they were;
    a NaN row leaves the other rows of its own expert."""
    c = Case(crowd(counts), 136, 72, 3, 3, seed=2)
    ye, saved, scale = c.forward(0, "int8")
    grads = c.backward(saved, scale)
    lo, hi = int(c.offset[1]), int(c.offset[2])
    c.xe[lo] = float("nan")
    c.xe[lo + 1] = float("inf")
    c.gy[lo] = float("nan")
    ye2, saved2, scale2 = c.forward(0, "int8")
    grads2 = c.backward(saved2, scale2)
    rest = [i for i in range(c.P) if i not in (lo, lo + 1)]
    assert torch.equal(ye2[rest], ye[rest]) and bool(ye2[lo].isnan().all()) and not bool(ye2[lo + 1].isfinite().any())
    assert torch.equal(saved2[rest], saved[rest]) and torch.equal(scale2[rest], scale[rest])
    assert bool(scale2[lo].isnan().all()) and bool((saved2[lo] == 0).all())
    assert torch.equal(grads2["grad_xe"][rest], grads["grad_xe"][rest])
    for n in ("grad_w_gate_up", "grad_w_down"):
        assert torch.equal(grads2[n][0], grads[n][0]) and torch.equal(grads2[n][2], grads[n][2])
        assert bool(grads2[n][1].isnan().all())
    c.w1[1] = float("nan")
    c.w2[1] = float("nan")
    ye3, saved3, scale3 = c.forward(0, "int8")
    rest = [i for i in range(c.P) if not lo <= i < hi]
    assert torch.equal(ye3[rest], ye[rest]) and bool(ye3[lo:hi].isnan().all())
    assert torch.equal(c.backward(saved3, scale3)["grad_xe"][rest], grads["grad_xe"][rest])


def test_far_pre_activations():
    """Gates far from zero: the sigmoid is 0 or 1, the cubic of GELU overflows, nothing becomes NaN."""
    for act in (0, 1):
        c = Case(crowd([40, 3]), 64, 32, 2, 2, seed=3)
        c.xe *= 1e4
        c.w1 *= 1e3
        ye, saved, scale = c.forward(act, "bf16")
        check_forward(c, ye, act, saved, scale)
        got = c.backward(saved, scale, act)
        check_backward(c, got, saved, scale, act)


def test_subnormal_rows():
    """bf16 subnormals are values, not zeros: a row scaled by 2^-130 comes back scaled."""
    c = Case(crowd([20]), 64, 32, 1, 1, seed=4)
    small = (c.xe.double() * 2.0 ** -130).to(torch.bfloat16)
    assert bool((small != 0).any())
    c.xe = small.contiguous()
    q, s = torch.empty(c.xe.shape, dtype=torch.int8, device="cuda"), \
        torch.empty((c.P, 2), dtype=torch.bfloat16, device="cuda")
    c.ms.moe_experts_pack8(c.xe, q, s)
    rq, rs = ref.pack8(c.xe.float().cpu())
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


# ---- 8-bit checkpoints on their own ----

@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 32), (3, 40), (5, 104), (64, 1024), (257, 72), (33, 7168),
                                       (1000, 24)])
def test_pack8(rows, cols):
    import moe_expert_token_amd as ms
    say(f"[experts] pack8 {rows} x {cols}")
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = bf16(gen, rows, cols) * torch.logspace(-30, 30, rows, device="cuda")[:, None].to(torch.bfloat16)
    x[rows // 2, : min(32, cols)] = 0
    groups = -(-cols // 32)
    q = torch.full((rows + 1, cols), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1, groups), SENTINEL, dtype=torch.bfloat16, device="cuda")
    back = torch.full((rows + 1, cols), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ms.moe_experts_pack8(x, q[:rows], s[:rows])
    ms.moe_experts_unpack8(q[:rows], s[:rows], back[:rows])
    rq, rs = ref.pack8(x.float().cpu())
    assert torch.equal(q[:rows].cpu(), rq) and torch.equal(s[:rows].cpu(), rs)
    want = ref.unpack8(rq, rs).float().to(torch.bfloat16)  # int8 * bf16 is exact in fp32
    assert torch.equal(back[:rows].cpu(), want)
    assert bool((q[rows:] == 77).all()) and bool((s[rows:] == SENTINEL).all()) and bool((back[rows:] == SENTINEL).all())


def test_pack8_of_what_is_not_finite_and_of_the_largest():
    import moe_expert_token_amd as ms
    x = torch.randn((4, 96), device="cuda").to(torch.bfloat16)
    x[0, 40], x[1, 5], x[1, 95] = float("nan"), float("inf"), float("-inf")
    x[2, :32] = torch.finfo(torch.bfloat16).max
    x[3, 64:] = 2.0 ** -133
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty((4, 3), dtype=torch.bfloat16, device="cuda")
    back = torch.empty_like(x)
    ms.moe_experts_pack8(x, q, s)
    ms.moe_experts_unpack8(q, s, back)
    rq, rs = ref.pack8(x.float().cpu())
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu().isnan(), rs.isnan())
    assert torch.equal(s.cpu().nan_to_num(7.0), rs.nan_to_num(7.0))
    for r, g in ((0, 1), (1, 0), (1, 2)):
        assert bool(back[r, 32 * g:32 * g + 32].isnan().all())
    assert int(back.isnan().sum()) == 96
    assert bool(back[2, :32].isfinite().all()) and float((back[2, :32].double() / x[2, :32].double() - 1).abs().max()) < 2.0 ** -7


# ---- 4-bit weights ----

def four_bit_weights(c, group):
    """Random 4-bit values, every one of the sixteen among them, and scales of either sign."""
    gen = c.gen
    q = [torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=gen)
         for s in ((c.E, 2 * c.I, c.H // 2), (c.E, c.H, c.I // 2))]
    s = [((torch.rand(t, device="cuda", generator=gen) + 0.5) / (4.6 * w ** 0.5) *
          torch.where(torch.rand(t, device="cuda", generator=gen) < 0.1, -1.0, 1.0)).to(torch.bfloat16)
         for t, w in (((c.E, 2 * c.I, c.H // group), c.H), ((c.E, c.H, c.I // group), c.I))]
    return q[0], s[0], q[1], s[1]


W4_SHAPES = [
    ("one row", crowd([0, 1, 0, 0]), 64, 32, 4, 2, 32),
    ("one group", routed(3, 4, 2), 128, 128, 4, 2, 128),
    ("one token", routed(1, 16, 8), 512, 256, 16, 4, 128),
    ("small groups", routed(17, 8, 2), 224, 96, 8, 2, 32),
    ("middle groups", routed(33, 8, 3), 320, 192, 8, 4, 64),
    ("row edges", crowd([15, 16, 17, 31, 32, 33, 0, 47, 48, 49, 64, 65, 1]), 384, 160, 13, 13, 32),
    ("odd chunks", routed(20, 6, 2), 1056, 544, 6, 2, 32),
    ("long sums", routed(12, 4, 2), 4224, 1920, 4, 2, 128),
    ("crowded", crowd([0, 300, 5]), 256, 384, 3, 1, 128),
    ("top-8 of 64", routed(40, 64, 8), 256, 128, 64, 8, 64),
]


@pytest.mark.parametrize("act", [0, 1], ids=["silu", "gelu"])
@pytest.mark.parametrize("name,idx,H,I,E,R,group", W4_SHAPES, ids=[s[0].replace(" ", "-") for s in W4_SHAPES])
def test_w4_forward(name, idx, H, I, E, R, group, act):
    say(f"[experts] w4 {name}")
    c = Case(idx, H, I, E, R, seed=len(name) + 7)
    q1, s1, q2, s2 = four_bit_weights(c, group)
    whole, ye = c.out(c.P, H)
    c.ms.moe_experts_ffn_w4_forward(c.plan, c.xe, q1, s1, q2, s2, ye, c.ws, group=group, act=act)
    w1, w2 = ref.four_bit(q1, s1, group), ref.four_bit(q2, s2, group)
    # products may be summed as (128 + q) - 136, whose magnitudes are up to 264 / 1 times those of q - 8 (at least
    # 1 where not zero, and zero weights still add their term): 17 terms in the place of one on average
    say(f"[experts] w4 {name}: of the bounds {check_forward(c, whole, act, w1=w1, w2=w2, terms=(64 * H, 64 * I))}")


def test_w4_expert_and_row_isolation():
    c = Case(crowd([3, 20, 4]), 256, 128, 3, 3, seed=2)
    q1, s1, q2, s2 = four_bit_weights(c, 64)
    _, ye = c.out(c.P, c.H)
    c.ms.moe_experts_ffn_w4_forward(c.plan, c.xe, q1, s1, q2, s2, ye, c.ws, group=64)
    first = ye.clone()
    lo, hi = int(c.offset[1]), int(c.offset[2])
    c.xe[lo] = float("nan")
    c.ms.moe_experts_ffn_w4_forward(c.plan, c.xe, q1, s1, q2, s2, ye, c.ws, group=64)
    rest = [i for i in range(c.P) if i != lo]
    assert torch.equal(ye[rest], first[rest]) and bool(ye[lo].isnan().all())
    s1[1], s2[1] = float("nan"), float("nan")
    c.ms.moe_experts_ffn_w4_forward(c.plan, c.xe, q1, s1, q2, s2, ye, c.ws, group=64)
    rest = [i for i in range(c.P) if not lo <= i < hi]
    assert torch.equal(ye[rest], first[rest]) and bool(ye[lo:hi].isnan().all())


@pytest.mark.parametrize("rows,cols,group", [(1, 32, 32), (7, 96, 32), (64, 256, 64), (33, 1152, 128), (300, 64, 64)])
def test_w4_quantize(rows, cols, group):
    import moe_expert_token_amd as ms
    gen = torch.Generator(device="cuda").manual_seed(rows)
    w = bf16(gen, rows, cols) * torch.logspace(-20, 20, rows, device="cuda")[:, None].to(torch.bfloat16)
    w[0, :group] = 0
    q = torch.full((rows + 1, cols // 2), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 1, cols // group), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ms.moe_experts_w4_quantize(w, q[:rows], s[:rows], group=group)
    t = w.float().cpu().unflatten(-1, (-1, group))
    scale = (t.abs().amax(-1) / 7).clamp(min=2.0 ** -126).to(torch.bfloat16)
    v = torch.round(t * (1 / scale.float())[..., None]).clamp(-8, 7).flatten(-2).to(torch.int64) + 8
    want = (v[:, 0::2] | (v[:, 1::2] << 4)).to(torch.uint8)
    assert torch.equal(s[:rows].cpu(), scale) and torch.equal(q[:rows].cpu(), want)
    assert bool((q[rows:] == 77).all()) and bool((s[rows:] == SENTINEL).all())
    # half a step, but where -8..7 ends above 7 (bf16's rounding of the scale: 2^-8 of 7 steps)
    err = (ref.four_bit(q[:rows], s[:rows], group).cpu() - w.double().cpu()).abs()
    wide = scale.double().repeat_interleave(group, -1)
    assert bool((err <= wide * (0.5 + 7 * 2.0 ** -8 + 2.0 ** -20)).all())


def test_w4_quantize_of_what_is_not_finite():
    import moe_expert_token_amd as ms
    w = torch.randn((2, 128), device="cuda").to(torch.bfloat16)
    w[0, 3], w[1, 127] = float("nan"), float("-inf")
    q = torch.empty((2, 64), dtype=torch.uint8, device="cuda")
    s = torch.empty((2, 2), dtype=torch.bfloat16, device="cuda")
    ms.moe_experts_w4_quantize(w, q, s, group=64)
    assert s.isnan().tolist() == [[True, False], [False, True]]
    assert bool((q[0, :32] == 0x88).all()) and bool((q[1, 32:] == 0x88).all())


# ---- the operators together, streams, graphs, refusals ----

def test_layer_step_from_tokens_to_gradients():
    """plan, dispatch, the block, combine, and the whole way back, with x kept in 8 bits, against 64 bits."""
    import moe_expert_token_amd as ms
    T, H, I, E, k, R = 200, 128, 64, 8, 2, 4
    idx, gates = synth.random_routing(np.random.default_rng(1), T, E, k)
    c = Case(idx, H, I, E, R, seed=11)
    x = bf16(c.gen, T, H)
    gout = bf16(c.gen, T, H)
    w = torch.from_numpy(gates).cuda()
    xq = torch.empty((T, H), dtype=torch.int8, device="cuda")
    xs = torch.empty((T, H // 32), dtype=torch.bfloat16, device="cuda")
    xr = torch.empty((T * min(k, R), H), dtype=torch.bfloat16, device="cuda")
    ye, out = torch.empty_like(c.xe), torch.empty_like(x)
    saved, scale = c.held("int8")
    ms.moe_experts_pack8(x, xq, xs)
    ms.moe_shuffle_dispatch(c.plan, x, xr, c.xe)
    ms.moe_experts_ffn_forward(c.plan, c.xe, c.w1, c.w2, ye, c.ws, saved=saved, saved_scale=scale)
    ms.moe_shuffle_combine(c.plan, ye, w, out)
    check_forward(c, torch.cat((ye, torch.full_like(ye[:1], SENTINEL))), 0, saved, scale)
    # the way back: x comes out of its checkpoint and is dispatched again
    back = torch.empty_like(x)
    ms.moe_experts_unpack8(xq, xs, back)
    ms.moe_shuffle_dispatch(c.plan, back, xr, c.xe)
    gye, gw = torch.empty_like(ye), torch.empty((T, k), dtype=torch.float32, device="cuda")
    ms.moe_shuffle_combine_backward(c.plan, gout, ye, w, gye, gw)
    c.gy = gye
    got = c.backward(saved, scale)
    check_backward(c, got, saved, scale, 0)
    gxr, gx = torch.empty_like(xr), torch.empty_like(x)
    ms.moe_shuffle_dispatch_backward(c.plan, got["grad_xe"][:c.P], gxr, gx)
    rows = ms.plan_array_views(c.plan)["comb_row"].long()
    want = got["grad_xe"].double()[rows].sum(1)
    # two bf16 roundings on the way (rank rows, token rows), of sums of at most two magnitudes each
    bound = 2 * ref.U * got["grad_xe"].double().abs()[rows].sum(1) * (1 + ref.U) + ref.TINY
    within(gx, want, bound, "grad_x")
    ywant = (ye.double()[rows] * w.double()[..., None]).sum(1)
    within(out, ywant, ref.U * ywant.abs() + ref.GAMMA(k) * (ye.double().abs()[rows] * w.double()[..., None]).sum(1) +
           ref.TINY, "out")


def test_forward_with_a_static_plan():
    import moe_expert_token_amd as ms
    c = Case(routed(64, 8, 2), 128, 64, 8, 4, seed=1)
    ye, _, _ = c.forward()
    c.plan = ms.moe_shuffle_plan_static(c.dims, c.idx)
    again, _, _ = c.forward()
    assert torch.equal(ye, again)


def test_two_streams_with_a_workspace_each():
    cases = [Case(routed(300 + 100 * i, 8, 2, seed=i), 256, 136, 8, 4, seed=i) for i in range(2)]
    want = []
    for c in cases:
        ye, saved, scale = c.forward(0, "int8")
        want.append((ye, c.backward(saved, scale)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            saved, scale = c.held("int8")
            _, ye = c.out(c.P, c.H)
            outs = [c.out(c.P, c.H)[1], c.out(c.E, 2 * c.I, c.H)[1], c.out(c.E, c.H, c.I)[1]]
            s.wait_stream(torch.cuda.current_stream())
            c.ms.moe_experts_ffn_forward(c.plan, c.xe, c.w1, c.w2, ye, c.ws, saved=saved, saved_scale=scale, stream=s)
            c.ms.moe_experts_ffn_backward(c.plan, c.gy, c.xe, c.w1, c.w2, saved, *outs, c.ws, saved_scale=scale,
                                          stream=s)
            got.append((ye, outs))
        torch.cuda.synchronize()
        for (ye, outs), (wy, wb), c in zip(got, want, cases):
            assert torch.equal(ye, wy[:c.P])
            for o, n in zip(outs, ("grad_xe", "grad_w_gate_up", "grad_w_down")):
                assert torch.equal(o, wb[n][:o.shape[0]]), n


@pytest.mark.parametrize("T", [3, 300], ids=["decode", "prefill"])
def test_replays_in_a_graph_with_new_routing(T):
    """Plan, block (bf16, 8-bit saved, 4-bit weights) and backward pass captured once; every replay on new ids and
    rows gives the bits of the same calls made eagerly."""
    import moe_expert_token_amd as ms
    H, I, E, k, R = 128, 96, 8, 2, 4
    c = Case(routed(T, E, k), H, I, E, R, seed=21)
    q1, s1, q2, s2 = four_bit_weights(c, 32)
    saved, scale = c.held("int8")
    ye, y4 = torch.zeros_like(c.xe), torch.zeros_like(c.xe)
    outs = [torch.zeros_like(c.xe), torch.zeros_like(c.w1), torch.zeros_like(c.w2)]

    def step():
        plan = ms.moe_shuffle_plan(c.dims, c.idx, c.plan_ws)
        ms.moe_experts_ffn_forward(plan, c.xe, c.w1, c.w2, ye, c.ws, saved=saved, saved_scale=scale)
        ms.moe_experts_ffn_backward(plan, c.gy, c.xe, c.w1, c.w2, saved, *outs, c.ws, saved_scale=scale)
        ms.moe_experts_ffn_w4_forward(plan, c.xe, q1, s1, q2, s2, y4, c.ws, group=32)
        return plan

    plans = [step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plans.append(step())
    held = [ye, y4, saved, scale] + outs
    for replay in range(4):
        c.idx.copy_(torch.from_numpy(routed(T, E, k, seed=50 + replay)))
        c.xe.normal_(0, 1, generator=c.gen)
        c.gy.normal_(0, 1, generator=c.gen)
        plans.append(step())
        torch.cuda.synchronize()
        want = [t.clone() for t in held]
        for t in held:
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(held, want):
            assert torch.equal(t, w), f"replay {replay}"


def test_runs_repeat_bit_for_bit():
    c = Case(routed(500, 8, 2), 264, 200, 8, 4, seed=31)
    first = None
    for _ in range(5):
        ye, saved, scale = c.forward(0, "bf16")
        now = [ye, saved] + list(c.backward(saved, scale).values())
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = first or now


def test_refusals_with_a_plan():
    """Every refusal that needs a plan's handle; nothing is launched and nothing written."""
    import moe_expert_token_amd as ms
    from moe_expert_token_amd import experts
    c = Case(routed(50, 8, 2), 64, 32, 8, 4)
    lib, h = experts._load(), c.plan.handle
    whole, ye = c.out(c.P, c.H)
    saved, scale = c.held("int8")
    n = c.ws.numel()

    def fwd(x=c.xe.data_ptr(), w1=c.w1.data_ptr(), w2=c.w2.data_ptr(), inter=32, act=0, y=ye.data_ptr(), sv=None,
            sc=None, ws=c.ws.data_ptr(), nb=n):
        return lib.moe_experts_ffn_forward(h, x, w1, w2, inter, act, y, sv, sc, ws, nb, None)

    assert fwd(x=None) == fwd(w1=None) == fwd(w2=None) == fwd(y=None) == fwd(ws=None) == ms.E_INVALID_ARG
    assert fwd(inter=0) == fwd(act=2) == fwd(act=-1) == ms.E_INVALID_ARG
    assert fwd(inter=12) == fwd(x=c.xe.data_ptr() + 2) == fwd(ws=c.ws.data_ptr() + 16) == ms.E_ALIGN
    assert fwd(sv=saved.data_ptr() + 8) == ms.E_ALIGN
    assert fwd(inter=1 << 20) == ms.E_OVERFLOW
    assert fwd(nb=c.P * 32 * 2 - 1) == ms.E_WORKSPACE
    assert fwd(sc=scale.data_ptr()) == ms.E_INVALID_ARG                  # a scale without saved
    assert fwd(y=c.xe.data_ptr()) == fwd(y=c.w2.data_ptr()) == ms.E_INVALID_ARG
    assert fwd(sv=c.xe.data_ptr()) == fwd(ws=c.w1.data_ptr()) == ms.E_INVALID_ARG
    # the plan's workspace is no scratch
    assert c.plan_ws.numel() > 256 and fwd(ws=c.plan_ws.data_ptr()) == fwd(y=c.plan_ws.data_ptr()) == ms.E_INVALID_ARG

    gx, g1, g2 = torch.empty_like(c.xe), torch.empty_like(c.w1), torch.empty_like(c.w2)

    def bwd(gy=c.gy.data_ptr(), x=c.xe.data_ptr(), w1=c.w1.data_ptr(), w2=c.w2.data_ptr(), sv=saved.data_ptr(),
            sc=scale.data_ptr(), a=gx.data_ptr(), b=g1.data_ptr(), d=g2.data_ptr(), ws=c.ws.data_ptr(), nb=n):
        return lib.moe_experts_ffn_backward(h, gy, x, w1, w2, 32, 0, sv, sc, a, b, d, ws, nb, None)

    assert bwd(gy=None) == bwd(x=None) == bwd(w1=None) == bwd(w2=None) == bwd(sv=None) == ms.E_INVALID_ARG
    assert bwd(a=c.gy.data_ptr()) == bwd(b=c.w1.data_ptr()) == bwd(d=c.w2.data_ptr()) == ms.E_INVALID_ARG
    assert bwd(a=g1.data_ptr()) == ms.E_INVALID_ARG
    assert bwd(d=g2.data_ptr() + 4) == ms.E_ALIGN
    assert bwd(nb=3 * c.P * 32 * 2 - 1) == ms.E_WORKSPACE
    assert bwd(a=None, b=None, d=None) == ms.OK                          # nothing asked for, nothing launched

    q1, s1, q2, s2 = four_bit_weights(c, 32)

    def w4(x=c.xe.data_ptr(), a=q1.data_ptr(), b=s1.data_ptr(), d=q2.data_ptr(), e=s2.data_ptr(), inter=32, group=32,
           y=ye.data_ptr(), nb=n):
        return lib.moe_experts_ffn_w4_forward(h, x, a, b, d, e, inter, group, 0, y, c.ws.data_ptr(), nb, None)

    assert w4(x=None) == w4(a=None) == w4(b=None) == w4(d=None) == w4(e=None) == w4(y=None) == ms.E_INVALID_ARG
    assert w4(group=16) == w4(group=0) == ms.E_INVALID_ARG
    assert w4(group=128) == w4(group=64) == w4(b=s1.data_ptr() + 4) == ms.E_ALIGN
    assert w4(nb=16) == ms.E_WORKSPACE
    assert w4(y=q1.data_ptr()) == ms.E_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((whole == SENTINEL).all())
