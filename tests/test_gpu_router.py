"""The router of many rows on the MI355X against its 64-bit definition: sizes
around each border, ties and near ties, rows that are zero, tiny, huge or not
finite, the backward pass, graphs, streams, and a training step through it."""

import pytest
import torch

import layer_ref as ref
from experts_ref import GAMMA

pytestmark = pytest.mark.gpu

SENTINEL = -12345.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_token_amd
    moe_expert_token_amd.load()


def ms():
    import moe_expert_token_amd
    return moe_expert_token_amd


def bf16(gen, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=gen)


def guarded(rows, cols, dtype, value):
    whole = torch.full((rows + 1, cols), value, dtype=dtype, device="cuda")
    return whole, whole[:rows]


class Router:
    def __init__(self, T, H, E, k, sigmoid=False, norm=True, bias=False, scale=1.0, seed=0):
        m = ms()
        self.T, self.H, self.E, self.k = T, H, E, k
        self.sigmoid, self.norm, self.scale = sigmoid, norm, scale
        gen = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.x = bf16(gen, T, H)
        self.w = bf16(gen, E, H, std=H ** -0.5)
        self.bias = torch.empty(E, device="cuda").normal_(0, 0.1, generator=gen) if bias else None
        self.grad = torch.empty(T, k, device="cuda").normal_(0, 1, generator=gen)
        self.dims = m.dims_of(T, H, E, k, 1)
        self.ws = torch.empty(m.moe_router_workspace_size(self.dims, True), dtype=torch.uint8, device="cuda")
        self.ws.fill_(0xff)

    def rule(self):
        m = ms()
        return m.RouterRule(m.SCORE_SIGMOID if self.sigmoid else m.SCORE_SOFTMAX, self.norm, self.scale, self.bias)

    def forward(self, logits=True, **kw):
        self.wholes = [guarded(self.T, self.k, torch.int32, -77), guarded(self.T, self.k, torch.float32, SENTINEL),
                       guarded(self.T, self.E, torch.float32, SENTINEL)]
        self.idx, self.gates, self.logits = (t[1] for t in self.wholes)
        ms().moe_router_forward(self.dims, self.rule(), self.x, self.w, self.idx, self.gates, self.ws,
                                logits=self.logits if logits else None, **kw)
        return self

    def guards_hold(self):
        for whole, _ in self.wholes:
            assert bool((whole[-1] == (-77 if whole.dtype == torch.int32 else SENTINEL)).all())

    def check(self, rows=None):
        """The forward call's results (of some rows)."""
        r = slice(None) if rows is None else rows
        x, w = self.x[r].double(), self.w.double()
        l = x @ w.T
        el = GAMMA(self.H) * (x.abs() @ w.abs().T) + ref.TINY
        far = (self.logits[r].double() - l).abs()
        assert bool((far <= el).all()), f"logits: {float((far / el).max()):.3g}"
        idx = ref.choose(l, self.k, self.sigmoid, self.bias)
        assert torch.equal(self.idx[r].long(), idx), f"{int((self.idx[r].long() != idx).any(1).sum())} rows' ids"
        gates, rel = ref.gates(l, idx, self.sigmoid, self.norm, self.scale)
        rel = rel + 4 * el.amax(1, keepdim=True)
        off = (self.gates[r].double() - gates).abs()
        assert bool((off <= rel * gates.abs() + 1e-37).all()), f"gates: {float((off / (rel * gates.abs() + 1e-37)).max())}"

    def backward(self, want=("grad_x", "grad_w"), grad_x_in=None, grad_logits=None, **kw):
        gx, gw = guarded(self.T, self.H, torch.bfloat16, SENTINEL), guarded(self.E, self.H, torch.bfloat16, SENTINEL)
        ms().moe_router_backward(self.dims, self.rule(), self.grad, self.logits, self.idx, self.x, self.w,
                                 gx[1] if "grad_x" in want else None, gw[1] if "grad_w" in want else None, self.ws,
                                 grad_x_in=grad_x_in, grad_logits=grad_logits, **kw)
        assert bool((gx[0][-1] == SENTINEL).all()) and bool((gw[0][-1] == SENTINEL).all())
        for name, t in (("grad_x", gx), ("grad_w", gw)):
            assert name in want or bool((t[0] == SENTINEL).all())
        return gx[1], gw[1]

    def check_backward(self, gx, gw, grad_x_in=None, grad_logits=None):
        dl, e_dl = ref.score_gradient(self.logits.double(), self.idx.long(), self.grad, self.sigmoid, self.norm, self.scale)
        if grad_logits is not None:
            dl = dl + grad_logits.double()
            e_dl = e_dl + ref.STEP * (dl.abs() + grad_logits.double().abs())
        wx, ex, ww, ew = ref.router_backward(self.x, self.w, dl, e_dl, grad_x_in)
        for got, want, err, name in ((gx, wx, ex, "grad_x"), (gw, ww, ew, "grad_w")):
            far = (got.double() - want).abs()
            assert bool((far <= err).all()), f"{name}: {float((far / err).max()):.3g} of the bound"


SHAPES = [  # T, H, E, k
    (1, 8, 1, 1), (1, 4096, 8, 2), (3, 72, 2, 2), (63, 64, 3, 2), (64, 520, 40, 6), (65, 1544, 64, 8), (200, 136, 65, 5),
    (257, 2048, 128, 8), (1000, 264, 130, 3), (300, 7168, 256, 8), (129, 512, 257, 8), (70, 520, 1023, 64), (4100, 128, 16, 4),
]
RULES = [dict(), dict(sigmoid=True, bias=True, scale=2.5), dict(norm=False, scale=0.5), dict(sigmoid=True, norm=False)]
NAMES = ["softmax", "bias", "plain", "sigmoid"]


@pytest.mark.parametrize("rule", RULES, ids=NAMES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_both_ways(shape, rule):
    c = Router(*shape, seed=sum(shape), **rule).forward()
    c.check()
    c.guards_hold()
    first = [c.idx.clone(), c.gates.clone()]
    add = bf16(c.gen, c.T, c.H, std=0.1)
    extra = torch.empty(c.T, c.E, device="cuda").normal_(0, 0.05, generator=c.gen)
    gx, gw = c.backward()
    c.check_backward(gx, gw)
    gx2, gw2 = c.backward(grad_x_in=add, grad_logits=extra)
    c.check_backward(gx2, gw2, add, extra)
    # each alone, and in place: the same bits
    assert torch.equal(c.backward(want=("grad_x",), grad_x_in=add, grad_logits=extra)[0], gx2)
    assert torch.equal(c.backward(want=("grad_w",), grad_logits=extra)[1], gw2)
    same = add.clone()
    ms().moe_router_backward(c.dims, c.rule(), c.grad, c.logits, c.idx, c.x, c.w, same, None, c.ws, grad_x_in=same,
                             grad_logits=extra)
    assert torch.equal(same, gx2)
    # without logits, and again
    c.forward(logits=False)
    assert torch.equal(c.idx, first[0]) and torch.equal(c.gates, first[1])
    assert bool((c.logits == SENTINEL).all())


@pytest.mark.parametrize("rule", RULES[:2], ids=NAMES[:2])
def test_large_batch(rule):
    """The DeepSeek-V3-like batch: every row's ids."""
    c = Router(8192, 7168, 256, 8, seed=1, **rule).forward()
    for lo in range(0, 8192, 1024):
        c.check(slice(lo, lo + 1024))


@pytest.mark.parametrize("rule", RULES, ids=NAMES)
@pytest.mark.parametrize("shape", [(8192, 7168, 256, 8), (2100, 7168, 300, 8), (300, 7168, 256, 8), (1, 7168, 8, 2), (63, 4096, 40, 6),
                                   (257, 1544, 64, 8), (1000, 264, 130, 3)], ids=lambda s: "-".join(map(str, s)))
def test_logits_within_their_bound(shape, rule):
    """What the choice of experts takes a logit to be off by at most is what it is off by at most; and gates are off by what that
    makes of them: twice a logit's of a normalized gate, or one of a softmax's, once of a plain sigmoid (e^(2 b) - 1 < 2.01 b)."""
    c = Router(*shape, seed=sum(shape) + 1, **rule).forward()
    for lo in range(0, c.T, 1024):
        r = slice(lo, lo + 1024)
        l = c.x[r].double() @ c.w.double().T
        bound = ref.logit_bound(c.x[r], c.w, c.T)
        far = (c.logits[r].double() - l).abs()
        assert bool((far <= bound).all()), f"{float((far / bound).max()):.3g} of the bound"
        gates, rel = ref.gates(l, c.idx[r].long(), c.sigmoid, c.norm, c.scale)
        rel = rel + 2.01 * bound.amax(1, keepdim=True)
        off = (c.gates[r].double() - gates).abs()
        assert bool((off <= rel * gates.abs() + 1e-37).all()), f"gates: {float((off / (rel * gates.abs() + 1e-37)).max())}"


@pytest.mark.parametrize("shape", [(8192, 7168, 256, 8), (2100, 7168, 300, 8), (300, 7168, 256, 8), (1, 7168, 8, 2), (63, 4096, 40, 6),
                                   (257, 1544, 64, 8), (65, 7176, 17, 3)], ids=lambda s: "-".join(map(str, s)))
def test_logits_of_whole_numbers(shape):
    """Products up to 64 of whole numbers, whose sums are exact in fp32 in any order (7176 64 < 2^24): every bit of the
    logits, so each product once, in the tail of H and at the borders of its parts too; ids with their ties."""
    c = Router(*shape, seed=sum(shape) + 2)
    c.x[:] = torch.randint(-8, 9, c.x.shape, device="cuda", generator=c.gen)
    c.w[:] = torch.randint(-8, 9, c.w.shape, device="cuda", generator=c.gen) / 64
    c.forward()
    l = c.x.double() @ c.w.double().T
    assert torch.equal(c.logits.double(), l)
    assert torch.equal(c.idx.long(), ref.choose(l, c.k, False))


@pytest.mark.parametrize("rule", RULES[1:3], ids=NAMES[1:3])
@pytest.mark.parametrize("shape", [(1024, 520, 200, 8), (1041, 1544, 256, 4), (1055, 8, 129, 2), (8200, 4104, 40, 2),
                                   (8207, 4104, 72, 3)], ids=lambda s: "-".join(map(str, s)))
def test_many_rows_backward(shape, rule):
    """grad_x in stripes of columns: rows and columns that end inside a tile, experts that end inside 32."""
    c = Router(*shape, seed=sum(shape), **rule).forward()
    add = bf16(c.gen, c.T, c.H, std=0.1)
    gx, gw = c.backward(grad_x_in=add)
    c.check_backward(gx, gw, add)
    same = add.clone()
    ms().moe_router_backward(c.dims, c.rule(), c.grad, c.logits, c.idx, c.x, c.w, same, None, c.ws, grad_x_in=same)
    assert torch.equal(same, gx)
    plain, _ = c.backward(want=("grad_x",))
    c.check_backward(plain, gw)


def test_values_that_are_not_finite_stay_in_their_rows():
    """In stripes, an infinite element of W reaches its column alone, a NaN gradient its row alone."""
    c = Router(1100, 512, 160, 4, norm=False, seed=15).forward()
    gx, _ = c.backward()
    c.w[3, 100] = float("inf")
    c.grad[50, 1] = float("nan")
    bad, _ = c.backward()
    rows = torch.arange(1100, device="cuda") != 50
    columns = torch.arange(512, device="cuda") != 100
    assert torch.equal(bad[rows][:, columns], gx[rows][:, columns])
    assert not bool(torch.isfinite(bad[rows, 100]).any()) and bool(torch.isnan(bad[50]).all())


@pytest.mark.parametrize("shape", [(1041, 1544, 200, 4), (1055, 72, 129, 2), (8207, 4104, 72, 3), (8200, 4104, 5, 2),
                                   (77, 136, 37, 3), (2050, 72, 30, 2)], ids=lambda s: "-".join(map(str, s)))
def test_what_lies_around_the_inputs(shape):
    """NaN before and after every input reach nothing: experts, rows and columns past the last are not looked at."""
    c = Router(*shape, seed=sum(shape)).forward()
    add = bf16(c.gen, c.T, c.H, std=0.1)
    want = [c.idx, c.gates, c.logits] + list(c.backward(grad_x_in=add))

    def inside(t, rows):
        whole = torch.full((t.shape[0] + 2 * rows, t.shape[1]), float("nan"), dtype=t.dtype, device="cuda")
        whole[rows:rows + t.shape[0]] = t
        return whole[rows:rows + t.shape[0]]

    c.x, c.w, add, c.grad = inside(c.x, 256), inside(c.w, 256), inside(add, 256), inside(c.grad, 256)
    c.forward()
    c.logits = inside(c.logits, 256)
    got = [c.idx, c.gates, c.logits] + list(c.backward(grad_x_in=add))
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def near_ties(c, size):
    """Rows whose keys differ by little: all experts share a row but for one element, where x is small."""
    c.w[:] = c.w[:1].clone()
    n = min(c.E, c.H)
    c.x[:, :n] = (torch.randn(c.T, n, device="cuda", generator=c.gen) * size).to(torch.bfloat16)
    at = torch.arange(n)
    c.w[at, at] = torch.randn(n, device="cuda", generator=c.gen).to(torch.bfloat16)


@pytest.mark.parametrize("size", [2.0 ** -6, 2.0 ** -12, 2.0 ** -18])
@pytest.mark.parametrize("E", [16, 200])
@pytest.mark.parametrize("rule", [dict(), dict(sigmoid=True, bias=True)], ids=["softmax", "bias"])
def test_keys_that_nearly_tie(size, E, rule):
    """From a few that 32 bits cannot order to more of them than a wave's lanes."""
    c = Router(300, 2048, E, 8, seed=E, **rule)
    near_ties(c, size)
    if c.bias is not None:
        c.bias.normal_(0, size, generator=c.gen)
    c.forward().check()


@pytest.mark.parametrize("at", [0, 9, 31])
@pytest.mark.parametrize("T,H", [(64, 256), (300, 7168), (2500, 4096), (8192, 7168)])
def test_ids_where_sums_round_one_way(T, H, at):
    """One large element and products of half a step for every eight of them: fp32 sums lose all of these, in one expert
    above the other, and the choice is still that of exact sums, whatever the large one's lead."""
    c = Router(T, H, 3, 1)
    c.x[:] = 2.0 ** -13
    c.w.zero_()
    c.w[0, :1792] = 2.0 ** -14  # true sums are up to 224 steps of 2^-23 apart, and leads up to 255
    c.w[1, :1792] = -2.0 ** -14
    c.x[:, at] = 1
    c.w[:2, at] = 1
    lead = (at + 1) % H
    c.x[:, lead] = (torch.arange(T, device="cuda") % 256).float() * 2.0 ** -16
    c.w[:, lead] = 0
    c.w[1, lead] = 2.0 ** -7
    c.forward()
    l = c.x.double() @ c.w.double().T
    want = ref.choose(l, 1, False)
    assert bool((want == 0).any()) and bool((want == 1).any())
    assert torch.equal(c.idx.long(), want)


@pytest.mark.parametrize("above", [True, False])
@pytest.mark.parametrize("below", [True, False])
@pytest.mark.parametrize("T", [70, 2100])
def test_ids_where_one_key_is_less_sure_than_its_neighbours(T, below, above):
    """Expert 0's logit is near 1 and its fp32 sum off by 55 2^-20, 1e-5 of the key; those of 1 and 2 are 42.5 and their keys off
    by a step at most, which the biases set: 1 is clear of 2 by 5e-6, and 0 comes out of fp32 beyond 1 (`above`: above both,
    else below) but is exactly within a step of 2, on the side where 2's fp32 key has it wrong."""
    c = Router(T, 448, 3, 2 if above else 1, sigmoid=True, bias=True)
    c.x[:] = 2.0 ** -13
    c.x[:, 9], c.x[:, 447] = 17, -16
    c.w.zero_()
    c.w[0] = -2.0 ** -10 if above else 2.0 ** -10  # sums of eight are half a step of 17, and lost
    c.w[0, 9] = c.w[0, 447] = 1
    c.w[1:, 9] = 2.5
    step = 2.0 ** -23  # of keys from 1 to 2
    # the key 1 + bias of expert 2 is rounded down by 3/8 of a step, or up; and 0's is an eighth to 3/8 from its exact one
    c.bias[2] = 2.0 ** -10 + (0.375 if below else 0.625) * step
    exact = 1 + c.bias[2].double()
    c.bias[1] = c.bias[2] + (5e-6 if above else -5e-6)
    s = ref.scores(c.x[:1].double() @ c.w.double().T, True)[0, 0]
    c.bias[0] = (exact + (-0.25 if below else 0.25) * step - s).float()
    off = float(s + c.bias[0].double() - exact) / step
    assert 0.1 < (-off if below else off) < 0.37
    c.forward()
    want = ref.choose(c.x.double() @ c.w.double().T, c.k, True, c.bias)
    assert want[0].tolist() == ([1] if above else []) + [2 if below else 0]
    assert torch.equal(c.idx.long(), want)


@pytest.mark.parametrize("down", [2.0 ** -70, 2.0 ** -100])
def test_weights_whose_squares_underflow(down):
    """Ids as those of the same weights, larger by a power of two; and of zeros, by index."""
    c = Router(200, 1024, 40, 4, seed=17)
    near_ties(c, 2.0 ** -10)
    ids = c.forward().idx.clone()
    c.check()
    c.w *= down
    assert torch.equal(c.forward().idx, ids)
    c.w[:, :] = 0
    assert c.forward().idx[5].tolist() == [0, 1, 2, 3]


def test_ids_do_not_depend_on_the_batch():
    c = Router(2000, 1024, 96, 6, sigmoid=True, bias=True, seed=3)
    near_ties(c, 2.0 ** -10)
    c.x[1000:] = bf16(c.gen, 1000, 1024)
    ids = c.forward().idx.clone()
    m = ms()
    for lo, n in ((0, 1), (990, 50), (1990, 10), (500, 700)):
        d = Router(n, 1024, 96, 6, sigmoid=True, seed=4)
        d.x, d.w, d.bias = c.x[lo:lo + n].contiguous(), c.w, c.bias
        assert torch.equal(d.forward().idx, ids[lo:lo + n])
        if n <= 64:  # and the layer's
            dims = m.dims_of(n, 1024, 96, 6, 1)
            ws = torch.empty(m.moe_layer_workspace_size(dims, 8), dtype=torch.uint8, device="cuda")
            w1, w2 = bf16(c.gen, 96, 16, 1024), bf16(c.gen, 96, 1024, 8)
            out, idx = torch.empty_like(d.x), torch.empty(n, 6, dtype=torch.int32, device="cuda")
            m.moe_layer_forward(dims, d.rule(), d.x, c.w, w1, w2, out, ws, topk_idx=idx)
            assert torch.equal(idx, ids[lo:lo + n])


@pytest.mark.parametrize("rule", RULES[:2], ids=NAMES[:2])
@pytest.mark.parametrize("E", [4, 8, 40])
@pytest.mark.parametrize("H", [64, 1000, 4096, 7168])
def test_sums_that_depend_on_their_order(H, E, rule):
    """Logits of 0, of products of 2^-40 to 2^40 each of which some other one cancels: what 64 bits leave of them goes by the
    order of the additions, and so do the ids.  They are the same of many rows, few and one, and by every form of the
    layer's scores."""
    m = ms()
    c = Router(2100, H, E, 3, seed=H + E, **rule)
    order = torch.randperm(H, device="cuda", generator=c.gen)
    one, other = order[:H // 2], order[H // 2:]
    for t in (c.x, c.w):
        t.mul_(torch.exp2(40 * torch.rand(t.shape, device="cuda", generator=c.gen) - 20).to(torch.bfloat16))
    c.x[:, other] = -c.x[:, one]
    c.w[:, other] = c.w[:, one]
    if c.bias is not None:
        c.bias.zero_()
    ids = c.forward().idx.clone()
    assert len(set(map(tuple, ids.tolist()))) > 3  # as the sums' ends fall
    for n in (1, 2, 3, 8, 40, 300):
        d = Router(n, H, E, 3, sigmoid=c.sigmoid, seed=4)
        d.x, d.w, d.bias = c.x[:n].contiguous(), c.w, c.bias
        assert torch.equal(d.forward().idx, ids[:n]), f"{n} rows"
        if n > 64:
            continue
        dims = m.dims_of(n, H, E, 3, 1)
        ws = torch.empty(m.moe_layer_workspace_size(dims, 8), dtype=torch.uint8, device="cuda")
        w1, w2 = torch.zeros(E, 16, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, H, 8, dtype=torch.bfloat16, device="cuda")
        out, idx = torch.empty_like(d.x), torch.empty(n, 3, dtype=torch.int32, device="cuda")
        m.moe_layer_forward(dims, d.rule(), d.x, d.w, w1, w2, out, ws, topk_idx=idx)
        assert torch.equal(idx, ids[:n]), f"layer of {n} rows"


@pytest.mark.parametrize("rule", RULES, ids=NAMES)
def test_ties_and_zero_rows(rule):
    c = Router(130, 256, 100, 5, seed=5, **rule)
    c.w[1::2] = c.w[0::2]  # pairs of equal experts
    c.x[7] = 0
    c.x[64:100] = 0
    c.forward().check()
    if c.bias is None:
        assert c.idx[7].tolist() == [0, 1, 2, 3, 4]
    c.bias = torch.zeros(100, device="cuda") if c.bias is not None else None
    c.forward().check()
    c.w.zero_()
    c.forward().check()
    gx, gw = c.backward()
    c.check_backward(gx, gw)


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e15, 1e25])
def test_rows_of_extreme_size(size):
    """Norms whose squares leave fp32 (down to products that do not): the choice is still that of exact sums."""
    c = Router(70, 512, 48, 6, seed=6)
    c.x[3:40] = (c.x[3:40].float() * size).to(torch.bfloat16)
    c.forward()
    l = c.x.double() @ c.w.double().T
    assert torch.equal(c.idx.long(), ref.choose(l, 6, False))


def test_rows_that_are_not_finite():
    c = Router(100, 256, 20, 4, seed=7)
    clean = c.forward()
    ids, gates = clean.idx.clone(), clean.gates.clone()
    c.x[5, 3] = float("nan")
    c.x[6, 4] = float("inf")
    c.forward()
    others = torch.ones(100, dtype=torch.bool, device="cuda")
    others[5:7] = False
    assert torch.equal(c.idx[others], ids[others]) and torch.equal(c.gates[others], gates[others])
    assert c.idx[5].tolist() == [0, 1, 2, 3]
    for t in (5, 6):
        row = c.idx[t].tolist()
        assert len(set(row)) == 4 and min(row) >= 0 and max(row) < 20
    # a bias of minus infinity takes an expert out; all but three: the others follow by index
    s = Router(50, 64, 30, 5, sigmoid=True, bias=True, seed=8)
    s.bias[:] = float("-inf")
    s.bias[[4, 9, 17]] = 0.0
    s.forward()
    assert bool((s.idx[:, 3:] == torch.tensor([0, 1], device="cuda")).all())
    assert torch.equal(s.idx.long(), ref.choose(s.x.double() @ s.w.double().T, 5, True, s.bias))


@pytest.mark.parametrize("T", [3, 2100])
def test_rows_that_are_not_finite_under_zero_weights(T):
    """0 times infinity or NaN is NaN, of every expert: whatever the bias, the ids are 0 .. k - 1, as the layer's are."""
    m = ms()
    c = Router(T, 256, 20, 4, sigmoid=True, bias=True, seed=18)
    c.w.zero_()
    c.x[0, 3], c.x[1, 200] = float("nan"), float("inf")
    c.forward()
    assert c.idx[:2].tolist() == [[0, 1, 2, 3]] * 2
    assert bool(c.logits[:2].isnan().all()) and bool((c.logits[2:] == 0).all())
    first = torch.sort(c.bias.double() + 0.5, descending=True, stable=True).indices[:4]
    assert bool((c.idx[2:].long() == first).all())
    for n in (1, 3):
        dims = m.dims_of(n, 256, 20, 4, 1)
        ws = torch.empty(m.moe_layer_workspace_size(dims, 8), dtype=torch.uint8, device="cuda")
        w1, w2 = bf16(c.gen, 20, 16, 256), bf16(c.gen, 20, 256, 8)
        out, idx = torch.empty(n, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 4, dtype=torch.int32, device="cuda")
        m.moe_layer_forward(dims, c.rule(), c.x[:n], c.w, w1, w2, out, ws, topk_idx=idx)
        assert torch.equal(idx, c.idx[:n])


def test_bad_ids_touch_nothing_else():
    c = Router(40, 128, 12, 3, seed=9).forward()
    good = c.backward()[0].clone()
    c.idx[7] = torch.tensor([-1, 12, 1 << 30], dtype=torch.int32, device="cuda")
    gx, gw = c.backward()
    others = torch.arange(40, device="cuda") != 7
    assert torch.equal(gx[others], good[others])
    assert bool((gx[7] == 0).all())  # nothing was chosen


def unit_weights(c):
    """Weights under which grad_x of columns 0 .. E - 1 is dl, rounded to bf16."""
    c.w.zero_()
    at = torch.arange(c.E)
    c.w[at, at] = 1


@pytest.mark.parametrize("T,E", [(31, 8), (1100, 160)])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_of_saturated_sigmoids(norm, T, E):
    """Chosen logits from -30 to 30: dl keeps its relative accuracy where 1 - s has few bits or none in fp32.  In dl are the
    roundings of the exponential (4 STEP), of three operations on it and of two on the gradient's side (normalized: two
    divisions more), in grad_x those to two parts (U^2) and of the output (U)."""
    c = Router(T, 256, E, 2, sigmoid=True, norm=norm, seed=16).forward()
    unit_weights(c)
    at = torch.linspace(-30, 30, T, device="cuda")
    c.idx[:, 0], c.idx[:, 1] = 3, E - 2
    c.logits[:, 3], c.logits[:, E - 2] = at, at.flip(0)
    c.grad[:, 0], c.grad[:, 1] = 1.25, -0.75
    gx, _ = c.backward(want=("grad_x",))
    s = 1 / (1 + torch.exp(-c.logits.double().gather(1, c.idx.long())))
    slope = s * (1 / (1 + torch.exp(c.logits.double().gather(1, c.idx.long()))))
    g = c.grad.double()
    if norm:
        total = s.sum(1, keepdim=True) + 1e-20
        g = ((g - g.flip(1)) * s.flip(1) + 1e-20 * g) / total / total  # g_j - sum_i g_i s_i / total, the s_j g_j taken out
    want = torch.zeros(T, 256, dtype=torch.float64, device="cuda").scatter_(1, c.idx.long(), g * slope)
    far = (gx.double() - want).abs()
    # normalized, the mean of g is off by the scores' 6 STEP, 7 of their sum, and three of product, sum and division, and
    # the difference rounds once
    err = (2.0 ** -8 * (1 + 2.0 ** -6) + 32 * ref.STEP) * want.abs()
    if norm:
        err += torch.zeros_like(err).scatter_(1, c.idx.long(), 20 * ref.STEP * 1.25 / total * slope)
    assert bool((far <= err).all()), f"{float((far / err.clamp(min=1e-300)).max()):.3g} of the bound"


@pytest.mark.parametrize("T,E", [(34, 8), (1105, 160), (17, 600)])
@pytest.mark.parametrize("rule", [dict(norm=False), dict(), dict(sigmoid=True)], ids=["plain", "softmax", "sigmoid"])
def test_gradient_where_one_score_is_nearly_all(rule, T, E):
    """The first of three chosen leads by up to 16 in the logits, so that the others' scores are 2^-23 of the sum: dl keeps its
    relative accuracy.  The gradients are such that no term of sum_i s_i (g_j - g_i) is against another.  A score is off by
    20 + E / 64 STEP at most (exponential 4, whole numbers' differences none, the sum's terms and additions, division), the
    sum of the chosen by as much and three, products and sums over the chosen by five: under 100 STEP together."""
    c = Router(T, 640, E, 3, seed=17, **rule).forward()
    unit_weights(c)
    lead = (torch.arange(T, device="cuda") % 17).float()
    top = 4.0 if c.sigmoid else 20.0
    c.logits[:] = (top - lead - 6)[:, None]
    for j, (e, down) in enumerate(((5, 0), (E - 1, lead), (0, lead + 1))):
        c.idx[:, j] = e
        c.logits[:, e] = top - down
    c.grad[:] = torch.tensor([1.25, -0.75, -0.75], device="cuda")
    gx, _ = c.backward(want=("grad_x",))
    l, at = c.logits.double(), c.idx.long()
    want, _ = ref.score_gradient(l, at, c.grad, c.sigmoid, c.norm, 1.0)
    s = ref.scores(l, c.sigmoid)
    mine, g = s.gather(1, at), c.grad.double()
    apart = (mine[:, None, :] * (g[:, :, None] - g[:, None, :]).abs()).sum(2)
    if c.norm:
        total = mine.sum(1, keepdim=True)
        size = torch.zeros_like(s).scatter_(1, at, apart / total ** 2)
    else:
        size = (mine * g.abs()).sum(1, keepdim=True).expand_as(s).scatter(1, at, apart + (1 - mine.sum(1, keepdim=True)) * g.abs())
    size = size * (s * (1 - s) if c.sigmoid else s)
    err = 2.0 ** -8 * (1 + 2.0 ** -6) * want.abs() + 100 * ref.STEP * size + ref.TINY
    if c.norm and not c.sigmoid:
        # of the experts not chosen it is -s_e sum_i ds_i s_i, 0 but for 1e-20 of the gradients; `want` has it as a sum in 64
        # bits of three terms of |g_i| s_i / D and less, in which 16 roundings of 2^-53 leave up to 2^-49 of those
        err += 2.0 ** -49 * s * (g.abs() * mine / total).sum(1, keepdim=True) / total
    far = (gx[:, :E].double() - want).abs()
    assert bool((far <= err).all()), f"{float((far / err).max()):.3g} of the bound"


def test_no_rows():
    m = ms()
    c = Router(4, 64, 8, 2, seed=10)
    dims = m.dims_of(0, 64, 8, 2, 1)
    ws = torch.empty(m.moe_router_workspace_size(dims, True), dtype=torch.uint8, device="cuda")
    i, f, l = (torch.empty(0, n, dtype=d, device="cuda") for n, d in ((2, torch.int32), (2, torch.float32), (8, torch.float32)))
    m.moe_router_forward(dims, c.rule(), c.x[:0], c.w, i, f, ws, logits=l)
    gw = torch.full((8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    m.moe_router_backward(dims, c.rule(), f, l, i, c.x[:0], c.w, c.x[:0].clone(), gw, ws)
    assert bool((gw == 0).all())


def test_graph_replays():
    """Forward and backward in one graph, new rows and weights between replays, eager work between them."""
    c = Router(500, 520, 40, 6, sigmoid=True, bias=True, seed=11)
    m, rule = ms(), c.rule()
    out = [torch.empty(500, 6, dtype=torch.int32, device="cuda"), torch.empty(500, 6, device="cuda"),
           torch.empty(500, 40, device="cuda"), torch.empty_like(c.x), torch.empty_like(c.w)]
    eager_ws = torch.empty_like(c.ws)

    def go(out, ws):
        m.moe_router_forward(c.dims, rule, c.x, c.w, out[0], out[1], ws, logits=out[2])
        m.moe_router_backward(c.dims, rule, c.grad, out[2], out[0], c.x, c.w, out[3], out[4], ws)

    go(out, c.ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(out, c.ws)
    for i in range(5):
        c.x.normal_(0, 1, generator=c.gen)
        c.w.normal_(0, 0.05, generator=c.gen)
        c.bias.normal_(0, 0.1, generator=c.gen)
        graph.replay()
        torch.cuda.synchronize()
        eager = [torch.empty_like(t) for t in out]
        go(eager, eager_ws)
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
    c.idx, c.gates, c.logits = out[:3]
    c.check()
    c.check_backward(out[3], out[4])


def test_two_streams_at_once():
    a, b = Router(700, 1024, 64, 4, seed=12), Router(300, 2048, 128, 8, sigmoid=True, bias=True, seed=13)
    want = []
    for c in (a, b):
        c.forward()
        want.append([c.idx.clone(), c.gates.clone()] + [t.clone() for t in c.backward()])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        got = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.forward()
                got.append([c.idx, c.gates] + list(c.backward()))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for g, w in zip(got, want):
            for x, y in zip(g, w):
                assert torch.equal(x, y)


def test_a_training_step():
    """Router, plan, dispatch, block, combine, and back; the gradients of x and of the router's weights against 64-bit
    autograd, then AdamW on all weights.  Each path has at most six bf16 roundings of 2^-8 of what they round (xe is
    exact): a gradient's error is held to 6 2^-8 of its norm."""
    m = ms()
    T, H, E, k, R, I = 300, 256, 8, 2, 4, 128
    c = Router(T, H, E, k, sigmoid=True, bias=True, seed=14)
    gen = c.gen
    w1, w2 = bf16(gen, E, 2 * I, H, std=H ** -0.5), bf16(gen, E, H, I, std=I ** -0.5)
    grad_out = bf16(gen, T, H)
    dims = m.dims_of(T, H, E, k, R)
    c.forward()
    plan_ws = torch.empty(m.moe_shuffle_workspace_size(dims), dtype=torch.uint8, device="cuda")
    plan = m.moe_shuffle_plan(dims, c.idx, plan_ws)
    P = T * k
    rows = {n: torch.empty(P, H, dtype=torch.bfloat16, device="cuda") for n in ("xr", "xe", "ye", "gye", "gxe", "gxr")}
    saved = torch.empty(P, 2 * I, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(m.moe_experts_ffn_workspace_size(dims, I, True), dtype=torch.uint8, device="cuda")
    out, gx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    gw = torch.empty(T, k, device="cuda")
    gw1, gw2, gwr = torch.empty_like(w1), torch.empty_like(w2), torch.empty_like(c.w)
    m.moe_shuffle_dispatch(plan, c.x, rows["xr"], rows["xe"])
    m.moe_experts_ffn_forward(plan, rows["xe"], w1, w2, rows["ye"], ws, saved=saved)
    m.moe_shuffle_combine(plan, rows["ye"], c.gates, out)
    m.moe_shuffle_combine_backward(plan, grad_out, rows["ye"], c.gates, rows["gye"], gw)
    m.moe_experts_ffn_backward(plan, rows["gye"], rows["xe"], w1, w2, saved, rows["gxe"], gw1, gw2, ws)
    m.moe_shuffle_dispatch_backward(plan, rows["gxe"], rows["gxr"], gx)
    m.moe_router_backward(c.dims, c.rule(), gw, c.logits, c.idx, c.x, c.w, gx, gwr, c.ws, grad_x_in=gx)
    # 64 bits on the CPU
    x, wr, a, b = (t.double().cpu().requires_grad_(True) for t in (c.x, c.w, w1, w2))
    s = torch.sigmoid(x @ wr.T)
    idx = c.idx.long().cpu()
    at = s.gather(1, idx)
    gates = at / (at.sum(1, keepdim=True) + 1e-20)
    total = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        pre = x[t] @ a[e].T
        y = (torch.nn.functional.silu(pre[:, :I]) * pre[:, I:]) @ b[e].T
        total = total.index_add(0, t, gates[t, j][:, None] * y)
    want = torch.autograd.grad(total, (x, wr, a, b), grad_out.double().cpu())
    for got, w, name in zip((gx, gwr, gw1, gw2), want, ("x", "w_router", "w_gate_up", "w_down")):
        far = float((got.double().cpu() - w).norm() / w.norm())
        assert far <= 6 * 2.0 ** -8, f"{name}: {far}"
    tensors, before = [], []
    for p, g in ((w1, gw1), (w2, gw2), (c.w, gwr)):
        master = p.float()
        tensors.append(dict(p=master, copy=p, g=g, m=torch.zeros_like(master), v=torch.zeros_like(master)))
        before.append(master.clone())
    m.moe_adamw_step(m.AdamwTensors(tensors), 1, 1e-2, weight_decay=0.0)
    for t, old in zip(tensors, before):
        # the first step is lr times the gradient's sign, wherever the gradient is far above eps
        far = t["g"].float().abs() > 1e-4
        move = (t["p"] - old)[far]
        assert bool(((move + 1e-2 * t["g"].float().sign()[far]).abs() <= 1e-2 * 1.1e-4 + 2.0 ** -23 * old[far].abs()).all())
        assert torch.equal(t["copy"], t["p"].to(torch.bfloat16))
