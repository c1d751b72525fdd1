"""The layer for few tokens on the MI355X against its 64-bit definition: sizes
around each border, crowded and empty experts, ties, rows that are not finite,
4-bit weights, graphs, streams, and the same layer step by step."""

import pytest
import torch

import experts_bounds as bounds
import layer_ref as ref

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


class Layer:
    def __init__(self, T, H, E, k, I, group=0, sigmoid=False, norm=True, bias=False, scale=1.0, act=0, seed=0):
        m = ms()
        self.T, self.H, self.E, self.k, self.I, self.group, self.act = T, H, E, k, I, group, act
        self.sigmoid, self.norm, self.scale = sigmoid, norm, scale
        gen = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.x = bf16(gen, T, H)
        self.w_router = bf16(gen, E, H, std=H ** -0.5)
        self.residual = bf16(gen, T, H)
        self.bias = torch.empty(E, device="cuda").normal_(0, 0.1, generator=gen) if bias else None
        w1, w2 = bf16(gen, E, 2 * I, H, std=H ** -0.5), bf16(gen, E, H, I, std=I ** -0.5)
        if group:
            self.weights = []
            for w in (w1, w2):
                q = torch.empty(w.shape[:-1] + (w.shape[-1] // 2,), dtype=torch.uint8, device="cuda")
                s = torch.empty(w.shape[:-1] + (w.shape[-1] // group,), dtype=torch.bfloat16, device="cuda")
                m.moe_experts_w4_quantize(w, q, s, group=group)
                self.weights += [q, s]
        else:
            self.weights = [w1, w2]
        self.dims = m.dims_of(T, H, E, k, 1)
        self.ws = torch.empty(m.moe_layer_workspace_size(self.dims, I), dtype=torch.uint8, device="cuda")
        self.ws.fill_(0xff)  # NaN and -1 wherever something is read before it is written

    def rule(self):
        m = ms()
        return m.RouterRule(m.SCORE_SIGMOID if self.sigmoid else m.SCORE_SOFTMAX, self.norm, self.scale, self.bias)

    def run(self, residual=True, ids=True, **kw):
        m = ms()
        self.whole, out = guarded(self.T, self.H, torch.bfloat16, SENTINEL)
        self.ids_whole, self.idx = guarded(self.T, self.k, torch.int32, -77)
        self.gates_whole, self.gates = guarded(self.T, self.k, torch.float32, SENTINEL)
        kept = dict(residual=self.residual if residual else None, act=self.act)
        if ids:
            kept.update(topk_idx=self.idx, topk_w=self.gates)
        kept.update(kw)
        call, more = (m.moe_layer_w4_forward, dict(group=self.group)) if self.group else (m.moe_layer_forward, {})
        call(self.dims, self.rule(), self.x, self.w_router, *self.weights, kept.pop("out", out), self.ws, **more, **kept)
        return out

    def pair(self, which, e):
        if self.group:
            return bounds.w4_weights(self.weights[2 * which][e], self.weights[2 * which + 1][e], self.group)
        return bounds.bf16_weights(self.weights[which][e])

    def expect(self, residual=True):
        l = ref.logits(self.x, self.w_router)
        idx = ref.choose(l, self.k, self.sigmoid, self.bias)
        w, rel = ref.gates(l, idx, self.sigmoid, self.norm, self.scale)
        rel = rel.expand_as(w)
        out, err = ref.layer(self.x, idx, w, rel, lambda e: self.pair(0, e), lambda e: self.pair(1, e), self.act,
                             self.residual if residual else None)
        return idx, w, rel, out, err

    def check(self, out, residual=True, ids=True):
        idx, w, rel, want, err = self.expect(residual)
        if ids:
            assert torch.equal(self.idx.long(), idx), "ids"
            far = (self.gates.double() - w).abs()
            assert bool((far <= rel * w.abs() + 1e-37).all()), f"gates: {float((far / (rel * w.abs() + 1e-37)).max())}"
            assert bool((self.ids_whole[self.T:] == -77).all()) and bool((self.gates_whole[self.T:] == SENTINEL).all())
        assert bool(torch.isfinite(out).all())
        worst = float(((out.double() - want).abs() / err).max())
        assert worst <= 1, f"out: {worst:.3g} of the bound"
        assert bool((self.whole[self.T:] == SENTINEL).all()), "a row past the last was written"


SHAPES = [  # T, H, E, k, I
    (1, 8, 1, 1, 8), (1, 128, 8, 2, 256), (2, 136, 5, 5, 72), (3, 2048, 16, 4, 1024), (1, 4096, 8, 2, 4096),
    (15, 264, 40, 6, 520), (16, 1544, 40, 6, 712), (17, 1544, 40, 6, 712), (33, 4104, 9, 3, 136), (64, 512, 64, 8, 256),
    (8, 64, 1024 - 1, 64, 40), (64, 64, 3, 1, 128), (64, 4096, 4, 4, 64), (48, 256, 300, 8, 128), (5, 128, 65, 3, 4224),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("rule", [dict(), dict(sigmoid=True, bias=True, scale=2.5), dict(norm=False, scale=0.5),
                                  dict(sigmoid=True, norm=False)], ids=["softmax", "bias", "plain", "sigmoid"])
def test_bf16(shape, rule):
    c = Layer(*shape, act=shape[1] % 3 % 2, seed=sum(shape), **rule)
    c.check(c.run())


@pytest.mark.parametrize("shape", [(3, 136, 5, 5, 72, 0), (1, 128, 8, 2, 256, 0), (17, 1544, 40, 6, 712, 0), (64, 64, 3, 1, 128, 0),
                                   (5, 128, 65, 3, 4224, 0), (4, 160, 6, 2, 96, 32), (2, 384, 9, 2, 640, 128),
                                   (40, 1088, 20, 4, 320, 64), (1, 4096, 8, 2, 512, 128)], ids=lambda s: "-".join(map(str, s)))
def test_what_lies_around_the_inputs(shape):
    """NaN before and after every input reach nothing."""
    *sizes, group = shape
    c = Layer(*sizes, group=group, seed=sum(shape))
    want = [c.run(), c.idx, c.gates]

    def inside(t):
        value = float("nan") if t.is_floating_point() else 0xff
        n, pad = t.numel(), 1 << 16
        whole = torch.full((n + 2 * pad,), value, dtype=t.dtype, device="cuda")
        whole[pad:pad + n] = t.flatten()
        return whole[pad:pad + n].view(t.shape)

    c.x, c.w_router, c.residual = inside(c.x), inside(c.w_router), inside(c.residual)
    c.weights = [inside(t) for t in c.weights]
    for g, w in zip([c.run(), c.idx, c.gates], want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 128, 8, 2, 256), (1, 7168, 16, 8, 2048), (7, 256, 5, 5, 384), (16, 640, 40, 6, 896),
                                   (17, 640, 40, 6, 896), (48, 1024, 64, 8, 512), (64, 4224, 3, 2, 4096),
                                   (2, 2048, 4, 2, 16384 + 128)], ids=lambda s: "-".join(map(str, s)))
def test_w4(shape, group):
    c = Layer(*shape, group=group, sigmoid=group == 64, bias=group == 64, act=group // 64 % 2, seed=sum(shape) + group)
    c.check(c.run())


@pytest.mark.parametrize("shape", [(1, 96, 8, 2, 160), (20, 160, 8, 2, 96)], ids=lambda s: "-".join(map(str, s)))
def test_w4_widths_that_end_inside_a_chunk(shape):
    c = Layer(*shape, group=32, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("group", [0, 32, 128])
def test_rows_of_16400_scales(group):
    """Longer rows of scales than the staging holds; wide sums."""
    H = 16384 + 128
    c = Layer(3, H, 2, 1, 128, group=group, seed=5)
    c.check(c.run())


@pytest.mark.parametrize("T", [16, 17, 31, 33, 63, 64])
@pytest.mark.parametrize("group", [0, 128])
def test_all_tokens_on_one_expert(T, group):
    """One expert with every token, the others with none or all of what is left."""
    c = Layer(T, 256, 7, 1, 384, group=group, seed=T)
    c.x = c.x.abs()
    c.w_router = torch.zeros_like(c.w_router)
    c.w_router[4] = 0.5
    c.check(c.run())
    assert bool((c.idx == 4).all())


def test_ties_go_to_the_lowest_index():
    c = Layer(9, 64, 130, 5, 64, seed=1)
    c.w_router[1::2] = c.w_router[0::2]  # pairs of equal experts
    c.x[3] = 0                           # all keys equal
    c.check(c.run())
    assert c.idx[3].tolist() == [0, 1, 2, 3, 4]
    first = c.idx[:, 0]
    assert bool((first % 2 == 0).all())
    assert torch.equal(c.idx[:, 1], first + 1)
    # equal scores far out, where a sigmoid is 1 or its key loses the logit
    s = Layer(4, 64, 16, 4, 64, sigmoid=True, bias=True, seed=2)
    s.bias.zero_()
    s.x = s.x.abs() * 100
    s.w_router = s.w_router.abs() * 100
    s.check(s.run())
    assert s.idx[0].tolist() == [0, 1, 2, 3]


def test_logits_that_nearly_tie():
    """Keys that differ by less than 32 bits resolve: the order is that of exact sums."""
    T, H, E = 16, 4096, 64
    c = Layer(T, H, E, 8, 64, seed=4)
    base = c.w_router[:1].clone()
    c.w_router[:] = base
    # one element of each row moves by a few bf16 steps where x is small
    c.x[:, :E] = (torch.randn(T, E, device="cuda", generator=c.gen) * 2.0 ** -18).to(torch.bfloat16)
    c.w_router[torch.arange(E), torch.arange(E)] = torch.randn(E, device="cuda", generator=c.gen).to(torch.bfloat16)
    l = ref.logits(c.x, c.w_router)
    top = l.sort(1, descending=True).values[:, :9]
    gap = (top[:, :-1] - top[:, 1:]).min()
    assert 0 < float(gap) < 2.0 ** -22 * float(l.abs().max())
    c.run()
    assert torch.equal(c.idx.long(), ref.choose(l, 8, False))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("group", [0, 32])
def test_a_row_that_is_not_finite_stays_alone(value, group):
    """The other tokens' bits do not change; the row's own ids are distinct and in range."""
    c = Layer(20, 256, 12, 4, 128, group=group, seed=6)
    clean = c.run().clone()
    ids = c.idx.clone()
    c.x[7, 100] = value
    out = c.run()
    others = torch.arange(20, device="cuda") != 7
    assert torch.equal(out[others], clean[others]) and torch.equal(c.idx[others], ids[others])
    row = sorted(c.idx[7].tolist())
    assert len(set(row)) == 4 and row[0] >= 0 and row[-1] < 12
    if value != value:
        assert row == [0, 1, 2, 3]  # no key is a number
        assert bool(torch.isnan(out[7]).all())


@pytest.mark.parametrize("group", [0, 64])
def test_other_tokens_do_not_matter(group):
    c = Layer(24, 512, 10, 3, 256, group=group, sigmoid=True, bias=True, seed=7)
    first = c.run().clone()
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        keep = torch.rand(24, device="cuda", generator=gen) < 0.5
        fresh = bf16(gen, 24, 512)
        c.x = torch.where(keep[:, None], c.x, fresh)
        out = c.run()
        assert torch.equal(out[keep], first[keep])
        c.check(out)
        first = out.clone()


def test_residual_forms():
    c = Layer(6, 136, 8, 2, 64, seed=8)
    c.check(c.run(residual=False), residual=False)
    want = c.run().clone()
    whole, out = guarded(6, 136, torch.bfloat16, SENTINEL)
    out.copy_(c.residual)
    m = ms()
    m.moe_layer_forward(c.dims, c.rule(), c.x, c.w_router, *c.weights, out, c.ws, residual=out)
    assert torch.equal(out, want)
    assert bool((whole[6:] == SENTINEL).all())
    without = c.run(ids=False)
    assert torch.equal(without, want)


def test_no_tokens():
    m = ms()
    c = Layer(4, 64, 8, 2, 64, seed=9)
    dims = m.dims_of(0, 64, 8, 2, 1)
    out = torch.full((4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_layer_forward(dims, c.rule(), c.x[:0], c.w_router, *c.weights, out[:0], c.ws)
    assert bool((out == 7).all())
    assert m.moe_layer_workspace_size(dims, 64) > 0


def test_strided_parts_of_a_cache_line_of_rows():
    """Rows at the start of a longer buffer, outputs in the middle of another."""
    c = Layer(3, 40, 4, 2, 24, seed=10)
    big = torch.zeros(10, 40, dtype=torch.bfloat16, device="cuda")
    big[2:5] = c.x
    c.x = big[2:5]
    c.check(c.run())


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T", [1, 20])
def test_graph_replays(T, group):
    """New rows, weights and routing between replays, with eager work and waits; every replay equals the eager call."""
    c = Layer(T, 512, 16, 4, 256, group=group, sigmoid=True, bias=True, seed=11)
    want_ws = torch.empty_like(c.ws)
    out = torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, 4, device="cuda")
    m, rule = ms(), c.rule()
    call, more = (m.moe_layer_w4_forward, dict(group=group)) if group else (m.moe_layer_forward, {})

    def go(out, ws):
        call(c.dims, rule, c.x, c.w_router, *c.weights, out, ws, residual=c.residual, topk_idx=idx, topk_w=gate, **more)

    go(out, c.ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(out, c.ws)
    for i in range(5):
        c.x.normal_(0, 1, generator=c.gen)
        c.bias.normal_(0, 0.2, generator=c.gen)
        out.fill_(SENTINEL)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        ids = idx.clone()
        eager = torch.empty_like(out)
        go(eager, want_ws)
        assert torch.equal(eager, out) and torch.equal(ids, idx)
        c.idx, c.gates = idx, gate
        c.whole = torch.cat((out, torch.full((1, 512), SENTINEL, dtype=torch.bfloat16, device="cuda")))
        c.check(out, ids=False)


def test_two_streams_at_once():
    """Calls that overlap in time, a workspace each."""
    a, b = Layer(8, 2048, 32, 4, 1024, seed=12), Layer(40, 1024, 16, 2, 2048, group=64, seed=13)
    want = [a.run().clone(), b.run().clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        outs = []
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                outs.append(c.run())
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for got, w in zip(outs, want):
            assert torch.equal(got, w)


@pytest.mark.parametrize("group", [0, 32])
def test_the_same_layer_step_by_step(group):
    """Ids and gates of the layer through plan, dispatch, the experts' block and combine: the same sums up to the
    rounding of y to bf16, which the bounds of both sides hold."""
    m = ms()
    c = Layer(30, 256, 12, 4, 160, group=group, seed=14)
    out = c.run(residual=False).clone()
    P = 30 * 4
    plan_ws = torch.empty(m.moe_shuffle_workspace_size(c.dims), dtype=torch.uint8, device="cuda")
    plan = m.moe_shuffle_plan(c.dims, c.idx, plan_ws)
    xr = torch.empty(30, 256, dtype=torch.bfloat16, device="cuda")
    xe, ye = (torch.empty(P, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.moe_shuffle_dispatch(plan, c.x, xr, xe)
    ws = torch.empty(m.moe_experts_ffn_workspace_size(c.dims, 160), dtype=torch.uint8, device="cuda")
    if group:
        m.moe_experts_ffn_w4_forward(plan, xe, *c.weights, ye, ws, group=group)
    else:
        m.moe_experts_ffn_forward(plan, xe, *c.weights, ye, ws)
    steps = torch.empty(30, 256, dtype=torch.bfloat16, device="cuda")
    m.moe_shuffle_combine(plan, ye, c.gates, steps)
    idx, w, rel, want, err = c.expect(residual=False)
    assert bool(((out.double() - want).abs() <= err).all())
    # y rounded: half a bf16 step of each term
    views = m.plan_array_views(plan)
    y = ye.double()[views["comb_row"].long().flatten()].view(30, 4, 256)
    slack = ref.U * (w.abs()[:, :, None] * y.abs()).sum(1) * 1.01
    assert bool(((steps.double() - want).abs() <= err + slack).all())
