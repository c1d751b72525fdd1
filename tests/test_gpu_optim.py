"""AdamW on the MI355X against its 64-bit definition: every type, sizes around
each border, many tensors, 8-bit states, values that are not finite, device
scalars, graphs, streams, and a chain with the experts' gradients."""

import pytest
import torch

import optim_ref as ref

pytestmark = pytest.mark.gpu

HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
GUARD = 64  # elements behind a tensor that nothing may write


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_expert_token_amd as ms
    ms.load()


def ms():
    import moe_expert_token_amd
    return moe_expert_token_amd


def guarded(values):
    """A copy with guard elements behind it: (whole, the part)."""
    whole = torch.empty(values.numel() + GUARD, dtype=values.dtype, device="cuda")
    whole.view(torch.uint8).fill_(77)
    whole[: values.numel()] = values
    return whole, whole[: values.numel()]


def make(n, gen, param="fp32", grad="fp32", eight=False, copy=False):
    """Parameters, gradients and states of a run in progress; a third of the gradients are zero."""
    def normal(std):
        return torch.empty(n, device="cuda").normal_(0, std, generator=gen)

    keep = torch.rand(n, device="cuda", generator=gen)
    t = {"p": normal(0.1), "g": normal(1e-2) * keep ** 4 * (keep > 0.3)}
    if param == "bf16":
        t["p"] = t["p"].to(torch.bfloat16)
    if grad == "bf16":
        t["g"] = t["g"].to(torch.bfloat16)
    if copy:
        t["copy"] = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = normal(3e-3) * keep ** 3, normal(5e-3).square() * keep ** 6
    if eight:
        for name, dtype, size in (("m", torch.uint8, n), ("v", torch.uint8, n), ("m_scale", torch.float32, -(-n // 128)),
                                  ("v_scale", torch.float32, -(-n // 128))):
            t[name] = torch.zeros(size, dtype=dtype, device="cuda")
        t["m_out"], t["v_out"] = m, v
    else:
        t["m"], t["v"] = m, v
    t = {k: guarded(x) for k, x in t.items()}
    part = {k: x[1] for k, x in t.items()}
    if eight:
        ms().moe_adamw_pack(ms().AdamwTensors([part]))
    return {k: x[0] for k, x in t.items()}, part


def state(part):
    """m and v as 64-bit values."""
    if "m_scale" in part:
        return ref.m_value(part["m"], part["m_scale"]), ref.s_value(part["v"], part["v_scale"]) ** 2
    return part["m"].double(), part["v"].double()


def near(got, want, bound, what):
    err = (got.double() - want).abs()
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.3g} of the bound"


def check(part, before, step, scale=1.0, **hyper):
    """`part` after a step from the values `before` = (p, g, m, v) in 64 bits."""
    h = dict(HYPER, **hyper)
    p, m, v, ep, em, ev = ref.adamw(*before, step, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"], scale)
    half = part["p"].dtype == torch.bfloat16
    near(part["p"], p, ep + (ref.U * (p.abs() + ep) if half else 0), "p")
    if "copy" in part:
        assert torch.equal(part["copy"], part["p"].to(torch.bfloat16))
    if "m_scale" not in part:
        near(part["m"], m, em, "m")
        near(part["v"], v, ev, "v")
        return
    gm, gv = state(part)
    near(gm, m, em * 1.125 + ref.m_slack(m, part["m_scale"]) + ref.TINY, "m")
    s = v.sqrt()
    es = torch.minimum(ev.sqrt(), ev / (2 * s).clamp_min(1e-300)) + 2 * ref.STEP * s
    near(gv.sqrt(), s, es * 1.05 + ref.s_slack(s, part["v_scale"]) + ref.TINY, "s")
    assert bool((gv[s > 1e-30] > 0).all()), "a root came back as zero"
    for values, top, name in ((m, 448, "m_scale"), (s, 8064, "v_scale")):
        want = ref.scales(values, top)
        slack = ref.scales(em if name == "m_scale" else es, top) + 4 * ref.STEP * want
        near(part[name], want, slack, name)


def values_of(part):
    return (part["p"].double(), part["g"].double()) + state(part)


def guards_hold(whole):
    for name, t in whole.items():
        raw = t[-GUARD:].contiguous().view(torch.uint8)
        assert bool((raw == 77).all()), f"{name}: written past its end"


KINDS = [("fp32", "fp32", False, False), ("fp32", "bf16", False, True), ("bf16", "bf16", False, False),
         ("bf16", "fp32", False, False), ("fp32", "fp32", True, True), ("fp32", "bf16", True, False),
         ("bf16", "bf16", True, False), ("bf16", "fp32", True, False)]


@pytest.mark.parametrize("param,grad,eight,copy", KINDS)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 127, 128, 129, 2047, 2049, 8191, 8192, 8193, 30001])
def test_steps(n, param, grad, eight, copy):
    gen = torch.Generator(device="cuda").manual_seed(n)
    whole, part = make(n, gen, param, grad, eight, copy)
    tensors = ms().AdamwTensors([part])
    for step in (1, 2, 1000):
        before = values_of(part)
        ms().moe_adamw_step(tensors, step, **HYPER)
        check(part, before, step)
    guards_hold(whole)


@pytest.mark.parametrize("count", [2, 40, 41, 97])
@pytest.mark.parametrize("eight", [False, True])
def test_many_tensors(count, eight):
    gen = torch.Generator(device="cuda").manual_seed(count)
    made = [make([0, 3, 200, 8193, 64, 20000][i % 6], gen, "fp32", "bf16", eight, i % 2 == 0) for i in range(count)]
    before = [values_of(part) for _, part in made]
    ms().moe_adamw_step(ms().AdamwTensors([part for _, part in made]), 7, **HYPER)
    for (whole, part), b in zip(made, before):
        if part["p"].numel():
            check(part, b, 7)
        guards_hold(whole)
    ms().moe_adamw_step(ms().AdamwTensors([]), 1, **HYPER)


@pytest.mark.parametrize("hyper", [dict(beta1=0.0), dict(beta2=0.0), dict(lr=0.0), dict(weight_decay=0.0),
                                   dict(eps=0.0, beta2=0.999), dict(beta1=0.99999, beta2=0.9999999)])
@pytest.mark.parametrize("eight", [False, True])
def test_hyperparameters(hyper, eight):
    gen = torch.Generator(device="cuda").manual_seed(1)
    whole, part = make(3001, gen, "fp32", "fp32", eight, True)
    if hyper.get("eps") == 0:  # 0 / 0 has no value
        part["g"].clamp_(min=1e-6)
    before = values_of(part)
    ms().moe_adamw_step(ms().AdamwTensors([part]), 3, **dict(HYPER, **hyper))
    check(part, before, 3, **hyper)


def test_first_step_of_zero_states():
    for eight in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(2)
        whole, part = make(1000, gen, "fp32", "bf16", eight)
        for name in ("m", "v", "m_scale", "v_scale"):
            if name in part:
                part[name].zero_()
        before = values_of(part)
        assert float(before[2].abs().max()) == 0 and float(before[3].max()) == 0
        ms().moe_adamw_step(ms().AdamwTensors([part]), 1, **HYPER)
        check(part, before, 1)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_gradients_that_are_not_finite(value):
    """The element's own parameter and states, and with 8 bits its group's states."""
    for eight in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(3)
        whole, part = make(1000, gen, "fp32", "fp32", eight)
        clean = {k: t.clone() for k, t in part.items()}
        part["g"][300] = value
        ms().moe_adamw_step(ms().AdamwTensors([part]), 5, **HYPER)
        ms().moe_adamw_step(ms().AdamwTensors([clean]), 5, **HYPER)
        others = torch.arange(1000, device="cuda") != 300
        assert torch.equal(part["p"][others], clean["p"][others])
        assert bool(torch.isnan(part["p"][300]))  # infinity over infinity
        m, v = state(part)
        if eight:
            group = torch.arange(1000, device="cuda") // 128 == 300 // 128
            assert bool(torch.isnan(m[group]).all()) and bool(torch.isnan(v[group]).all())
            for name in ("m", "v", "m_scale", "v_scale"):
                keep = ~group if not name.endswith("scale") else torch.arange(8, device="cuda") != 300 // 128
                assert torch.equal(part[name][keep], clean[name][keep])
        else:
            assert not bool(torch.isfinite(m[300])) and not bool(torch.isfinite(v[300]))
            assert torch.equal(part["m"][others], clean["m"][others])


def test_pack_and_unpack():
    """Every code comes back to itself; values between codes go to the nearest; tiny, huge and zero groups."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    # all codes, each group with its largest: the step is exact where top is 448 and 8064 times a power of two
    codes_m = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)
    codes_m = codes_m[(codes_m & 127) != 127]
    codes_s = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)
    rows_m, rows_s = [], []
    for part in (codes_m[:127], codes_m[127:254], codes_m[200:254]):
        rows_m.append(torch.cat((part, torch.full((128 - part.numel(),), 0x7e, dtype=torch.uint8, device="cuda"))))
    for part in (codes_s[:127], codes_s[127:254], codes_s[129:256]):
        rows_s.append(torch.cat((part, torch.full((128 - part.numel(),), 255, dtype=torch.uint8, device="cuda"))))
    m, v = torch.cat(rows_m), torch.cat(rows_s)
    n = m.numel()
    steps = torch.tensor([1.0, 2.0 ** -20, 2.0 ** 30], device="cuda")
    part = dict(m=m.clone(), v=v.clone(), m_scale=steps.clone(), v_scale=steps.clone(),
                m_out=torch.empty(n, device="cuda"), v_out=torch.empty(n, device="cuda"))
    tensors = ms().AdamwTensors([part])
    ms().moe_adamw_unpack(tensors)
    assert torch.equal(part["m_out"].double(), ref.m_value(m, steps))
    assert torch.equal(part["v_out"].double(), ref.s_value(v, steps) ** 2)
    for name in ("m", "v", "m_scale", "v_scale"):
        part[name].zero_()
    ms().moe_adamw_pack(tensors)
    assert torch.equal(part["m"] & 127, m & 127)  # a zero may lose its sign
    assert torch.equal(part["m"][m & 127 != 0], m[m & 127 != 0])
    assert torch.equal(part["v"], v) and torch.equal(part["m_scale"], steps) and torch.equal(part["v_scale"], steps)
    half = dict(part, m_out=torch.empty(n, dtype=torch.bfloat16, device="cuda"),
                v_out=torch.empty(n, dtype=torch.bfloat16, device="cuda"))
    ms().moe_adamw_unpack(ms().AdamwTensors([half]))
    assert torch.equal(half["m_out"], part["m_out"].to(torch.bfloat16))
    assert torch.equal(half["v_out"], part["v_out"].to(torch.bfloat16))
    # random values of every size
    n = 128 * 64 + 5
    exponent = torch.randint(-140, 100, (-(-n // 128),), device="cuda", generator=gen)
    size = (2.0 ** exponent.double()).repeat_interleave(128)[:n]
    spread = 10.0 ** (-4 * torch.rand(n, device="cuda", generator=gen))
    a = (torch.randn(n, device="cuda", generator=gen) * spread * size).float()
    b = ((torch.randn(n, device="cuda", generator=gen) * spread).double().abs() * size.clamp(2.0 ** -60, 2.0 ** 60)).float()
    b[:128] = 0
    a[128:256] = 0
    whole = {k: guarded(t) for k, t in dict(m=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                                            v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                                            m_scale=torch.zeros(-(-n // 128), device="cuda"),
                                            v_scale=torch.zeros(-(-n // 128), device="cuda"), m_out=a,
                                            v_out=b.square()).items()}
    part = {k: t[1] for k, t in whole.items()}
    ms().moe_adamw_pack(ms().AdamwTensors([part]))
    m, s = part["m_out"].double(), part["v_out"].double().sqrt()
    near(ref.m_value(part["m"], part["m_scale"]), m, ref.m_slack(m, part["m_scale"]) + 1e-300, "m")
    near(ref.s_value(part["v"], part["v_scale"]), s, ref.s_slack(s, part["v_scale"]) + 4 * ref.STEP * s + 1e-300, "s")
    assert torch.equal(part["v"] == 0, s == 0)
    guards_hold({k: t[0] for k, t in whole.items()})


def test_negative_second_moments_and_bad_groups_pack():
    n = 256
    part = dict(m=torch.ones(n, dtype=torch.uint8, device="cuda"), v=torch.ones(n, dtype=torch.uint8, device="cuda"),
                m_scale=torch.ones(2, device="cuda"), v_scale=torch.ones(2, device="cuda"),
                m_out=torch.ones(n, device="cuda"), v_out=torch.full((n,), -1.0, device="cuda"))
    part["m_out"][200] = float("inf")
    ms().moe_adamw_pack(ms().AdamwTensors([part]))
    assert bool((part["v"] == 0).all())
    assert bool((part["m"][:128] == 0x7e).all()) and bool(torch.isnan(part["m_scale"][1]))


def test_device_scalars_and_graph():
    """A captured step follows the step's number, the rate and the gradients' factor; each replay equals eager steps."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    for eight in (False, True):
        _, part = make(20001, gen, "fp32", "bf16", eight, True)
        twin = {k: t.clone() for k, t in part.items()}
        lr = torch.zeros(1, device="cuda")
        step = torch.zeros(1, dtype=torch.int64, device="cuda")
        scale = torch.zeros(1, device="cuda")
        tensors, eager = ms().AdamwTensors([part]), ms().AdamwTensors([twin])
        hyper = {k: v for k, v in HYPER.items() if k != "lr"}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ms().moe_adamw_step(tensors, 0, 0.0, lr_device=lr, step_device=step, grad_scale=scale, **hyper)
        for i in range(1, 6):
            part["g"].normal_(0, 1e-2, generator=gen)
            twin["g"].copy_(part["g"])
            rate, factor = 1e-3 / i, 0.5 * i
            lr.fill_(rate)
            step.fill_(i)
            scale.fill_(factor)
            before = values_of(twin)
            graph.replay()
            torch.cuda.synchronize()
            ms().moe_adamw_step(eager, i, float(lr), grad_scale=scale, **hyper)
            for name in part:
                assert torch.equal(part[name], twin[name]), (name, i)
            check(twin, before, i, scale=float(scale), lr=float(lr))
            assert float(lr) != 0


def test_other_stream():
    gen = torch.Generator(device="cuda").manual_seed(6)
    _, part = make(50000, gen, "fp32", "bf16", False, True)
    twin = {k: t.clone() for k, t in part.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ms().moe_adamw_step(ms().AdamwTensors([part]), 4, stream=side, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    ms().moe_adamw_step(ms().AdamwTensors([twin]), 4, **HYPER)
    for name in part:
        assert torch.equal(part[name], twin[name])


def test_repeats_are_equal_and_split_does_not_matter():
    """Whole groups may be split over tensors as one likes: the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    _, part = make(128 * 300, gen, "fp32", "bf16", True)
    twin = {k: t.clone() for k, t in part.items()}
    ms().moe_adamw_step(ms().AdamwTensors([part]), 4, **HYPER)
    cuts = [0, 1, 66, 67, 200, 300]
    pieces = [{k: t[a:b] if k.endswith("scale") else t[128 * a:128 * b] for k, t in twin.items()}
              for a, b in zip(cuts, cuts[1:])]
    ms().moe_adamw_step(ms().AdamwTensors(pieces), 4, **HYPER)
    for name in part:
        assert torch.equal(part[name], twin[name])


def test_more_than_2_to_the_31_elements():
    """Offsets past 32 bits: the ends of a long tensor against the same values in a short one."""
    n = (1 << 31) + 128 * 3 + 17
    gen = torch.Generator(device="cuda").manual_seed(8)
    long = {"p": torch.zeros(n, dtype=torch.bfloat16, device="cuda"), "g": torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
            "m": torch.zeros(n, dtype=torch.uint8, device="cuda"), "v": torch.zeros(n, dtype=torch.uint8, device="cuda"),
            "m_scale": torch.zeros(-(-n // 128), device="cuda"), "v_scale": torch.zeros(-(-n // 128), device="cuda")}
    _, short = make(128 * 4 + 17, gen, "bf16", "bf16", True)
    at = n - 128 * 4 - 17
    for name in long:
        (long[name][at // 128:] if name.endswith("scale") else long[name][at:]).copy_(short[name])
    ms().moe_adamw_step(ms().AdamwTensors([long]), 9, **HYPER)
    ms().moe_adamw_step(ms().AdamwTensors([{k: short[k] for k in long}]), 9, **HYPER)
    for name in long:
        assert torch.equal(long[name][at // 128:] if name.endswith("scale") else long[name][at:], short[name]), name
    assert float(long["p"][:at:1001].abs().max()) == 0


def test_8_bit_states_follow_fp32_ones():
    """Two hundred steps on a noisy quadratic: the second moments that 8 bits hold stay near those of fp32 states, and
    do not stand still (an 8-bit scale would hold them at their first size)."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    n = 128 * 64
    whole, a = make(n, gen, "fp32", "fp32", True)
    _, b = make(n, gen, "fp32", "fp32", False)
    size = torch.rand(n, device="cuda", generator=gen) * 0.9 + 0.1
    for t in (a, b):
        for name in ("m", "v", "m_scale", "v_scale"):
            if name in t:
                t[name].zero_()
    b["p"].copy_(a["p"])
    eight, wide = ms().AdamwTensors([a]), ms().AdamwTensors([b])
    for step in range(1, 201):
        a["g"].normal_(0, 1.0 if step <= 20 else 0.1, generator=gen).mul_(size)
        b["g"].copy_(a["g"])
        ms().moe_adamw_step(eight, step, 1e-3, 0.9, 0.98)
        ms().moe_adamw_step(wide, step, 1e-3, 0.9, 0.98)
    _, va = state(a)
    ratio = va.sqrt() / b["v"].double().sqrt()
    mean = float(ratio.log().mean().exp())
    print("roots of second moments, 8 bits over fp32: geometric mean", mean, "spread", float(ratio.log().std()))
    # a root is held to 2^-6 and moves by a hundredth a step: it follows with a lag, and not by a factor of three, as
    # the first twenty steps' size would be
    assert 0.5 < mean < 2
