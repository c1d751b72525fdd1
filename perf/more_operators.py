"""What stands around the experts' block, as measured work.

  layer   a whole mixture-of-experts layer for a few tokens: router, experts
          (weights "bf16", or "w4": 4 bits with group scales) and combine
  router  logits, top-k ids and gates of a batch; with `train` its backward
          pass too, from the gates' gradients to those of rows and weights
  adamw   a step over many tensors at once, states in 32 bits or in 8 (then
          followed by unpacking the states, as a checkpoint does)

`run` computes them with elementary torch operations in 32 bits (in 64 where
the choice of experts hangs on them), or, where `own` is true, through this
repository's package.
"""

import math

import torch

own = False

GROUP_STATE = 128  # elements that share a scale in 8-bit optimizer states
BETA1, BETA2, EPS, DECAY, LR, STEP = 0.9, 0.999, 1e-8, 0.1, 1e-3, 1000


def listed():
    return [
        # one token through the widths of the bench's 256-token batch: nothing but latency
        dict(name="layer-tiny", op="layer", weights="bf16", T=1, H=128, E=8, k=2, I=256, act="silu", score="softmax",
             norm=True),
        # a decode step of four sequences through wide experts: the weights' bytes count
        dict(name="layer-decode", op="layer", weights="bf16", T=4, H=4096, E=8, k=2, I=14336, act="silu",
             score="softmax", norm=True),
        # speculative decoding at odd widths: sigmoid scores with a bias, rows that do not fill a tile
        dict(name="layer-ragged", op="layer", weights="bf16", T=37, H=1544, E=40, k=6, I=712, act="gelu",
             score="sigmoid", norm=True),
        # one token through 4-bit experts of the DeepSeek-V3-like widths: the latency of a single sequence
        dict(name="layer-w4-one", op="layer", weights="w4", T=1, H=7168, E=256, k=8, I=2048, group=128, act="silu",
             score="sigmoid", norm=True),
        # a decode step of 48 sequences there: most experts have a row or two
        dict(name="layer-w4-decode", op="layer", weights="w4", T=48, H=7168, E=256, k=8, I=2048, group=128,
             act="silu", score="sigmoid", norm=True),
        # the router of a chunk of a prompt, for inference
        dict(name="router-chunk", op="router", train=False, T=256, H=4096, E=8, k=2, score="softmax", norm=True),
        # the router of the DeepSeek-V3-like batch of the bench, for inference
        dict(name="router-deepseek", op="router", train=False, T=8192, H=7168, E=256, k=8, score="sigmoid",
             norm=True),
        # its training step
        dict(name="router-train-deepseek", op="router", train=True, T=8192, H=7168, E=256, k=8, score="sigmoid",
             norm=True),
        # a training step of odd sizes, plain softmax gates
        dict(name="router-train-ragged", op="router", train=True, T=1999, H=1544, E=40, k=6, score="softmax",
             norm=False),
        # a small model's step: forty tensors from a bias of 6 elements on, fp32 parameters and gradients
        dict(name="adamw-small", op="adamw", state="fp32", param="fp32", grad="fp32", H=520, E=6, I=136, layers=8),
        # experts of the 8-bit-checkpoint training step: fp32 parameters with their bf16 copy, fp32 states
        dict(name="adamw-experts", op="adamw", state="fp32", param="fp32+bf16", grad="bf16", H=2048, E=16, I=1000,
             layers=2),
        # the DeepSeek-V3-like widths on 32 experts, 8-bit states
        dict(name="adamw-deepseek-8bit", op="adamw", state="8bit", param="fp32+bf16", grad="bf16", H=7168, E=32,
             I=2048, layers=1),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["layer", "layer", "w4", "router", "router", "adamw"])
    act = rng.choice(["silu", "silu", "gelu"])
    score = rng.choice(["softmax", "sigmoid"])
    norm = rng.choice([True, True, False])
    if op == "adamw":
        H, E, I = 8 * log_int(8, 512), log_int(1, 16), 8 * log_int(8, 512)
        return dict(op=op, state=rng.choice(["fp32", "8bit"]), param=rng.choice(["fp32", "fp32+bf16", "bf16"]),
                    grad=rng.choice(["bf16", "bf16", "fp32"]), H=H, E=E, I=I,
                    layers=max(1, min(rng.randint(1, 12), int(4e8 / (3 * E * H * I)))))
    if op == "router":
        E, train = log_int(2, 256), rng.choice([True, False])
        # one normalized gate is constant: it has no gradient
        k = rng.randint(2 if train and norm else 1, min(8, E))
        return dict(op=op, train=train, T=log_int(1, 8192), H=8 * log_int(8, 896), E=E, k=k, score=score, norm=norm)
    E = log_int(2, 128)
    case = dict(op="layer", weights="bf16", T=log_int(1, 64), H=8 * log_int(8, 512), E=E, k=rng.randint(1, min(8, E)),
                I=8 * log_int(8, 512), act=act, score=score, norm=norm)
    if op == "w4":
        group = rng.choice([32, 64, 128])
        case.update(weights="w4", group=group, H=group * log_int(2, 4096 // group), I=group * log_int(2, 4096 // group))
    return case


def _normal(gen, shape, std, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _gate_scale(case):
    return 2.5 if case["score"] == "sigmoid" else 1.0


def _sizes(case):
    """Elements of each parameter of a layer: experts, router, its bias, a norm."""
    H, E, I = case["H"], case["E"], case["I"]
    return [E * 2 * I * H, E * H * I, E * H, E, H]


def _prepare_adamw(case, gen):
    """One buffer for each kind of value, as programs keep parameters; a tensor is a part of it, and starts at a whole
    group. What lies behind a tensor's end is zero."""
    sizes = _sizes(case) * case["layers"]
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // GROUP_STATE) * GROUP_STATE)
    total = at[-1]
    inside = torch.ones(total, dtype=torch.bool, device="cuda")
    for lo, n, hi in zip(at, sizes, at[1:]):
        inside[lo + n: hi] = False
    s = dict(case=case, p=_normal(gen, (total,), 0.02, torch.float32).mul_(inside))
    # gradients differ in size from element to element; where nothing was routed they are zero
    g = _normal(gen, (total,), 1e-3, torch.float32).mul_(inside)
    g *= torch.rand(total, device="cuda", generator=gen) ** 3
    g[: total // 16] = 0
    m, v = g * 0.3, g * g * 0.5
    m += _normal(gen, (total,), 1e-4, torch.float32).mul_(inside)
    v += _normal(gen, (total,), 1e-4, torch.float32).mul_(inside).square_()
    s["g"] = g if case["grad"] == "fp32" else g.to(torch.bfloat16)
    if case["param"] != "fp32":
        half = s["p"].to(torch.bfloat16)
        s["p" if case["param"] == "bf16" else "copy"] = half
    if case["state"] == "8bit":
        s["m"], s["m_scale"] = _pack_m(m)
        s["v"], s["v_scale"] = _pack_s(v.sqrt_())
        s["m_out"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    else:
        s["m"], s["v"] = m, v
    if own:
        import moe_expert_token_amd as ms

        def tensors(*names):
            return ms.AdamwTensors([{name: s[name][lo // GROUP_STATE: hi // GROUP_STATE] if name.endswith("scale")
                                     else s[name][lo: lo + n] for name in names if name in s}
                                    for lo, n, hi in zip(at, sizes, at[1:])])

        s["list"] = tensors("p", "copy", "g", "m", "v", "m_scale", "v_scale")
        if case["state"] == "8bit":
            s["states"] = tensors("m", "v", "m_scale", "v_scale", "m_out", "v_out")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    T, H, E, k = (case[n] for n in "T H E k".split())
    s = dict(case=case)
    s["x"] = _normal(gen, (T, H), 1.0)
    s["w_router"] = _normal(gen, (E, H), 1.0 / math.sqrt(H))
    # what balances sigmoid scores; softmax has none
    s["bias"] = _normal(gen, (E,), 0.05, torch.float32) if case["score"] == "sigmoid" else None
    if case["op"] == "router" and case["train"]:
        s["grad_topk_w"] = _normal(gen, (T, k), 1.0, torch.float32)
        # of the size that the gates' part has
        s["grad_x_in"] = _normal(gen, (T, H), 0.01)
    if case["op"] == "layer":
        I = case["I"]
        s["residual"] = _normal(gen, (T, H), 1.0)
        if case["weights"] == "w4":
            g = case["group"]
            s["q_gate_up"] = torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, device="cuda", generator=gen)
            s["q_down"] = torch.randint(0, 256, (E, H, I // 2), dtype=torch.uint8, device="cuda", generator=gen)
            # a uniform 4-bit value has a standard deviation of 4.6
            for name, n, w in (("s_gate_up", 2 * I, H), ("s_down", H, I)):
                sc = torch.rand((E, n, w // g), device="cuda", generator=gen) + 0.5
                s[name] = (sc / (4.6 * math.sqrt(w))).to(torch.bfloat16)
        else:
            s["w_gate_up"] = _normal(gen, (E, 2 * I, H), 1.0 / math.sqrt(H))
            s["w_down"] = _normal(gen, (E, H, I), 1.0 / math.sqrt(I))
    if own:
        import moe_expert_token_amd as ms
        dims = s["dims"] = ms.dims_of(T, H, E, k, 1)
        s["rule"] = ms.RouterRule(scoring=ms.SCORE_SOFTMAX if case["score"] == "softmax" else ms.SCORE_SIGMOID,
                                  normalize=case["norm"], scale=_gate_scale(case), bias=s["bias"])
        if case["op"] == "layer":
            nbytes = ms.moe_layer_workspace_size(dims, case["I"])
            s["out"] = torch.empty_like(s["x"])
        else:
            nbytes = ms.moe_router_workspace_size(dims, backward=case["train"])
            s["logits"] = torch.empty((T, E), dtype=torch.float32, device="cuda")
            if case["train"]:
                s["grad_x"] = torch.empty_like(s["x"])
                s["grad_w_router"] = torch.empty_like(s["w_router"])
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        s["topk_idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["topk_w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    return s


# ---- the plain forms ----

def _scores(case, l):
    return torch.softmax(l, dim=1) if case["score"] == "softmax" else 1 / (1 + torch.exp(-l))


def _route(s):
    """Logits in 64 bits, ids by falling key (ties to the lowest index), scores of the chosen, gates."""
    case = s["case"]
    l = s["x"].double() @ s["w_router"].double().T
    score = _scores(case, l)
    key = l if s["bias"] is None else score + s["bias"].double()
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, : case["k"]]
    w = score.gather(1, idx)
    if case["norm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return l, idx, w * _gate_scale(case)


def _slope(act):
    """(c0, c1) of the gate's sigmoid argument a(g) = c0 g + c1 g^3: g * sigmoid(a(g)) is SiLU, or GELU's tanh form."""
    return (1.0, 0.0) if act == "silu" else (2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715)


def _weights(s, name, used):
    if s["case"]["weights"] == "bf16":
        return s["w_" + name][used].float()
    q, scale = s["q_" + name][used], s["s_" + name][used]
    v = torch.stack((q & 15, q >> 4), dim=-1).reshape(q.shape[0], q.shape[1], -1).float() - 8
    return v * scale.float().repeat_interleave(s["case"]["group"], dim=-1)


def _layer(s):
    case = s["case"]
    T, k, H = case["T"], case["k"], case["H"]
    _, idx, w = _route(s)
    w = w.float()
    # pairs in the order of their experts, each expert's rows from 0 on
    order = torch.argsort(idx.flatten(), stable=True)
    count = torch.bincount(idx.flatten(), minlength=case["E"])
    used = count.nonzero().view(-1)
    expert = idx.flatten()[order]
    slot = (count > 0).long().cumsum(0)[expert] - 1
    place = torch.arange(T * k, device="cuda") - (count.cumsum(0) - count)[expert]
    x = torch.zeros((used.numel(), int(count.max()), H), device="cuda")
    x[slot, place] = s["x"][order // k].float()
    g, u = torch.bmm(x, _weights(s, "gate_up", used).transpose(1, 2)).chunk(2, dim=2)
    c0, c1 = _slope(case["act"])
    h = g / (1 + torch.exp(-(c0 * g + c1 * g * g * g))) * u
    y = torch.bmm(h, _weights(s, "down", used).transpose(1, 2))[slot, place]
    rows = torch.empty_like(y)
    rows[order] = y
    out = s["residual"].float() + (w[:, :, None] * rows.view(T, k, H)).sum(1)
    return dict(out=out.to(torch.bfloat16), topk_idx=idx.to(torch.int32), topk_w=w)


def _router(s):
    case = s["case"]
    l, idx, w = _route(s)
    out = dict(logits=l.float(), topk_idx=idx.to(torch.int32), topk_w=w.float())
    if not case["train"]:
        return out
    score = _scores(case, l.float())
    at, g = score.gather(1, idx), s["grad_topk_w"] * _gate_scale(case)
    if case["norm"]:
        total = at.sum(1, keepdim=True) + 1e-20
        g = (g - (g * at).sum(1, keepdim=True) / total) / total
    if case["score"] == "sigmoid":
        dl = torch.zeros_like(score).scatter_(1, idx, g * at * (1 - at))
    else:
        dl = torch.zeros_like(score).scatter_(1, idx, g)
        dl = score * (dl - (g * at).sum(1, keepdim=True))
    out["grad_x"] = (s["grad_x_in"].float() + dl @ s["w_router"].float()).to(torch.bfloat16)
    out["grad_w_router"] = (dl.T @ s["x"].float()).to(torch.bfloat16)
    return out


def _grouped(t):
    """[groups, GROUP_STATE], zeros behind the last element, and each group's largest magnitude."""
    t = torch.nn.functional.pad(t, (0, -t.numel() % GROUP_STATE)).view(-1, GROUP_STATE)
    return t, t.abs().amax(1)


def _pack_m(m):
    """The first moment: e4m3 of the quotient by a fp32 step, the group's largest magnitude / 448."""
    rows, top = _grouped(m)
    step = (top / 448).clamp(min=2.0 ** -126)
    code = (rows * (1 / step)[:, None]).to(torch.float8_e4m3fn)
    return code.view(-1)[: m.numel()].view(torch.uint8).clone(), step


def _pack_s(s):
    """The root of the second moment over a fp32 step (the group's largest / 8064) as (32 + c % 32) 2^(c // 32) with the
    nearest c from 1 to 255, the even one of two; 0 for 0."""
    rows, top = _grouped(s)
    step = (top / 8064).clamp(min=2.0 ** -126)
    bits = (rows * (1 / step)[:, None]).view(torch.int32)
    code = (((bits + 0x1ffff + ((bits >> 18) & 1)) >> 18) - (132 << 5)).clamp(1, 255)
    code = torch.where(rows > 0, code, torch.zeros_like(code))
    return code.view(-1)[: s.numel()].to(torch.uint8), step


def _wide(step, n):
    return step.repeat_interleave(GROUP_STATE)[:n]


def _unpack_m(code, step):
    return code.view(torch.float8_e4m3fn).float() * _wide(step, code.numel())


def _unpack_s(code, step):
    c = code.to(torch.int32)
    t = torch.where(c > 0, ((c + (132 << 5)) << 18).view(torch.float32), torch.zeros((), device="cuda"))
    return t * _wide(step, code.numel())


def _adamw(s):
    eight = s["case"]["state"] == "8bit"
    g = s["g"].float()
    m = (_unpack_m(s["m"], s["m_scale"]) if eight else s["m"]) * BETA1 + g * (1 - BETA1)
    v = (_unpack_s(s["v"], s["v_scale"]).square_() if eight else s["v"]) * BETA2 + g * g * (1 - BETA2)
    root = v.sqrt()
    p = s["p"].float() * (1 - LR * DECAY)
    p -= (LR / (1 - BETA1 ** STEP)) * m / (root / math.sqrt(1 - BETA2 ** STEP) + EPS)
    s["p"].copy_(p)
    if "copy" in s:
        s["copy"].copy_(p)
    if eight:
        for value, pack in ((m, _pack_m), (root, _pack_s)):
            name = "m" if pack is _pack_m else "v"
            code, step = pack(value)
            s[name].copy_(code)
            s[name + "_scale"].copy_(step)
        s["m_out"].copy_(_unpack_m(s["m"], s["m_scale"]))
        s["v_out"].copy_(_unpack_s(s["v"], s["v_scale"]).square_())
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    names = ("p", "copy", "m_out", "v_out") if s["case"]["state"] == "8bit" else ("p", "copy", "m", "v")
    return {name: s[name] for name in names if name in s}


def _plain(s):
    if s["case"]["op"] == "layer":
        return _layer(s)
    return _router(s) if s["case"]["op"] == "router" else _adamw(s)


# ---- the package's calls ----

def _own(s):
    import moe_expert_token_amd as ms
    case = s["case"]
    if case["op"] == "adamw":
        ms.moe_adamw_step(s["list"], step=STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY)
        if case["state"] == "8bit":
            ms.moe_adamw_unpack(s["states"])
        return _adamw_out(s)
    if case["op"] == "router":
        ms.moe_router_forward(s["dims"], s["rule"], s["x"], s["w_router"], s["topk_idx"], s["topk_w"], s["ws"],
                              logits=s["logits"])
        names = ["logits", "topk_idx", "topk_w"]
        if case["train"]:
            ms.moe_router_backward(s["dims"], s["rule"], s["grad_topk_w"], s["logits"], s["topk_idx"], s["x"],
                                   s["w_router"], s["grad_x"], s["grad_w_router"], s["ws"], grad_x_in=s["grad_x_in"])
            names += ["grad_x", "grad_w_router"]
        return {n: s[n] for n in names}
    act = ms.ACT_SILU if case["act"] == "silu" else ms.ACT_GELU_TANH
    kept = dict(residual=s["residual"], topk_idx=s["topk_idx"], topk_w=s["topk_w"], act=act)
    if case["weights"] == "w4":
        ms.moe_layer_w4_forward(s["dims"], s["rule"], s["x"], s["w_router"], s["q_gate_up"], s["s_gate_up"],
                                s["q_down"], s["s_down"], s["out"], s["ws"], group=case["group"], **kept)
    else:
        ms.moe_layer_forward(s["dims"], s["rule"], s["x"], s["w_router"], s["w_gate_up"], s["w_down"], s["out"],
                             s["ws"], **kept)
    return {n: s[n] for n in ("out", "topk_idx", "topk_w")}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    H, E = case["H"], case["E"]
    if case["op"] == "adamw":
        n = case["layers"] * sum(_sizes(case))
        param = {"fp32": 8, "fp32+bf16": 10, "bf16": 4}[case["param"]] + (2 if case["grad"] == "bf16" else 4)
        # 8 bits: two codes read and written, scales, and the way back to bf16
        return dict(bytes=n * (param + (16 if case["state"] == "fp32" else 4 + 6 + 24 / GROUP_STATE)), flops=0)
    T, k = case["T"], case["k"]
    if case["op"] == "router":
        nbytes = 2 * T * H + 2 * E * H + 4 * T * E + 8 * T * k
        if not case["train"]:
            return dict(bytes=nbytes, flops=2 * T * E * H)
        # again x and the weights, logits, ids and gates' gradients; grad_x in and out, the weights' gradient
        return dict(bytes=2 * nbytes + 4 * T * H + 2 * E * H, flops=6 * T * E * H)
    weights = 3 * H * case["I"]
    # experts that have a row, on average over even routing
    used = E * (1 - (1 - k / E) ** T)
    held = 2 if case["weights"] == "bf16" else 0.5 + 2 / case["group"]
    return dict(bytes=used * weights * held + 2 * E * H + 6 * T * H + 8 * T * k,
                flops=2 * T * k * weights + 2 * T * E * H)


# ---- the definition, in 64 bits ----

def _exact_gates(case, s, t):
    """One token: logits, ids in falling order of their keys, scores, gates."""
    l = s["w_router"].double().mv(s["x"][t].double())
    if case["score"] == "softmax":
        e = torch.exp(l - l.max())
        score = e / e.sum()
    else:
        score = torch.sigmoid(l)
    key = (l if s["bias"] is None else score + s["bias"].double()).tolist()
    idx = sorted(range(case["E"]), key=lambda e: (-key[e], e))[: case["k"]]
    at = score[idx]
    scale = _gate_scale(case)
    return l, idx, score, (scale * at / (at.sum() + 1e-20) if case["norm"] else scale * at)


def _exact_layer(case, s):
    I = case["I"]
    c0, c1 = _slope(case["act"])
    out, gates, ids, pairs = s["residual"].double().clone(), [], [], {}
    for t in range(case["T"]):
        _, idx, _, w = _exact_gates(case, s, t)
        gates.append(w)
        ids.append(idx)
        for j, e in enumerate(idx):
            pairs.setdefault(e, []).append((t, j))

    def weight(name, e):
        if case["weights"] == "bf16":
            return s["w_" + name][e].double()
        q, sc = s["q_" + name][e].long(), s["s_" + name][e].double()
        v = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = q % 16 - 8, q // 16 - 8
        return (v.view(q.shape[0], -1, case["group"]) * sc[:, :, None]).view(q.shape[0], -1)

    for e, rows in pairs.items():
        t = [r[0] for r in rows]
        pre = s["x"][t].double() @ weight("gate_up", e).T
        g, u = pre[:, :I], pre[:, I:]
        y = (g * torch.sigmoid(c0 * g + c1 * g ** 3) * u) @ weight("down", e).T
        out[t] += torch.stack([gates[a][b] for a, b in rows])[:, None] * y
    return dict(out=out, topk_idx=torch.tensor(ids, dtype=torch.int32, device="cuda"), topk_w=torch.stack(gates))


def _exact_router(case, s):
    l = torch.matmul(s["x"].double(), s["w_router"].double().T)
    score = (l - l.logsumexp(1, keepdim=True)).exp() if case["score"] == "softmax" else torch.sigmoid(l)
    key = l if s["bias"] is None else score + s["bias"].double()
    idx = key.topk(case["k"], dim=1).indices
    # gates as a function of the logits, its gradient by torch
    leaf = l.clone().requires_grad_(True)
    sc = torch.softmax(leaf, 1) if case["score"] == "softmax" else torch.sigmoid(leaf)
    w = sc.gather(1, idx)
    if case["norm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = w * _gate_scale(case)
    out = dict(logits=l, topk_idx=None, topk_w=w.detach())
    if case["train"]:
        (dl,) = torch.autograd.grad(w, leaf, s["grad_topk_w"].double())
        out["grad_x"] = s["grad_x_in"].double() + torch.matmul(dl, s["w_router"].double())
        out["grad_w_router"] = torch.matmul(dl.T.contiguous(), s["x"].double())
    return out


def _exact_adamw(case, s):
    eight = case["state"] == "8bit"
    parts = dict(p=[], m=[], v=[])
    size = 1 << 24  # a multiple of the group: bounds the room that 64 bits take
    for lo in range(0, s["p"].numel(), size):
        cut, groups = slice(lo, lo + size), slice(lo // GROUP_STATE, (lo + size) // GROUP_STATE)
        g, p = s["g"][cut].double(), s["p"][cut].double()
        if eight:
            m = s["m"][cut].view(torch.float8_e4m3fn).double().view(-1, GROUP_STATE)
            m = (m * s["m_scale"][groups].double()[:, None]).view(-1)
            c = s["v"][cut].long().view(-1, GROUP_STATE)
            root = torch.where(c > 0, (32 + c % 32) * 2.0 ** (c // 32).double(), 0.0)
            v = ((root * s["v_scale"][groups].double()[:, None]) ** 2).view(-1)
        else:
            m, v = s["m"][cut].double(), s["v"][cut].double()
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        parts["p"].append(p - LR * DECAY * p
                          - LR * (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS))
        if not eight:
            parts["m"].append(m)
            parts["v"].append(v)
    out = dict(p=torch.cat(parts["p"]))
    if "copy" in s:
        out["copy"] = out["p"]
    if eight:  # what 8 bits hold of a value next to a border is either neighbour: no exact value
        return {**out, "m_out": None, "v_out": None}
    return {**out, "m": torch.cat(parts["m"]), "v": torch.cat(parts["v"])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    return _exact_layer(case, s) if case["op"] == "layer" else _exact_router(case, s)
