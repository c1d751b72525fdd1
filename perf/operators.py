"""The experts' own operators between dispatch and combine, as measured work.

Four passes over expert-major rows (what dispatch leaves in xe):

  forward     the gated feed-forward block of every expert, bf16 weights
  train       the same with its pre-activations saved, then its backward pass;
              `saved` says how they are held in between: bf16, or 8 bits
  w4          the block for few tokens, 4-bit weights with group scales
  checkpoint  8-bit activation checkpoints on their own: rows packed to 8 bits
              and unpacked again

`run` computes them with elementary torch operations in 32 bits, or, where
`own` is true, through this repository's package.
"""

import math

import torch

own = False

GROUP8 = 32  # elements that share a scale in an 8-bit checkpoint


def listed():
    return [
        # the 256-token batch of the bench: launches and latency count
        dict(name="forward-tiny", op="forward", T=256, H=128, E=8, k=2, R=4, I=256, act="silu", skew=0.0),
        # a decode step of four sequences through wide experts: the weights' bytes count
        dict(name="forward-decode", op="forward", T=4, H=4096, E=8, k=2, R=8, I=14336, act="silu", skew=0.0),
        # odd widths, popular and empty experts, a ragged last tile everywhere
        dict(name="forward-ragged", op="forward", T=1999, H=1544, E=40, k=6, R=8, I=712, act="gelu", skew=1.2),
        # the DeepSeek-V3-like batch of the bench, 256 rows an expert on average
        dict(name="forward-deepseek", op="forward", T=8192, H=7168, E=256, k=8, R=32, I=2048, act="silu", skew=0.0),
        # a training step of the Mixtral-like batch: few wide experts, large products
        dict(name="train-mixtral", op="train", saved="bf16", T=4096, H=4096, E=8, k=2, R=8, I=14336, act="silu",
             skew=0.0),
        # a training step of odd sizes, experts without a row among them
        dict(name="train-ragged", op="train", saved="bf16", T=777, H=1160, E=48, k=3, R=4, I=520, act="gelu",
             skew=1.2),
        # a training step of the DeepSeek-V3-like widths on 32 experts, 8-bit checkpoints
        dict(name="train-deepseek-8bit", op="train", saved="int8", T=4096, H=7168, E=32, k=8, R=4, I=2048,
             act="silu", skew=0.0),
        # a smaller training step with 8-bit checkpoints, groups that end inside a tile
        dict(name="train-small-8bit", op="train", saved="int8", T=1500, H=2048, E=16, k=4, R=4, I=1000, act="silu",
             skew=0.0),
        # the activations of the DeepSeek-V3-like batch, packed and unpacked
        dict(name="checkpoint-deepseek", op="checkpoint", rows=8192, cols=7168),
        # one token through 4-bit experts: the latency of a single sequence
        dict(name="w4-one-token", op="w4", T=1, H=7168, E=256, k=8, R=32, I=2048, group=128, act="silu", skew=0.0),
        # a decode step of 48 sequences: most experts have a row or two
        dict(name="w4-decode", op="w4", T=48, H=7168, E=256, k=8, R=32, I=2048, group=128, act="silu", skew=0.0),
        # speculative or chunked decoding: many rows for few experts, small groups
        dict(name="w4-chunk", op="w4", T=203, H=4096, E=8, k=2, R=8, I=14336, group=32, act="silu", skew=0.0),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["forward", "forward", "train", "train", "w4", "w4", "checkpoint"])
    if op == "checkpoint":
        return dict(op=op, rows=log_int(1, 8192), cols=8 * log_int(1, 896))
    R = rng.choice([1, 2, 4, 8])
    E = R * rng.choice([1, 2, 4, 8, 16] if op == "w4" else [1, 2, 3, 6, 8])
    k = rng.randint(1, min(8, E))
    skew = rng.choice([0.0, 0.0, 1.2])
    act = rng.choice(["silu", "silu", "gelu"])
    if op == "w4":
        group = rng.choice([32, 64, 128])
        return dict(op=op, T=log_int(1, 256), H=group * log_int(2, 4096 // group), E=E, k=k, R=R,
                    I=group * log_int(2, 4096 // group), group=group, act=act, skew=skew)
    case = dict(op=op, T=log_int(1, 4096), H=8 * log_int(8, 512), E=E, k=k, R=R, I=8 * log_int(8, 512), act=act,
                skew=skew)
    if op == "train":
        case["saved"] = rng.choice(["bf16", "int8"])
    return case


def _normal(gen, shape, std):
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return t.normal_(0.0, std, generator=gen)


def _routing(case, gen):
    """Top-k of Gumbel-perturbed popularities: k distinct experts a token."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen).clamp_(1e-9, 1 - 1e-7)))
    logits += -case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return logits.topk(k, dim=1).indices.to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "checkpoint":
        x = _normal(gen, (case["rows"], case["cols"]), 1.0)
        # activations have a few channels that are far larger than the others
        big = torch.rand(case["cols"], device="cuda", generator=gen) < 0.01
        x[:, big] *= 30
        s["x"] = x
        if own:
            groups = -(-case["cols"] // GROUP8)
            s["q"] = torch.empty(x.shape, dtype=torch.int8, device="cuda")
            s["scale"] = torch.empty((case["rows"], groups), dtype=torch.bfloat16, device="cuda")
            s["back"] = torch.empty_like(x)
        return s

    T, H, E, k, R, I = (case[n] for n in "T H E k R I".split())
    rows = T * k
    s["idx"] = _routing(case, gen)
    count = torch.bincount(s["idx"].view(-1).long(), minlength=E)
    s["offset"] = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), count.cumsum(0)])
    # where the plain form puts each row: (place among the experts with rows, place in its expert)
    s["used"] = count.nonzero().view(-1)
    s["cap"] = int(count.max())
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), count)
    s["slot"] = (count > 0).long().cumsum(0)[expert] - 1
    s["place"] = torch.arange(rows, device="cuda") - s["offset"][expert]
    s["xe"] = _normal(gen, (rows, H), 1.0)
    if case["op"] == "w4":
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
    if case["op"] == "train":
        s["grad_ye"] = _normal(gen, (rows, H), 1.0)
    if own:
        import moe_expert_token_amd as ms
        dims = ms.dims_of(T, H, E, k, R)
        plan_ws = torch.empty(ms.moe_shuffle_workspace_size(dims), dtype=torch.uint8, device="cuda")
        s["plan"] = ms.moe_shuffle_plan(dims, s["idx"], plan_ws)
        train = case["op"] == "train"
        s["ws"] = torch.empty(ms.moe_experts_ffn_workspace_size(dims, I, backward=train), dtype=torch.uint8,
                              device="cuda")
        s["ye"] = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
        if train:
            eight = case["saved"] == "int8"
            s["saved"] = torch.empty((rows, 2 * I), dtype=torch.int8 if eight else torch.bfloat16, device="cuda")
            s["scale"] = torch.empty((rows, 2, -(-I // GROUP8)), dtype=torch.bfloat16, device="cuda") \
                if eight else None
            s["grad_xe"] = torch.empty_like(s["xe"])
            s["grad_w_gate_up"] = torch.empty_like(s["w_gate_up"])
            s["grad_w_down"] = torch.empty_like(s["w_down"])
    return s


# ---- the plain form, in 32 bits ----

def _slope(act):
    """(c0, c1) of the gate's sigmoid argument a(g) = c0 g + c1 g^3: g * sigmoid(a(g)) is SiLU, or GELU's tanh form."""
    return (1.0, 0.0) if act == "silu" else (2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715)


def _gate(g, act):
    """The gate's activation and its derivative."""
    c0, c1 = _slope(act)
    sig = 1 / (1 + torch.exp(-(c0 * g + c1 * g * g * g)))
    return g * sig, sig + g * sig * (1 - sig) * (c0 + 3 * c1 * g * g)


def _spread(s, rows):
    """Expert-major rows -> [experts with rows, most rows, width] in 32 bits, zeros behind each expert's last."""
    t = torch.zeros((s["used"].numel(), s["cap"], rows.shape[1]), device="cuda")
    t[s["slot"], s["place"]] = rows.float()
    return t


def _weights(s, w):
    return (w if s["used"].numel() == w.shape[0] else w[s["used"]]).float()


def _by_expert(s, w):
    """Gradients of the experts with rows -> of all, zero for those without, in bf16."""
    if s["used"].numel() == s["case"]["E"]:
        return w.to(torch.bfloat16)
    out = torch.zeros((s["case"]["E"],) + w.shape[1:], dtype=torch.bfloat16, device="cuda")
    out[s["used"]] = w.to(torch.bfloat16)
    return out


def _four_bit(s, q, scale):
    """Two 4-bit values a byte, the even column low; a value v stands for (v - 8) * its group's scale."""
    q, scale = (t if s["used"].numel() == t.shape[0] else t[s["used"]] for t in (q, scale))
    v = torch.stack((q & 15, q >> 4), dim=-1).reshape(q.shape[0], q.shape[1], -1).float() - 8
    return v * scale.float().repeat_interleave(s["case"]["group"], dim=-1)


def _eight_bit(t):
    """The values that an 8-bit checkpoint of t's rows holds: along each row GROUP8 elements share a bf16 scale,
    the least bf16 value that is no less than their largest magnitude over 127; 8 bits hold the quotient's nearest."""
    width = t.shape[-1]
    t = torch.nn.functional.pad(t, (0, -width % GROUP8)).unflatten(-1, (-1, GROUP8))
    step = (t.abs().amax(-1, keepdim=True) / 127).clamp(min=2.0 ** -126)
    step = ((step.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)
    return (torch.round(t * (1 / step)).clamp(-127, 127) * step).flatten(-2)[..., :width]


def _plain(s):
    case = s["case"]
    if case["op"] == "checkpoint":
        return _eight_bit(s["x"].float()).to(torch.bfloat16)
    act, at = case["act"], (s["slot"], s["place"])
    x = _spread(s, s["xe"])
    if case["op"] == "w4":
        w_gate_up = _four_bit(s, s["q_gate_up"], s["s_gate_up"])
    else:
        w_gate_up = _weights(s, s["w_gate_up"])
    gu = torch.bmm(x, w_gate_up.transpose(1, 2))
    g, u = gu.chunk(2, dim=2)
    h = _gate(g, act)[0] * u
    w_down = _four_bit(s, s["q_down"], s["s_down"]) if case["op"] == "w4" else _weights(s, s["w_down"])
    ye = torch.bmm(h, w_down.transpose(1, 2))[at].to(torch.bfloat16)
    if case["op"] != "train":
        return ye
    if case["saved"] == "int8":
        g, u = _eight_bit(g), _eight_bit(u)
    else:
        g, u = g.to(torch.bfloat16).float(), u.to(torch.bfloat16).float()
    gy = _spread(s, s["grad_ye"])
    a, da = _gate(g, act)
    h = a * u
    dh = torch.bmm(gy, w_down)
    dgu = torch.cat((dh * u * da, dh * a), dim=2)
    return dict(ye=ye,
                grad_xe=torch.bmm(dgu, w_gate_up)[at].to(torch.bfloat16),
                grad_w_gate_up=_by_expert(s, torch.bmm(dgu.transpose(1, 2), x)),
                grad_w_down=_by_expert(s, torch.bmm(gy.transpose(1, 2), h)))


# ---- the package's calls ----

def _own(s):
    import moe_expert_token_amd as ms
    case = s["case"]
    if case["op"] == "checkpoint":
        ms.moe_experts_pack8(s["x"], s["q"], s["scale"])
        ms.moe_experts_unpack8(s["q"], s["scale"], s["back"])
        return s["back"]
    act = ms.ACT_SILU if case["act"] == "silu" else ms.ACT_GELU_TANH
    if case["op"] == "w4":
        ms.moe_experts_ffn_w4_forward(s["plan"], s["xe"], s["q_gate_up"], s["s_gate_up"], s["q_down"], s["s_down"],
                                      s["ye"], s["ws"], group=case["group"], act=act)
        return s["ye"]
    if case["op"] == "forward":
        ms.moe_experts_ffn_forward(s["plan"], s["xe"], s["w_gate_up"], s["w_down"], s["ye"], s["ws"], act=act)
        return s["ye"]
    ms.moe_experts_ffn_forward(s["plan"], s["xe"], s["w_gate_up"], s["w_down"], s["ye"], s["ws"], saved=s["saved"],
                               saved_scale=s["scale"], act=act)
    ms.moe_experts_ffn_backward(s["plan"], s["grad_ye"], s["xe"], s["w_gate_up"], s["w_down"], s["saved"],
                                s["grad_xe"], s["grad_w_gate_up"], s["grad_w_down"], s["ws"], saved_scale=s["scale"],
                                act=act)
    return {n: s[n] for n in ("ye", "grad_xe", "grad_w_gate_up", "grad_w_down")}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    if case["op"] == "checkpoint":
        n = case["rows"] * case["cols"]
        # read bf16, write 8 bits and a scale a group; then the way back
        return dict(bytes=6 * n + 4 * case["rows"] * -(-case["cols"] // GROUP8), flops=0)
    T, H, E, k, I = (case[n] for n in "T H E k I".split())
    rows = T * k
    weights = 3 * H * I
    # experts that have a row, on average over even routing (all of them in a large batch)
    used = E * (1 - (1 - k / E) ** T)
    if case["op"] == "w4":
        return dict(bytes=used * weights * (0.5 + 2 / case["group"]) + 4 * rows * H, flops=2 * rows * weights)
    if case["op"] == "forward":
        return dict(bytes=2 * used * weights + 4 * rows * H, flops=2 * rows * weights)
    held = rows * 2 * I * (2 if case["saved"] == "bf16" else 1 + 2 / GROUP8)
    # forward: xe, weights, ye, what is saved; backward: grad_ye, xe, weights, saved, three gradients
    return dict(bytes=2 * used * weights * 2 + 2 * E * weights + 2 * rows * H * 5 + 2 * held,
                flops=6 * rows * weights)


# ---- the definition, in 64 bits ----

def _exact8(t):
    """As the definition has it, a group at a time along the row."""
    parts = []
    for part in t.split(GROUP8, dim=1):
        top = part.abs().amax(dim=1, keepdim=True)
        # the least bf16 value not below top / 127, never under the least normal one: 8 significant bits, upwards
        m, e = torch.frexp((top / 127).clamp_min(2.0 ** -126))
        step = torch.ldexp(torch.ceil(m * 256), e - 8)
        parts.append(torch.round(part / step).clamp(-127, 127) * step)
    return torch.cat(parts, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        return _exact8(s["x"].double())
    c0, c1 = _slope(case["act"])
    E, H, I = case["E"], case["H"], case["I"]
    offset = s["offset"].tolist()

    def weight(name, e):
        if case["op"] != "w4":
            return s["w_" + name][e].double()
        q, sc = s["q_" + name][e].long(), s["s_" + name][e].double()
        v = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = q % 16 - 8, q // 16 - 8
        return (v.view(q.shape[0], -1, case["group"]) * sc[:, :, None]).view(q.shape[0], -1)

    ye = torch.zeros((s["xe"].shape[0], H), dtype=torch.float64, device="cuda")
    train = case["op"] == "train"
    if train:
        grad_xe = torch.zeros_like(ye)
        grad_w_gate_up = torch.zeros((E, 2 * I, H), dtype=torch.float64, device="cuda")
        grad_w_down = torch.zeros((E, H, I), dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = offset[e], offset[e + 1]
        if lo == hi:
            continue
        x, w1, w2 = s["xe"][lo:hi].double(), weight("gate_up", e), weight("down", e)
        g, u = x @ w1[:I].T, x @ w1[I:].T
        ye[lo:hi] = (g * torch.sigmoid(c0 * g + c1 * g ** 3) * u) @ w2.T
        if not train:
            continue
        if case["saved"] == "int8":
            g, u = _exact8(g), _exact8(u)
        else:
            g, u = g.to(torch.bfloat16).double(), u.to(torch.bfloat16).double()
        sig = torch.sigmoid(c0 * g + c1 * g ** 3)
        gy = s["grad_ye"][lo:hi].double()
        dh = gy @ w2
        dgate = sig * (1 + g * (1 - sig) * (c0 + 3 * c1 * g ** 2))
        dg, du = dh * u * dgate, dh * g * sig
        grad_xe[lo:hi] = dg @ w1[:I] + du @ w1[I:]
        grad_w_gate_up[e, :I], grad_w_gate_up[e, I:] = dg.T @ x, du.T @ x
        grad_w_down[e] = gy.T @ (g * sig * u)
    if not train:
        return ye
    return dict(ye=ye, grad_xe=grad_xe, grad_w_gate_up=grad_w_gate_up, grad_w_down=grad_w_down)
