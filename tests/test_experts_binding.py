"""The binding of the experts' block refuses tensors that the kernels cannot
read: in host memory, or of a floating type other than bf16.  No call here
reaches the library (the plan's handle is null, and each refusal names the
tensor, which the library cannot)."""

import pytest
import torch

T, H, E, K, R, I, G = 5, 64, 8, 2, 4, 32, 32
P = T * K


def _ms():
    import moe_expert_token_amd as ms
    return ms


def bf(*s):
    return torch.empty(s, dtype=torch.bfloat16)


def byte(*s):
    return torch.empty(s, dtype=torch.int8)


def calls(ms):
    """name -> (function, arguments in host memory that fit in every other way)."""
    plan = ms.Plan(None, ms.dims_of(T, H, E, K, R), None, None)
    plan.handle = 0
    ws = torch.empty(1 << 16, dtype=torch.uint8)
    rows, up, down = bf(P, H), bf(E, 2 * I, H), bf(E, H, I)
    return {
        "forward": (ms.moe_experts_ffn_forward,
                    dict(plan=plan, xe=rows, w_gate_up=up, w_down=down, ye=bf(P, H), workspace=ws,
                         saved=byte(P, 2 * I), saved_scale=bf(P, 2, 1))),
        "backward": (ms.moe_experts_ffn_backward,
                     dict(plan=plan, grad_ye=rows, xe=bf(P, H), w_gate_up=up, w_down=down, saved=bf(P, 2 * I),
                          grad_xe=bf(P, H), grad_w_gate_up=bf(E, 2 * I, H), grad_w_down=bf(E, H, I), workspace=ws)),
        "w4": (ms.moe_experts_ffn_w4_forward,
               dict(plan=plan, xe=rows, q_gate_up=byte(E, 2 * I, H // 2), s_gate_up=bf(E, 2 * I, H // G),
                    q_down=byte(E, H, I // 2), s_down=bf(E, H, I // G), ye=bf(P, H), workspace=ws, group=G)),
        "quantize": (ms.moe_experts_w4_quantize, dict(w=bf(4, H), q=byte(4, H // 2), scale=bf(4, H // G), group=G)),
        "pack": (ms.moe_experts_pack8, dict(x=bf(4, H), q=byte(4, H), scale=bf(4, H // 32))),
        "unpack": (ms.moe_experts_unpack8, dict(q=byte(4, H), scale=bf(4, H // 32), x=bf(4, H))),
    }


class Elsewhere:
    """What a tensor on another GPU says of itself."""
    is_cuda, device = True, "cuda:1"

    def get_device(self):
        return 1


class Stream:
    device_index = 0


def test_tensors_and_plans_of_another_device_are_refused():
    ms = _ms()
    from moe_expert_token_amd import experts
    with pytest.raises(ms.MoeShuffleError) as e:
        experts._on_gpu("f", Stream(), xe=None, ye=Elsewhere())
    assert e.value.code == ms.E_INVALID_ARG and "ye" in str(e.value) and "cuda:1" in str(e.value)
    stream = Stream()
    stream.device_index = 1
    experts._on_gpu("f", stream, ye=Elsewhere(), none=None)  # the stream's device, whatever the current one is


@pytest.mark.parametrize("name", ["forward", "backward", "w4"])
def test_the_plans_workspace_is_held_to_the_same_device(name, monkeypatch):
    ms = _ms()
    from moe_expert_token_amd import experts
    seen = {}
    monkeypatch.setattr(experts, "_on_gpu", lambda func, stream, **tensors: seen.update(tensors))
    monkeypatch.setattr(experts, "_stream", lambda stream: None)
    f, args = calls(ms)[name]
    args["plan"].workspace = torch.empty(8, dtype=torch.uint8)
    refusal(ms, f, args)  # by the library: the handle is null
    assert any(t is args["plan"].workspace for t in seen.values())


NAMES = ["forward", "backward", "w4", "quantize", "pack", "unpack"]


def refusal(ms, f, args):
    with pytest.raises(ms.MoeShuffleError) as e:
        f(**args)
    assert e.value.code == ms.E_INVALID_ARG
    return str(e.value)


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_are_refused(name, monkeypatch):
    ms = _ms()
    from moe_expert_token_amd import experts
    monkeypatch.setattr(experts, "_load", lambda: pytest.fail("the library was called with a host address"))
    f, args = calls(ms)[name]
    assert "GPU" in refusal(ms, f, args)


@pytest.mark.parametrize("name", NAMES)
def test_other_floating_types_are_refused(name, monkeypatch):
    """fp16 has bf16's size and another meaning; float8 likewise beside int8."""
    ms = _ms()
    from moe_expert_token_amd import experts
    monkeypatch.setattr(experts, "_load", lambda: pytest.fail("the library was called"))
    f, args = calls(ms)[name]
    for key, t in args.items():
        if not isinstance(t, torch.Tensor) or key == "workspace":
            continue
        other = t.view(torch.float16 if t.element_size() == 2 else torch.float8_e4m3fn)
        text = refusal(ms, f, {**args, key: other})
        assert key in text and "float" in text, (key, text)
        # other views of the same bits are not refused for their type
        same = t.view(torch.int16 if t.element_size() == 2 else torch.uint8)
        assert "GPU" in refusal(ms, f, {**args, key: same})
