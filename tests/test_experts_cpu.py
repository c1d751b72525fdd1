"""The experts' block on the CPU: the header's functions, every refusal that
needs no GPU, and the 64-bit reference against differences."""

import ctypes
import os
import re

import pytest
import torch

import experts_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _lib():
    import moe_expert_token_amd as ms
    from moe_expert_token_amd import experts
    return ms, experts._load()


def test_every_declared_symbol_is_exported():
    ms, lib = _lib()
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_experts.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_experts_\w+)\s*\(", text)))
    assert names == sorted(ms.EXPERTS_EXPORTS)
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value


def test_header_is_c99(tmp_path):
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "moe_experts.h"\nint main(void) { return MOE_EXPERTS_ACT_SILU; }\n')
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-c", str(src), "-o", str(tmp_path / "t.o")], check=True)


def _size(ms, *dims, inter, backward=False):
    return ms.moe_experts_ffn_workspace_size(ms.dims_of(*dims), inter, backward)


def test_workspace_size():
    ms, _ = _lib()
    # h [P, I] bf16; the backward pass has [dg du] and h
    assert _size(ms, 100, 64, 8, 2, 4, inter=128) == 200 * 128 * 2
    assert _size(ms, 100, 64, 8, 2, 4, inter=128, backward=True) == 3 * 200 * 128 * 2
    assert 0 < _size(ms, 0, 64, 8, 2, 4, inter=128) <= 256
    # one call fits the workspace of the other direction
    assert _size(ms, 3, 64, 8, 2, 4, inter=8) <= _size(ms, 3, 64, 8, 2, 4, inter=8, backward=True)


@pytest.mark.parametrize("dims,inter,code", [
    ((4, 64, 8, 2, 4), 0, "E_INVALID_ARG"), ((4, 64, 8, 2, 4), -8, "E_INVALID_ARG"),
    ((4, 64, 8, 2, 4), 12, "E_ALIGN"), ((4, 12, 8, 2, 4), 8, "E_ALIGN"),
    ((4, 64, 8, 9, 4), 8, "E_INVALID_ARG"), ((4, 64, 8, 2, 4), 1 << 20, "E_OVERFLOW"),
    ((4, 1 << 20, 8, 2, 4), 8, "E_OVERFLOW"),
    ((1 << 24, 64, 8, 8, 4), 1 << 14, "E_OVERFLOW"),          # P * I / 32 at 2^36
    (((1 << 27) - 10, 8, 16, 16, 4), 8, "E_OVERFLOW"),        # P = 2^31 - 160, within 1024 of 2^31
    ((4, 1 << 19, 512, 2, 4), 1 << 19, "E_OVERFLOW"),         # tiles of the weight gradients
])
def test_workspace_size_refusals(dims, inter, code):
    ms, _ = _lib()
    with pytest.raises(ms.MoeShuffleError) as e:
        _size(ms, *dims, inter=inter)
    assert e.value.code == getattr(ms, code)


def test_null_plan_is_refused():
    ms, lib = _lib()
    p = 0x100000
    assert lib.moe_experts_ffn_forward(None, p, p, p, 8, 0, p, None, None, p, 1 << 20, None) == ms.E_INVALID_ARG
    assert lib.moe_experts_ffn_backward(None, p, p, p, p, 8, 0, p, None, p, p, p, p, 1 << 20, None) == ms.E_INVALID_ARG
    assert lib.moe_experts_ffn_w4_forward(None, p, p, p, p, p, 32, 32, 0, p, p, 1 << 20, None) == ms.E_INVALID_ARG


@pytest.mark.parametrize("f", ["moe_experts_pack8", "moe_experts_unpack8"])
def test_pack_refusals(f):
    ms, lib = _lib()
    a, b, c = 0x100000, 0x200000, 0x300000  # x, q, scale; never dereferenced: every call is refused

    def call(x, q, s, rows, cols):
        args = (x, rows, cols, q, s) if f.endswith("_pack8") else (q, s, rows, cols, x)
        return getattr(lib, f)(*args, None)

    assert call(None, None, None, 0, 64) == ms.OK          # no rows: nothing to do
    assert call(a, b, c, -1, 64) == ms.E_INVALID_ARG
    assert call(a, b, c, 4, 0) == ms.E_INVALID_ARG
    assert call(a, b, c, 4, 12) == ms.E_ALIGN
    assert call(a + 8, b, c, 4, 64) == ms.E_ALIGN
    assert call(a, b + 8, c, 4, 64) == ms.E_ALIGN
    assert call(a, b, c + 2, 4, 64) == ms.E_ALIGN
    assert call(None, b, c, 4, 64) == ms.E_INVALID_ARG
    assert call(a, None, c, 4, 64) == ms.E_INVALID_ARG
    assert call(a, b, None, 4, 64) == ms.E_INVALID_ARG
    assert call(a, a + 256, c, 4, 64) == ms.E_INVALID_ARG   # q inside x (4 * 64 * 2 bytes)
    assert call(a, b, a + 16, 4, 64) == ms.E_INVALID_ARG    # scale inside x
    assert call(a, b, c, 1 << 36, 64) == ms.E_OVERFLOW
    assert call(a, b, c, (1 << 31), 4096) == ms.E_OVERFLOW


def test_w4_quantize_refusals():
    ms, lib = _lib()
    a, b, c = 0x100000, 0x200000, 0x300000

    def call(w=a, rows=4, cols=128, group=64, q=b, s=c):
        return lib.moe_experts_w4_quantize(w, rows, cols, group, q, s, None)

    assert call(rows=0, w=None, q=None, s=None) == ms.OK
    assert call(rows=-1) == ms.E_INVALID_ARG
    assert call(group=48) == ms.E_INVALID_ARG
    assert call(group=0) == ms.E_INVALID_ARG
    assert call(cols=96) == ms.E_ALIGN
    assert call(w=a + 4) == ms.E_ALIGN
    assert call(w=None) == ms.E_INVALID_ARG
    assert call(q=a) == ms.E_INVALID_ARG
    assert call(s=b + 16) == ms.E_INVALID_ARG
    assert call(rows=1 << 38) == ms.E_OVERFLOW


def test_binding_refuses_tensors_that_do_not_fit():
    """Shape, element size and contiguity are checked before the library is called (host tensors suffice)."""
    ms, _ = _lib()
    T, H, E, k, R, I = 5, 64, 8, 2, 4, 32
    plan = ms.Plan(None, ms.dims_of(T, H, E, k, R), None, None)
    plan.handle = 0  # not a plan: a call that passed the checks would be refused by the library too
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(xe=bf(T * k, H), w_gate_up=bf(E, 2 * I, H), w_down=bf(E, H, I), ye=bf(T * k, H),
                workspace=torch.empty(1 << 16, dtype=torch.uint8))

    def refused(**change):
        with pytest.raises(ms.MoeShuffleError) as e:
            ms.moe_experts_ffn_forward(plan, **{**good, **change})
        assert e.value.code == ms.E_INVALID_ARG
        return str(e.value)

    assert "xe" in refused(xe=bf(T * k - 1, H))
    assert "xe" in refused(xe=torch.empty(T * k, H))                     # fp32
    assert "xe" in refused(xe=bf(H, T * k).t())                          # strided
    assert "w_gate_up" in refused(w_gate_up=bf(E, I, H))
    assert "w_down" in refused(w_down=bf(E - 1, H, I))
    assert "three axes" in refused(w_down=bf(E * H, I))
    assert "ye" in refused(ye=bf(T * k, H + 8))
    assert "saved" in refused(saved=bf(T * k, I))
    assert "saved" in refused(saved_scale=bf(T * k, 2, 1))
    assert "saved" in refused(saved=bf(T * k, 2 * I), saved_scale=bf(T * k, 2, 1))   # int8 with a scale
    assert "saved_scale" in refused(saved=torch.empty(T * k, 2 * I, dtype=torch.int8), saved_scale=bf(T * k, 2, 2))
    plan.handle = None
    assert "destroyed" in refused()


@pytest.mark.parametrize("act", [0, 1])
def test_reference_gradients_against_differences(act):
    """The reference's gradients are those of its forward pass: central differences, error O(step^2)."""
    gen = torch.Generator().manual_seed(act)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    n, H, I = 5, 12, 7
    x, w1, w2, gy = rnd(n, H), rnd(2 * I, H) / 3, rnd(H, I) / 3, rnd(n, H)
    f = ref.forward(x, w1, w2, act)
    b = ref.backward(gy, x, w1, w2, f["g"], f["u"], act)
    for name, t in (("grad_xe", x), ("grad_w_gate_up", w1), ("grad_w_down", w2)):
        v, eps = rnd(*t.shape), 1e-5
        loss = []
        for sign in (1, -1):
            args = [(x if t is not x else x + sign * eps * v), (w1 if t is not w1 else w1 + sign * eps * v),
                    (w2 if t is not w2 else w2 + sign * eps * v)]
            loss.append(float((ref.forward(*args, act)["y"] * gy).sum()))
        got, want = float((b[name] * v).sum()), (loss[0] - loss[1]) / (2 * eps)
        assert abs(got - want) <= 1e-7 * (1 + abs(want)), (name, got, want)


def test_reference_pack_holds_its_bound():
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((6, 100), generator=gen) * torch.logspace(-30, 30, 6)[:, None]
    q, step = ref.pack8(x)
    back = ref.unpack8(q, step)
    # half a step, and what the quotient's two roundings move a tie by
    bound = step.double().repeat_interleave(32, -1)[:, :100] * (0.5 + 127 * 2.0 ** -23)
    assert bool(((back - x.double()).abs() <= bound).all())
    assert int(q.abs().max()) <= 127
