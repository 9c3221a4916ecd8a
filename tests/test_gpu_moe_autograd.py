"""GPU: the operators of experts and adapters have no backward pass, so they refuse
tensors that a gradient is asked of, and tell autograd what they write."""
import pytest
import torch

import moe_ref as X

pytestmark = pytest.mark.gpu


def operands(lib):
    index = torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32, device="cuda")
    f = lambda *s: (torch.arange(torch.Size(s).numel(), device="cuda") % 7 - 3).view(s).to(torch.bfloat16)  # noqa: E731
    return lib.group_rows(index, 2), dict(out=f(5, 40), x=f(5, 64), lora_a=f(2, 8, 64), lora_b=f(2, 40, 8),
                                          scales=torch.tensor([0.5, 2.0], device="cuda"))


def lora(lib, groups, t):
    return lib.lora_add(t["out"], t["x"], t["lora_a"], t["lora_b"], groups, scales=t["scales"])


@pytest.mark.parametrize("name", ["out", "x", "lora_a", "lora_b", "scales"])
def test_lora_refuses_gradients(gpu_lib, name):
    groups, t = operands(gpu_lib)
    before = t["out"].clone()
    t[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name}.*backward"):
        lora(gpu_lib, groups, t)
    torch.cuda.synchronize()
    assert torch.equal(t["out"].detach(), before)
    # where no gradient is recorded, they are tensors as any
    want = lora(gpu_lib, *operands(gpu_lib))
    with torch.no_grad():
        assert torch.equal(lora(gpu_lib, groups, t).detach(), want)
    with torch.inference_mode():
        t["out"] = before.clone()
        assert torch.equal(lora(gpu_lib, groups, t), want)


def test_lora_refuses_an_out_of_a_graph(gpu_lib):
    """The projection's own output, where its weight is trained: written in place
    its gradient would be of other values."""
    groups, t = operands(gpu_lib)
    weight = torch.ones(40, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    t["out"] = t["out"] * weight
    with pytest.raises(ValueError, match="out.*backward"):
        lora(gpu_lib, groups, t)


def test_others_refuse_gradients(gpu_lib):
    lib = gpu_lib
    z, b = torch.ones(3, 8, device="cuda"), torch.ones(8, device="cuda")
    groups = lib.group_rows(torch.tensor([[0, 1], [1, 0], [1, 1]], dtype=torch.int32, device="cuda"), 2)
    y, w = torch.ones(6, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 2, device="cuda")
    s = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    for name, t, call in (("logits", z, lambda: lib.moe_route(z, 2, bias=b)), ("bias", b, lambda: lib.moe_route(z, 2, bias=b)),
                          ("y", y, lambda: lib.moe_combine(y, groups, w, shared=s)), ("weights", w, lambda: lib.moe_combine(y, groups, w, shared=s)),
                          ("shared", s, lambda: lib.moe_combine(y, groups, w, shared=s))):
        t.requires_grad_()
        with pytest.raises(ValueError, match=f"{name}.*backward"):
            call()
        with torch.no_grad():
            call()
        t.requires_grad_(False)
        call()


def test_writes_are_counted(gpu_lib):
    """What is written in place, or to a tensor passed in, gets another version, so
    that a graph that had kept it says so."""
    lib = gpu_lib
    groups, t = operands(lib)
    version = t["out"]._version
    lora(lib, groups, t)
    assert t["out"]._version > version
    leaf = torch.ones(5, 40, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    kept = (leaf * t["out"]).sum()
    lora(lib, groups, t)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()
    index = torch.tensor([[0, 1], [1, -1], [1, 0]], dtype=torch.int32, device="cuda")
    plan = lib.group_rows(index, 2)
    codes, words = torch.zeros(3, 256, dtype=torch.uint8, device="cuda"), torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    w, ws = torch.zeros(2, 256, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 2, 2, dtype=torch.uint8, device="cuda")
    y = torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda")
    e = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    for outs, call in (
            ((e(3, 2, t=f32), e(3, 2, t=i32)), lambda o: lib.moe_route(torch.ones(3, 8, device="cuda"), 2, weights=o[0], experts=o[1])),
            ((e(3, t=i32), e(6, t=i32), e(3, 2, t=i32)), lambda o: lib.group_rows(index, 2, out=o)),
            ((e(6, 256),), lambda o: lib.fp8_grouped_gemm_1x128_128x128(codes, words, w, ws, plan, gather=True, out=o[0])),
            ((e(6, 128, t=u8), e(6, 1, t=i32)), lambda o: lib.fp8_grouped_swiglu_1x128(codes, words, w, ws, plan, gather=True, q=o[0], q_scales=o[1])),
            ((e(3, 64),), lambda o: lib.moe_combine(y, plan, torch.ones(3, 2, device="cuda"), out=o[0]))):
        was = [o._version for o in outs]
        call(outs)
        assert all(o._version > v for o, v in zip(outs, was))


def test_tensors_of_inference_mode(gpu_lib):
    """Tensors made in inference mode have no version; they are written in and out
    of it as before."""
    with torch.inference_mode():
        groups, t = operands(gpu_lib)
    want, _ = X.lora(t["out"].cpu(), t["x"].cpu(), t["lora_a"].cpu(), t["lora_b"].cpu(), groups.offsets.cpu(), groups.rows.cpu(), t["scales"].cpu())
    got = lora(gpu_lib, groups, t)      # whole numbers of at most 15 bits, rounded to bf16
    assert bool(((got.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
