"""TensorList: a list whose tensors have got other memory since it was made is refused."""
import math

import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe

pytestmark = pytest.mark.gpu


def calls(tl):
    return (lambda: moe.moe_grad_sumsq(tl), lambda: moe.moe_grad_norm(tl), lambda: moe.moe_grad_clip(tl, 1.0))


def change(how, t):
    if how == "memory":
        t.data = torch.ones(t.numel(), device="cuda", dtype=t.dtype)
    elif how == "type":
        t.data = t.data.bfloat16()
    elif how == "fewer values":
        t.data = t.data[:10]
    elif how == "freed":
        t.untyped_storage().resize_(0)
    else:
        t.set_(torch.ones(t.numel(), device="cuda", dtype=t.dtype).untyped_storage(), 0, (t.numel(),))


@pytest.mark.parametrize("which", ["tensor", "output"])
@pytest.mark.parametrize("how", ["memory", "type", "fewer values", "freed", "set"])
def test_other_memory_is_refused(how, which):
    ts = [torch.ones(100, device="cuda"), torch.ones(5000, device="cuda")]
    outs = [torch.empty_like(t) for t in ts]
    tl = moe.TensorList(ts, outs)
    assert float(moe.moe_grad_clip(tl, 1.0)) == pytest.approx(math.sqrt(5100))
    change(how, (ts if which == "tensor" else outs)[1])
    for call in calls(tl):
        with pytest.raises(ValueError, match="make it again"):
            call()


def test_a_module_that_changes_its_type():
    layer = torch.nn.Linear(64, 64).cuda()
    layer(torch.ones(2, 64, device="cuda")).sum().backward()
    grads = [p.grad for p in layer.parameters()]
    tl = moe.TensorList(grads)
    norm = float(moe.moe_grad_norm(tl))
    layer.bfloat16()  # in place, the gradients too
    if any(g.dtype != torch.float32 for g in grads):
        with pytest.raises(ValueError):
            moe.moe_grad_norm(tl)
    assert float(moe.moe_grad_norm([p.grad for p in layer.parameters()])) == pytest.approx(norm, rel=2.0 ** -7)


def test_values_that_change_in_place_are_taken():
    t = torch.ones(3000, device="cuda")
    tl = moe.TensorList([t, torch.empty(0, device="cuda")])
    t.mul_(2)
    assert float(moe.moe_grad_norm(tl)) == pytest.approx(2 * math.sqrt(3000))
    t.requires_grad_()
    assert float(moe.moe_grad_norm(tl)) == pytest.approx(2 * math.sqrt(3000))
