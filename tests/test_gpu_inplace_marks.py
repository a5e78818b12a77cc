"""Tensors that the training calls write to are marked as changed: autograd refuses a
backward pass that needs the values they held."""
import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref
from mixture_experts_ffn_sort_b200 import train

pytestmark = pytest.mark.gpu


def refused(t, call):
    """`call` overwrites t, which a graph has saved."""
    x = torch.ones_like(t, requires_grad=True)
    out = (x * t).sum()
    before = t._version
    call()
    assert t._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward()


def test_outputs_that_are_given():
    T, H, K, E = 12, 40, 3, 8
    ids, off, inv = (t.cuda() for t in ref.routes(T, K, E, 0.1, 1))
    x, y, w = torch.randn((T, H), device="cuda"), torch.randn((T * K, H), device="cuda"), torch.rand((T, K), device="cuda")
    lg = torch.randn((T, E), device="cuda")
    rows, toks = torch.zeros_like(y), torch.zeros_like(x)
    dw, dlg, norm = torch.zeros_like(w), torch.zeros_like(lg), torch.zeros((), device="cuda")
    refused(rows, lambda: moe.moe_permute(x, inv, off, x_sorted=rows))
    refused(toks, lambda: moe.moe_permute_bwd(y, inv, T, dx=toks))
    refused(toks, lambda: moe.moe_unpermute(y, inv, w, out=toks))
    refused(rows, lambda: moe.moe_unpermute_bwd(x, y, inv, w, off, dy_sorted=rows))
    refused(dw, lambda: moe.moe_unpermute_bwd(x, y, inv, w, off, dtopk_w=dw))
    refused(dlg, lambda: moe.moe_route_bwd(lg, ids, w, dlogits=dlg))
    refused(norm, lambda: moe.moe_grad_sumsq([x], norm=norm))
    inputs = (x, y, w, lg, inv, off, ids)
    before = [t._version for t in inputs]
    moe.moe_permute(x, inv, off), moe.moe_unpermute(y, inv, w), moe.moe_unpermute_bwd(x, y, inv, w, off)
    moe.moe_route_bwd(lg, ids, w), moe.moe_grad_norm([x, y])
    assert [t._version for t in inputs] == before


@pytest.mark.parametrize("sizes", [[50], [40_000, 30], [20_000_000]])
def test_clipping(sizes):
    ts = [torch.ones(n, device="cuda") for n in sizes]
    for t in ts:
        refused(t, lambda: moe.moe_grad_clip(ts, 0.5))
        refused(t, lambda: moe.moe_grad_clip(ts, 0.5, sumsq=moe.moe_grad_sumsq(ts)))
    outs = [torch.zeros_like(t) for t in ts]
    tl = moe.TensorList(ts, outs)
    kept = [t._version for t in ts]
    refused(outs[0], lambda: moe.moe_grad_clip(tl, 0.5))
    assert [t._version for t in ts] == kept
    p = torch.nn.Parameter(torch.ones(300, device="cuda"))
    p.grad = torch.ones(300, device="cuda")
    refused(p.grad, lambda: train.clip_grad_norm([p], 0.1))
    base = torch.ones(100, device="cuda")  # a view's mark is its base's
    refused(base, lambda: moe.moe_grad_clip([base[10:20]], 0.1))


def test_inference_tensors():
    with torch.inference_mode():
        t = torch.ones(100, device="cuda")
        assert float(moe.moe_grad_clip([t], 1.0)) == 10.0
    assert float(moe.moe_grad_clip([t], 0.5)) == pytest.approx(1.0)
    assert torch.allclose(t.norm(), torch.tensor(0.5, device="cuda"))
