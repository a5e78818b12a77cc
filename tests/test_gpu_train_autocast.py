"""The routed layer in an autocast region: its gate product and the router's gradients stay in fp32."""
import pytest
import torch

import _train_ref as ref
from mixture_experts_ffn_sort_b200 import train

pytestmark = pytest.mark.gpu


def scale(rows, offsets):
    return rows * 2


@pytest.mark.parametrize("cast", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dtype,H", [(torch.float32, 96), (torch.bfloat16, 72), (torch.bfloat16, 128)])
def test_layer(dtype, H, cast):
    T, E, K = 40, 8, 2
    layer = train.RoutedLayer(H, E, K, scale, dtype=dtype)
    x = torch.randn((T, H), generator=ref.gen(1)).to(dtype).cuda().requires_grad_()
    dout = torch.randn((T, H), generator=ref.gen(2)).to(dtype).cuda()
    want = layer(x)
    grads = torch.autograd.grad(want, (x, layer.w_router), dout)
    with torch.autocast("cuda", dtype=cast):
        got = layer(x)
    assert torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(got, (x, layer.w_router), dout), grads))


def test_backward_of_the_router_within_the_region():
    T, H, E, K = 40, 128, 8, 2
    x = torch.randn((T, H), generator=ref.gen(3)).bfloat16().cuda().requires_grad_()
    wr = torch.randn((E, H), generator=ref.gen(4)).bfloat16().cuda().requires_grad_()
    dw = torch.randn((T, K), generator=ref.gen(5)).cuda()
    want = torch.autograd.grad(train.router(x, wr, K)[1], (x, wr), dw)
    with torch.autocast("cuda", dtype=torch.float16):
        got = torch.autograd.grad(train.router(x, wr, K)[1], (x, wr), dw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
