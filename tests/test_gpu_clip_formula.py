"""moe_grad_clip's factor where the norm is 0: min(1, max_norm / (0 + eps)), and 1 for 0 / 0."""
import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [5, 300_001, 40_000_001])
@pytest.mark.parametrize("max_norm,eps,factor", [(0.0, 1e-6, 0.0), (0.0, 0.0, 1.0), (1.0, 0.0, 1.0), (1.0, 4.0, 0.25),
                                                 (1.0, 1e-6, 1.0)])
def test_a_norm_of_zero_from_elsewhere(n, max_norm, eps, factor):
    x = torch.randn(n, device="cuda")
    before = x.clone()
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    assert float(moe.moe_grad_clip([x], max_norm, eps, sumsq=zero)) == 0.0
    assert torch.equal(x, before * factor)
    # The same with a norm that is the tensors' own.
    z = torch.zeros(n, device="cuda")
    assert float(moe.moe_grad_clip([z], max_norm, eps)) == 0.0 and (z == 0).all()
