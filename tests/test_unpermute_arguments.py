"""moe_unpermute takes its number of tokens from topk_w [T, K]: other shapes are refused
(before the device is looked at, so on CPU tensors)."""
import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe


@pytest.mark.parametrize("shape", [(12,), (6, 2, 1), (1, 6, 2), ()])
def test_weights_of_another_shape(shape):
    y, inv = torch.zeros((12, 8)), torch.arange(12, dtype=torch.int32)
    with pytest.raises(ValueError, match="topk_w must be"):
        moe.moe_unpermute(y, inv, torch.ones(shape))
