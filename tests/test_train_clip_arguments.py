"""train.clip_grad_norm's argument: one parameter, a list or a generator of them (on the
CPU, the library's call replaced by a stand-in)."""
import pytest
import torch

from mixture_experts_ffn_sort_b200 import train


@pytest.fixture
def clipped(monkeypatch):
    lists = []
    monkeypatch.setattr(train, "moe_grad_clip", lambda tensors, max_norm, eps: lists.append(list(tensors)))
    return lists


@pytest.mark.parametrize("shape", [(4, 3), (5,), ()])
def test_one_parameter(clipped, shape):
    p = torch.nn.Parameter(torch.ones(shape))
    p.grad = torch.full(shape, 2.0)
    train.clip_grad_norm(p, 1.0)
    assert len(clipped) == 1 and len(clipped[0]) == 1 and clipped[0][0] is p.grad


def test_several(clipped):
    ps = [torch.nn.Parameter(torch.ones(3)) for _ in range(3)]
    ps[0].grad, ps[2].grad = torch.ones(3), torch.zeros(3)
    train.clip_grad_norm(ps, 1.0)
    train.clip_grad_norm(iter(ps), 1.0)
    for got in clipped:
        assert len(got) == 2 and got[0] is ps[0].grad and got[1] is ps[2].grad
