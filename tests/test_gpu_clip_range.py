"""moe_grad_clip where max_norm / norm is below fp32's normal numbers: the scaled
values keep the accuracy of the others.  Bounds as in test_gpu_grad_clip.py: the
norm and the factor are off by at most 10 2^-24, and the product is rounded to
the tensor's type (fp32 results below its normal numbers twice, by half of its
smallest number in all but a 2^-24 of the value)."""
import math

import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref
from _train_ref import HALF, TINY, U32

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def huge(n, dtype, seed):
    """Values of 3e37 to 3e38, either sign."""
    g = ref.gen(seed)
    v = (torch.rand(n, generator=g) * 0.9 + 0.1) * 3e38
    return torch.where(torch.rand(n, generator=g) < 0.5, v, -v).to(dtype).cuda()


# One launch by a cluster; two launches; the two of a list of 64 MB and more.
@pytest.mark.parametrize("sizes", [[1], [1000, 77], [100_003] * 12, [40_000_001]])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("max_norm", [1.0, 1e-30, 1e-37, 2.0 ** -149])
def test_factors_below_the_normal_numbers(sizes, dtype, max_norm):
    ts = [huge(n, dtype, i) for i, n in enumerate(sizes)]
    before = [t.double() for t in ts]
    norm = math.sqrt(sum(float(b.square().sum()) for b in before))
    assert max_norm / norm < 2.0 ** -126
    got = float(moe.moe_grad_clip(ts, max_norm, eps=0.0))
    if norm > torch.finfo(F).max:
        assert got == math.inf  # in fp32; the factor has the norm in fp64
    else:
        assert abs(got - norm) <= 6 * U32 * norm
    for t, b in zip(ts, before):
        want = b * (max_norm / norm)
        err = 10 * U32 * want.abs()
        assert ((t.double() - want).abs() <= HALF[dtype] * (want.abs() + err) + err + TINY[dtype]).all()


def test_into_other_memory_and_with_a_sum_from_elsewhere():
    x = huge(5000, F, 9)
    out = torch.empty(5001, device="cuda")[1:]  # aligned otherwise
    norm = math.sqrt(float(x.double().square().sum()))
    moe.moe_grad_clip(moe.TensorList([x], [out]), 1.0, eps=0.0)
    want = x.double() / norm
    assert ((out.double() - want).abs() <= 12 * U32 * want.abs()).all()
    # A norm far beyond fp32: 1e60, so that even 3e38 comes out at 3e-22.
    moe.moe_grad_clip([x], 1.0, eps=0.0, sumsq=torch.full((), 1e120, dtype=torch.float64, device="cuda"))
    want = want * norm / 1e60
    assert ((x.double() - want).abs() <= 12 * U32 * want.abs()).all()
