"""Clipping of small lists, which a cluster of blocks does in one launch, on SMs
that other streams keep busy: the same bits as on a quiet GPU.  Lists of one or
two chunks leave most blocks of the cluster without work, so that they reach the
exchange of sums first."""
import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [[1], [4000], [8193, 3], [131072 - 64], [4096] * 32])
def test_small_lists_beside_other_streams(sizes):
    T, H, K, E = 1500, 4095, 8, 32
    _, off, inv = (t.cuda() for t in ref.routes(T, K, E, 0.1, 3))
    g = torch.Generator(device="cuda").manual_seed(3)
    y = torch.randn((T * K, H), generator=g, device="cuda").bfloat16()
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    w = torch.rand((T, K), generator=g, device="cuda")
    grads = [torch.randn(n, generator=g, device="cuda") for n in sizes]
    outs = [torch.empty_like(t) for t in grads]
    tl = moe.TensorList(grads, outs)
    norm = moe.moe_grad_clip(tl, 0.5)
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    norms = []
    for it in range(20):
        with torch.cuda.stream(streams[0]):
            moe.moe_unpermute_bwd(x, y, inv, w, off)
        with torch.cuda.stream(streams[1]):
            moe.moe_unpermute(y, inv, w)
        with torch.cuda.stream(streams[2]):
            for _ in range(10):
                for t in outs:
                    t.fill_(7.0)
                norms.append(moe.moe_grad_clip(tl, 0.5))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), it
    assert all(torch.equal(n, norm) for n in norms)
