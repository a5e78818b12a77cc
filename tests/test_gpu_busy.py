"""Calls on SMs that other streams keep busy: every result has the same bits as
on a quiet GPU.  Kernels that share an SM with a memory-bound one see their
loads from shared memory wait, which shows a ring stage that is refilled before
it has been read."""
import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref
from mixture_experts_ffn_sort_b200 import workloads as wl

pytestmark = pytest.mark.gpu

SIZES = [(3000, 4096, 8, 32), (2500, 4095, 9, 32), (4000, 1500, 12, 32)]


def rows_of(T, H, K, E, seed):
    _, off, inv = ref.routes(T, K, E, 0.1, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (inv.cuda(), off.cuda(), torch.randn((T * K, H), generator=g, device="cuda").bfloat16(),
            torch.rand((T, K), generator=g, device="cuda"),
            torch.randn((T, H), generator=g, device="cuda").bfloat16())


def row_calls(inv, off, y, w, x):
    out = moe.moe_unpermute(y, inv, w, x)
    dx = moe.moe_permute_bwd(y, inv, x.shape[0])
    dy, dw = moe.moe_unpermute_bwd(x, y, inv, w, off)
    return out, dx, dy, dw, moe.moe_grad_norm([out, dx])


@pytest.fixture(scope="module")
def layer_data():
    w = wl.make_workload("decode_skew")
    dev = torch.device("cuda")
    return (w.shape, moe.Experts.from_host(w.routed, dev),
            torch.from_numpy(w.x.view("int16")).view(torch.bfloat16).to(dev), torch.from_numpy(w.logits).to(dev))


@pytest.mark.parametrize("mode", ["HYBRID", "DECODE", "PREFILL", "W8A8"])
def test_layer_beside_row_calls(layer_data, mode):
    shape, routed, x, logits = layer_data
    layer = moe.MoEFFN(routed, shape.T, shape.K, mode=getattr(moe, "MOE_MODE_" + mode, moe.MOE_MODE_AUTO),
                       w8a8=mode == "W8A8")
    sets = [rows_of(*s, seed) for seed, s in enumerate(SIZES)]
    quiet = [row_calls(*s) for s in sets]
    out = layer(x, logits).clone()
    y = layer.y_sorted.clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(len(sets) + 1)]
    for it in range(60):
        busy = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                busy.append(row_calls(*s))
        with torch.cuda.stream(streams[-1]):
            layer(x, logits)
        torch.cuda.synchronize()
        assert torch.equal(layer.y_sorted, y) and torch.equal(layer.out, out), it
        for got, want in zip(busy, quiet):
            assert all(torch.equal(a, b) for a, b in zip(got, want)), it
    assert layer.status.item() == 0
