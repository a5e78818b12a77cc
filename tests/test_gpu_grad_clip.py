"""moe_grad_sumsq, moe_grad_norm and moe_grad_clip against plain 64-bit forms.

Tolerances: up to 8 squares are added in fp32 (8 roundings of 2^-24), the rest
in fp64, so the sum of squares is within 9 2^-24 and the norm (the root, and
its rounding to fp32) within 6 2^-24.  The factor adds its rounding and the
product one more; the result is rounded once to its type."""
import math

import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref
from _train_ref import HALF, TINY, U32

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def tensors(sizes, dtypes, seed, scale=1.0, offset=0):
    """Views that start at odd places of one buffer each."""
    g = ref.gen(seed)
    got = []
    for i, n in enumerate(sizes):
        k = (i + offset) % 9
        buf = (torch.randn(n + k + 3, generator=g) * scale).to(dtypes[i % len(dtypes)]).cuda()
        got.append(buf[k:k + n])
    return got


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check_clip(ts, max_norm, outs=None, eps=1e-6):
    before = [t.clone() for t in ts]
    norm = norm64(before)
    got = moe.moe_grad_clip(moe.TensorList(ts, outs), max_norm, eps)
    assert abs(float(got) - norm) <= 6 * U32 * norm
    factor = min(1.0, max_norm / (norm + eps))
    for b, t, o in zip(before, ts, ts if outs is None else outs):
        want = b.double() * factor
        err = 10 * U32 * want.abs()
        assert ((o.double() - want).abs() <= HALF[b.dtype] * (want.abs() + err) + err + TINY[b.dtype]).all()
        if outs is not None:
            assert torch.equal(t, b)
        if factor == 1.0:
            assert torch.equal(o, b)


SETS = [[1], [0], [3, 0, 5], [4096, 8192, 8193], [7, 1000, 65537, 12, 300001], [16384, 1, 2, 3] * 5,
        [129] * 70]


@pytest.mark.parametrize("dtypes", [[BF], [HF], [F], [BF, F, HF]])
@pytest.mark.parametrize("sizes", SETS)
def test_norm_and_clip(sizes, dtypes):
    ts = tensors(sizes, dtypes, 1)
    norm = norm64(ts)
    assert abs(float(moe.moe_grad_norm(ts)) - norm) <= 6 * U32 * norm
    s = moe.moe_grad_sumsq(ts)
    assert s.dtype == torch.float64 and s.shape == () and abs(float(s) - norm ** 2) <= 9 * U32 * norm ** 2
    check_clip(ts, 0.5 * norm if norm else 1.0)          # in place
    check_clip(tensors(sizes, dtypes, 2), 1e9)           # nothing to clip
    check_clip(tensors(sizes, dtypes, 3), 0.25, tensors(sizes, dtypes, 4))           # into others, alike aligned
    check_clip(tensors(sizes, dtypes, 3), 0.25, tensors(sizes, dtypes, 4, offset=1))  # and otherwise aligned
    check_clip(tensors(sizes, dtypes, 5), 0.0)


def test_more_tensors_than_one_launch_takes():
    sizes = [37 + 5 * i % 911 for i in range(2311)]
    for dtypes in ([BF], [F, HF]):
        check_clip(tensors(sizes, dtypes, 7), 3.0)
        ts = tensors(sizes, dtypes, 8)
        assert abs(float(moe.moe_grad_norm(ts)) - norm64(ts)) <= 6 * U32 * norm64(ts)


@pytest.mark.parametrize("dtypes", [[BF], [HF], [F], [HF, F]])
@pytest.mark.parametrize("sizes", [[262144 - 9], [262144], [8192] * 32, [8192] * 31 + [8193], [1] * 32, [1] * 33,
                                   [0] * 40 + [5, 7], [131072, 1, 131000], [4088, 4096, 4104] * 10])
def test_a_cluster_of_blocks_and_just_beyond(sizes, dtypes):
    """Lists of about 32 chunks of 16 KB, which one launch clips."""
    check_clip(tensors(sizes, dtypes, 31), 1.5)
    check_clip(tensors(sizes, dtypes, 32), 1e9)
    check_clip(tensors(sizes, dtypes, 33), 0.5, tensors(sizes, dtypes, 34))
    check_clip(tensors(sizes, dtypes, 35), 0.5, tensors(sizes, dtypes, 36, offset=1))
    # The norm of the one launch and that of the sum alone are the same number to fp64.
    ts = tensors(sizes, dtypes, 37)
    s = float(moe.moe_grad_sumsq(ts))
    assert abs(float(moe.moe_grad_clip(ts, 1e9)) - math.sqrt(s)) <= U32 * math.sqrt(s) * 1.001


@pytest.mark.parametrize("n", [31, 32, 33, 127, 128, 129, 256, 257, 511, 512, 513, 999, 1000, 1001, 2000, 2001])
def test_every_size_of_table(n):
    """Small tensors, some of them empty, with a long one among them."""
    sizes = [(7 * i) % 53 for i in range(n)]
    sizes[n // 2] = 70001
    check_clip(tensors(sizes, [BF, F], n), 2.0)
    ts = tensors(sizes, [HF], n + 1)
    assert abs(float(moe.moe_grad_norm(ts)) - norm64(ts)) <= 6 * U32 * norm64(ts)
    check_clip(ts, 1.0, tensors(sizes, [HF], n + 2))


def test_large_lists_in_one_and_in_several_tables():
    """Over 64 MB, where the sum and the scaling are cut differently."""
    for sizes in ([40_000_001], [90_001] * 400, [20_011] * 1700 + [3, 0, 5_000_000]):
        check_clip(tensors(sizes, [BF], len(sizes)), 1.0)
        ts = tensors(sizes, [F], len(sizes))
        total = moe.moe_grad_sumsq(ts)
        assert abs(float(total) - norm64(ts) ** 2) <= 9 * U32 * norm64(ts) ** 2
        before = [t.clone() for t in ts[:3]]
        moe.moe_grad_clip(ts, 1.0, sumsq=total)
        for t, b in zip(ts, before):
            want = b.double() / (float(total) ** 0.5 + 1e-6)
            assert ((t.double() - want).abs() <= 12 * U32 * want.abs()).all()


def test_large_tensors():
    """More chunks than a grid has blocks, and an element past 2^31 (4.3 GB)."""
    check_clip(tensors([50_000_001, 30_000_000], [BF, F], 9), 1.0)
    big = torch.zeros(2 ** 31 + 100, dtype=BF, device="cuda")
    big[5], big[-1] = 3.0, 4.0
    assert float(moe.moe_grad_norm([big])) == 5.0
    moe.moe_grad_clip([big], 2.5, eps=0.0)
    assert float(big[5]) == 1.5 and float(big[-1]) == 2.0


@pytest.mark.parametrize("scale", [1e25, 1e-25, 1e-30, 1e30])
@pytest.mark.parametrize("dtype", [BF, F])
def test_squares_outside_fp32(scale, dtype):
    check_clip(tensors([1000, 77, 20000], [dtype], 11, scale=scale), 0.1 * scale, eps=0.0)
    mixed = tensors([1000], [dtype], 12) + tensors([1000], [dtype], 13, scale=scale)
    check_clip(mixed, 1.0)


def test_zeros_and_no_tensors():
    z = torch.zeros(5000, device="cuda")
    assert float(moe.moe_grad_clip([z], 0.0, eps=0.0)) == 0 and (z == 0).all()
    assert float(moe.moe_grad_norm([])) == 0 and float(moe.moe_grad_clip([], 1.0)) == 0
    assert float(moe.moe_grad_sumsq([torch.empty(0, device="cuda")])) == 0


def test_infinity_and_nan_follow_the_formula():
    a, b = torch.ones(300, device="cuda"), torch.ones(50, dtype=BF, device="cuda")
    b[3] = math.inf
    assert float(moe.moe_grad_clip([a, b], 1.0)) == math.inf
    assert (a == 0).all() and math.isnan(b[3]) and (b[4:] == 0).all()
    c = torch.ones(300, device="cuda")
    c[7] = math.nan
    d = torch.ones(5, dtype=HF, device="cuda")
    assert math.isnan(moe.moe_grad_clip([c, d], 1.0)) and torch.isnan(c).all() and torch.isnan(d).all()


def test_same_result_every_time():
    ts = tensors([300001, 5, 70000] * 9, [BF, F], 15)
    tl = moe.TensorList(ts)
    first = moe.moe_grad_sumsq(tl)
    assert all(torch.equal(first, moe.moe_grad_sumsq(tl)) for _ in range(5))


def test_a_sum_of_squares_from_elsewhere():
    a, b = tensors([5000, 70], [F], 17), tensors([900], [BF], 18)
    total = moe.moe_grad_sumsq(a) + moe.moe_grad_sumsq(b)
    norm = norm64(a + b)
    before = a[0].double().clone()
    assert abs(float(moe.moe_grad_clip(a, 2.0, sumsq=total)) - norm) <= 6 * U32 * norm
    want = before * (2.0 / (norm + 1e-6))
    assert ((a[0].double() - want).abs() <= 12 * U32 * want.abs()).all()


def test_dense_in_another_order():
    base = torch.randn((40, 70, 3), device="cuda")
    check_clip([base.permute(2, 0, 1)], 1.0)
    check_clip([torch.randn((33, 21), device="cuda").t()], 1.0, [torch.empty((33, 21), device="cuda").t()])
    for bad in (base[:, ::2], base[:, :, :1], torch.ones(1, device="cuda").expand(4)):
        with pytest.raises(ValueError):
            moe.moe_grad_norm([bad])


@pytest.mark.parametrize("sizes", [[20000, 333, 4], [900001, 77, 40000], [333] * 50, [50_000_000]])
def test_stream_and_graphs_side_by_side(sizes):
    """Two captured graphs replayed at once on two streams, and a call on another stream."""
    sets = [tensors(sizes, [BF, F], s) for s in (21, 22)]
    keep = [[t.clone() for t in ts] for ts in sets]
    want = [norm64(ts) for ts in sets]
    moe.moe_grad_clip(tensors([10], [F], 1), 1.0)
    graphs, norms = [], []
    for ts in sets:
        tl = moe.TensorList(ts)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(moe.moe_grad_clip(tl, 1.0))
        graphs.append((g, tl))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for ts, k in zip(sets, keep):
            for t, b in zip(ts, k):
                t.copy_(b)
        torch.cuda.synchronize()
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for n, w in zip(norms, want):
            assert abs(float(n) - w) <= 6 * U32 * w
    for ts, w in zip(sets, want):
        assert abs(norm64(ts) - 1.0) <= 2 * HALF[BF]
    ts = tensors([5000], [F], 23)
    streams[0].wait_stream(torch.cuda.current_stream())
    n = moe.moe_grad_norm(ts, stream=streams[0])
    streams[0].synchronize()
    assert abs(float(n) - norm64(ts)) <= 6 * U32 * norm64(ts)


def test_refusals():
    t = torch.ones(100, device="cuda")
    for bad in ([t.double()], [t.cpu()], [t, t.int()]):
        with pytest.raises(ValueError):
            moe.TensorList(bad)
    with pytest.raises(ValueError):
        moe.TensorList([t], [])
    with pytest.raises(ValueError):
        moe.TensorList([t], [torch.ones(100, dtype=BF, device="cuda")])
    for tensors_, outs in (([t, t], None), ([t[:60], t[59:]], None), ([t[:50], t[50:]], [t[50:], t[:50]]),
                           ([t[:50], t[60:90]], [t[10:60], t[60:90]])):
        with pytest.raises(moe.MoEError):
            moe.TensorList(tensors_, outs)
    for args in ((math.nan,), (-1.0,), (math.inf,), (1.0, -1.0), (1.0, math.nan)):
        with pytest.raises(moe.MoEError):
            moe.moe_grad_clip([t], *args)
    with pytest.raises(ValueError):
        moe.moe_grad_clip([t], 1.0, sumsq=torch.ones((), device="cuda"))
