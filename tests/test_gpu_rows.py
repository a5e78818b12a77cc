"""moe_permute, moe_unpermute and their gradients against plain 64-bit forms.

Tolerances: a copy is exact.  A sum of K products in fp32, in any order, is off
by at most (K + 1) 2^-24 times the sum of the magnitudes, and the result is
rounded once to the row type.  A dot product over H columns goes through at
most H/32 + 32 fp32 additions in a row."""
import math

import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref
from _train_ref import DTYPES, HALF, TINY, U32

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1, 1), (1, 2048, 8, 256), (7, 3, 2, 5), (33, 30, 4, 9), (64, 64, 8, 8), (130, 1030, 6, 64),
         (5, 515, 32, 40), (257, 2048, 3, 16), (40, 4100, 9, 12), (3, 24, 17, 4),
         # Long rows of many tokens, at every alignment.
         (520, 1030, 6, 64), (1100, 515, 3, 8), (300, 4100, 9, 12), (129, 4097, 32, 40), (2100, 261, 2, 4),
         (1030, 512, 17, 24)]


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def close(got, want, err, dtype):
    """|got - want| <= the fp32 error `err` and one rounding to dtype."""
    bound = HALF[dtype] * (want.abs() + err) + err + TINY[dtype]
    d = (got.double().cpu() - want).abs()
    assert (d <= bound).all(), "off by %g of the bound" % (d / bound).max()


def setup(T, H, K, E, dtype, drop, seed=0):
    ids, off, inv = ref.routes(T, K, E, drop, seed)
    g = ref.gen(seed + 1)
    x = torch.randn((T, H), generator=g).to(dtype)
    y = torch.randn((T * K, H), generator=g).to(dtype)
    w = torch.rand((T, K), generator=g)
    w[torch.rand((T, K), generator=g) < 0.1] = 0.0
    return ids, off, inv, x, y, w


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("T,H,K,E", SIZES)
def test_permute(T, H, K, E, drop, dtype):
    ids, off, inv, x, _, _ = setup(T, H, K, E, dtype, drop)
    # The library's own sort gives these maps.
    o2, _, i2 = moe.moe_sort(ids.cuda(), E)
    assert torch.equal(o2.cpu(), off) and torch.equal(i2.cpu(), inv)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = moe.moe_permute(x.cuda(), inv.cuda(), off.cuda(), status=status)
    want = ref.permute(x, inv, K)
    assert torch.equal(bits(out.cpu()), bits(want)) and status.item() == 0
    # Without the offsets the rows behind the last one stay as they were.
    out = torch.full((T * K, H), 7.0, dtype=dtype, device="cuda")
    moe.moe_permute(x.cuda(), inv.cuda(), x_sorted=out)
    n = int(off[-1])
    assert torch.equal(bits(out[:n].cpu()), bits(want[:n])) and (out[n:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("T,H,K,E", SIZES)
def test_unpermute_and_permute_bwd(T, H, K, E, drop, dtype):
    _, off, inv, x, y, w = setup(T, H, K, E, dtype, drop)
    terms = ref.weighted(y, inv, w, T)
    err = (K + 2) * U32 * terms.abs().sum(1)
    close(moe.moe_unpermute(y.cuda(), inv.cuda(), w.cuda()), terms.sum(1), err, dtype)
    want = terms.sum(1) + x.double()
    err = (K + 2) * U32 * (terms.abs().sum(1) + x.double().abs())
    close(moe.moe_unpermute(y.cuda(), inv.cuda(), w.cuda(), x.cuda()), want, err, dtype)
    terms = ref.weighted(y, inv, None, T)
    close(moe.moe_permute_bwd(y.cuda(), inv.cuda(), T), terms.sum(1), (K + 2) * U32 * terms.abs().sum(1), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 0.97])
@pytest.mark.parametrize("T,H,K,E", [
    (1300, 4097, 5, 64), (2500, 1031, 10, 64), (3000, 514, 17, 40), (400, 2050, 32, 40), (12301, 2049, 1, 8),
    (1100, 4096, 16, 32), (4099, 1024, 17, 40), (600, 8192, 32, 40), (8200, 2048, 4, 8), (2400, 5000, 7, 12)])
def test_unpermute_of_many_long_rows(T, H, K, E, drop, dtype):
    """64 MB and more, where the rows go through shared memory (24 MB for rows that do not
    start on 16 bytes); against 64-bit sums on the GPU, slot by slot."""
    _, off, inv = ref.routes(T, K, E, drop, T)
    inv = inv.cuda()
    g = torch.Generator(device="cuda").manual_seed(H)
    y = torch.randn((T * K, H), generator=g, device="cuda").to(dtype)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    w = torch.rand((T, K), generator=g, device="cuda")
    w[torch.rand((T, K), generator=g, device="cuda") < 0.05] = 0.0
    y[int(off[-1]):] = math.nan  # behind the last row: not read
    y[inv[(inv >= 0) & (w.view(-1) == 0)].long()] = math.inf  # hidden by a weight of 0
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    size, plain, plain_size = torch.zeros_like(want), torch.zeros_like(want), torch.zeros_like(want)
    clean = torch.where(y.isfinite(), y, 0)
    for j in range(K):
        p = inv.view(T, K)[:, j]
        rows = torch.where((p >= 0)[:, None], clean[p.clamp(min=0).long()].double(), 0.0)
        plain += rows
        plain_size += rows.abs()
        want += rows * w[:, j, None]
        size += rows.abs() * w[:, j, None]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for got, exp, mag in ((moe.moe_unpermute(y, inv, w, status=status), want, size),
                          (moe.moe_unpermute(y, inv, w, x, status=status), want + x.double(), size + x.double().abs()),
                          (moe.moe_permute_bwd(clean, inv, T, status=status), plain, plain_size)):
        err = (K + 2) * U32 * mag
        bound = HALF[dtype] * (exp.abs() + err) + err + TINY[dtype]
        assert ((got.double() - exp).abs() <= bound).all()
    assert status.item() == 0
    # Corrupt positions among them.
    bad = inv.clone()
    bad[5], bad[T * K - 1], bad[T * K // 2] = T * K, -7, 2 ** 31 - 1
    cut = torch.where((bad < 0) | (bad >= T * K), -1, bad)
    assert torch.equal(moe.moe_permute_bwd(clean, bad, T, status=status), moe.moe_permute_bwd(clean, cut, T))
    assert status.item() == moe.MOE_STATUS_BAD_MAP


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("T,H,K,E", SIZES)
def test_unpermute_bwd(T, H, K, E, drop, dtype):
    _, off, inv, dout, y, w = setup(T, H, K, E, dtype, drop)
    n = int(off[-1])
    y[n:] = math.nan  # rows behind the last one are not read
    dy, dw = moe.moe_unpermute_bwd(dout.cuda(), y.cuda(), inv.cuda(), w.cuda(), off.cuda())
    r = (inv >= 0).nonzero()[:, 0]
    want = torch.zeros((T * K, H), dtype=torch.float64)
    want[inv[r].long()] = dout.double()[r // K] * w.double().view(-1)[r, None]
    close(dy, want, U32 * want.abs(), dtype)
    assert (dy[n:] == 0).all()
    prod = torch.zeros((T * K, H), dtype=torch.float64)
    prod[r] = dout.double()[r // K] * y.double()[inv[r].long()]
    d = (dw.double().cpu().view(-1) - prod.sum(1)).abs()
    assert (d <= (H / 32 + 32) * U32 * prod.abs().sum(1)).all()
    # One gradient at a time gives the same bits.
    dy1, none = moe.moe_unpermute_bwd(dout.cuda(), None, inv.cuda(), w.cuda(), off.cuda(), need_dw=False)
    assert none is None and torch.equal(bits(dy1), bits(dy))
    none, dw1 = moe.moe_unpermute_bwd(dout.cuda(), y.cuda(), inv.cuda(), w.cuda(), off.cuda(), need_dy=False)
    assert none is None and torch.equal(dw1, dw)


def test_unpermute_bwd_leaves_rows_without_the_offsets():
    _, off, inv, dout, y, w = setup(20, 40, 4, 8, torch.bfloat16, 0.5)
    dy = torch.full_like(y, 3.0).cuda()
    moe.moe_unpermute_bwd(dout.cuda(), None, inv.cuda(), w.cuda(), need_dw=False, dy_sorted=dy)
    n = int(off[-1])
    assert (dy[n:] == 3).all() and not (dy[:n] == 3).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_weight_of_zero_hides_its_row(bad, dtype):
    T, H, K = 6, 72, 4
    _, off, inv, dout, y, w = setup(T, H, K, 8, dtype, 0.0, seed=5)
    w = w + 0.1
    w[:, 2] = 0.0
    w[3] = 0.0  # a token with nothing left
    hidden = inv.view(T, K)[w == 0].long()
    clean = moe.moe_unpermute(y.cuda(), inv.cuda(), w.cuda())
    y2 = y.clone()
    y2[hidden] = bad
    out = moe.moe_unpermute(y2.cuda(), inv.cuda(), w.cuda())
    assert torch.equal(bits(out), bits(clean)) and (out[3] == 0).all()
    dout[1] = bad
    dy, dw = moe.moe_unpermute_bwd(dout.cuda(), y2.cuda(), inv.cuda(), w.cuda(), off.cuda())
    assert (dy[hidden.cuda()] == 0).all()
    # The weight's own gradient is the product with the row, whatever the weight.
    assert torch.isfinite(dw.cpu()[w != 0].view(-1)[:3]).all() and not torch.isfinite(dw[0, 2])


def test_corrupt_positions_are_skipped_and_reported():
    T, H, K = 9, 136, 3
    _, off, inv, x, y, w = setup(T, H, K, 4, torch.float32, 0.0, seed=7)
    bad = inv.clone()
    bad[4], bad[11], bad[20] = T * K, -2, 2 ** 31 - 1
    dropped = torch.where((bad < 0) | (bad >= T * K), -1, bad)
    w = w + 0.1
    for call in (lambda m, s: moe.moe_permute(x.cuda(), m, x_sorted=torch.zeros_like(y).cuda(), status=s),
                 lambda m, s: moe.moe_unpermute(y.cuda(), m, w.cuda(), status=s),
                 lambda m, s: moe.moe_permute_bwd(y.cuda(), m, T, status=s),
                 lambda m, s: moe.moe_unpermute_bwd(x.cuda(), y.cuda(), m, w.cuda(), status=s,
                                                    dy_sorted=torch.zeros_like(y).cuda())[0]):
        s1, s2 = torch.zeros((2, 4), dtype=torch.int32, device="cuda").unbind()
        a, b = call(bad.cuda(), s1[:1]), call(dropped.to(torch.int32).cuda(), s2[:1])
        assert torch.equal(a, b)
        assert s1[0] == moe.MOE_STATUS_BAD_MAP and s2[0] == 0


@pytest.mark.parametrize("H", [64, 35])
def test_linear_in_its_rows_and_weights(H):
    """Differences of the forward pass equal the gradients (it is linear in y and in w)."""
    T, K = 11, 5
    _, off, inv, dout, y, w = setup(T, H, K, 16, torch.float32, 0.2, seed=9)
    w = w + 0.1
    g = ref.gen(3)
    vy, vw = torch.randn(y.shape, generator=g), torch.randn(w.shape, generator=g)
    dy, dw = moe.moe_unpermute_bwd(dout.cuda(), y.cuda(), inv.cuda(), w.cuda(), off.cuda())
    f = lambda a, b: (moe.moe_unpermute(a.cuda(), inv.cuda(), b.cuda()).double().cpu() * dout.double()).sum()  # noqa: E731
    size = float((ref.weighted(y.abs() + vy.abs(), inv, w + vw.abs(), T).sum(1) * dout.double().abs()).sum())
    tol = 4 * (H + K + 8) * U32 * size
    assert abs(f(y + vy, w) - f(y - vy, w) - 2 * (dy.double().cpu() * vy).sum()) <= tol
    assert abs(f(y, w + vw) - f(y, w - vw) - 2 * (dw.double().cpu() * vw).sum()) <= tol


def test_rows_past_32_bit_offsets():
    """T*K*H = 2.2e9 elements, rows of 16896 bytes."""
    T, K, H, E = 16384, 16, 8448, 64
    ids = torch.rand((T, E), device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
    off, srt, inv = moe.moe_sort(ids, E)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    xs = moe.moe_permute(x, inv, off)
    for p in (0, 1, T * K // 2, T * K - 2, T * K - 1):
        assert torch.equal(xs[p], x[srt[p] // K])
    # Each token's 16 equal rows add up exactly, whatever the order.
    dx = moe.moe_permute_bwd(xs, inv, T)
    assert torch.equal(dx, 16 * x)
    w = torch.full((T, K), 0.5, device="cuda")
    assert torch.equal(moe.moe_unpermute(xs, inv, w), 8 * x)
    dy, dw = moe.moe_unpermute_bwd(x, xs, inv, w, off, dy_sorted=torch.empty_like(xs))
    for p in (0, T * K // 2, T * K - 1):
        assert torch.equal(dy[p], 0.5 * x[srt[p] // K])
    want = x.double().square().sum(1)
    assert ((dw.double() - want[:, None]).abs() <= (H / 32 + 32) * U32 * want[:, None]).all()


def test_no_tokens_and_no_kept_routes():
    x = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    inv = torch.empty(0, dtype=torch.int32, device="cuda")
    w = torch.empty((0, 4), device="cuda")
    assert moe.moe_permute(x, inv).shape == (0, 16)
    assert moe.moe_unpermute(x, inv, w).shape == (0, 16)
    assert moe.moe_permute_bwd(x, inv, 0).shape == (0, 16)
    dy, dw = moe.moe_unpermute_bwd(x, x, inv, w)
    assert dy.shape == (0, 16) and dw.shape == (0, 4)
    assert moe.moe_unpermute_bwd(x, x, inv, w, need_dy=False, need_dw=False) == (None, None)


def test_another_stream_and_a_captured_graph():
    T, H, K, E = 50, 520, 4, 16
    _, off, inv, x, y, w = (t.cuda() for t in setup(T, H, K, E, torch.bfloat16, 0.3))
    want = (moe.moe_permute(x, inv, off), moe.moe_unpermute(y, inv, w), moe.moe_permute_bwd(y, inv, T),
            *moe.moe_unpermute_bwd(x, y, inv, w, off))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (moe.moe_permute(x, inv, off, stream=side), moe.moe_unpermute(y, inv, w, stream=side),
           moe.moe_permute_bwd(y, inv, T, stream=side), *moe.moe_unpermute_bwd(x, y, inv, w, off, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = (moe.moe_permute(x, inv, off), moe.moe_unpermute(y, inv, w), moe.moe_permute_bwd(y, inv, T),
               *moe.moe_unpermute_bwd(x, y, inv, w, off))
    x.neg_()
    y.neg_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, -b) for a, b in zip(cap[:4], want[:4])) and torch.equal(cap[4], want[4])


def test_refusals():
    _, off, inv, x, y, w = (t.cuda() for t in setup(8, 32, 2, 4, torch.bfloat16, 0.0))
    for call in (lambda: moe.moe_permute(x.double(), inv), lambda: moe.moe_permute(x.t(), inv),
                 lambda: moe.moe_permute(x, inv[:-1]), lambda: moe.moe_permute(x, inv.long()),
                 lambda: moe.moe_permute(x, inv.cpu()), lambda: moe.moe_permute(x.cpu(), inv),
                 lambda: moe.moe_permute(x, inv, x_sorted=y.float()),
                 lambda: moe.moe_permute(x, inv, x_sorted=y[:-1]),
                 lambda: moe.moe_unpermute(y, inv, w.half()), lambda: moe.moe_unpermute(y[:-1], inv, w),
                 lambda: moe.moe_unpermute(y, inv, w, x.half()), lambda: moe.moe_unpermute(y, inv[1:], w),
                 lambda: moe.moe_permute_bwd(y, inv, 5), lambda: moe.moe_unpermute_bwd(x, None, inv, w),
                 lambda: moe.moe_unpermute_bwd(x, y[1:], inv, w), lambda: moe.moe_unpermute_bwd(x, y, inv, w[1:])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_unpermute(y, inv, w, out=y[:8]), lambda: moe.moe_unpermute(y, inv, w, x, out=x),
                 lambda: moe.moe_unpermute_bwd(x, y, inv, w, dy_sorted=y)):
        with pytest.raises(moe.MoEError):
            call()
    with pytest.raises(moe.MoEError):  # rows that do not start on 16 bytes
        moe.moe_permute(torch.empty(8 * 32 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 32), inv)
