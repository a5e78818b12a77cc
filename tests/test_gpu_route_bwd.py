"""moe_route_bwd against the 64-bit gradient of the route weights.

Tolerance: a score is off by a few fp32 roundings and by the rounding of
l - l_max, |l - l_max| 2^-24; its sums over K choices (and E logits, E/32 in a
row, for the full softmax) add one each.  With c the count of them,
|d - exact| <= c 2^-24 scaling (|G_j| + sum_i |G_i| q_i) q_j.  The 64-bit form
itself goes through the whole row's softmax: where the formula gives 0 or
nearly, its terms of up to scaling |G| cancel only to a few of their own
roundings of 2^-53 (2^-48 sum |G| is allowed for up to 32 of them)."""
import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref
from _train_ref import U32

pytestmark = pytest.mark.gpu

VARIANTS = [(score, renorm, scaling) for score in (0, 1) for renorm in (True, False) for scaling in (1.0, 2.5)]


def data(T, E, K, seed, spread=1.0, mask=0.0):
    g = ref.gen(seed)
    logits = torch.randn((T, E), generator=g) * spread
    ids = logits.topk(K, dim=1).indices.to(torch.int32)
    dw = torch.randn((T, K), generator=g)
    zm = (torch.rand((T, K), generator=g) < mask).to(torch.uint8) if mask else None
    return logits, ids, dw, zm


def exact(logits, ids, dw, score, renorm, scaling, zm):
    l64 = logits.double().requires_grad_()
    w = ref.route_weights(l64, ids, score, renorm, scaling, zm)
    g = torch.autograd.grad(w, l64, dw.double())[0]
    with torch.no_grad():
        G = (dw if zm is None else dw.masked_fill(zm.bool(), 0.0)).double().abs()
        s = torch.sigmoid(l64) if score else torch.softmax(l64, 1)
        mine = s.gather(1, ids.long())
        q = mine / mine.sum(1, keepdim=True) if renorm else mine
        # The bound's q_j (|G_j| + sum) at the chosen experts; p_e sum elsewhere (full softmax).
        total = (G * q).sum(1, keepdim=True)
        size = torch.zeros_like(s) if score or renorm else s * total
        size.scatter_(1, ids.long(), q * (G + total))
        spread = float((logits.max() - logits.min()))
        c = 48 + logits.shape[1] / 32 + ids.shape[1] + spread
        own = 2.0 ** -48 * scaling * G.sum(1, keepdim=True)  # the 64-bit form's rounding
    return g, c * U32 * scaling * size + own


def check(logits, ids, dw, score, renorm, scaling, zm):
    want, bound = exact(logits, ids, dw, score, renorm, scaling, zm)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = moe.moe_route_bwd(logits.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renorm, scaling=scaling,
                            zero_mask=None if zm is None else zm.cuda(), status=status,
                            dlogits=torch.full_like(logits, 9.0).cuda())
    d = (got.double().cpu() - want).abs()
    assert (d <= bound + 1e-38).all(), "off by %g of the bound" % (d / (bound + 1e-38)).max()
    assert status.item() == 0
    return got


@pytest.mark.parametrize("score,renorm,scaling", VARIANTS)
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 8), (5, 7, 3), (64, 256, 8), (33, 512, 10), (9, 1024, 32),
                                   (130, 100, 6), (17, 33, 2)])
def test_against_64_bits(T, E, K, score, renorm, scaling):
    check(*data(T, E, K, T + E)[:3], score, renorm, scaling, None)
    lg, ids, dw, zm = data(T, E, K, T + E + 1, spread=4.0, mask=0.3)
    dw[zm.bool()] = float("nan")  # a masked weight's gradient is not looked at
    check(lg, ids, torch.where(zm.bool(), 0.0, dw), score, renorm, scaling, zm)
    a = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renorm, scaling=scaling,
                          zero_mask=zm.cuda())
    assert torch.isfinite(a).all()


@pytest.mark.parametrize("score,renorm,scaling", VARIANTS)
def test_against_differences_of_the_forward_pass(score, renorm, scaling):
    """Central differences of moe_route_ex with a step of 2^-6 along random directions: off by
    at most h^2/6 times a third derivative (below 2 for these scores and unit
    directions) and by the weights' rounding, 1e-5 (the routing test's) / h."""
    T, E, K, h = 40, 24, 4, 2.0 ** -6
    lg, ids, dw, _ = data(T, E, K, 3)
    lg.scatter_(1, ids.long(), lg.gather(1, ids.long()) + 5.0 + torch.arange(K, 0, -1))
    cfg = dict(score=score, renormalize=renorm, scaling=scaling)
    grad = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda(), **cfg).double().cpu()
    for k in range(4):
        v = torch.randn((T, E), generator=ref.gen(50 + k))
        v = v / v.norm(dim=1, keepdim=True)
        (i1, w1), (i2, w2) = (moe.moe_route_ex((lg + s * h * v).cuda(), K, **cfg) for s in (1, -1))
        assert torch.equal(i1.cpu(), ids) and torch.equal(i2.cpu(), ids)
        diff = ((w1 - w2).double().cpu() * dw.double()).sum(1) / (2 * h)
        tol = scaling * dw.double().abs().sum(1) * (2 * h * h / 6 + 1e-5 / h)
        assert ((diff - (grad * v.double()).sum(1)).abs() <= tol).all()


def test_bias_and_groups_choose_only():
    lg, ids, dw, _ = data(20, 64, 8, 11)
    kw = dict(score=1, scaling=2.5)
    a = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda(), **kw)
    b = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda(), sel_bias=torch.randn(64).cuda(), n_group=8, topk_group=4,
                          **kw)
    assert torch.equal(a, b)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_missing_and_repeated_choices(score, renorm):
    lg, ids, dw, _ = data(12, 16, 4, 13)
    ids[0] = -1
    ids[1, 2] = 16
    ids[2, 1:3] = -5
    ids[4, 3] = ids[4, 0]
    ids[5] = ids[5, 0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renorm, status=status)
    assert status.item() == moe.MOE_STATUS_BAD_ID
    for t in range(12):
        on = (ids[t] >= 0) & (ids[t] < 16)
        if not on.any():
            assert (got[t] == 0).all()
            continue
        row = slice(t, t + 1)
        want, bound = exact(lg[row], ids[row][:, on], dw[row][:, on], score, renorm, 1.0, None)
        # A repeated expert's bound is that of its choices together.
        bound = bound.max() * 4 + 1e-30
        assert ((got[row].double().cpu() - want).abs() <= bound).all()


def test_scores_far_out():
    """Chosen logits 200 apart (softmax) and scores that all vanish in fp32 (sigmoid): finite gradients."""
    lg = torch.tensor([[100.0, -100.0, 0.0, 50.0], [-150.0, -160.0, -200.0, -300.0]])
    ids = torch.tensor([[0, 3], [0, 1]], dtype=torch.int32)
    dw = torch.tensor([[1.0, -2.0], [3.0, 4.0]])
    for score, renorm, scaling in VARIANTS:
        got = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renorm, scaling=scaling)
        assert torch.isfinite(got).all()
    want, bound = exact(lg, ids, dw, 0, True, 1.0, None)
    got = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda())
    assert ((got.double().cpu() - want).abs() <= bound + 1e-38).all()


@pytest.mark.parametrize("score,renorm,scaling", VARIANTS)
def test_masked_logits(score, renorm, scaling):
    """Experts masked by -inf or the lowest value: chosen or not, they get no gradient; a token
    whose chosen experts are all masked gets none at all.  NaN stays in its own row."""
    lowest = torch.finfo(torch.float32).min
    T, E, K = 8, 12, 4
    lg, ids, dw, _ = data(T, E, K, 23)
    masked = torch.ones((T, E), dtype=torch.bool).scatter_(1, ids.long(), False)
    lg[:4] = torch.where(masked[:4], torch.tensor([float("-inf"), lowest, float("-inf"), lowest])[:, None], lg[:4])
    lg[1, ids[1, 3]] = float("-inf")  # fewer experts left than choices
    lg[2, ids[2].long()] = float("-inf")
    lg[2] = float("-inf")
    lg[5, ids[5, 0]] = float("nan")
    cfg = dict(score=score, renormalize=renorm, scaling=scaling)
    got = moe.moe_route_bwd(lg.cuda(), ids.cuda(), dw.cuda(), **cfg).cpu()
    assert torch.isfinite(got[[0, 1, 2, 3, 4, 6, 7]]).all()
    assert (got[2] == 0).all() and got[1, ids[1, 3]] == 0 and not torch.isfinite(got[5]).all()
    assert (got[:2][masked[:2]] == 0).all()
    rows = torch.tensor([0, 3, 4, 6, 7])
    want, bound = exact(lg[rows].clamp(min=-1e4), ids[rows], dw[rows], score, renorm, scaling, None)
    assert ((got[rows].double() - want).abs() <= bound + 1e-38).all()


def test_stream_graph_and_refusals():
    lg, ids, dw, _ = (None if t is None else t.cuda() for t in data(70, 128, 6, 17))
    want = moe.moe_route_bwd(lg, ids, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_route_bwd(lg, ids, dw, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = moe.moe_route_bwd(lg, ids, dw)
    dw.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap, -want)
    assert moe.moe_route_bwd(lg[:0], ids[:0], dw[:0]).shape == (0, 128)
    for call in (lambda: moe.moe_route_bwd(lg.half(), ids, dw), lambda: moe.moe_route_bwd(lg, ids.long(), dw),
                 lambda: moe.moe_route_bwd(lg, ids, dw[:, 1:]), lambda: moe.moe_route_bwd(lg, ids[1:], dw),
                 lambda: moe.moe_route_bwd(lg, ids, dw, zero_mask=ids), lambda: moe.moe_route_bwd(lg.cpu(), ids, dw)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moe.moe_route_bwd(lg, ids, dw, score=7), lambda: moe.moe_route_bwd(lg, ids, dw, dlogits=lg),
                 lambda: moe.moe_route_bwd(lg, ids, dw, scaling=0.0)):
        with pytest.raises(moe.MoEError):
            call()
