"""The training calls together: the differentiable functions and RoutedLayer
against a plain 64-bit layer, with its gradients and their clipping."""
import math

import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe
import _train_ref as ref
from _train_ref import HALF, U32
from mixture_experts_ffn_sort_b200 import ep, train

pytestmark = pytest.mark.gpu


class Experts(torch.nn.Module):
    """One matrix and a tanh for every expert, in plain torch."""

    def __init__(self, E, H, dtype, seed):
        super().__init__()
        w = torch.randn((E, H, H), generator=ref.gen(seed)) * H ** -0.5
        self.w = torch.nn.ParameterList([torch.nn.Parameter(w[e].to(dtype).cuda()) for e in range(E)])

    def forward(self, x, offsets):
        ends = offsets.tolist()
        rows = [torch.tanh(x[a:b] @ w) for a, b, w in zip(ends, ends[1:], self.w)]
        return torch.cat(rows + [torch.zeros_like(x[ends[-1]:])])


def plain(layer, x, ids, zero_mask, cfg):
    """The same layer in fp64 with the choice held fixed: every token through every expert."""
    p = {n: q.detach().double().cpu().requires_grad_() for n, q in layer.named_parameters()}
    x = x.detach().double().cpu().requires_grad_()
    wr = p["w_router"]
    w = ref.route_weights(x @ wr.t(), ids, cfg.get("score", 0), cfg.get("renormalize", True), cfg.get("scaling", 1.0),
                          zero_mask)
    every = torch.stack([torch.tanh(x @ p["experts.w.%d" % e]) for e in range(layer.n_experts)], 1)
    out = (every.gather(1, ids.long()[:, :, None].expand(-1, -1, x.shape[1])) * w[:, :, None]).sum(1)
    if layer.shared is not None:
        out = out + torch.tanh(x @ p["shared.w"])
    return out, x, p


class Shared(torch.nn.Module):
    def __init__(self, H, dtype):
        super().__init__()
        self.w = torch.nn.Parameter((torch.randn((H, H), generator=ref.gen(77)) * H ** -0.5).to(dtype).cuda())

    def forward(self, x):
        return torch.tanh(x @ self.w)


CFGS = [{}, dict(score=1, scaling=2.5), dict(renormalize=False), dict(score=1, renormalize=False)]


@pytest.mark.parametrize("cfg", CFGS)
@pytest.mark.parametrize("dtype,T,H,E,K,shared,mask", [
    (torch.float32, 37, 40, 6, 3, True, 0.2), (torch.float32, 1, 128, 8, 2, False, 0.0),
    (torch.bfloat16, 50, 128, 16, 4, True, 0.1), (torch.bfloat16, 9, 72, 5, 2, False, 0.0)])
def test_layer_and_its_gradients(dtype, T, H, E, K, shared, mask, cfg):
    """fp32: products of length H and the sums after them, rounded a few times each on the way
    forward and back, 2^-24 (H + 64) relative in norm at most.  bf16: about twelve roundings
    to bf16 one after another (2^-8 each at most), in every output and gradient.
    The factor of 4: the norms of intermediates that cancel in part."""
    layer = train.RoutedLayer(H, E, K, Experts(E, H, dtype, 5), Shared(H, dtype) if shared else None, cfg, dtype)
    assert layer.fused_router() == (dtype == torch.bfloat16 and H % 64 == 0)
    g = ref.gen(T + H)
    x = torch.randn((T, H), generator=g).to(dtype).cuda().requires_grad_()
    zm = (torch.rand((T, K), generator=g) < mask).cuda() if mask else None
    dout = torch.randn((T, H), generator=g).to(dtype)
    torch.backends.cuda.matmul.allow_tf32 = False
    out = layer(x, zm)
    out.backward(dout.cuda())
    plan = layer.plan
    ids = (torch.searchsorted(plan.expert_offsets, plan.inv_route, right=True) - 1).view(T, K).to(torch.int32).cpu()
    want, x64, p64 = plain(layer, x, ids, None if zm is None else zm.cpu(), cfg)
    want.backward(dout.double())
    tol = 4 * (U32 * (H + 64) if dtype == torch.float32 else 12 * HALF[dtype])
    pairs = [(out, want, "out"), (x.grad, x64.grad, "x")]
    pairs += [(q.grad, p64[n].grad, n) for n, q in layer.named_parameters() if not n.startswith("experts")]
    pairs.append((torch.stack([q.grad for q in layer.experts.w]),
                  torch.stack([p64["experts.w.%d" % e].grad if p64["experts.w.%d" % e].grad is not None else
                               torch.zeros((H, H), dtype=torch.float64) for e in range(E)]), "experts"))
    for got, exp, name in pairs:
        assert got is not None, name
        off = float((got.detach().double().cpu() - exp.detach()).norm())
        assert off <= tol * float(exp.detach().norm()) + 1e-30, (name, off, float(exp.norm()))
    # Clipping all of them by their norm.
    params = list(layer.parameters())
    before = [q.grad.double().clone() for q in params]
    norm = math.sqrt(sum(float(b.square().sum()) for b in before))
    got = train.clip_grad_norm(params, 0.5 * norm)
    assert abs(float(got) - norm) <= 6 * U32 * norm
    for q, b in zip(params, before):
        assert ((q.grad.double() - 0.5 * b).abs() <= (HALF[dtype] + 20 * U32) * b.abs() + 1e-6 * b.abs() / norm).all()


def test_gradients_that_are_not_wanted():
    H, E, K, T = 64, 4, 2, 12
    _, off, inv = ref.routes(T, K, E, 0.2, 3)
    plan = train.RoutePlan(off.cuda(), None, inv.cuda(), T, K, E)
    y = torch.randn((T * K, H), device="cuda", requires_grad=True)
    w = torch.rand((T, K), device="cuda", requires_grad=True)
    sh = torch.randn((T, H), device="cuda", requires_grad=True)
    dout = torch.randn((T, H), device="cuda")
    full = torch.autograd.grad(train.unpermute(y, w, plan, sh), (y, w, sh), dout)
    assert torch.equal(full[2], dout)
    assert torch.equal(torch.autograd.grad(train.unpermute(y, w.detach(), plan), y, dout)[0], full[0])
    assert torch.equal(torch.autograd.grad(train.unpermute(y.detach(), w, plan), w, dout)[0], full[1])
    assert torch.equal(torch.autograd.grad(train.unpermute(y.detach(), w.detach(), plan, sh), sh, dout)[0], dout)
    # A broadcast gradient, as a sum's is.
    a = torch.autograd.grad(train.unpermute(y, w, plan).sum(), (y, w))
    b = torch.autograd.grad(train.unpermute(y, w, plan), (y, w), torch.ones((T, H), device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    x = torch.randn((T, H), device="cuda", requires_grad=True)
    train.permute(x, plan).sum().backward()
    kept = (inv.view(T, K) >= 0).sum(1).float()
    assert torch.equal(x.grad.cpu(), kept[:, None].expand(T, H))


def test_dropped_routes_give_zero_rows_and_no_gradient():
    T, H, K, E = 20, 48, 3, 4
    ids, off, inv = ref.routes(T, K, E, 0.5, 9)
    plan = train.sort_plan(ids.cuda(), E)
    assert torch.equal(plan.inv_route.cpu(), inv)
    x = torch.randn((T, H), device="cuda", requires_grad=True)
    xs = train.permute(x, plan)
    n = int(off[-1])
    assert (xs[n:] == 0).all()
    dxs = torch.full_like(xs, math.nan)
    dxs[:n] = 1.0
    g = torch.autograd.grad(xs, x, dxs)[0]
    assert torch.isfinite(g).all()


def test_slices_and_gradients_that_start_anywhere():
    """Rows of 6 bytes out of the middle of larger tensors, gradients of a concatenation."""
    T, H, K, E = 21, 3, 2, 4
    _, off, inv = ref.routes(T, K, E, 0.2, 5)
    plan = train.RoutePlan(off.cuda(), None, inv.cuda(), T, K, E)
    big = torch.randn((T * K + 9, H), device="cuda").half()
    wide = torch.rand((T + 3, K), device="cuda")
    x, y, w, sh = big[1:T + 1], big[5:T * K + 5], wide[1:T + 1], big[3:T + 3]
    args = [t.clone().requires_grad_() for t in (x, y, w, sh)]
    sliced = [t.detach().requires_grad_() for t in (x, y, w, sh)]
    head = torch.randn((5, H), device="cuda").half()
    grads = []
    for a, b, c, d in (args, sliced):
        xs, out = train.permute(a, plan), train.unpermute(b, c, plan, d)
        loss = (torch.cat([head, xs]).float().square().sum() + torch.cat([head, out]).float().square().sum())
        grads.append(torch.autograd.grad(loss, (a, b, c, d)))
    assert all(torch.equal(p, q) for p, q in zip(*grads))
    lg = torch.randn((T + 2, E + 1), device="cuda")
    ids, rw = train.route(lg[1:T + 1, 1:].requires_grad_(), K)
    i2, r2 = moe.moe_route(lg[1:T + 1, 1:].clone(), K)
    assert torch.equal(ids, i2) and torch.equal(rw, r2)


def test_no_tokens():
    layer = train.RoutedLayer(64, 8, 2, Experts(8, 64, torch.bfloat16, 1))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    out = layer(x)
    out.sum().backward()
    assert out.shape == (0, 64) and x.grad.shape == (0, 64) and (layer.w_router.grad == 0).all()


def test_forward_and_backward_in_a_graph():
    """One captured step (no eager graph of the same leaves is alive), replayed on new rows."""
    T, H, E, K = 64, 128, 8, 2
    wr = (torch.randn((E, H), device="cuda") * H ** -0.5).bfloat16().requires_grad_()
    x = torch.randn((T, H), device="cuda").bfloat16().requires_grad_()

    def step():
        ids, w = train.router(x, wr, K)
        plan = train.sort_plan(ids, E)
        y = train.permute(x, plan) * 2
        out = train.unpermute(y, w, plan)
        gx, gw = torch.autograd.grad(out.float().square().sum(), (x, wr))
        norm = moe.moe_grad_clip([gx, gw], 1.0)
        return out.detach(), gx, gw, norm

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = step()
    with torch.no_grad():
        x.copy_(torch.randn((T, H), device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in cap]
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_sharded_norm_without_a_group():
    """One rank: the expert and the replicated gradients count once each."""
    a = [torch.randn(500, device="cuda"), torch.randn((7, 9), device="cuda").bfloat16()]
    b = [torch.randn(40, device="cuda")]
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in a + b))
    before = [t.double().clone() for t in a + b]
    got = ep.clip_grad_norm(a, b, 1.0)
    assert abs(float(got) - norm) <= 8 * U32 * norm
    for t, q in zip(a + b, before):
        assert ((t.double() - q / norm).abs() <= (HALF[t.dtype] + 30 * U32 + 1e-6 / norm) * q.abs() / norm).all()


def test_a_capture_that_forks_and_joins():
    """The calls on two captured streams, joined, and replayed on new values."""
    T, H, K, E = 90, 264, 4, 8
    ids, off, inv = (t.cuda() for t in ref.routes(T, K, E, 0.2, 21))
    x, y = torch.randn((T, H), device="cuda"), torch.randn((T * K, H), device="cuda")
    w, lg = torch.rand((T, K), device="cuda"), torch.randn((T, E), device="cuda")

    def left():
        return [moe.moe_permute(x, inv, off), *moe.moe_unpermute_bwd(x, y, inv, w, off)]

    def right():
        return [moe.moe_unpermute(y, inv, w), moe.moe_route_bwd(lg, ids, w), moe.moe_grad_norm([x, y])]

    def both():
        a, b = left(), right()
        return a + b + [moe.moe_unpermute(a[0], inv, w), a[1] * 2]

    both()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b = right()
        a = left()
        torch.cuda.current_stream().wait_stream(side)
        cap = a + b + [moe.moe_unpermute(a[0], inv, w), a[1] * 2]
    for t in (x, y, w, lg):
        t.copy_(torch.randn_like(t))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(cap, both()))


def test_calls_from_several_threads():
    """Four host threads, each on a stream of its own, with lists and rows of their own."""
    import threading
    T, H, K, E = 64, 520, 4, 8
    failures = []

    def work(k):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                _, off, inv = (t.cuda() for t in ref.routes(T, K, E, 0.2, 30 + k))
                x = torch.randn((T, H), generator=ref.gen(k)).cuda()
                w = torch.rand((T, K), generator=ref.gen(k)).cuda()
                want = None
                for _ in range(30):
                    xs = moe.moe_permute(x, inv, off)
                    out = moe.moe_unpermute(xs, inv, w)
                    dy, dw = moe.moe_unpermute_bwd(out, xs, inv, w, off)
                    got = [xs, out, dy, dw, moe.moe_grad_clip([dy.clone(), dw.clone()], 1.0)]
                    if want is None:
                        want = got
                    elif not all(torch.equal(p, q) for p, q in zip(got, want)):
                        failures.append(k)
                try:
                    moe.moe_permute(x, inv[:-1])
                    failures.append("accepted")
                except ValueError:
                    pass
        except Exception as e:  # reported below
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
