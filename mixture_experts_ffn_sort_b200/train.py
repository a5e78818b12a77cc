"""Training the routed layer around expert products of the caller's own: the
library's routing, row and gradient calls as differentiable functions.

    plan        = sort_plan(ids, E)                    moe_sort
    ids, w      = route(logits, K, ...)                moe_route_ex   / moe_route_bwd
    ids, w      = router(x, w_router, K, ...)          moe_router     / moe_route_bwd and two matrix products
    x_sorted    = permute(x, plan)                     moe_permute    / moe_permute_bwd
    out         = unpermute(y_sorted, w, plan, ...)    moe_unpermute  / moe_unpermute_bwd

The steps are those of the Nemotron-H page's sorted path
(spark_model/layers/nemotron_moe.rs, `prefill`, steps 2 and 5) and the NKI
library's Router Top-K, Permute Routed Tokens and Top-K Reduce.  RoutedLayer
runs them in order around a function of the sorted rows; clip_grad_norm clips
its gradients (and any others) by their global norm.

Every function runs on the current stream.  Gradients of gradients are not
defined.  A step may be captured in a CUDA graph after a first one, with
torch.autograd.grad, or with backward() as long as no eager graph of the same
leaves is alive.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Callable, Iterable, Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import (MOE_SCORE_SOFTMAX, moe_grad_clip, moe_permute, moe_permute_bwd, moe_route_bwd, moe_route_ex, moe_router,
               moe_sort, moe_unpermute, moe_unpermute_bwd)


@dataclass
class RoutePlan:
    """What moe_sort leaves of T tokens' K choices among E experts: expert e's
    rows are expert_offsets[e] .. expert_offsets[e + 1] of the sorted ones."""

    expert_offsets: torch.Tensor
    sorted_route: torch.Tensor
    inv_route: torch.Tensor
    T: int
    K: int
    E: int


def _base(t: torch.Tensor) -> torch.Tensor:
    """t as the library takes it: contiguous from a 16-byte boundary on (a slice of a
    larger tensor, such as the gradient of a concatenation, may start anywhere)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def sort_plan(topk_ids: torch.Tensor, E: int, status: Optional[torch.Tensor] = None) -> RoutePlan:
    """Sort the choices topk_ids [T, K] i32 by expert (an id outside [0, E) is a
    dropped route: it has no row)."""
    T, K = topk_ids.shape
    off, srt, inv = moe_sort(_base(topk_ids), E, status)
    return RoutePlan(off, srt, inv, T, K, E)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, K, zero_mask, cfg):
        ids, w = moe_route_ex(logits, K, zero_mask=zero_mask, **cfg)
        ctx.save_for_backward(logits, ids, zero_mask)
        ctx.cfg = cfg
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        logits, ids, zero_mask = ctx.saved_tensors
        return moe_route_bwd(logits, ids, _base(dw), zero_mask=zero_mask, **ctx.cfg), None, None, None


def route(logits: torch.Tensor, K: int, score: int = MOE_SCORE_SOFTMAX, sel_bias: Optional[torch.Tensor] = None,
          n_group: int = 1, topk_group: Optional[int] = None, renormalize: bool = True, scaling: float = 1.0,
          zero_mask: Optional[torch.Tensor] = None):
    """moe_route_ex with a gradient: logits [T, E] f32 -> (topk_ids, topk_w)."""
    cfg = dict(score=score, sel_bias=sel_bias, n_group=n_group, topk_group=topk_group, renormalize=renormalize,
               scaling=scaling)
    return _Route.apply(_base(logits), K, _mask(zero_mask), cfg)


def _product(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """a @ b in fp32, in an autocast region too (there the product would be rounded to 16 bits)."""
    with torch.autocast("cuda", enabled=False):
        return a.float() @ b.float()


def _mask(zero_mask):
    if zero_mask is None:
        return None
    zero_mask = zero_mask.contiguous()
    return zero_mask.view(torch.uint8) if zero_mask.dtype == torch.bool else zero_mask


class _Router(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_router, K, zero_mask, cfg):
        logits = torch.empty((x.shape[0], w_router.shape[0]), dtype=torch.float32, device=x.device)
        ids, w = moe_router(x, w_router, K, zero_mask=zero_mask, logits=logits, **cfg)
        ctx.save_for_backward(x, w_router, logits, ids, zero_mask)
        ctx.cfg = cfg
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        x, w_router, logits, ids, zero_mask = ctx.saved_tensors
        dlogits = moe_route_bwd(logits, ids, _base(dw), zero_mask=zero_mask, **ctx.cfg)
        # The gate GEMM's own gradients: two plain products, in fp32 like its logits.
        dx = _product(dlogits, w_router).to(x.dtype) if ctx.needs_input_grad[0] else None
        dwr = _product(dlogits.t(), x).to(w_router.dtype) if ctx.needs_input_grad[1] else None
        return dx, dwr, None, None, None


def router(x: torch.Tensor, w_router: torch.Tensor, K: int, score: int = MOE_SCORE_SOFTMAX,
           sel_bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: Optional[int] = None,
           renormalize: bool = True, scaling: float = 1.0, zero_mask: Optional[torch.Tensor] = None):
    """moe_router with gradients: x [T, H] bf16 and w_router [E, H] bf16 -> (topk_ids, topk_w)."""
    cfg = dict(score=score, sel_bias=sel_bias, n_group=n_group, topk_group=topk_group, renormalize=renormalize,
               scaling=scaling)
    return _Router.apply(_base(x), _base(w_router), K, _mask(zero_mask), cfg)


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, inv_route, expert_offsets):
        ctx.save_for_backward(inv_route)
        ctx.T = x.shape[0]
        return moe_permute(x, inv_route, expert_offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dx_sorted):
        (inv_route,) = ctx.saved_tensors
        return moe_permute_bwd(_base(dx_sorted), inv_route, ctx.T), None, None


def permute(x: torch.Tensor, plan: RoutePlan) -> torch.Tensor:
    """Token rows [T, H] -> rows sorted by expert [T*K, H] (zeros behind the last one)."""
    return _Permute.apply(_base(x), plan.inv_route, plan.expert_offsets)


class _Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y_sorted, topk_w, y_shared, inv_route, expert_offsets):
        need_dw = ctx.needs_input_grad[1]
        ctx.save_for_backward(y_sorted if need_dw else None, topk_w, inv_route, expert_offsets)
        return moe_unpermute(y_sorted, inv_route, topk_w, y_shared)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y_sorted, topk_w, inv_route, expert_offsets = ctx.saved_tensors
        need_dy, need_dw, need_shared = ctx.needs_input_grad[:3]
        dy, dw = moe_unpermute_bwd(_base(dout), y_sorted, inv_route, topk_w, expert_offsets, need_dy, need_dw)
        return dy, dw, dout if need_shared else None, None, None


def unpermute(y_sorted: torch.Tensor, topk_w: torch.Tensor, plan: RoutePlan,
              y_shared: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Sorted rows [T*K, H] and route weights [T, K] (and the shared expert's rows [T, H]) -> [T, H]."""
    return _Unpermute.apply(_base(y_sorted), _base(topk_w), None if y_shared is None else _base(y_shared), plan.inv_route, plan.expert_offsets)


class RoutedLayer(torch.nn.Module):
    """A routed layer that trains: router -> sort -> permute -> experts ->
    unpermute (+ shared expert).

    experts: a function (or module) of (x_sorted [T*K, H], expert_offsets
    [E+1] i32) -> y_sorted [T*K, H] in x's type; expert e's rows are
    expert_offsets[e] .. expert_offsets[e+1].  shared: a function of x [T, H] ->
    [T, H], or None.  route_cfg: keyword arguments of moe_route_ex.  w_router
    is a parameter [E, H] of `dtype`; bf16 rows whose sizes moe_router takes
    are routed by it, others by a plain gate product in fp32 and moe_route_ex.
    """

    def __init__(self, hidden: int, n_experts: int, top_k: int, experts: Callable, shared: Optional[Callable] = None,
                 route_cfg: Optional[dict] = None, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.hidden, self.n_experts, self.top_k = hidden, n_experts, top_k
        self.experts, self.shared = experts, shared
        self.route_cfg = dict(route_cfg) if route_cfg else {}
        self.w_router = torch.nn.Parameter(torch.randn(n_experts, hidden, device=device).mul_(hidden ** -0.5).to(dtype))
        self.plan: Optional[RoutePlan] = None  # the last forward's

    def fused_router(self) -> bool:
        return self.w_router.dtype == torch.bfloat16 and self.hidden % 64 == 0 and \
            self.hidden <= 16384 and self.n_experts <= 512

    def forward(self, x: torch.Tensor, zero_mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        if self.fused_router() and x.dtype == torch.bfloat16:
            ids, w = router(x, self.w_router, self.top_k, zero_mask=zero_mask, **self.route_cfg)
        else:
            ids, w = route(_product(x, self.w_router.t()), self.top_k, zero_mask=zero_mask, **self.route_cfg)
        self.plan = plan = sort_plan(ids, self.n_experts)
        y = self.experts(permute(x, plan), plan.expert_offsets)
        return unpermute(y, w, plan, None if self.shared is None else self.shared(x))


def clip_grad_norm(parameters: Union[torch.Tensor, Iterable[torch.Tensor]], max_norm: float,
                   eps: float = 1e-6) -> torch.Tensor:
    """Clip the parameters' gradients (or one parameter's) in place by their
    global 2-norm; returns the norm before that, f32 [] on the device (no host
    synchronisation).  Parameters without a gradient are passed over; expert
    gradients that other ranks hold are ep.clip_grad_norm's."""
    if isinstance(parameters, torch.Tensor):  # not its rows, which have no gradients of their own
        parameters = [parameters]
    return moe_grad_clip([p.grad for p in parameters if p.grad is not None], max_norm, eps)
