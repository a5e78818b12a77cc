"""Host-side contract checks of the training calls (CPU only: every call here
returns from validation, none reaches a kernel)."""
import ctypes

import pytest
import torch

import mixture_experts_ffn_sort_b200 as moe

P = ctypes.c_void_p
A, B, C, D = P(0x100000), P(0x200000), P(0x300000), P(0x400000)


@pytest.fixture(scope="module")
def L():
    from mixture_experts_ffn_sort_b200 import build
    build.build()
    return moe.lib()


def err(L):
    return L.moe_last_error().decode()


def permute(L, x=A, inv=B, n=None, T=4, K=2, H=16, dt=0, out=C, status=None):
    return L.moe_permute(x, inv, n, T, K, H, dt, out, status, None)


def unpermute(L, y=A, inv=B, w=None, sh=None, T=4, K=2, H=16, dt=0, out=C, status=None):
    return L.moe_unpermute(y, inv, w, sh, T, K, H, dt, out, status, None)


def unpermute_bwd(L, dout=A, y=B, inv=C, w=None, n=None, T=4, K=2, H=16, dt=0, dy=D, dw=P(0x500000), status=None):
    return L.moe_unpermute_bwd(dout, y, inv, w, n, T, K, H, dt, dy, dw, status, None)


@pytest.mark.parametrize("call", [permute, unpermute, unpermute_bwd])
def test_rows_sizes_and_types(L, call):
    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(K=0), dict(K=33), dict(dt=3), dict(dt=-1)):
        assert call(L, **kw) == moe.MOE_ERR_INVALID_ARG and err(L)
    for H in (0, -8, 65537):
        assert call(L, H=H) == moe.MOE_ERR_UNSUPPORTED_SHAPE and "H=%d" % H in err(L)
    assert call(L, T=0) == moe.MOE_OK and err(L) == ""
    assert call(L, inv=None) == moe.MOE_ERR_INVALID_ARG
    assert call(L, inv=P(0x200004)) == moe.MOE_ERR_MISALIGNED
    assert call(L, status=P(0x200002)) == moe.MOE_ERR_MISALIGNED


def test_permute_refusals(L):
    assert permute(L, x=None) == moe.MOE_ERR_INVALID_ARG
    assert permute(L, out=None) == moe.MOE_ERR_INVALID_ARG
    assert permute(L, x=P(0x100002)) == moe.MOE_ERR_MISALIGNED
    assert permute(L, n=P(0x100002)) == moe.MOE_ERR_MISALIGNED
    # 4 rows of 32 bytes in, 8 out: an output that starts within the input, or the other way round.
    assert permute(L, out=A) == moe.MOE_ERR_INVALID_ARG and "overlaps" in err(L)
    assert permute(L, out=P(0x100000 + 112)) == moe.MOE_ERR_INVALID_ARG
    assert permute(L, x=P(0x300000 + 240)) == moe.MOE_ERR_INVALID_ARG
    assert permute(L, out=B) == moe.MOE_ERR_INVALID_ARG


def test_unpermute_refusals(L):
    assert unpermute(L, y=None) == moe.MOE_ERR_INVALID_ARG
    assert unpermute(L, out=None) == moe.MOE_ERR_INVALID_ARG
    for kw in (dict(y=P(0x100008)), dict(w=P(0x600004)), dict(sh=P(0x600008)), dict(out=P(0x300008))):
        assert unpermute(L, **kw) == moe.MOE_ERR_MISALIGNED
    for kw in (dict(out=A), dict(out=P(0x100000 + 240)), dict(sh=C), dict(w=C), dict(out=B)):
        assert unpermute(L, **kw) == moe.MOE_ERR_INVALID_ARG and "overlaps" in err(L)


def test_unpermute_bwd_refusals(L):
    assert unpermute_bwd(L, dout=None) == moe.MOE_ERR_INVALID_ARG
    assert unpermute_bwd(L, dy=None, dw=None) == moe.MOE_ERR_INVALID_ARG
    assert unpermute_bwd(L, y=None) == moe.MOE_ERR_INVALID_ARG and "y_sorted" in err(L)
    for kw in (dict(dout=P(0x100008)), dict(y=P(0x200008)), dict(w=P(0x600004)), dict(dy=P(0x400008)),
               dict(dw=P(0x500004)), dict(n=P(0x500002))):
        assert unpermute_bwd(L, **kw) == moe.MOE_ERR_MISALIGNED
    for kw in (dict(dy=A), dict(dy=B), dict(dy=C), dict(dw=A), dict(dw=B), dict(w=P(0x500000)), dict(dw=D)):
        assert unpermute_bwd(L, **kw) == moe.MOE_ERR_INVALID_ARG and "overlap" in err(L)


def test_route_bwd_refusals(L):
    def call(lg=A, ids=B, dw=C, T=4, E=16, K=4, cfg=None, zm=None, out=D, status=None):
        return L.moe_route_bwd(lg, ids, dw, T, E, K, cfg, zm, out, status, None)

    def cfg(score=0, n_group=1, topk_group=1, renorm=1, scaling=1.0, bias=None):
        return ctypes.byref(moe._RouteConfig(score, bias, n_group, topk_group, renorm, scaling))

    for kw in (dict(T=-1), dict(K=17), dict(K=0), dict(lg=None), dict(ids=None), dict(dw=None), dict(out=None),
               dict(cfg=cfg(score=2)), dict(cfg=cfg(renorm=2)), dict(cfg=cfg(scaling=0.0)), dict(cfg=cfg(n_group=3)),
               dict(out=A), dict(out=B), dict(out=C), dict(zm=D)):
        assert call(**kw) == moe.MOE_ERR_INVALID_ARG and err(L), kw
    assert call(E=1025) == moe.MOE_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(lg=P(0x100004)), dict(ids=P(0x200004)), dict(dw=P(0x300008)), dict(out=P(0x400008)),
               dict(status=P(0x500001))):
        assert call(**kw) == moe.MOE_ERR_MISALIGNED
    assert call(T=0, lg=None, ids=None, dw=None, out=None) == moe.MOE_OK


def refs(*rows):
    r = (moe._TensorRef * max(len(rows), 1))()
    for i, (data, out, numel, dtype) in enumerate(rows):
        r[i] = moe._TensorRef(data, out, numel, dtype, 0)
    return r, len(rows)


def test_grad_workspace(L):
    assert L.moe_grad_workspace_bytes(0) == 0 and L.moe_grad_workspace_bytes(-3) == 0
    one = L.moe_grad_workspace_bytes(1)
    assert one > 0 and one % 8 == 0
    assert L.moe_grad_workspace_bytes(100000) > one


def test_grad_list_refusals(L):
    ws = P(0x800000)
    need = L.moe_grad_workspace_bytes(4)

    def sumsq(r, n, out=P(0x700000), norm=None, ws=ws, need=need):
        return L.moe_grad_sumsq(r, n, out, norm, ws, need, None)

    def clip(r, n, s=None, max_norm=1.0, eps=1e-6, norm=None, ws=ws, need=need):
        return L.moe_grad_clip(r, n, s, max_norm, eps, norm, ws, need, None)

    good = (0x100000, 0x100000, 10, 1)
    for bad, code in (((0x100000, 0x100000, 10, 3), moe.MOE_ERR_INVALID_ARG),
                      ((0x100000, 0x100000, -1, 1), moe.MOE_ERR_INVALID_ARG),
                      ((None, 0x100000, 10, 1), moe.MOE_ERR_INVALID_ARG),
                      ((0x100002, 0x100000, 10, 1), moe.MOE_ERR_MISALIGNED),
                      ((0x100001, 0x100000, 10, 0), moe.MOE_ERR_MISALIGNED),
                      ((0x100000, 0x100000, 1 << 44, 1), moe.MOE_ERR_UNSUPPORTED_SHAPE)):
        r, n = refs((0x200000, 0x200000, 4, 0), bad)
        for call in (sumsq, clip):
            assert call(r, n) == code, bad
        assert L.moe_grad_refs_check(r, n) == code
    r, n = refs((0x100000, None, 10, 1))
    assert clip(r, n) == moe.MOE_ERR_INVALID_ARG
    r, n = refs((0x100000, 0x100002, 10, 1))
    assert clip(r, n) == moe.MOE_ERR_MISALIGNED
    r, n = refs(good)
    assert sumsq(r, -1) == moe.MOE_ERR_INVALID_ARG and clip(None, 1) == moe.MOE_ERR_INVALID_ARG
    assert sumsq(r, n, out=None) == moe.MOE_ERR_INVALID_ARG
    assert sumsq(r, n, out=P(0x700004)) == moe.MOE_ERR_MISALIGNED
    assert clip(r, n, s=P(0x700004)) == moe.MOE_ERR_MISALIGNED
    assert sumsq(r, n, ws=None) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert clip(r, n, need=need - 1) == moe.MOE_ERR_WORKSPACE_TOO_SMALL and "need" in err(L)
    assert sumsq(r, n, ws=P(0x800008)) == moe.MOE_ERR_MISALIGNED
    for kw in (dict(max_norm=float("nan")), dict(max_norm=-1.0), dict(eps=float("inf")), dict(eps=-1.0)):
        assert clip(r, n, **kw) == moe.MOE_ERR_INVALID_ARG
    r[0].reserved = 1
    assert sumsq(r, n) == moe.MOE_ERR_INVALID_ARG


def test_grad_list_overlaps(L):
    def check(*rows):
        return L.moe_grad_refs_check(*refs(*rows))

    a = 0x100000
    assert check() == moe.MOE_OK and check((0, 0, 0, 1)) == moe.MOE_OK
    assert check((a + 40, a + 40, 10, 1), (a, a, 10, 1)) == moe.MOE_OK           # side by side, in any order
    assert check((a, a, 10, 1), (a, a, 10, 1)) == moe.MOE_ERR_INVALID_ARG        # the same tensor twice
    assert check((a, a, 11, 1), (a + 40, a + 40, 10, 1)) == moe.MOE_ERR_INVALID_ARG
    assert check((a, a, 100, 1), (a + 8, a + 8, 1, 0)) == moe.MOE_ERR_INVALID_ARG and "overlaps" in err(L)
    b = 0x200000
    assert check((a, b, 10, 1), (a + 40, b + 40, 10, 1)) == moe.MOE_OK
    assert check((a, b, 10, 1), (b + 36, b + 36, 10, 1)) == moe.MOE_ERR_INVALID_ARG   # an output over a tensor
    assert check((a, b, 10, 1), (a + 40, b, 10, 1)) == moe.MOE_ERR_INVALID_ARG        # two outputs
    assert check((a, a + 20, 10, 1)) == moe.MOE_ERR_INVALID_ARG                       # an output over its own tensor
    assert check((a, None, 10, 1), (b, None, 10, 1)) == moe.MOE_OK
    many = [(a + 8 * i, a + 8 * i, 2, 1) for i in range(3000)]
    assert check(*many[::-1]) == moe.MOE_OK
    assert check(*many[::-1], (a + 8 * 1500 + 4, a + 8 * 1500 + 4, 1, 1)) == moe.MOE_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    x, inv = torch.zeros((4, 8)), torch.zeros(8, dtype=torch.int32)
    w, lg = torch.zeros((4, 2)), torch.zeros((4, 8))
    for call in (lambda: moe.moe_permute(x, inv), lambda: moe.moe_permute_bwd(torch.zeros((8, 8)), inv, 4),
                 lambda: moe.moe_unpermute(torch.zeros((8, 8)), inv, w),
                 lambda: moe.moe_unpermute_bwd(x, torch.zeros((8, 8)), inv, w),
                 lambda: moe.moe_route_bwd(lg, inv.view(4, 2), w)):
        with pytest.raises(ValueError):
            call()
