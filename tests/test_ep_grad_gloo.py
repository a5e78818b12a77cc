"""ep.clip_grad_norm over a world-size-2 gloo group on CPU, the library's calls
replaced by plain 64-bit stand-ins: every rank clips by the norm over both
ranks' expert gradients and one copy of the replicated ones, also a rank that
holds no expert gradient."""
import math
import os
import socket
import sys

import torch
import torch.multiprocessing as mp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def _grads(rank):
    g = torch.Generator().manual_seed(rank)
    own = [torch.randn(n, generator=g) for n in ([30, 7] if rank == 0 else [])]
    g = torch.Generator().manual_seed(99)
    return own, [torch.randn(50, generator=g)]


class _List:
    def __init__(self, tensors, out=None, device=None):
        self.tensors, self.device = list(tensors), device or torch.device("cpu")


def _sumsq(t):
    ts = t.tensors if isinstance(t, _List) else t
    return sum((x.double().square().sum() for x in ts), torch.zeros((), dtype=torch.float64))


def _clip(t, max_norm, eps, sumsq):
    norm = sumsq.sqrt()
    for x in t.tensors:
        x.mul_(min(1.0, max_norm / (float(norm) + eps)))
    return norm.float()


def _rank_main(rank, world, port, q):
    import torch.distributed as dist
    from datetime import timedelta

    from mixture_experts_ffn_sort_b200 import ep
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=timedelta(seconds=60))
    try:
        ep.TensorList, ep.moe_grad_sumsq, ep.moe_grad_clip = _List, _sumsq, _clip
        own, shared = _grads(rank)
        before = [t.clone() for t in own + shared]
        every = _grads(0)[0] + _grads(1)[0] + shared
        want = math.sqrt(sum(float(t.double().square().sum()) for t in every))
        norm = ep.clip_grad_norm(own, shared, 0.5)
        assert abs(float(norm) - want) <= 1e-6 * want, (float(norm), want)
        for t, b in zip(own + shared, before):
            assert torch.allclose(t, b * (0.5 / want), rtol=1e-5, atol=0)
        q.put((rank, "ok"))
    except Exception:  # reported to the parent
        import traceback
        q.put((rank, traceback.format_exc()[-2000:]))
    finally:
        dist.destroy_process_group()


def test_norm_over_the_ranks():
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    procs = [ctx.Process(target=_rank_main, args=(r, 2, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    res = dict(q.get(timeout=120) for _ in procs)
    for p in procs:
        p.join(timeout=60)
    assert res == {0: "ok", 1: "ok"}, res
