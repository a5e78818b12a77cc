"""ep.clip_grad_norm over a world-size-2 gloo group on CPU: every rank clips by
the same bits, also where the ranks' sums of the replicated gradients differ in
their last ones (as they do when the tensors start at different places).  The
library's calls are replaced by stand-ins, whose sum adds a rank's own rounding."""
import os
import socket
import sys

import torch
import torch.multiprocessing as mp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


class _List:
    def __init__(self, tensors, out=None, device=None):
        self.tensors, self.device = list(tensors), device or torch.device("cpu")


def _rank_main(rank, world, port, q):
    import torch.distributed as dist
    from datetime import timedelta

    from mixture_experts_ffn_sort_b200 import ep
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=timedelta(seconds=60))
    try:
        def sumsq(t):
            ts = t.tensors if isinstance(t, _List) else t
            exact = sum((x.double().square().sum() for x in ts), torch.zeros((), dtype=torch.float64))
            return exact * (1 + rank * 2.0 ** -26)

        used = []

        def clip(t, max_norm, eps, sumsq):
            used.append(sumsq.item())
            return sumsq.sqrt().float()

        ep.TensorList, ep.moe_grad_sumsq, ep.moe_grad_clip = _List, sumsq, clip
        g = torch.Generator().manual_seed(99)
        shared = [torch.randn(1000, generator=g)]
        own = [torch.randn(30, generator=torch.Generator().manual_seed(rank))] if rank else []
        ep.clip_grad_norm(own, shared, 0.5)
        ep.clip_grad_norm([], shared, 0.5)
        ep.clip_grad_norm(own, [], 0.5)
        q.put((rank, used))
    except Exception:  # reported to the parent
        import traceback
        q.put((rank, traceback.format_exc()[-2000:]))
    finally:
        dist.destroy_process_group()


def test_every_rank_uses_the_same_bits():
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
    assert res[0] == res[1] and len(res[0]) == 3, res
    # The replicated gradients count once.
    shared = float(torch.randn(1000, generator=torch.Generator().manual_seed(99)).double().square().sum())
    assert abs(res[0][1] - shared) <= 1e-6 * shared
