"""The operators that train a routed layer, as cases: rows sorted by expert and
back with their gradients, the router's gradient, and the global gradient norm
with clipping.  listed() says for each case what it stands for; draw() gives
more of the same ranges.

A case's "op" is one call:
  permute         x [T, H] -> rows sorted by expert [T*K, H]
  permute_bwd     its gradient: [T*K, H] -> [T, H]
  unpermute       sorted rows and route weights (and the shared expert's rows) -> [T, H]
  unpermute_bwd   its gradients: of the sorted rows and of the route weights
  route_bwd       the gradient of the route weights -> the gradient of the logits
  clip            a list of gradients -> its 2-norm and the clipped gradients
Routes have ids in [0, E), or -1 for a share `drop` of them: those have no
sorted row (position -1), and the rows behind the last sorted one are zeros.
"""
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def _rows(name, op, T, H, K, E, dtype, drop=0.0, zero=0.0, shared=False):
    return {"name": name, "op": op, "T": T, "H": H, "K": K, "E": E, "dtype": dtype, "drop": drop, "zero": zero,
            "shared": shared}


def _route(name, T, E, K, score, renorm, scaling, zero):
    return {"name": name, "op": "route_bwd", "T": T, "E": E, "K": K, "score": score, "renorm": renorm,
            "scaling": scaling, "zero": zero}


def _clip(name, count, least, most, dtype, norm):
    return {"name": name, "op": "clip", "count": count, "least": least, "most": most, "dtype": dtype, "norm": norm}


def listed():
    return [
        # One token of the decode configuration: the latency of a call.
        _rows("permute one token", "permute", 1, 2048, 8, 256, "bf16"),
        # A training or prefill batch of 8192 tokens of width 4096, 512 experts, top-10.
        _rows("permute prefill", "permute", 8192, 4096, 10, 512, "bf16"),
        # Odd sizes (rows that no 16-byte load fits), routes dropped by a capacity limit.
        _rows("permute_bwd odd, dropped", "permute_bwd", 777, 1030, 6, 128, "f16", drop=0.1),
        # The large prefill: 32768 tokens of width 8192; the rows pass 2^31 elements.
        _rows("permute_bwd large", "permute_bwd", 32768, 8192, 10, 512, "bf16"),
        # The decode batch.
        _rows("unpermute decode", "unpermute", 64, 2048, 8, 256, "bf16"),
        # The prefill batch in half precision with a shared expert and 1 % zero-weight routes.
        _rows("unpermute prefill", "unpermute", 8192, 4096, 10, 512, "f16", zero=0.01, shared=True),
        # A small fine-tuning batch in fp32.
        _rows("unpermute_bwd small", "unpermute_bwd", 512, 2048, 8, 256, "f32"),
        # The prefill batch.
        _rows("unpermute_bwd prefill", "unpermute_bwd", 8192, 4096, 10, 512, "bf16", zero=0.01),
        # The decode batch through the softmax router.
        _route("route_bwd decode", 64, 256, 8, "softmax", True, 1.0, 0.0),
        # 32768 tokens through the sigmoid router with a routed scaling factor.
        _route("route_bwd large", 32768, 512, 10, "sigmoid", True, 2.5, 0.01),
        # A router and a few small tensors beside it, fp32.
        _clip("clip few", 9, 1000, 524288, "f32", 1.0),
        # Gate, up and down of 256 experts of 512 x 2048, and the router: 805 million values.
        _clip("clip experts", 769, 1048576, 1048576, "bf16", 1.0),
    ]


def _spread(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["permute", "permute_bwd", "unpermute", "unpermute_bwd", "route_bwd", "clip"])
    if op == "route_bwd":
        E = _spread(rng, 8, 1024)
        return _unnamed(_route("", _spread(rng, 1, 32768), E, min(E, rng.randint(1, 16)),
                               rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, rng.choice([1.0, 2.5]),
                               rng.choice([0.0, 0.01])))
    if op == "clip":
        count = _spread(rng, 1, 1537)
        least = _spread(rng, 1, 65536)
        most = min(_spread(rng, least, 1 << 24), max(least, (1 << 28) // count))
        return _unnamed(_clip("", count, least, most, rng.choice(list(TYPES)), rng.choice([1.0, 1e6])))
    K = rng.randint(1, 16)
    H = _spread(rng, 8, 8192)
    if rng.random() < 0.5:
        H = max(8, H // 64 * 64)
    T = max(1, min(_spread(rng, 1, 32768), 300_000_000 // (K * H)))
    return _unnamed(_rows("", op, T, H, K, _spread(rng, max(8, K), 1024), rng.choice(list(TYPES)),
                          rng.choice([0.0, 0.0, 0.1, 0.9]), rng.choice([0.0, 0.01]),
                          op == "unpermute" and rng.random() < 0.5))


def _unnamed(case):
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _random(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    # Drawn in pieces in fp32, so that large tensors need no second copy of their size.
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return out


def _choices(g, T, E, K):
    """Router logits with unequal experts, and each token's K distinct best."""
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    return logits, logits.topk(K, dim=1).indices


def _mask(g, shape, share):
    return torch.rand(shape, generator=g, device="cuda") < share


def prepare(case, seed):
    g = _random(seed)
    s = {"case": case}
    if case["op"] == "clip":
        return _prepare_clip(case, g, s)
    T, K, E = case["T"], case["K"], case["E"]
    logits, ids = _choices(g, T, E, K)
    zero = _mask(g, (T, K), case["zero"])
    if case["op"] == "route_bwd":
        s["logits"], s["ids"] = logits, ids.to(torch.int32)
        s["zero_mask"] = zero.to(torch.uint8) if case["zero"] else None
        s["dw"] = torch.randn((T, K), generator=g, device="cuda")
        return s
    # The maps that a sort of the routes by expert leaves: stable, dropped routes last.
    ids = torch.where(_mask(g, (T, K), case["drop"]), E, ids).view(-1)
    order = torch.sort(ids, stable=True).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * K, device="cuda")
    s["inv"] = torch.where(ids == E, -1, inv).to(torch.int32)
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    w = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), dim=1)
    s["w"] = torch.where(zero, 0.0, w)
    dtype, H = TYPES[case["dtype"]], case["H"]
    if case["op"] in ("permute", "unpermute_bwd"):
        s["tokens"] = _normal(g, (T, H), dtype)
    if case["op"] != "permute":
        s["sorted"] = _normal(g, (T * K, H), dtype)
    s["shared"] = _normal(g, (T, H), dtype) if case["shared"] else None
    return s


def _prepare_clip(case, g, s):
    # Tensor sizes over the logarithm of their range (by multiples of the golden ratio, in no
    # order); each tensor starts where the last one ended, at any element, as views of a flat
    # gradient buffer do.
    u = torch.arange(1, case["count"] + 1, dtype=torch.float64) * 0.6180339887498949 % 1
    sizes = (case["least"] * (case["most"] / case["least"]) ** u).round().long().tolist()
    s["sizes"] = sizes
    flat = _normal(g, (sum(sizes),), TYPES[case["dtype"]])
    flat *= 0.01
    s["grads"] = list(flat.split(sizes))
    s["clipped"] = torch.empty_like(flat)
    if own:
        import mixture_experts_ffn_sort_b200 as moe
        # The list of gradients that a training loop keeps, with the place of the clipped ones.
        s["list"] = moe.TensorList(s["grads"], out=list(s["clipped"].split(sizes)))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import mixture_experts_ffn_sort_b200 as moe
    c = s["case"]
    op = c["op"]
    if op == "permute":
        return moe.moe_permute(s["tokens"], s["inv"], s["offsets"])
    if op == "permute_bwd":
        return moe.moe_permute_bwd(s["sorted"], s["inv"], c["T"])
    if op == "unpermute":
        return moe.moe_unpermute(s["sorted"], s["inv"], s["w"], s["shared"])
    if op == "unpermute_bwd":
        return moe.moe_unpermute_bwd(s["tokens"], s["sorted"], s["inv"], s["w"], s["offsets"])
    if op == "route_bwd":
        score = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        return moe.moe_route_bwd(s["logits"], s["ids"], s["dw"], score=score, renormalize=c["renorm"],
                                 scaling=c["scaling"], zero_mask=s["zero_mask"])
    return {"norm": moe.moe_grad_clip(s["list"], c["norm"]), "grads": s["clipped"]}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route_bwd":
        return _route_bwd_plain(s)
    if c["op"] == "clip":
        return _clip_plain(s)
    T, K, H = c["T"], c["K"], c["H"]
    dtype = TYPES[c["dtype"]]
    inv = s["inv"].long()
    valid = inv >= 0
    if c["op"] == "permute":
        out = torch.zeros((T * K + 1, H), dtype=dtype, device="cuda")
        at = torch.where(valid, inv, T * K)  # dropped routes go to a row that is cut off
        out[at] = s["tokens"].repeat_interleave(K, dim=0)
        out[T * K] = 0
        return out[:T * K]
    here = inv.clamp(min=0)
    if c["op"] == "permute_bwd":
        rows = s["sorted"][here].float() * valid[:, None]
        return rows.view(T, K, H).sum(1).to(dtype)
    w = s["w"].view(-1) * valid
    if c["op"] == "unpermute":
        out = (s["sorted"][here].float() * w[:, None]).view(T, K, H).sum(1)
        if s["shared"] is not None:
            out += s["shared"].float()
        return out.to(dtype)
    dout = s["tokens"].float().repeat_interleave(K, dim=0)
    dw = ((s["sorted"][here].float() * dout).sum(1) * valid).view(T, K)
    dy = torch.zeros((T * K + 1, H), dtype=dtype, device="cuda")
    dy[torch.where(valid, inv, T * K)] = (w[:, None] * dout).to(dtype)
    return dy[:T * K], dw


def _route_bwd_plain(s):
    c = s["case"]
    ids, dw = s["ids"].long(), s["dw"]
    if s["zero_mask"] is not None:
        dw = torch.where(s["zero_mask"] != 0, 0.0, dw)
    if c["score"] == "softmax":
        e = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-s["logits"]))
    mine = p.gather(1, ids)
    total = mine.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(mine[:, :1])
    # d w_j / d s_j, and the part of the common divisor.
    ds = c["scaling"] * dw / total
    if c["renorm"]:
        ds = ds - c["scaling"] * (dw * mine).sum(1, keepdim=True) / (total * total)
    dp = torch.zeros_like(p).scatter_add_(1, ids, ds)
    if c["score"] == "sigmoid":
        return dp * p * (1 - p)
    return p * (dp - (dp * p).sum(1, keepdim=True))


def _clip_plain(s):
    c = s["case"]
    every = torch.cat(s["grads"]).float()
    norm = every.square().sum(dtype=torch.float64).sqrt()
    factor = torch.clamp(c["norm"] / (norm + 1e-6), max=1.0).float()
    return {"norm": norm.float(), "grads": (every * factor).to(TYPES[c["dtype"]])}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "clip":
        mean = case["least"]
        if case["most"] > case["least"]:
            from math import log
            mean = (case["most"] - case["least"]) / log(case["most"] / case["least"])
        n = case["count"] * mean
        return {"bytes": 2 * n * SIZES[case["dtype"]] + 4, "flops": 3 * n}
    T, K = case["T"], case["K"]
    R = T * K
    if op == "route_bwd":
        read = T * case["E"] if case["score"] == "softmax" and not case["renorm"] else R
        return {"bytes": 4 * (2 * R + read + T * case["E"]) + (R if case["zero"] else 0), "flops": 10 * R}
    b, H = SIZES[case["dtype"]], case["H"]
    kept = R * (1 - case["drop"])
    if op == "permute":
        return {"bytes": b * H * (T + R) + 4 * R, "flops": 0}
    if op == "permute_bwd":
        return {"bytes": b * H * (T + kept) + 4 * R, "flops": kept * H}
    if op == "unpermute":
        return {"bytes": b * H * (T + kept + (T if case["shared"] else 0)) + 8 * R, "flops": 2 * kept * H}
    return {"bytes": b * H * (T + kept + R) + 12 * R, "flops": 3 * kept * H}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in s["grads"]:
            total += torch.dot(g.double(), g.double())
        norm = torch.sqrt(total)
        scale = case["norm"] / (norm + 1e-6)
        scale = scale if scale < 1 else torch.ones_like(scale)
        return {"norm": norm, "grads": torch.cat([g.double() * scale for g in s["grads"]])}
    if op == "route_bwd":
        # Through the forward pass, differentiated in 64 bits.
        logits = s["logits"].double().requires_grad_()
        score = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, dim=1)
        w = torch.take_along_dim(score, s["ids"].long(), 1)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = w * case["scaling"]
        if s["zero_mask"] is not None:
            w = w.masked_fill(s["zero_mask"].bool(), 0.0)
        return torch.autograd.grad(w, logits, s["dw"].double())[0]
    T, K, H = case["T"], case["K"], case["H"]
    inv = s["inv"].view(T, K).long()
    if op == "permute" or op == "unpermute_bwd":
        out = torch.zeros((T * K, H), dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        for j in range(K):
            t = (inv[:, j] >= 0).nonzero()[:, 0]
            p = inv[t, j]
            if op == "permute":
                out[p] = s["tokens"][t].double()
            else:
                out[p] = s["tokens"][t].double() * s["w"][t, j, None].double()
                dw[t, j] = torch.einsum("th,th->t", s["tokens"][t].double(), s["sorted"][p].double())
        return out if op == "permute" else (out, dw)
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for j in range(K):
        t = (inv[:, j] >= 0).nonzero()[:, 0]
        row = s["sorted"][inv[t, j]].double()
        out[t] += row if op == "permute_bwd" else row * s["w"][t, j, None].double()
    return out if s["shared"] is None else out + s["shared"].double()
