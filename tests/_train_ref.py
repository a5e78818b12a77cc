"""Plain 64-bit forms of the training operators, and inputs for their tests."""
import torch

# Half a step of each type, relative to the value, and half of its smallest subnormal.
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
U32 = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def routes(T, K, E, drop, seed):
    """Ids [T, K] i32 (distinct where K <= E; -1 for dropped routes) and moe_sort's maps, on the CPU."""
    g = gen(seed)
    if K <= E:
        ids = torch.rand((T, E), generator=g).argsort(1)[:, :K]
    else:
        ids = torch.randint(0, E, (T, K), generator=g)
    ids = torch.where(torch.rand((T, K), generator=g) < drop, -1, ids).to(torch.int32)
    flat = torch.where(ids < 0, E, ids).view(-1).long()
    order = torch.sort(flat, stable=True).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * K)
    inv = torch.where(flat == E, -1, inv).to(torch.int32)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return ids, off, inv


def permute(x, inv, K):
    out = torch.zeros((x.shape[0] * K, x.shape[1]), dtype=x.dtype)
    r = (inv >= 0).nonzero()[:, 0]
    out[inv[r].long()] = x[r // K]
    return out


def weighted(y, inv, w, T):
    """w[t, j] * y[inv[t, j]] in fp64, [T, K, H]; 0 for dropped routes and weights of 0."""
    rows = y.double()[inv.clamp(min=0).long()]
    ww = torch.ones(inv.numel(), dtype=torch.float64) if w is None else w.double().view(-1)
    on = (inv >= 0) & (ww != 0)
    return torch.where(on[:, None], rows * ww[:, None], 0.0).view(T, -1, y.shape[1])


def route_weights(logits, ids, score, renormalize, scaling, zero_mask=None):
    """The route weights of a given choice, fp64 and differentiable."""
    s = torch.sigmoid(logits) if score else torch.softmax(logits, dim=1)
    w = s.gather(1, ids.long())
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    w = w * scaling
    return w if zero_mask is None else w.masked_fill(zero_mask.bool(), 0.0)
