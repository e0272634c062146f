"""Plain 64-bit forms of the sequence operators, written from their formulas,
and bounds on what their kernels may be off by.

Roundings as in tests/training_reference.py: U[dtype] is the unit roundoff, an
fp32 sum of n terms is off by at most n 2^-23 times the sum of their magnitudes.
"""
import math
from typing import NamedTuple, Optional

import torch

from tests.training_reference import E32, Bounded, U


# ---- embedding ---------------------------------------------------------------------

def embedding(tokens, weight, scale, padding):
    flat = tokens.reshape(-1)
    inside = (flat >= 0) & (flat < weight.shape[0])
    x = weight.double()[flat.clamp(0, weight.shape[0] - 1)] * scale
    x[~inside] = math.nan
    if padding is not None:
        x[flat == padding] = 0
    return x.reshape(*tokens.shape, -1)


def embedding_grad(grad, tokens, vocab, scale, padding, base=None):
    """A Bounded: products of fp32 with the scale, sums of a token's rows."""
    flat, g = tokens.reshape(-1), grad.double().reshape(-1, grad.shape[-1])
    keep = (flat >= 0) & (flat < vocab)
    if padding is not None:
        keep &= flat != padding
    out = torch.zeros(vocab, g.shape[1], dtype=torch.float64, device=g.device)
    size, count = out.clone(), torch.zeros(vocab, dtype=torch.float64, device=g.device)
    out.index_add_(0, flat[keep], g[keep] * scale)
    size.index_add_(0, flat[keep], (g[keep] * scale).abs())
    count.index_add_(0, flat[keep], torch.ones_like(flat[keep], dtype=torch.float64))
    off = (count[:, None] + 2) * E32 * size
    if base is not None:
        out, off = out + base.double(), off + E32 * (size + base.double().abs())
    return Bounded(out, off)


# ---- attention ----------------------------------------------------------------------

class Case(NamedTuple):
    """What a call is made of, flat: q [T, H, D], k and v [T, Hk, D]."""
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    scale: float
    causal: bool = True
    softcap: float = 0.0
    slopes: Optional[torch.Tensor] = None
    offsets: Optional[list] = None      # documents; else runs of `sequence`
    sequence: int = 0
    prefix: Optional[list] = None


def mask(c: Case):
    T = c.q.shape[0]
    m = torch.zeros(T, T, dtype=torch.bool)
    ends = c.offsets if c.offsets is not None else list(range(0, T + 1, c.sequence))
    for d, (a, b) in enumerate(zip(ends, ends[1:])):
        if b <= a:
            continue
        n = b - a
        block = torch.ones(n, n, dtype=torch.bool)
        if c.causal:
            block = block.tril()
            if c.prefix is not None:
                block[:, :min(max(c.prefix[d], 0), n)] = True
        m[a:b, a:b] = block
    return m.to(c.q.device)


def _scores(c: Case, seen):
    """Scores [H, T, T] with zeros where not seen, ds/d(q . k), their error."""
    H, Hk = c.q.shape[1], c.k.shape[1]
    # what is not in any document may hold anything
    alive = seen.any(1)
    clean = [torch.where(alive[:, None, None], t.double(), 0.0) for t in (c.q, c.k, c.v)]
    q, k, v = clean[0].transpose(0, 1), *(t.transpose(0, 1).repeat_interleave(H // Hk, 0)
                                          for t in clean[1:])
    D = q.shape[2]
    z = c.scale * (q @ k.transpose(1, 2))
    off = D * E32 * c.scale * (q.abs() @ k.abs().transpose(1, 2)) + 4 * E32 * z.abs()
    slope = torch.ones_like(z)
    if c.softcap:
        t = torch.tanh(z / c.softcap)
        z, slope = c.softcap * t, 1 - t * t
        # tanh of an argument off by that, itself off by 2^-20
        off = off + c.softcap * 2.0 ** -20 + 4 * E32 * z.abs()
    if c.slopes is not None:
        at = torch.arange(q.shape[1], device=q.device, dtype=torch.float64)
        bias = c.slopes.double()[:, None, None] * (at[:, None] - at).abs()
        z = z - bias
        off = off + 4 * E32 * (bias.abs() + z.abs())
    return q, k, v, torch.where(seen, z, 0.0), slope, torch.where(seen, off, 0.0)


def attention(c: Case):
    """(out, lse) as Bounded [T, H, D] and [T, H], and which rows see nothing."""
    seen = mask(c)
    q, k, v, z, _, off = _scores(c, seen)
    n = seen.sum(1).double()
    empty = n == 0
    z = torch.where(seen, z, -math.inf)
    lse = torch.logsumexp(z, 2)
    a = torch.where(seen, (z - torch.where(empty, 0.0, lse)[..., None]).exp(), 0.0)
    out = a @ v
    u = U.get(c.q.dtype, 2.0 ** -53)
    # a weight: its score, its exponent's rounding and the exponential's, its own
    # rounding for the product; the sum of weights: the same but for the last
    rel = off + 2 * E32 * (8 + torch.where(seen, (z - z.amax(2, keepdim=True).clamp(min=-1e30)).abs(), 0.0))
    total = (a * rel).sum(2, keepdim=True) + (n[:, None] + 16) * E32
    small = 2.0 ** -32 if c.q.dtype == torch.float16 else 0.0    # below the smallest fp16
    out_off = (a * (rel + u)) @ v.abs() + total * (a @ v.abs()) \
        + (n[:, None] + 64) * E32 * (a @ v.abs()) + small * (seen.double() @ v.abs())
    lse_off = off.amax(2) + total[..., 0] + 8 * E32 * (1 + lse.abs())
    rows = lambda t: t.transpose(0, 1)      # noqa: E731
    lse = torch.where(empty, 0.0, lse)
    lse_off = torch.where(empty, 0.0, lse_off)
    return Bounded(rows(out), rows(out_off)), Bounded(rows(lse), rows(lse_off)), empty


def attention_grad(c: Case, grad_out, out, lse):
    """{name: Bounded} of the gradients; out and lse are inputs."""
    seen = mask(c)
    alive = seen.any(1)
    q, k, v, z, slope, off = _scores(c, seen)
    H, Hk, D = c.q.shape[1], c.k.shape[1], c.q.shape[2]
    go, o = (torch.where(alive[:, None, None], t.double(), 0.0).transpose(0, 1) for t in (grad_out, out))
    ls = torch.where(alive[:, None], lse.double(), 0.0).t()[..., None]
    p = torch.where(seen, (z - ls).exp(), 0.0)
    u, half = U.get(c.q.dtype, 2.0 ** -53), c.q.dtype == torch.float16
    # a weight: its score, the rounding of its exponent, the exponential
    rel = off + 2 * E32 * (8 + z.abs() + ls.abs())
    dp = go @ v.transpose(1, 2)
    delta = (go * o).sum(2, keepdim=True)
    dp_off = D * E32 * (go.abs() @ v.abs().transpose(1, 2) + (go * o).abs().sum(2, keepdim=True))
    ds = p * (dp - delta) * slope
    ds_off = p * slope * dp_off + p * (dp - delta).abs() * (slope * (rel + 8 * E32) + 2.0 ** -19 * (slope < 1))
    ds_off = ds_off + u * (ds.abs() + ds_off)
    if half:
        ds_off = ds_off + seen * (2.0 ** -24 * grad_out.double()[alive].abs().max() if alive.any() else 0.0)
    p_off = p * (rel + u) + (seen * 2.0 ** -34 if half else 0.0)
    n = seen.sum(1).double()[:, None]          # keys of a query
    m = seen.sum(0).double()[:, None] * (H // Hk)
    dq = Bounded(c.scale * (ds @ k), c.scale * (ds_off @ k.abs() + (n + 64) * E32 * (ds.abs() @ k.abs())))
    dk = (c.scale * (ds.transpose(1, 2) @ q),
          c.scale * (ds_off.transpose(1, 2) @ q.abs() + (m + 64) * E32 * (ds.abs().transpose(1, 2) @ q.abs())))
    dv = (p.transpose(1, 2) @ go,
          p_off.transpose(1, 2) @ go.abs() + (m + 64) * E32 * (p.transpose(1, 2) @ go.abs()))

    def shared(t):      # over the query heads that share one
        return t.view(Hk, H // Hk, *t.shape[1:]).sum(1).transpose(0, 1)

    rows = lambda t: t.transpose(0, 1)      # noqa: E731
    tail = 8 * E32
    return {"q": Bounded(rows(dq.value), rows(dq.off + tail * dq.value.abs())),
            "k": Bounded(shared(dk[0]), shared(dk[1] + tail * dk[0].abs())),
            "v": Bounded(shared(dv[0]), shared(dv[1] + tail * dv[0].abs()))}
