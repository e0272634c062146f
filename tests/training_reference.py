"""Plain 64-bit forms of the training operators, written from their formulas,
and bounds on what a 32-bit evaluation with 16-bit operands may be off by.

Roundings: U[dtype] is the unit roundoff.  An fp32 sum of n terms, in any
order, is off by at most n 2^-23 times the sum of their magnitudes (twice the
unit roundoff, which also covers the tensor cores' truncation of addends).
"""
from typing import NamedTuple

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
E32 = 2.0 ** -23


class Bounded(NamedTuple):
    value: torch.Tensor
    off: torch.Tensor     # how far an evaluation may be, before its own rounding

    def holds(self, got, what=""):
        """Asserts that `got` is the value within the bound and its rounding."""
        u = U[got.dtype]
        limit = self.off * (1 + u) + self.value.abs() * u + TINY[got.dtype]
        far = (got.double() - self.value).abs()
        bad = ~(far <= limit)
        assert not bad.any(), (what, int(bad.sum()), float((far / limit.clamp(min=1e-300)).max()))


# ---- loss ------------------------------------------------------------------------

class Xent(NamedTuple):
    loss: torch.Tensor
    row_loss: torch.Tensor
    lse: torch.Tensor
    grad_x: torch.Tensor
    grad_w: torch.Tensor
    dz: torch.Tensor


def xent(x, w, y, *, mean, ignore=-100, scale=1.0):
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    keep = y != ignore
    at = torch.where(keep, y, 0)[:, None]
    row = torch.where(keep, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    share = 1.0 / max(1, int(keep.sum())) if mean else 1.0
    dz = (z - lse[:, None]).exp()
    dz = dz.scatter_add(1, at, -torch.ones_like(lse)[:, None])
    dz = torch.where(keep[:, None], dz, torch.zeros_like(dz)) * (share * scale)
    x = torch.where(keep[:, None], x, torch.zeros_like(x))
    return Xent(row.sum() * share, row, lse, dz @ w, dz.t() @ x, dz)


def xent_bounds(x, w, y, dtype, *, mean, ignore=-100, scale=1.0):
    """What the kernel's outputs are held to: dict of Bounded."""
    r = xent(x, w, y, mean=mean, ignore=ignore, scale=scale)
    D, V = x.shape[1], w.shape[0]
    keep = y != ignore
    share = 1.0 / max(1, int(keep.sum())) if mean else 1.0
    # a logit's fp32 sum; the difference to the largest one, times log2 e, and
    # exp2 of it: 2^-21 relative for each unit of the exponent's size
    z_off = D * E32 * (x.abs() @ w.abs().t())
    top_off = z_off.max(1).values
    # the sum of exponentials: 128 in a piece, the pieces, each off by its logits
    lse_off = top_off + (V / 64 + 192) * E32 + 8 * E32 * (1 + r.lse.abs())
    row_off = torch.where(keep, 2 * lse_off + 4 * E32 * (1 + r.row_loss.abs()), 0.0)
    # dz: a probability off by its logit and lse, kept in fp16 (2^-11, 2^-25 of
    # the piece's largest), rounded to the operand's type
    p = (x @ w.t() - r.lse[:, None]).exp() * (share * scale)
    p = torch.where(keep[:, None], p, torch.zeros_like(p))
    p_off = p * (z_off + lse_off[:, None] + 32 * E32 + 2.0 ** -11)
    p_off += torch.where(keep[:, None], share * scale * 2.0 ** -25, 0.0)
    p_off += U[dtype] * r.dz.abs()
    if dtype == torch.float16:
        p_off += share * scale * 2.0 ** -40      # fp16 dz, held times 2^15
    xk = torch.where(keep[:, None], x, torch.zeros_like(x))
    gx_off = p_off @ w.abs() + V * E32 * (r.dz.abs() @ w.abs())
    gw_off = p_off.t() @ xk.abs() + x.shape[0] * E32 * (r.dz.abs().t() @ xk.abs())
    return {"loss": Bounded(r.loss, row_off.sum() * share + 4 * E32 * r.loss.abs()),
            "row_loss": Bounded(r.row_loss, row_off), "lse": Bounded(r.lse, lse_off),
            "grad_x": Bounded(r.grad_x, gx_off + 8 * E32 * r.grad_x.abs()),
            "grad_w": Bounded(r.grad_w, gw_off + 8 * E32 * r.grad_w.abs())}


# ---- block norms ------------------------------------------------------------------

class Norm(NamedTuple):
    h_out: torch.Tensor
    x_out: torch.Tensor
    r1: torch.Tensor
    r2: torch.Tensor


def _rows(gate, rows, width, like):
    if gate is None:
        return torch.ones(rows, width, dtype=torch.float64, device=like.device)
    return gate[torch.arange(rows, device=like.device) // (rows // gate.shape[0])]


def block_norm(f, h, pre, post, gate, alpha, eps):
    r1 = None
    n = f
    if post is not None:
        r1 = (f.square().mean(1) + eps).rsqrt()
        n = f * r1[:, None] * post
    h_out = h + alpha * _rows(gate, *f.shape, f) * n
    r2 = (h_out.square().mean(1) + eps).rsqrt()
    return Norm(h_out, h_out * r2[:, None] * pre, r1, r2)


def block_norm_bounds(f, h, pre, post, gate, alpha, eps):
    r = block_norm(f, h, pre, post, gate, alpha, eps)
    D = f.shape[1]
    part = (alpha * _rows(gate, *f.shape, f) * (f if post is None else f * r.r1[:, None] * post)).abs()
    # mean and rsqrt of a sum of squares: half of D terms' error, plus a few roundings
    rel = (D / 2 + 8) * E32
    h_off = part * (rel + 6 * E32) + E32 * r.h_out.abs()
    # r2 sees h_out's error through its own sum
    r2_rel = rel + ((r.h_out.abs() * h_off).mean(1) * r.r2.square())
    out = {"h_out": Bounded(r.h_out, h_off), "r2": Bounded(r.r2, r.r2 * r2_rel),
           "x_out": Bounded(r.x_out, (h_off * r.r2[:, None] * pre.abs())
                            + r.x_out.abs() * (r2_rel[:, None] + 4 * E32))}
    if post is not None:
        out["r1"] = Bounded(r.r1, r.r1 * rel)
    return out


def block_norm_grad(gh, gx, f, h_out, r1, r2, pre, post, gate, alpha):
    """{name: Bounded} of the gradients; h_out and the rstds are inputs."""
    rows, D = gx.shape
    gamma = _rows(gate, rows, D, gx)
    hh, g = h_out * r2[:, None], gx * pre
    e = gh + r2[:, None] * (g - hh * (g * hh).mean(1, keepdim=True))
    n = f if post is None else f * r1[:, None] * post
    a = alpha * gamma * (1.0 if post is None else post)
    t, fh = a * e, f if post is None else f * r1[:, None]
    df = t if post is None else r1[:, None] * (t - fh * (t * fh).mean(1, keepdim=True))
    # magnitudes of what is added up, and the sums' errors
    many = (D + 16) * E32
    m1 = (g * hh).abs().mean(1, keepdim=True)
    size = gh.abs() + r2[:, None] * (g.abs() + hh.abs() * m1)
    e_off = 8 * E32 * size + many * r2[:, None] * hh.abs() * m1
    # the second mean as S2 - S3 S1: all three sums' magnitudes count
    s2 = (a * fh * (gh.abs() + r2[:, None] * g.abs())).abs().mean(1, keepdim=True)
    s3 = (a * fh * hh).abs().mean(1, keepdim=True) * r2[:, None] * m1 * 1.0
    if post is None:
        df_off = 6 * E32 * t.abs() + a.abs() * e_off
    else:
        mean_off = many * (s2 + 3 * s3) + (a * fh * e_off).abs().mean(1, keepdim=True)
        df_off = r1[:, None] * (8 * E32 * (t.abs() + fh.abs() * (s2 + s3)) + a.abs() * e_off
                                + fh.abs() * mean_off)

    def over_rows(terms, off):
        return Bounded(terms.sum(0), off.sum(0) + (rows + 16) * E32 * terms.abs().sum(0))

    out = {"h": Bounded(e, e_off), "f": Bounded(df, df_off),
           "pre": over_rows(gx * hh, 4 * E32 * (gx * hh).abs())}
    dn = alpha * gamma * e
    if post is not None:
        out["post"] = over_rows(dn * fh, (alpha * gamma * fh).abs() * (e_off + 6 * E32 * e.abs()))
    if gate is not None:
        per = rows // gate.shape[0]
        terms = (alpha * n * e).view(-1, per, D)
        off = ((alpha * n).abs() * (e_off + 6 * E32 * e.abs())).view(-1, per, D)
        out["gate"] = Bounded(terms.sum(1), off.sum(1) + (per + 16) * E32 * terms.abs().sum(1))
    return out


# ---- 8-bit checkpoints ---------------------------------------------------------------

GROUP = 128
SMALLEST = 2.0 ** -100


def groups_of(x):
    """[rows, groups, 128], zeros beyond the width."""
    rows, D = x.shape
    wide = x.new_zeros(rows, -(-D // GROUP) * GROUP)
    wide[:, :D] = x
    return wide.view(rows, -1, GROUP)


def _towards_zero(x):
    """fp32 of non-negative 64-bit values, rounded towards zero."""
    near = x.float()
    below = torch.nextafter(near, torch.zeros_like(near))
    return torch.where(near.double() > x, below, near)


def codes(x):
    """Codes and scales as two fp32 operations each give them, on the CPU."""
    v = groups_of(x.detach().cpu().float())
    a = v.abs().amax(2, keepdim=True)
    seven = torch.full_like(a, 127.0)
    finite, kept = torch.isfinite(a), a >= SMALLEST
    inverse = torch.where(kept & finite, seven / a, torch.zeros_like(a))
    q = torch.round(torch.where(finite, v, torch.zeros_like(v)) * inverse)
    scale = torch.where(finite, torch.where(kept, _towards_zero(a.double() / 127), torch.zeros_like(a)),
                        torch.full_like(a, float("nan")))
    return q.view(x.shape[0], -1)[:, :x.shape[1]].to(torch.int8), scale[:, :, 0]


def values(q, scale):
    D = q.shape[1]
    return q.double() * scale.double().repeat_interleave(GROUP, 1)[:, :D]
