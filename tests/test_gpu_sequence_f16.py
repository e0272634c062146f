"""Attention's backward pass in fp16: gradients of very different sizes in one
call, and values that could overflow on the way, against the 64-bit forms.

The kernel holds p times 2^10 and ds times a power of two that brings a bound of
its row to 2^14, so that what underflows is below 2^-38 of the bound: far
below the 2^-24 of the document's largest grad_out that the 64-bit form's bound
allows, unless sums of a |v| row are beyond 2^13."""
import math

import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from tests import sequence_reference as ref
from tests.test_gpu_sequence import F16, _case, _gen, _no_wait_gave_up, _options, _rand, _shaped  # noqa: F401

pytestmark = pytest.mark.gpu


def _backward(c, go):
    kw = _options(c)
    shaped = [_shaped(c, t) for t in (c.q, c.k, c.v)]
    r = fadam.attention(*shaped, **kw)
    return r, fadam.attention_backward(go.view(r.out.shape), *shaped, r.out, r.lse, **kw)


@pytest.mark.parametrize("H,Hk", [(2, 2), (6, 2)])
@pytest.mark.parametrize("kw", [{}, dict(causal=False), dict(softcap=20.0)])
def test_documents_whose_gradients_differ_by_2_to_the_16(H, Hk, kw):
    """Each against its own 64-bit form, whose bound knows the document's own
    largest gradient only; documents share tiles, and heads are split over CTAs."""
    for offsets in ([0, 37, 165, 400, 900], None):
        ends = offsets or [0, 225, 450, 675, 900]
        c = _case(900, H, Hk, 64, F16, seed=8, size=0.3, offsets=offsets, sequence=225, **kw)
        go = _rand(_gen(3), *c.q.shape)
        for d, size in enumerate((2.0 ** -10, 2.0 ** 6, 2.0 ** -4, 2.0 ** -9)):
            go[ends[d]:ends[d + 1]] *= size
        go = go.to(F16)
        r, grads = _backward(c, go)
        for a, b in zip(ends, ends[1:]):
            rows = slice(a, b)
            alone = c._replace(q=c.q[rows], k=c.k[rows], v=c.v[rows], offsets=None, sequence=b - a)
            want = ref.attention_grad(alone, go[rows], r.out.view(c.q.shape)[rows], r.lse.view(-1, H)[rows])
            for name in "qkv":
                got = getattr(grads, name).reshape(getattr(c, name).shape)
                want[name].holds(got[rows], f"grad_{name} of {a}")


def test_queries_whose_gradients_differ_by_2_to_the_16():
    """grad_q's rows, each with its own grad_out's size."""
    c = _case(500, 2, 1, 64, F16, seed=9, size=0.3)
    sizes = 2.0 ** (-16.0 * torch.rand(500, 1, 1, generator=_gen(1), device="cuda") + 5)
    go = (_rand(_gen(3), *c.q.shape).clamp(-4, 4) * sizes).to(F16)
    r, grads = _backward(c, go)
    # rows by themselves: the bound's largest grad_out is theirs
    for some in range(0, 500, 49):
        mine = torch.zeros_like(go)
        mine[some] = go[some]
        want = ref.attention_grad(c, mine, r.out.view(c.q.shape), r.lse.view(500, 2))["q"]
        got = grads.q.view(c.q.shape)[some]
        ref.Bounded(want.value[some], want.off[some]).holds(got, f"grad_q of {some}")


def test_an_infinite_gradient_leaves_other_documents_their_bits():
    """No tile of 128 tokens is shared: what an infinity or a NaN does to its own
    document's gradients, it does not change the factor of another one's."""
    c = _case(640, 2, 1, 64, F16, seed=8, size=0.3, offsets=[0, 128, 500])
    go = (_rand(_gen(3), *c.q.shape) * 1e-3).to(F16)
    _, want = _backward(c, go)
    for value in (math.inf, math.nan):
        bad = go.clone()
        bad[77, 1, 3] = value
        _, got = _backward(c, bad)
        for a, b in zip(want, got):
            assert torch.equal(a.view(640, -1)[128:], b.view(640, -1)[128:])
        assert not torch.isfinite(got.q.view(c.q.shape)[77, 1]).any() and not torch.isfinite(got.k[:128]).all()


@pytest.mark.parametrize("size", [130.0, 300.0, 3000.0, 60000.0])
def test_large_values_do_not_overflow(size):
    """Every element of v of this size, and grad_out with its signs: go . v is up
    to 64 * 60000 times go.  (The bound: 2^-38 of the row's, twice the sum of |v|
    times the largest |grad_out|.)"""
    c = _case(300, 2, 1, 64, F16, seed=5, size=0.5)
    signs = torch.where(_rand(_gen(2), 300, 1, 64) > 0, 1.0, -1.0)
    c = c._replace(v=(signs * size * (0.5 + 0.5 * torch.rand(300, 1, 64, generator=_gen(4), device="cuda"))).to(F16))
    # small enough for the gradients themselves to be in fp16's range
    go = (signs * (1.0 + 0.1 * _rand(_gen(3), *c.q.shape)) * 2.0 ** -6 * min(1.0, 300.0 / size)).to(F16)
    r, grads = _backward(c, go)
    out, lse = r.out.view(c.q.shape), r.lse.view(300, 2)
    want = ref.attention_grad(c, go, out, lse)
    less = 2.0 ** -38 * 2 * float(go.double().abs().max() * c.v.double().abs().sum(2).max())
    seen = ref.mask(c).double()
    for name, other in (("q", c.k.double().abs().expand(-1, 2, -1)), ("k", c.q.double().abs().sum(1, keepdim=True))):
        of = seen if name == "q" else seen.t()
        more = c.scale * less * torch.einsum("ij,jhd->ihd", of, other)
        want[name] = ref.Bounded(want[name].value, want[name].off + more)
    for name in "qkv":
        got = getattr(grads, name).reshape(getattr(c, name).shape)
        assert torch.isfinite(got).all()
        want[name].holds(got, "grad_" + name)
