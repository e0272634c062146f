"""Attention at the ends of what its arguments allow, against the 64-bit forms."""
import math

import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from tests import sequence_reference as ref
from tests.test_gpu_sequence import BF16, F16, _case, _check, _gen, _no_wait_gave_up, _options, _rand, _shaped  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [1e4, 1e9, 1e12, 1e15])
def test_attention_wide_caps(softcap):
    """Caps far beyond the scores, which then are what they are without one, and
    products that come near such a cap."""
    c = _case(300, 4, 2, 64, BF16, seed=1, softcap=softcap)
    shaped = [_shaped(c, t) for t in (c.q, c.k, c.v)]
    r = fadam.attention(*shaped, **_options(c))
    # tanh(y) is y but for y^3 / 3, and y is below 1e-2
    out, lse, _ = ref.attention(c._replace(softcap=0.0))
    cubes = float((c.scale * torch.einsum("ihd,jhd->hij", c.q.double(), c.k.double().repeat_interleave(2, 1))).abs()
                  .max()) ** 3 / 3 / softcap ** 2
    ref.Bounded(lse.value, lse.off + cubes).holds(r.lse.view(300, 4), "lse")
    ref.Bounded(out.value, out.off + 2 * cubes * c.v.double().abs().max()).holds(r.out.view(c.q.shape), "out")
    # up to about a quarter of the cap and beyond it
    for top in (0.2, 1.0):
        big = math.sqrt(top * softcap / 32.0)
        c = ref.Case(*((_rand(_gen(i), 200, h, 64) * s).to(BF16) for i, (h, s) in enumerate(((4, big), (2, big), (2, 1.0)))),
                     1.0, softcap=softcap, sequence=200)
        shaped = [_shaped(c, t) for t in (c.q, c.k, c.v)]
        r = fadam.attention(*shaped, **_options(c))
        _, lse, _ = ref.attention(c)
        lse.holds(r.lse.view(200, 4), f"lse of scores up to {top} caps")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_row_of_scores_that_are_all_minus_infinity_is_not_an_empty_one(dtype):
    """exp(s - lse) of the formula is then exp(-inf + inf): NaN, out and its
    gradients, as with a score of +infinity; not the zeros of a row that sees
    nothing."""
    for offsets in (None, [0, 300]):
        c = _case(300, 2, 1, 64, dtype, seed=4, offsets=offsets)
        c.k[:6, 0, 3] = -1.5
        c.q[5, 1, 3] = math.inf
        shaped = [_shaped(c, t) for t in (c.q, c.k, c.v)]
        kw = _options(c)
        r = fadam.attention(*shaped, **kw)
        out, lse = r.out.view(c.q.shape), r.lse.view(300, 2)
        assert torch.isnan(out[5, 1]).all() and float(lse[5, 1]) == -math.inf
        assert torch.isfinite(out[:5]).all() and torch.isfinite(out[5, 0]).all() and torch.isfinite(out[6:]).all()
        go = torch.full_like(r.out, 1e-2)
        d = fadam.attention_backward(go, *shaped, r.out, r.lse, **kw)
        assert torch.isnan(d.q.view(c.q.shape)[5, 1]).all()
        assert not torch.isfinite(d.k).all() and not torch.isfinite(d.v).all()
    # a row of no document beside them keeps its zeros
    c = _case(300, 2, 1, 64, dtype, seed=4, offsets=[10, 290])
    c.k[10:16, 0, 3] = -1.5
    c.q[15, 1, 3] = math.inf
    r = fadam.attention(c.q, c.k, c.v, **_options(c))
    assert torch.isnan(r.out[15, 1]).all() and (r.out[:10] == 0).all() and (r.lse[:10] == -math.inf).all()


@pytest.mark.parametrize("H,Hk", [(35, 35), (36, 18), (56, 56)])
def test_attention_tiles_in_order_of_their_work(H, Hk):
    """Several sequences and documents of one to two CTAs to an SM, whose tiles
    are sorted by their work: one head or two to a CTA."""
    for kw in (dict(sequence=200), dict(sequence=200, prefix=[0, 30, 200, 1, 128, 77]),
               dict(offsets=[10, 40, 700, 701, 1190]), dict(offsets=[0, 0, 300, 1200]), dict(offsets=[600, 650])):
        _check(_case(1200, H, Hk, 16, BF16, seed=H, **kw))


@pytest.mark.parametrize("T,H,Hk,D,dtype,kw", [
    (8192, 2, 1, 128, BF16, {}), (8192, 1, 1, 64, F16, dict(softcap=30.0)), (8100, 1, 1, 128, F16, dict(bias=True)),
    (6000, 2, 2, 72, BF16, dict(causal=False)), (8192, 2, 1, 64, BF16, dict(offsets=[5, 900, 8190], prefix=[400, 5000]))])
def test_attention_walks_over_many_tiles(T, H, Hk, D, dtype, kw):
    """Up to 64 tiles of keys or queries, and twice as many where heads share
    their keys: rings and barriers go round many times."""
    _check(_case(T, H, Hk, D, dtype, seed=T, **kw))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_query_of_one_key_has_no_gradient_by_its_score(dtype):
    """Its weight is 1 whatever its score: grad_q is 0, not what grad_out . v and
    grad_out . out differ by in their roundings, and so is grad_k in a document of
    one token."""
    cases = [(_case(T, H, Hk, D, dtype, seed=T, sequence=1, **kw), slice(0, T), slice(0, T))
             for T, H, Hk, D, kw in ((1, 1, 1, 128, {}), (2, 3, 3, 128, dict(causal=False)), (7, 32, 8, 64, dict(softcap=50.0)),
                                     (300, 6, 2, 72, dict(bias=True)))]
    some = list(range(0, 140)) + [200, 400]
    cases.append((_case(400, 4, 2, 64, dtype, seed=3, offsets=some), [*range(0, 139), 139, 200], slice(0, 139)))
    cases.append((_case(300, 4, 2, 64, dtype, seed=3, sequence=150), [0, 150], slice(0, 0)))
    for c, queries, keys in cases:
        r, d = _check(c)
        assert (d.q.reshape(c.q.shape)[queries] == 0).all()
        assert (d.k.reshape(c.k.shape)[keys] == 0).all()
        assert (d.v != 0).any()
