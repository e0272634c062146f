"""The sequence operators on the GPU against their 64-bit forms, within bounds
derived from their roundings (tests/sequence_reference.py), at the sizes,
masks, layouts and values where they can go wrong."""
import math
import os
import subprocess
import sys

import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from tests import sequence_reference as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    assert fadam.ops_status() == 0


# ---- embedding ------------------------------------------------------------------------

def _tokens(gen, vocab, *shape):
    rank = torch.exp(torch.rand(*shape, generator=gen, device="cuda") * math.log(vocab + 1))
    return (rank.long() - 1).clamp(0, vocab - 1)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,D,V", [(1, 8, 1), (1, 4096, 50), (3, 1, 5), (17, 72, 100), (257, 130, 31),
                                   (700, 2056, 999), (5000, 64, 300), (4, 5001, 7)])
def test_embedding_sizes(T, D, V, dtype):
    g = _gen(T + D)
    w, t = _rand(g, V, D).to(dtype), _tokens(g, V, T)
    for scale in (1.0, 45.25):
        want = ref.embedding(t, w, scale, None)
        for out in (None, F32):
            x = fadam.embedding(t, w, scale=scale, dtype=out)
            assert x.dtype is (out or dtype)
            ref.Bounded(want, torch.zeros_like(want)).holds(x)      # one rounding


def test_embedding_padding_and_bad_tokens():
    w = _rand(_gen(1), 10, 72).to(BF16)
    t = torch.tensor([[0, 3, -1], [10, 9, 2**40], [-2**60, 3, 3]], device="cuda")
    x = fadam.embedding(t, w, padding_index=3)
    assert x.shape == (3, 3, 72)
    bad = torch.tensor([[0, 0, 1], [1, 0, 1], [1, 0, 0]], dtype=torch.bool, device="cuda")
    assert torch.isnan(x[bad]).all() and torch.isfinite(x[~bad]).all()
    assert (x[t == 3] == 0).all() and torch.equal(x[0, 0], w[0]) and torch.equal(x[1, 1], w[9])
    # a padding index outside the vocabulary
    y = fadam.embedding(t, w, padding_index=-1)
    assert (y[0, 2] == 0).all() and torch.equal(y[0, 1], w[3])


def test_embedding_strided_weight():
    big = torch.full((40, 200), float("nan"), dtype=BF16, device="cuda")
    t = torch.arange(30, device="cuda").view(2, 15)
    for c0, D in ((8, 128), (3, 75), (1, 64)):
        w = big[5:35, c0:c0 + D]
        w.copy_(_rand(_gen(c0), 30, D))
        assert torch.equal(fadam.embedding(t, w).view(30, D), w)


@pytest.mark.parametrize("kind", [(BF16, BF16), (F16, F16), (F32, F32), (BF16, F32), (F16, F32),
                                  (F32, BF16), (F32, F16)])
@pytest.mark.parametrize("T,D,V", [(1, 8, 1), (1, 100, 7), (5, 1, 3), (64, 72, 9), (1000, 130, 31),
                                   (3000, 256, 40000), (2500, 2056, 17), (4, 5001, 2000)])
def test_embedding_grad_sizes(T, D, V, kind):
    g = _gen(T + D + V)
    grad, t = _rand(g, T, D).to(kind[0]), _tokens(g, V, T)
    base = _rand(g, V, D).to(kind[1])
    for scale in (1.0, 3.7):
        out = torch.full((V, D), float("nan"), dtype=kind[1], device="cuda")
        assert fadam.embedding_weight_grad(grad, t, scale=scale, out=out) is out
        want = ref.embedding_grad(grad, t, V, scale, None)
        want.holds(out, "grad_w")
        untouched = torch.bincount(t, minlength=V) == 0
        assert (out[untouched] == 0).all()
        again = fadam.embedding_weight_grad(grad, t, V, scale=scale) if kind[0] is kind[1] else None
        assert again is None or torch.equal(again, out)       # the same bits
        out.copy_(base)
        fadam.embedding_weight_grad(grad, t, scale=scale, out=out, accumulate=True, padding_index=0)
        ref.embedding_grad(grad, t, V, scale, 0, base).holds(out, "accumulated")
        assert torch.equal(out[untouched], base[untouched]) and torch.equal(out[0], base[0])


@pytest.mark.parametrize("tokens", ["one", "two", "none", "bad", "ordered", "every"])
def test_embedding_grad_distributions(tokens):
    T, D, V = 5000, 136, 3001
    g = _gen(7)
    t = {"one": torch.full((T,), 1234), "two": torch.arange(T) % 2 * (V - 1), "none": torch.zeros(T),
         "bad": torch.arange(T) - 2500, "ordered": torch.arange(T) * V // T,
         "every": torch.arange(T).flip(0) % V}[tokens].long().cuda()
    if tokens == "bad":
        t[::7] = 2**62
        t[1::7] = -2**62
    grad = _rand(g, T, D).to(BF16)
    pad = 0 if tokens == "none" else None
    out = fadam.embedding_weight_grad(grad, t, V, padding_index=pad)
    ref.embedding_grad(grad, t, V, 1.0, pad).holds(out)


def test_embedding_grad_order_is_fixed():
    """A token's rows are added in their order: the same bits with other tokens
    between them, as long as the groups are cut alike."""
    T, D = 4096, 64
    grad = _rand(_gen(3), T, D)
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    one = fadam.embedding_weight_grad(grad, t, 5)
    for _ in range(3):
        assert torch.equal(fadam.embedding_weight_grad(grad, t, 5), one)


def test_embedding_grad_strides_and_shapes():
    g = _gen(9)
    for cols, c0, D in ((256, 8, 128), (101, 3, 75)):
        big = torch.full((60, cols), float("nan"), dtype=F32, device="cuda")
        grad = _rand(g, 6, 10, cols).to(BF16)[:, :, c0:c0 + D]
        t = _tokens(g, 50, 6, 10)
        view = big[5:55, c0:c0 + D]
        fadam.embedding_weight_grad(grad, t, out=view)
        ref.embedding_grad(grad, t, 50, 1.0, None).holds(view)
        view.fill_(float("nan"))
        assert torch.isnan(big).all()
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    out = torch.ones(4, 8, device="cuda")
    fadam.embedding_weight_grad(torch.empty(0, 8, device="cuda"), empty, out=out, accumulate=True)
    assert (out == 1).all()
    fadam.embedding_weight_grad(torch.empty(0, 8, device="cuda"), empty, out=out)
    assert (out == 0).all()
    assert fadam.embedding(empty, out).shape == (0, 8)


def test_embedding_grad_of_a_large_vocabulary():
    """More tokens than 152 ranges of 1024."""
    V, T, D = 400_003, 3000, 16
    g = _gen(2)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[:3] = torch.tensor([0, V - 1, V - 1])
    grad = _rand(g, T, D)
    ref.embedding_grad(grad, t, V, 1.0, None).holds(fadam.embedding_weight_grad(grad, t, V))


# ---- attention --------------------------------------------------------------------------

def _case(T, H, Hk, D, dtype, seed=0, size=1.3, **kw):
    g = _gen(seed)
    q, k, v = (_rand(g, T, h, D) * s for h, s in ((H, size), (Hk, size), (Hk, 1.0)))
    if kw.pop("bias", False):
        kw["slopes"] = 2.0 ** (-6.0 * torch.arange(1, H + 1, device="cuda") / H)
    return ref.Case(q.to(dtype), k.to(dtype), v.to(dtype), D ** -0.5, **{"sequence": T, **kw})


def _options(c):
    as_ints = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(causal=c.causal, scale=c.scale, softcap=c.softcap, slopes=c.slopes,
                documents=as_ints(c.offsets), prefix=as_ints(c.prefix))


def _shaped(c, t):
    return t if c.offsets is not None else t.view(-1, c.sequence, *t.shape[1:])


def _check(c, seed=1, q=None, k=None, v=None, go=None, size=1e-2):
    """Forward and backward of a case, by tensors of any layout."""
    shaped = [_shaped(c, t) if given is None else given for t, given in ((c.q, q), (c.k, k), (c.v, v))]
    kw = _options(c)
    r = fadam.attention(*shaped, **kw)
    out, lse, empty = ref.attention(c)
    flat_out, flat_lse = r.out.reshape(c.q.shape), r.lse.reshape(c.q.shape[:2])
    assert (flat_out[empty] == 0).all() and (flat_lse[empty] == -math.inf).all()
    out.holds(flat_out, "out")
    lse.holds(torch.where(empty[:, None], 0.0, flat_lse), "lse")
    if go is None:
        go = (_rand(_gen(seed), *c.q.shape) * size).to(c.q.dtype).view(r.out.shape)
    d = fadam.attention_backward(go, *shaped, r.out, r.lse, **kw)
    want = ref.attention_grad(c, go.reshape(c.q.shape), flat_out, flat_lse)
    for name in "qkv":
        got = getattr(d, name)
        assert got.shape == shaped["qkv".index(name)].shape
        want[name].holds(got.reshape(getattr(c, name).shape), "grad_" + name)
    return r, d


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,H,Hk,D", [
    (1, 1, 1, 8), (1, 4, 2, 128), (2, 2, 1, 64), (31, 3, 3, 16), (127, 2, 2, 72), (128, 4, 1, 128),
    (129, 2, 1, 64), (200, 6, 3, 24), (256, 1, 1, 128), (257, 5, 1, 120), (385, 2, 2, 40),
    (600, 8, 2, 80), (1000, 2, 2, 128)])
def test_attention_sizes(T, H, Hk, D, dtype):
    for causal in (True, False):
        _check(_case(T, H, Hk, D, dtype, seed=T + D, causal=causal))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 88, 128])
@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(bias=True), dict(softcap=20.0, bias=True),
                                dict(softcap=5.0, size=4.0), dict(softcap=0.5, size=2.0, bias=True)])
def test_attention_caps_and_biases(dtype, D, kw):
    """Scores far below the cap, and far beyond it."""
    for causal in (True, False):
        _check(_case(333, 4, 2, D, dtype, seed=D, causal=causal, **kw))


DOCUMENTS = [
    [0, 400], [0, 1, 2, 3, 400], [0, 128, 256, 400], [0, 127, 129, 129, 300, 400], [0, 0, 400, 400],
    [37, 200, 390], [0, 100], [399, 400], [150, 150, 150], [0], [400], list(range(0, 401, 5)),
    [0, 130, 131, 350]]


@pytest.mark.parametrize("offsets", DOCUMENTS)
@pytest.mark.parametrize("causal", [True, False])
def test_attention_documents(offsets, causal):
    for dtype, D in ((BF16, 128), (F16, 48)):
        _check(_case(400, 4, 2, D, dtype, seed=len(offsets), causal=causal, offsets=offsets,
                     softcap=25.0 if D == 48 else 0.0, bias=D == 128))


@pytest.mark.parametrize("offsets,prefix", [
    (None, [0, 1, 200]), (None, [100, 37, 199]), (None, [-5, 1000, 128]), ([0, 300, 450, 600], [150, 150, 0]),
    ([0, 1, 1, 500], [1, 3, 129]), ([20, 250, 590], [130, 340])])
def test_attention_prefixes(offsets, prefix):
    for dtype, D in ((BF16, 64), (F16, 128)):
        _check(_case(600, 2, 1, D, dtype, seed=3, offsets=offsets, prefix=prefix, sequence=200))


@pytest.mark.parametrize("H,Hk", [(65, 65), (66, 33)])
def test_attention_tiles_as_they_come(H, Hk):
    """Several sequences and documents of more than two CTAs to an SM, whose
    tiles are not sorted by their work: one head or two to a CTA."""
    for kw in (dict(sequence=200), dict(sequence=200, prefix=[0, 30, 200, 1, 128, 77]),
               dict(offsets=[10, 40, 700, 701, 1190])):
        _check(_case(1200, H, Hk, 16, BF16, seed=H, **kw))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_padding_may_hold_anything(dtype):
    """Rows outside all documents, before and behind them, of q, k, v, grad_out
    and out: infinities and NaN there reach nothing."""
    bad = torch.tensor([math.nan, math.inf, -math.inf, 60000.0], device="cuda")
    for offsets in ([40, 130, 333], [0, 200], [129, 130]):
        c = _case(400, 4, 2, 128, dtype, seed=5, offsets=offsets)
        pad = torch.ones(400, dtype=torch.bool, device="cuda")
        pad[offsets[0]:offsets[-1]] = False
        for t in (c.q, c.k, c.v):
            t[pad] = bad.to(dtype).repeat(t.shape[2] // 4).expand(int(pad.sum()), t.shape[1], -1)
        go = (_rand(_gen(4), *c.q.shape) * 1e-2).to(dtype)
        go[pad] = math.nan
        r, d = _check(c, go=go)
        for t in d:
            assert (t[pad] == 0).all()
        r.out[pad] = math.inf      # what a user may have put there
        kw = _options(c)
        again = fadam.attention_backward(go, c.q, c.k, c.v, r.out, r.lse, **kw)
        for a, b in zip(d, again):
            assert torch.equal(a, b)


def test_attention_without_tokens():
    e = torch.empty(2, 0, 4, 64, dtype=BF16, device="cuda")
    r = fadam.attention(e, e, e)
    assert r.out.shape == e.shape and r.lse.shape == (2, 0, 4)
    d = fadam.attention_backward(e, e, e, e, r.out, r.lse)
    assert all(t.shape == e.shape for t in d)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_layouts(dtype):
    B, S, H, Hk, D = 3, 150, 4, 2, 64
    g = _gen(11)
    fused = _rand(g, B, S, H + 2 * Hk, D).to(dtype)
    q, k, v = fused.split([H, Hk, Hk], 2)
    flat = [t.reshape(B * S, -1, D) for t in (q, k, v)]
    c = ref.Case(*flat, D ** -0.5, sequence=S)
    go = (_rand(g, B, S, 2 * H, D) * 1e-2).to(dtype)[:, :, ::2]
    _check(c, q=q, k=k, v=v, go=go)
    # heads outside, tokens inside; one sequence
    by_head = [_rand(g, h, S, D).to(dtype).transpose(0, 1) for h in (H, Hk, Hk)]
    c = ref.Case(*(t.contiguous() for t in by_head), D ** -0.5, sequence=S)
    go = (_rand(g, H, S, D) * 1e-2).to(dtype).transpose(0, 1)
    r, d = _check(c, q=by_head[0], k=by_head[1], v=by_head[2], go=go)
    # out as another program may lay it out
    out = r.out.transpose(0, 1).contiguous().transpose(0, 1)
    e = fadam.attention_backward(go, *by_head, out, r.lse, scale=c.scale)
    for a, b in zip(d, e):
        assert torch.equal(a, b)
    # inside a larger buffer whose other columns hold NaN
    big = torch.full((S, H + 1, D + 16), float("nan"), dtype=dtype, device="cuda")
    inner = big[:, :H, 8:8 + D]
    inner.copy_(by_head[0])
    _check(c, q=inner, k=by_head[1], v=by_head[2], go=go)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_growing_and_large_scores(dtype):
    """Each tile of keys raises the rows' maximum, a little or by much."""
    for grow, T in ((0.02, 700), (1.0, 500)):
        c = _case(T, 2, 1, 64, dtype, seed=2, size=1.0)
        along = _rand(_gen(9), 64)
        k = c.k.float() + along * torch.arange(T, device="cuda")[:, None, None] * grow * 0.05
        c = c._replace(k=k.to(dtype), q=(c.q.float() + along).to(dtype))
        _check(c)
        _check(c._replace(causal=False))
    # one key that outweighs all others, met first or last
    for at in (0, 299):
        c = _case(300, 2, 2, 128, dtype, seed=6, causal=False)
        c.k[at] = (c.q[5].float() * 20).to(dtype)
        _check(c)


def test_attention_fp16_gradients_of_any_size():
    """grad_out far below fp16's normal numbers times the rows' weights, and far
    above 1; rows whose weights are spread over many keys."""
    for size in (2.0 ** -20, 1e-4, 300.0):
        _check(_case(900, 2, 1, 64, F16, seed=8, size=0.3), size=size)
    c = _case(300, 2, 1, 64, F16, seed=8)
    zero = torch.zeros(1, 300, 2, 64, dtype=F16, device="cuda")
    r = fadam.attention(*(_shaped(c, t) for t in (c.q, c.k, c.v)))
    d = fadam.attention_backward(zero, *(_shaped(c, t) for t in (c.q, c.k, c.v)), r.out, r.lse)
    assert all((t == 0).all() for t in d)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_passes_infinities_on(dtype):
    """An overflow in what comes back makes the gradients not finite, so that the
    shard's screen skips the step; a bad query row reaches no other row's output."""
    c = _case(300, 2, 1, 64, dtype, seed=4)
    q, k, v = (_shaped(c, t) for t in (c.q, c.k, c.v))
    r = fadam.attention(q, k, v)
    for value in (math.inf, math.nan):
        go = torch.full_like(r.out, 1e-2)
        go[0, 77, 1, 3] = value
        d = fadam.attention_backward(go, q, k, v, r.out, r.lse)
        assert not torch.isfinite(d.q[0, 77, 1]).any() and not torch.isfinite(d.v[0, :78]).all()
        assert not torch.isfinite(d.k).all()
        bad = q.clone()
        bad[0, 40, 0, 0] = value
        s = fadam.attention(bad, k, v)
        assert not torch.isfinite(s.out[0, 40, 0]).any()
        keep = torch.ones(300, dtype=torch.bool, device="cuda")
        keep[40] = False
        assert torch.equal(s.out[0, keep], r.out[0, keep]) and torch.equal(s.out[0, 40, 1], r.out[0, 40, 1])
        # documents that share no 128 tokens with the bad row's
        offsets = torch.tensor([0, 128, 300], dtype=torch.int32, device="cuda")
        kk = k.clone()
        kk[0, 130] = value
        a, b = (fadam.attention(q, x, v, documents=offsets) for x in (k, kk))
        assert torch.equal(a.out[0, :128], b.out[0, :128]) and not torch.isfinite(b.out[0, 130:]).any()


def test_attention_bad_documents_stay_in_bounds():
    """Offsets that decrease or lie outside: any result, within the outputs."""
    c = _case(300, 2, 1, 64, BF16, seed=4)
    for offsets in ([0, 200, 100, 300], [-50, 100, 1000], [500, 600], [300, 0], [2**31 - 1, -2**31]):
        docs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        r = fadam.attention(c.q, c.k, c.v, documents=docs)
        d = fadam.attention_backward(c.q, c.q, c.k, c.v, r.out, r.lse, documents=docs)
        assert all(t.shape == s.shape for t, s in zip(d, (c.q, c.k, c.v)))
    torch.cuda.synchronize()


def test_attention_over_thousands_of_documents():
    """More documents than a block keeps the offsets of; each a few tokens long."""
    T, H, D = 11_000, 2, 16
    g = _gen(7)
    lengths = torch.randint(0, 4, (7000,), generator=torch.Generator().manual_seed(1)).tolist()
    offsets = [0]
    for n in lengths:
        if offsets[-1] + n <= T - 17:
            offsets.append(offsets[-1] + n)
    assert len(offsets) > 4096
    q, k, v, go = (_rand(g, T, H, D).to(BF16) for _ in range(4))
    docs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    prefix = torch.ones(len(offsets) - 1, dtype=torch.int32, device="cuda")
    r = fadam.attention(q, k, v, documents=docs, prefix=prefix)
    d = fadam.attention_backward(go, q, k, v, r.out, r.lse, documents=docs, prefix=prefix)
    for first in (0, 3000, len(offsets) - 200):      # a stretch of documents, as tokens of their own
        part = offsets[first:first + 190]
        rows = slice(part[0], part[-1])
        c = ref.Case(*(t[rows] for t in (q, k, v)), D ** -0.5, offsets=[o - part[0] for o in part])
        out, lse, _ = ref.attention(c)
        out.holds(r.out[rows], "out")
        lse.holds(r.lse[rows], "lse")
        want = ref.attention_grad(c, go[rows], r.out[rows], r.lse[rows])
        for name in "qkv":
            want[name].holds(getattr(d, name)[rows], "grad_" + name)
    assert (r.out[offsets[-1]:] == 0).all() and all((t[offsets[-1]:] == 0).all() for t in d)


def test_two_threads_two_streams():
    """Two shapes from two host threads at once: the same bits as alone."""
    import threading
    cases = [_case(900, 4, 2, 128, BF16, seed=1, offsets=[0, 300, 870]), _case(650, 6, 3, 64, F16, seed=2, bias=True)]
    work = []
    for c in cases:
        shaped = [_shaped(c, t) for t in (c.q, c.k, c.v)]
        kw = _options(c)
        r = fadam.attention(*shaped, **kw)
        work.append((shaped, kw, r, fadam.attention_backward(r.out, *shaped, r.out, r.lse, **kw)))
    torch.cuda.synchronize()
    errors = []

    def body(shaped, kw, r, d):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(200):
                    s = fadam.attention(*shaped, **kw)
                    e = fadam.attention_backward(s.out, *shaped, s.out, s.lse, **kw)
                stream.synchronize()
            for a, b in zip((*r, *d), (*s, *e)):
                assert torch.equal(a, b)
        except BaseException as e:      # reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=body, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


def test_attention_against_differences():
    """The gradients against differences of the 64-bit form's loss along one
    direction: the two formulas, not the roundings (a few percent of bf16's)."""
    c = _case(200, 4, 2, 64, BF16, seed=12, softcap=4.0, bias=True, offsets=[0, 90, 190], prefix=[20, 50])
    kw = _options(c)
    r = fadam.attention(c.q, c.k, c.v, **kw)
    go = _rand(_gen(2), *c.q.shape).to(BF16)
    d = fadam.attention_backward(go, c.q, c.k, c.v, r.out, r.lse, **kw)
    for name in "qkv":
        t = getattr(c, name)
        step = _rand(_gen(5), *t.shape).double() * 1e-3
        far = [(ref.attention(c._replace(**{name: t.double() + s * step}))[0].value * go.double()).sum()
               for s in (-1, 1)]
        along = (getattr(d, name).double() * step).sum()
        # ds and p are rounded to 2^-8 at random: of n products their mean error goes as n^-1/2
        spread = 2.0 ** -8 * ((getattr(d, name).double() * step) ** 2).sum().sqrt() * 4
        assert abs((far[1] - far[0]) / 2 - along) < 4 * spread + 1e-3 * abs(along), name


def test_attention_is_deterministic_and_capturable():
    c = _case(700, 8, 2, 128, BF16, seed=1, offsets=[0, 300, 650], softcap=30.0)
    kw = _options(c)
    go = (_rand(_gen(3), *c.q.shape) * 1e-2).to(BF16)
    r = fadam.attention(c.q, c.k, c.v, **kw)
    d = fadam.attention_backward(go, c.q, c.k, c.v, r.out, r.lse, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s = fadam.attention(c.q, c.k, c.v, **kw)
        e = fadam.attention_backward(go, c.q, c.k, c.v, s.out, s.lse, **kw)
    side.synchronize()
    for a, b in zip((*r, *d), (*s, *e)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = fadam.attention(c.q, c.k, c.v, **kw)
        e = fadam.attention_backward(go, c.q, c.k, c.v, s.out, s.lse, **kw)
    c.q.mul_(0.5)
    graph.replay()
    r = fadam.attention(c.q, c.k, c.v, **kw)
    d = fadam.attention_backward(go, c.q, c.k, c.v, r.out, r.lse, **kw)
    for a, b in zip((*r, *d), (*s, *e)):
        assert torch.equal(a, b)


def test_two_graphs_replayed_side_by_side():
    """Workspaces of two captured graphs are apart."""
    cases = [_case(600, 4, 1, 64, F16, seed=s, offsets=[0, 100 * s, 600]) for s in (1, 2)]
    go = (_rand(_gen(3), 600, 4, 64) * 1e-2).to(F16)
    w = torch.randint(0, 50, (600,), generator=_gen(4), device="cuda")
    graphs, kept, want = [], [], []
    options = [_options(c) for c in cases]      # (a graph's inputs live as long as it does)
    for c, kw in zip(cases, options):
        def body():
            r = fadam.attention(c.q, c.k, c.v, **kw)
            d = fadam.attention_backward(go, c.q, c.k, c.v, r.out, r.lse, **kw)
            return (*r, *d, fadam.embedding_weight_grad(d.q.view(600, -1), w, 50))
        want.append([t.clone() for t in body()])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(body())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for have, w_ in zip(kept, want):
        for a, b in zip(have, w_):
            assert torch.equal(a, b)


def test_the_first_call_of_a_process_may_be_captured():
    code = """
import torch
import adamw_optimizer_step_persistent_gb300 as fadam
q = torch.randn(200, 4, 64, device="cuda").bfloat16()
w = torch.randn(100, 256, device="cuda").bfloat16()
t = torch.randint(0, 100, (200,), device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    x = fadam.embedding(t, w)
    r = fadam.attention(x.view(200, 4, 64), q, q)
    d = fadam.attention_backward(r.out, x.view(200, 4, 64), q, q, r.out, r.lse)
    g = fadam.embedding_weight_grad(d.q.view(200, 256), t, 100)
graph.replay()
torch.cuda.synchronize()
s = fadam.attention(fadam.embedding(t, w).view(200, 4, 64), q, q)
assert torch.equal(r.out, s.out) and torch.isfinite(g).all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=240,
                   env=dict(os.environ, PYTHONPATH=root))


# ---- offsets beyond 32 bits -----------------------------------------------------------------

def test_embedding_beyond_2_to_the_31_elements():
    V, T, D = 270_000, 262_200, 8192
    w = torch.zeros(V, D, dtype=BF16, device="cuda")
    at = torch.tensor([0, 1, 262_144, V - 1], device="cuda")
    w[at] = _rand(_gen(1), 4, D).to(BF16)
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    t[-4:] = at
    t[:-4] = 5
    x = fadam.embedding(t, w)
    assert torch.equal(x[-4:], w[at]) and not x[:-4].any()
    grad = torch.zeros(T, D, dtype=BF16, device="cuda")
    grad[-4:] = x[-4:]
    grad[7] = 1.0
    del x
    out = fadam.embedding_weight_grad(grad, t, V)
    assert torch.equal(out[at], w[at]) and (out[5] == 1).all() and not out[6:262_144].any()


def test_attention_beyond_2_to_the_31_elements():
    T, H, D = 140_000, 128, 128
    g = _gen(6)
    q = torch.randn(T, H, D, generator=g, device="cuda", dtype=BF16)
    k = torch.randn(T, 1, D, generator=g, device="cuda", dtype=BF16)
    offsets = list(range(0, T, 50)) + [T]
    docs = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    r = fadam.attention(q, k, k, documents=docs)
    d = fadam.attention_backward(q, q, k, k, r.out, r.lse, documents=docs)
    for a in (0, 69_950, 139_900):
        rows = slice(a, a + 50)
        c = ref.Case(q[rows].clone(), k[rows].clone(), k[rows].clone(), D ** -0.5, sequence=50)
        out, lse, _ = ref.attention(c)
        out.holds(r.out[rows], "out")
        lse.holds(r.lse[rows], "lse")
        want = ref.attention_grad(c, q[rows], r.out[rows], r.lse[rows])
        for name in "qkv":
            want[name].holds(getattr(d, name)[rows], "grad_" + name)


# ---- all of them together ------------------------------------------------------------------

def _model_loss(w, tokens, targets, ends, model):
    """The example's model in 64 bits, by plain operations."""
    def rms(x, weight):
        return x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * weight

    alpha, H, Hk, D = model.alpha, model.heads, model.kv_heads, model.head
    T = tokens.shape[0]
    at = torch.arange(T, device="cuda")
    doc = torch.bucketize(at, torch.tensor(ends, device="cuda"), right=True)
    seen = (doc[:, None] == doc) & (at[:, None] >= at)
    h = w["embed"][tokens]
    x = rms(h, w["norm0"])
    for b in range(model.blocks):
        q, k, v = (x @ w[f"qkv{b}"].t()).view(T, -1, D).transpose(0, 1).split([H, Hk, Hk])
        k, v = (t.repeat_interleave(H // Hk, 0) for t in (k, v))
        s = 30.0 * torch.tanh(q @ k.transpose(1, 2) / (30.0 * D ** 0.5))
        s = s - model.slopes.double()[:, None, None] * (at[:, None] - at).abs()
        o = torch.softmax(s.masked_fill(~seen, -math.inf), 2) @ v
        f = o.transpose(0, 1).reshape(T, -1) @ w[f"out{b}"].t()
        h = h + alpha * w[f"gatea{b}"] * rms(f, w[f"posta{b}"])
        y = rms(h, w[f"prea{b}"])
        f = torch.relu(y @ w[f"up{b}"].t()) @ w[f"down{b}"].t()
        h = h + alpha * w[f"gatem{b}"] * rms(f, w[f"postm{b}"])
        x = rms(h, w[f"prem{b}"])
    z = x @ w["head"].t()
    keep = targets != -1
    return (torch.logsumexp(z, 1) - z.gather(1, targets.clamp(min=0)[:, None])[:, 0])[keep].mean()


def test_a_model_of_all_operators_has_the_gradients_of_its_formula():
    """Every gradient of the example's model against autograd's in 64 bits.  On
    the way through the two blocks a value is rounded some forty times to bf16
    (2^-9 of it on average) and kept in 8 bits five times (about as much): their
    errors add up as roots of sums of squares to 45^(1/2) 2^-9 = 1.3% of a
    gradient, held to 5% of its norm.  Behind a perceptron's relu (going back) its
    mask counts too: an argument that is off by 1.3% of its standard deviation
    has another sign with probability atan(0.013) / pi = 0.41%, and the 8-bit code
    of an activation below 1/254 of its group's largest (some three deviations) is
    zero, 0.4 * 3 / 254 = 0.47% of the arguments.  Of the half that pass, 0.88 /
    50 = 1.8% are then wrong by their whole gradient: 13% of its norm, from each
    of the two.  The sum with the residual stream's own gradient is off by less,
    so gradients behind a relu are held to 5% + 13% = 18%."""
    from examples import train_step
    model = train_step.Model(vocab=90, width=128, hidden=200, blocks=2, heads=4, kv_heads=2)
    g = _gen(5)
    tokens, ends = _tokens(g, 90, 300), [0, 37, 165, 166, 300]
    targets = torch.randint(0, 90, (300,), generator=g, device="cuda")
    targets[::7] = -1
    documents = torch.tensor(ends, dtype=torch.int32, device="cuda")
    loss = model.step(tokens, targets, documents)
    w = {n: t.double().requires_grad_() for n, t in model.w.items()}
    want = _model_loss(w, tokens, targets, ends[1:-1], model)
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 0.02 * float(want.detach())
    for name, grad in model.grads.items():
        far = (grad.double() - w[name].grad).norm() / w[name].grad.norm()
        assert far < (0.05 if name in ("head", "down1", "postm1", "prem1", "gatem1") else 0.18), (name, float(far))
    # a second micro-batch is added
    first = {n: t.clone() for n, t in model.grads.items()}
    model.step(tokens, targets, documents, first=False)
    for name, grad in model.grads.items():
        assert (grad - 2 * first[name]).norm() <= 2.0 ** -20 * first[name].norm(), name
