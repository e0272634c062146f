"""Calls of the sequence operators have to give what they give alone: whatever
ran before them in the same memory, whatever lies beside what they see."""
import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from tests.test_gpu_sequence import BF16, F16, _case, _gen, _no_wait_gave_up, _options, _rand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_back_to_back_calls_in_the_same_workspace(dtype):
    """Calls that follow one another without a wait get the same workspace from
    the allocator: each has the bits that it has alone, with other queries,
    statistics, gradients, documents and prefixes in it than the one before."""
    cuts = [[0, 900], [0, 1, 130, 897], [60, 400, 401, 850], [0, 128, 256, 640], [333, 334, 900], [0, 0, 500]]
    calls = []
    for i, offsets in enumerate(cuts):
        n = len(offsets) - 1
        c = _case(900, 6, 2, 128, dtype, seed=i, offsets=offsets, prefix=[37 * i] * n, softcap=20.0 * (i % 2))
        go = (_rand(_gen(i), *c.q.shape) * 10.0 ** -i).to(dtype)
        calls.append((c, go, _options(c)))

    def run(c, go, kw):
        r = fadam.attention(c.q, c.k, c.v, **kw)
        return (*r, *fadam.attention_backward(go, c.q, c.k, c.v, r.out, r.lse, **kw))

    alone = []
    for call in calls:
        torch.cuda.synchronize()
        alone.append(run(*call))
    torch.cuda.synchronize()
    order = torch.randint(0, len(calls), (120,), generator=torch.Generator().manual_seed(1)).tolist()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(3):
        got = [run(*calls[i]) for i in order]
        for i, g in zip(order, got):
            for a, b in zip(alone[i], g):
                wrong += (a.view(torch.uint8) != b.view(torch.uint8)).sum()
    assert int(wrong) == 0


def _all(c, go):
    kw = _options(c)
    r = fadam.attention(c.q, c.k, c.v, **kw)
    return (*r, *fadam.attention_backward(go, c.q, c.k, c.v, r.out, r.lse, **kw))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bias", [False, True])
def test_capped_scores_have_their_bits_whatever_lies_beside_them(dtype, bias):
    """Small scores of a row that sees few of its tile; beside it, not seen, what
    is far beyond the cap.  (The cap is below the growth at which a row's
    reference maximum is raised.)"""
    def case(offsets):
        return _case(400, 4, 2, 64, dtype, seed=5, size=0.3, softcap=2.0, offsets=offsets, bias=bias)

    def large(n, seed):
        return [(_rand(_gen(seed + i), n, h, 64) * 40).to(dtype) for i, h in enumerate((4, 2, 2))]

    go = (_rand(_gen(4), 400, 4, 64) * 1e-2).to(dtype)
    # padding, of finite numbers and of any
    c = case([40, 130, 333])
    want = _all(c, go)
    live = slice(40, 333)
    for fill in (None, float("inf"), float("nan")):
        for rows in (slice(0, 40), slice(333, 400)):
            n = rows.stop - rows.start
            for t, x in zip((c.q, c.k, c.v), large(n, 7)):
                t[rows] = x if fill is None else fill
        for a, b in zip(want, _all(c, go)):
            assert torch.equal(a[live], b[live])
    # a document in the same tiles
    c = case([0, 70, 200, 400])
    want = _all(c, go)
    for t, x in zip((c.q, c.k, c.v), large(130, 9)):
        t[70:200] = x
    for a, b in zip(want, _all(c, go)):
        for rows in (slice(0, 70), slice(200, 400)):
            assert torch.equal(a[rows], b[rows])
    # later tokens of the same document
    c = case([0, 400])
    kw = _options(c)
    want = fadam.attention(c.q, c.k, c.v, **kw)
    for t, x in zip((c.q, c.k, c.v), large(250, 11)):
        t[150:] = x
    for a, b in zip(want, fadam.attention(c.q, c.k, c.v, **kw)):
        assert torch.equal(a[:150], b[:150])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kw", [{}, dict(bias=True), dict(softcap=60.0)])
def test_rows_have_their_bits_whatever_their_neighbours_grow_to(dtype, kw):
    """Rows whose scores grow a little from tile to tile, beside rows whose scores
    grow by much: those of another document, and later ones of their own."""
    c = _case(700, 4, 2, 64, dtype, seed=6, size=0.8, offsets=[0, 300, 330, 700], **kw)
    along = _rand(_gen(9), 64)
    small = c.k.float() + along * (torch.arange(700, device="cuda")[:, None, None] // 128) * 0.1
    c = c._replace(k=small.to(dtype), q=(c.q.float() + 0.3 * along).to(dtype))
    kw = _options(c)
    want = fadam.attention(c.q, c.k, c.v, **kw)
    # a document of 30 tokens whose tile holds the others' rows
    large = c._replace(k=c.k.clone(), q=c.q.clone())
    large.k[300:330] *= 6
    large.q[300:330] *= 6
    for a, b in zip(want, fadam.attention(large.q, large.k, large.v, **kw)):
        assert torch.equal(a[:300], b[:300]) and torch.equal(a[330:], b[330:])
    # later tokens of a document: they see the tiles that earlier ones see, with larger scores
    large = c._replace(q=c.q.clone())
    large.q[600:] *= 5
    for a, b in zip(want, fadam.attention(large.q, large.k, large.v, **kw)):
        assert torch.equal(a[:600], b[:600])


@pytest.mark.parametrize("many", [1, 700, 3000])
def test_an_embedding_sum_does_not_change_with_the_tokens_between_its_rows(many):
    """A token's rows are added in their order, by groups that the sorted list is
    cut into: other tokens' rows between them, whose places in that list lie
    behind, change no bit."""
    T, D, V = 4096, 72, 50
    rows = _rand(_gen(3), T, D)
    together = torch.full((T,), 31, dtype=torch.int64, device="cuda")
    together[:many] = 4
    want = fadam.embedding_weight_grad(rows, together, V)
    for seed in range(4):
        at = torch.randperm(T, generator=torch.Generator().manual_seed(seed))
        first = at[:many].sort().values.cuda()
        rest = at[many:].sort().values.cuda()
        tokens, spread = torch.empty_like(together), torch.empty_like(rows)
        tokens[first], tokens[rest] = 4, 5 + torch.arange(T - many, device="cuda") % 45
        spread[first], spread[rest] = rows[:many], rows[many:]
        got = fadam.embedding_weight_grad(spread, tokens, V)
        assert torch.equal(got[4], want[4])


def test_calls_of_two_threads_have_their_bits_every_time():
    """Two shapes from two host threads at once: every call's results, not the
    last one's alone."""
    import threading
    cases = [_case(900, 4, 2, 128, BF16, seed=1, offsets=[0, 300, 870], softcap=9.0),
             _case(650, 6, 3, 64, F16, seed=2, offsets=[20, 600], bias=True)]
    tokens = torch.randint(0, 40, (650,), generator=_gen(4), device="cuda")

    def run(c, kw):
        r = fadam.attention(c.q, c.k, c.v, **kw)
        d = fadam.attention_backward(r.out, c.q, c.k, c.v, r.out, r.lse, **kw)
        return (*r, *d, fadam.embedding_weight_grad(d.q[:650].flatten(1), tokens, 40))

    work = [(c, _options(c)) for c in cases]
    alone = [run(*w) for w in work]
    wrong = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in work]
    torch.cuda.synchronize()
    errors = []

    def body(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(150):
                    for a, b in zip(alone[i], run(*work[i])):
                        wrong[i] += (a.view(torch.uint8) != b.view(torch.uint8)).sum()
                stream.synchronize()
        except BaseException as e:      # reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=body, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    assert [int(w) for w in wrong] == [0, 0]
