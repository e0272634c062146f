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
