"""The example's model as it was called before it had documents."""
import pytest
import torch

from tests.test_gpu_sequence import _gen, _no_wait_gave_up, _tokens  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_step_without_documents_is_one_of_a_single_document():
    from examples import train_step
    model = train_step.Model(vocab=90, width=128, hidden=200, blocks=2)
    g = _gen(5)
    tokens = _tokens(g, 90, 200)
    targets = torch.randint(0, 90, (200,), generator=g, device="cuda")
    loss = model.step(tokens, targets)
    grads = {n: t.clone() for n, t in model.grads.items()}
    whole = model.step(tokens, targets, torch.tensor([0, 200], dtype=torch.int32, device="cuda"))
    assert torch.equal(loss, whole)
    for name, grad in model.grads.items():
        assert torch.equal(grad, grads[name]), name
    model.step(tokens, targets, first=False)
