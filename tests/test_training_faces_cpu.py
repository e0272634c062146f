"""What the training operators' Python face says to shapes without elements."""
import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam


def test_norms_of_no_width_with_a_gate_are_refused():
    e, p = torch.zeros(4, 0, dtype=torch.bfloat16), torch.zeros(0, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fadam.block_norm(e, e, p, gate=torch.zeros(1, 0, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fadam.block_norm_backward(None, e, e, e, None, torch.zeros(4), p,
                                  gate=torch.zeros(1, 0, dtype=torch.bfloat16))
