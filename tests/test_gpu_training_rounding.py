"""Where the training operators' own rounding would show.  Each input makes
every other rounding exact or small, so that the bounds are those of the one
step that is looked at."""
import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    assert fadam.ops_status() == 0


# ---- loss and dz of confident rows at large logits --------------------------------------

def _confident(dtype, x0, step):
    """One row whose logits are x0 * 100 + d, all exact in fp32: d = 0 for the
    target, -8 step and less elsewhere."""
    V, D = 600, 64
    d = -8.0 * step - (torch.arange(V, device="cuda") % 64) * (step / 8)
    y = torch.tensor([317], device="cuda")
    d[317] = 0.0
    w = torch.zeros(V, D, dtype=dtype, device="cuda")
    w[:, 0], w[:, 1] = 100.0, d
    x = torch.zeros(1, D, dtype=dtype, device="cuda")
    x[0, 0], x[0, 1] = x0, 1.0
    assert torch.equal(w[:, 1].float(), d.float())
    return x, w, y, d.double()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("x0", [128.0, -128.0, 64.0, 1.0])
@pytest.mark.parametrize("step", [1.0, 0.5, 0.25])
def test_xent_confident_row_at_large_logits(dtype, x0, step):
    x, w, y, d = _confident(dtype, x0, step)
    gw = torch.empty(w.shape, dtype=F32, device="cuda")
    r = fadam.linear_cross_entropy(x, w, y, reduction="sum", grad_weight=gw)
    e = d.exp()
    e[317] = 0.0
    rest = e.sum()                            # of the exponentials beside the target's 1
    # an exponential of an exact difference: its argument times log2 e rounded
    # (|d| <= 16: 2^-20 relative), 2^-22 for the function; a piece's 32 additions to a
    # lane, 8 more, the row's 5, each half a unit of the sum; the logarithm's unit
    off = rest * 2.0 ** -19 + 48 * 2.0 ** -24 * (1 + rest)
    loss = torch.log1p(rest)
    assert abs(r.row_loss.double()[0] - loss) <= off
    assert abs(r.loss.double() - loss) <= off
    # dW of one row is dz times the row, and x0 is a power of two: dz itself
    dz = gw[:, 0].double() / x0
    p = d.exp() / (1 + rest)
    want = p.clone()
    want[317] -= 1.0
    far = (dz - want).abs()
    # kept in fp16 (2^-11, 2^-25 of the piece's largest), the row's sum, dz's own rounding
    limit = p * (2.0 ** -11 + 2.0 ** -18) + 2.0 ** -25 + U[dtype] * want.abs() + 2.0 ** -40
    limit[317] = off + 2.0 ** -24 + U[dtype] * want[317].abs() + 2.0 ** -40
    assert (far <= limit).all(), float((far / limit).max())
