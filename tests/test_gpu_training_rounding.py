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


# ---- long sums of one sign ---------------------------------------------------------------

# A chunk of a sum is at most 23 steps of 64 terms, 92 additions of 16 terms on the
# tensor cores, each of which may lose two units of the sum so far (the addends'
# alignment and the result's); the chunks are added in fp32, rounded to nearest.
def _sum_off(terms):
    return (2 * 92 + -(-terms // 768) / 2 + 2) * 2.0 ** -23


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_weight_grad_sums_long_columns(dtype):
    T, N, D = 40000, 1024, 4864             # 76 whole tiles: no split along the rows
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = (torch.rand(T, N, generator=g, device="cuda") + 0.5).to(dtype)
    # groups whose largest element is 127: scales of 1, whole numbers
    x = torch.randint(64, 127, (T, D), generator=g, device="cuda").to(dtype)
    x[:, ::128] = 127
    k = fadam.checkpoint8(x)
    assert torch.equal(k.codes, x.to(torch.int8))
    out = torch.empty(N, D, dtype=F32, device="cuda")
    fadam.checkpoint8_weight_grad(dy, k, out=out)
    want = dy.double().t() @ x.double()
    far = (out.double() - want).abs() / want
    assert far.max() <= _sum_off(T), float(far.max())


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_sums_long_columns(dtype):
    T, D, V = 16384, 4864, 1024             # dW: 76 whole tiles, 16384 rows
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.exp(2 * torch.randn(T, D, generator=g, device="cuda")).clamp(max=1000).to(dtype)
    w = torch.zeros(V, D, dtype=dtype, device="cuda")
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    gw = torch.empty(V, D, dtype=F32, device="cuda")
    fadam.linear_cross_entropy(x, w, y, reduction="sum", grad_weight=gw)
    # every probability is 2^-10: dz is exact
    want = x.double().sum(0) * 2.0 ** -10
    far = (gw[1:].double() - want).abs() / want
    assert far.max() <= _sum_off(T) + 2.0 ** -23, float(far.max())


def test_xent_sums_long_rows():
    T, D, V = 1024, 4864, 131072            # dx: 76 whole tiles, 131072 entries
    g = torch.Generator(device="cuda").manual_seed(3)
    size = torch.rand(D, generator=g, device="cuda") + 1.0
    w = (torch.rand(V, D, generator=g, device="cuda") * size).to(F16)
    w[0] = 0.0
    x = torch.zeros(T, D, dtype=F16, device="cuda")
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    r = fadam.linear_cross_entropy(x, w, y, reduction="sum")
    want = torch.stack([w[:, i:i + 256].double().mean(0) for i in range(0, D, 256)]).view(-1)
    far = (r.grad_x.double() - want) / want
    assert far.abs().max() <= U[F16] + _sum_off(V)
    # the outputs' own rounding, to nearest, averages out over the columns: 2^-11 in
    # 4864 independent ones, six standard deviations of a uniform error
    assert far[0].mean().abs() <= _sum_off(V) + 6 * 2.0 ** -11 / 3 ** 0.5 / D ** 0.5, float(far[0].mean())
    assert torch.equal(r.grad_x, r.grad_x[:1].expand_as(r.grad_x))


# ---- kept values beyond fp16's range -------------------------------------------------------

@pytest.mark.parametrize("kept", [BF16, F32])
@pytest.mark.parametrize("size", [1.0, 1e6, 1e30])
def test_weight_grad_of_wide_values_from_fp16(kept, size):
    T, N, D = 300, 130, 264
    g = torch.Generator(device="cuda").manual_seed(4)
    dy = (torch.randn(T, N, generator=g, device="cuda") * 1e-3).to(F16)
    x = (torch.randn(T, D, generator=g, device="cuda") * size).to(kept)
    k = fadam.checkpoint8(x)
    out = torch.empty(N, D, dtype=F32, device="cuda")
    fadam.checkpoint8_weight_grad(dy, k, out=out)
    v = k.codes.double() * k.scales.double().repeat_interleave(128, 1)[:, :D]
    each = dy.double().abs().t() @ v.abs()
    # values rounded to 11 bits (2^-25 of the largest below its 2^-14th), fp32 sums
    off = each * (2.0 ** -11 + T * 2.0 ** -23) + dy.double().abs().sum(0)[:, None] * v.abs().max() * 2.0 ** -24
    far = (out.double() - dy.double().t() @ v).abs()
    assert (far <= off).all(), float((far / off).max())
    # a group that is not finite is NaN, and only where it belongs
    k.scales[7, 1] = float("nan")
    fadam.checkpoint8_weight_grad(dy, k, out=out)
    assert torch.isnan(out[:, 128:256]).all() and torch.isfinite(out[:, :128]).all()
