"""The training operators on the GPU against their 64-bit forms, within bounds
derived from their roundings (tests/training_reference.py), at the sizes,
masks, layouts and values where they can go wrong."""
import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from tests import training_reference as ref

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


# ---- cross entropy ----------------------------------------------------------------

def _xent_case(T, D, V, dtype, seed=0, ignored=0.25):
    g = _gen(seed)
    w = (_rand(g, V, D) * (2.0 / D ** 0.5)).to(dtype)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = (_rand(g, T, D) + 2.0 * torch.rand(T, 1, generator=g, device="cuda") * w[y].float()).to(dtype)
    y = torch.where(torch.rand(T, generator=g, device="cuda") < ignored, -100, y)
    return x, w, y


def _check_xent(r, x, w, y, *, mean, ignore=-100, scale=1.0, base=None):
    bounds = ref.xent_bounds(x.double(), w.double(), y, x.dtype, mean=mean, ignore=ignore, scale=scale)
    for name in ("loss", "row_loss", "lse"):
        bounds[name].holds(getattr(r, name), name)
    if r.grad_x is not None:
        bounds["grad_x"].holds(r.grad_x, "grad_x")
        want = bounds["grad_w"]
        if base is not None:
            want = ref.Bounded(want.value + base.double(), want.off + 2.0 ** -23 * base.double().abs())
        want.holds(r.grad_weight, "grad_w")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,D,V", [
    (1, 8, 1), (1, 64, 7), (1, 512, 1000), (2, 72, 129), (3, 1, 5), (127, 130, 257), (128, 256, 128),
    (129, 64, 4096), (256, 1000, 999), (257, 72, 5003), (300, 520, 130), (700, 33, 777)])
def test_xent_sizes(T, D, V, dtype):
    x, w, y = _xent_case(T, D, V, dtype, seed=T + D + V)
    for mean in (True, False):
        r = fadam.linear_cross_entropy(x, w, y, reduction="mean" if mean else "sum")
        _check_xent(r, x, w, y, mean=mean)
    alone = fadam.linear_cross_entropy(x, w, y, reduction="sum", grads=False)
    assert alone.grad_x is None and alone.grad_weight is None
    for name in ("loss", "row_loss", "lse"):     # the same kernels, the same bits
        assert torch.equal(getattr(alone, name), getattr(r, name))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_many_tiles(dtype):
    x, w, y = _xent_case(1100, 192, 40007, dtype, seed=5, ignored=0.1)
    r = fadam.linear_cross_entropy(x, w, y)
    _check_xent(r, x, w, y, mean=True)
    again = fadam.linear_cross_entropy(x, w, y)
    for a, b in zip(r, again):
        assert torch.equal(a, b)


def test_xent_every_target_position():
    V = 300
    x, w, _ = _xent_case(V, 64, V, BF16, seed=3)
    y = torch.arange(V, device="cuda")
    _check_xent(fadam.linear_cross_entropy(x, w, y, reduction="sum"), x, w, y, mean=False)


@pytest.mark.parametrize("chunk", [1, 100, 256, 512])
@pytest.mark.parametrize("wide", [False, True])
def test_xent_chunks_of_rows(chunk, wide):
    x, w, y = _xent_case(600, 136, 1000, BF16, seed=9)
    if chunk == 1:
        x, y = x[:5].contiguous(), y[:5].contiguous()
    out = torch.empty(1000, 136, dtype=F32 if wide else BF16, device="cuda")
    r = fadam.linear_cross_entropy(x, w, y, chunk_rows=chunk, grad_weight=out)
    assert r.grad_weight is out
    _check_xent(r, x, w, y, mean=True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D", [64, 75])
def test_xent_accumulates(dtype, wide, D):
    x, w, y = _xent_case(200, D, 333, dtype, seed=11)
    base = _rand(_gen(4), 333, D).to(F32 if wide else dtype)
    for chunk in (0, 64):
        out = base.clone()
        r = fadam.linear_cross_entropy(x, w, y, grad_weight=out, accumulate=True, loss_scale=128.0,
                                       chunk_rows=chunk)
        _check_xent(r, x, w, y, mean=True, scale=128.0, base=base)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_strides_and_alignment(dtype):
    x0, w0, y = _xent_case(130, 96, 500, dtype, seed=2)

    def inside(t, rows, cols, r0, c0):
        big = torch.full((rows, cols), float("nan"), dtype=t.dtype, device="cuda")
        v = big[r0:r0 + t.shape[0], c0:c0 + t.shape[1]]
        v.copy_(t)
        return v, big

    for cols, c0 in ((128, 8), (128, 16), (101, 3), (99, 1)):   # bulk-readable rows, and not
        x, _ = inside(x0, 140, cols, 5, c0)
        w, _ = inside(w0, 510, cols, 2, c0)
        gw, big = inside(torch.zeros_like(w0), 520, cols, 4, c0)
        r = fadam.linear_cross_entropy(x, w, y, grad_weight=gw)
        _check_xent(r, x, w, y, mean=True)
        big[4:504, c0:c0 + 96] = float("nan")
        assert torch.isnan(big).all()      # nothing written around the view
    x3 = x0.view(2, 65, 96)
    r3 = fadam.linear_cross_entropy(x3, w0, y.view(2, 65))
    assert r3.grad_x.shape == x3.shape and r3.lse.shape == (2, 65)
    _check_xent(r3._replace(grad_x=r3.grad_x.view(130, 96), row_loss=r3.row_loss.view(-1),
                            lse=r3.lse.view(-1)), x0, w0, y, mean=True)


def test_xent_ignored_rows_have_no_influence():
    x, w, y = _xent_case(200, 64, 300, BF16, seed=6, ignored=0.5)
    clean = fadam.linear_cross_entropy(x, w, y)
    dirty = x.clone()
    dirty[(y == -100).nonzero()[::3, 0]] = float("nan")
    dirty[(y == -100).nonzero()[1::3, 0]] = float("inf")
    dirty[(y == -100).nonzero()[2::3, 0]] = torch.finfo(BF16).min
    r = fadam.linear_cross_entropy(dirty, w, y)
    for name in ("loss", "row_loss", "grad_x", "grad_weight"):
        assert torch.equal(getattr(clean, name), getattr(r, name)), name
    assert (r.grad_x[y == -100] == 0).all() and (r.row_loss[y == -100] == 0).all()


def test_xent_all_rows_ignored():
    x, w, y = _xent_case(70, 64, 300, F16, seed=6, ignored=2.0)
    for reduction in ("mean", "sum"):
        r = fadam.linear_cross_entropy(x, w, y, reduction=reduction)
        assert r.loss == 0 and (r.grad_x == 0).all() and (r.grad_weight == 0).all()


def test_xent_other_ignore_index():
    x, w, y = _xent_case(64, 64, 100, BF16, ignored=0.0)
    y[:20] = 7
    _check_xent(fadam.linear_cross_entropy(x, w, y, ignore_index=7), x, w, y, mean=True, ignore=7)


@pytest.mark.parametrize("target", [300, -1, 2 ** 40])
def test_xent_target_outside_the_vocabulary_is_nan(target):
    x, w, y = _xent_case(40, 64, 300, BF16, ignored=0.0)
    y[3] = target
    r = fadam.linear_cross_entropy(x, w, y)
    assert torch.isnan(r.loss) and torch.isnan(r.row_loss[3]) and torch.isnan(r.grad_x[3]).all()
    rest = torch.arange(40, device="cuda") != 3
    assert torch.isfinite(r.row_loss[rest]).all() and torch.isfinite(r.grad_x[rest]).all()
    assert torch.isnan(r.grad_weight).all()


def test_xent_rows_that_are_not_finite():
    x, w, y = _xent_case(40, 64, 300, BF16, ignored=0.0)
    x[5, 3], x[9, 0] = float("inf"), float("nan")
    r = fadam.linear_cross_entropy(x, w, y)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[5] = bad[9] = True
    assert torch.isnan(r.lse[bad]).all() and torch.isnan(r.grad_x[bad]).all()
    assert torch.isfinite(r.lse[~bad]).all() and torch.isfinite(r.grad_x[~bad]).all()


def test_xent_extreme_logits():
    """Logits of +-1000 and more: a target that is certain, one that is
    hopeless, and pieces of the vocabulary whose exponentials all vanish."""
    V, D = 600, 64
    w = torch.zeros(V, D, dtype=BF16, device="cuda")
    w[:, 0] = torch.linspace(-8, 8, V, device="cuda")
    x = torch.zeros(4, D, dtype=BF16, device="cuda")
    x[:, 0] = torch.tensor([200.0, -200.0, 0.0, 1.0], device="cuda")
    y = torch.tensor([V - 1, V - 1, 5, 9], device="cuda")
    r = fadam.linear_cross_entropy(x, w, y, reduction="sum")
    _check_xent(r, x, w, y, mean=False)
    assert r.row_loss[1] > 3000


def test_xent_no_rows():
    w = torch.ones(50, 16, dtype=BF16, device="cuda")
    x, y = w.new_empty(0, 16), torch.empty(0, dtype=torch.int64, device="cuda")
    r = fadam.linear_cross_entropy(x, w, y)
    assert r.loss == 0 and r.grad_x.shape == (0, 16) and (r.grad_weight == 0).all()
    out = torch.ones(50, 16, device="cuda")
    fadam.linear_cross_entropy(x, w, y, grad_weight=out, accumulate=True)
    assert (out == 1).all()


def test_xent_gradients_against_differences():
    """Directional differences of the 64-bit loss against the kernel's gradients."""
    x, w, y = _xent_case(60, 64, 200, F16, seed=8)
    r = fadam.linear_cross_entropy(x, w, y, reduction="sum")
    b = ref.xent_bounds(x.double(), w.double(), y, F16, mean=False)
    h, g = 1e-5, _gen(1)
    for at, grad, off, f in (
            (x, r.grad_x, b["grad_x"], lambda v: ref.xent(v, w.double(), y, mean=False).loss),
            (w, r.grad_weight, b["grad_w"], lambda v: ref.xent(x.double(), v, y, mean=False).loss)):
        d = torch.randn(at.shape, generator=g, device="cuda", dtype=torch.float64)
        slope = (f(at.double() + h * d) - f(at.double() - h * d)) / (2 * h)
        limit = ((off.off + off.value.abs() * ref.U[F16]) * d.abs()).sum() + 1e-6 * slope.abs()
        assert abs(slope - (grad.double() * d).sum()) <= limit


# ---- 8-bit checkpoints ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,D", [(1, 1), (1, 128), (3, 127), (2, 129), (5, 8), (40, 1000), (7, 4096),
                                 (4, 5000), (33, 1005), (6000, 264), (2000, 2048)])
def test_checkpoint_codes_and_values(T, D, dtype):
    g = _gen(T * D)
    x = (_rand(g, T, D) * torch.exp(2 * _rand(g, T, D))).to(dtype)
    k = fadam.checkpoint8(x)
    q, s = ref.codes(x)
    assert torch.equal(k.codes.cpu(), q) and torch.equal(k.scales.cpu(), s)
    back = fadam.checkpoint8_restore(k)
    v = ref.values(k.codes, k.scales)
    assert back.dtype == dtype and torch.equal(back, v.float().to(dtype))
    top = ref.groups_of(x.double()).abs().amax(2).repeat_interleave(128, 1)[:, :D]
    assert ((v - x.double()).abs() <= top / 254 + top * 2.0 ** -23).all()     # the header's bound


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("D", [512, 511])
def test_checkpoint_special_values(D, dtype):
    x = torch.zeros(9, D, dtype=dtype, device="cuda")
    x[1, :128] = 1.0
    x[2, 5] = float("inf")
    x[3, 130] = float("nan")
    x[4, 300] = float("-inf")
    x[5] = torch.finfo(dtype).max
    x[6] = -torch.finfo(dtype).max
    x[6, 0] = torch.finfo(dtype).max
    if dtype != F16:
        x[7] = 2.0 ** -101          # too small to be kept
        x[8] = 2.0 ** -100
    x[7, 200] = -0.0
    k = fadam.checkpoint8(x)
    q, s = ref.codes(x)
    assert torch.equal(torch.isnan(k.scales.cpu()), torch.isnan(s))
    fine = ~torch.isnan(s)
    assert torch.equal(k.scales.cpu()[fine], s[fine])
    back = fadam.checkpoint8_restore(k)
    groups = torch.isnan(s).repeat_interleave(128, 1)[:, :D].cuda()
    assert torch.isnan(back[groups]).all() and torch.isfinite(back[~groups]).all()
    # a group's largest element is off by the rounding of its scale alone
    for row in (1, 5, 6):
        if dtype == F32:
            assert ((back[row].double() - x[row].double()).abs() <= 2.0 ** -23 * x[row].double().abs()).all()
        else:
            assert torch.equal(back[row], x[row])
    assert (back[0] == 0).all()


@pytest.mark.parametrize("c0,cols", [(8, 80), (3, 80), (1, 77)])
def test_checkpoint_strided_rows(c0, cols):
    big = torch.full((50, cols), float("nan"), dtype=BF16, device="cuda")
    x = big[4:44, c0:c0 + 64]
    x.copy_(_rand(_gen(1), 40, 64))
    k = fadam.checkpoint8(x)
    q, s = ref.codes(x)
    assert torch.equal(k.codes.cpu(), q) and torch.equal(k.scales.cpu(), s)
    t = _rand(_gen(2), 3, 8, 2, 64)[:, :, 1]        # evenly strided leading dimensions
    assert torch.equal(fadam.checkpoint8(t).codes, fadam.checkpoint8(t.contiguous()).codes)


def _check_wgrad(out, dy, k, base=None):
    x = ref.values(k.codes.view(-1, k.codes.shape[-1]), k.scales.view(-1, k.scales.shape[-1]))
    dy = dy.reshape(-1, dy.shape[-1])
    size = dy.double().abs().t() @ x.abs()
    want = dy.double().t() @ x
    off = size * (ref.U[dy.dtype] + dy.shape[0] * 2.0 ** -23)
    if base is not None:
        want, off = want + base.double(), off + 2.0 ** -23 * base.double().abs()
    ref.Bounded(want, off).holds(out, "grad_w")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,N,D", [(1, 1, 1), (1, 8, 128), (16, 33, 100), (64, 256, 256), (65, 257, 300),
                                   (777, 130, 514), (1500, 64, 72), (3000, 300, 264)])
def test_weight_grad(T, N, D, dtype):
    g = _gen(T + N + D)
    dy = _rand(g, T, N).to(dtype)
    k = fadam.checkpoint8(_rand(g, T, D).to(dtype))
    out = fadam.checkpoint8_weight_grad(dy, k)
    _check_wgrad(out, dy, k)
    assert torch.equal(out, fadam.checkpoint8_weight_grad(dy, k))
    wide = torch.empty(N, D, dtype=F32, device="cuda")
    _check_wgrad(fadam.checkpoint8_weight_grad(dy, k, out=wide), dy, k)
    for base in (_rand(g, N, D), _rand(g, N, D).to(dtype)):
        acc = base.clone()
        fadam.checkpoint8_weight_grad(dy, k, out=acc, accumulate=True)
        _check_wgrad(acc, dy, k, base)


def test_weight_grad_strides_and_leading_dimensions():
    g = _gen(0)
    big = torch.full((70, 130), float("nan"), dtype=BF16, device="cuda")
    for c0 in (8, 1):
        dy = big[3:67, c0:c0 + 96]
        dy.copy_(_rand(g, 64, 96))
        k = fadam.checkpoint8(_rand(g, 64, 200).to(BF16))
        room = torch.full((100, 203), float("nan"), device="cuda")
        out = room[2:98, 2:202]
        _check_wgrad(fadam.checkpoint8_weight_grad(dy, k, out=out), dy, k)
        out.fill_(float("nan"))
        assert torch.isnan(room).all()
    dy3, x3 = _rand(g, 2, 32, 96).to(BF16), _rand(g, 2, 32, 200).to(BF16)
    k = fadam.checkpoint8(x3)
    _check_wgrad(fadam.checkpoint8_weight_grad(dy3, k), dy3, k)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,N,D", [(64, 512, 512), (200, 2304, 2064), (1, 300, 4096), (4097, 1000, 1040),
                                   (1027, 4096, 4112), (2500, 8192, 256), (9000, 257, 400), (640, 256, 16)])
def test_weight_grad_takes_codes_wherever_they_lie(T, N, D, dtype):
    """The codes' alignment decides how they are read, not what is computed."""
    g = _gen(T + N)
    dy = _rand(g, T, N).to(dtype)
    k = fadam.checkpoint8(_rand(g, T, D).to(dtype))
    k.scales[T // 2] *= 37.5
    moved = torch.empty(T * D + 1, dtype=torch.int8, device="cuda")[1:].view(T, D)
    moved.copy_(k.codes)
    other = k._replace(codes=moved)
    for out in (dtype, F32):
        a, b = (torch.empty(N, D, dtype=out, device="cuda") for _ in range(2))
        fadam.checkpoint8_weight_grad(dy, k, out=a)
        fadam.checkpoint8_weight_grad(dy, other, out=b)
        assert torch.equal(a, b)
    _check_wgrad(a, dy, k)


def test_weight_grad_no_rows():
    k = fadam.checkpoint8(torch.empty(0, 24, dtype=BF16, device="cuda"))
    dy = torch.empty(0, 16, dtype=BF16, device="cuda")
    assert (fadam.checkpoint8_weight_grad(dy, k) == 0).all()
    out = torch.ones(16, 24, device="cuda")
    assert (fadam.checkpoint8_weight_grad(dy, k, out=out, accumulate=True) == 1).all()


# ---- block norms --------------------------------------------------------------------------

def _norm_case(rows, D, block, residual, params, post, gates, seed=0):
    g = _gen(seed)
    c = torch.exp(0.5 * _rand(g, D))
    a = {"f": (_rand(g, rows, D) * c).to(block), "h": (_rand(g, rows, D) * 2 * c.flip(0)).to(residual),
         "pre": (1 + 0.2 * _rand(g, D)).to(params),
         "post": (1 + 0.2 * _rand(g, D)).to(params) if post else None,
         "gate": (0.5 + 0.3 * _rand(g, gates, D)).to(params) if gates else None}
    a["gh"], a["gx"] = _rand(g, rows, D).to(residual), _rand(g, rows, D).to(block)
    return a


def _d(t):
    return None if t is None else t.double()


def _check_norm(a, alpha=0.7, eps=1e-5, kept=False):
    n = fadam.block_norm(a["f"], a["h"], a["pre"], post_weight=a["post"], gate=a["gate"],
                         residual_scale=alpha, eps=eps, checkpoint=kept)
    D = a["f"].shape[-1]
    want = ref.block_norm_bounds(_d(a["f"]).reshape(-1, D), _d(a["h"]).reshape(-1, D), _d(a["pre"]),
                                 _d(a["post"]), _d(a["gate"]), alpha, eps)
    for name, got in (("h_out", n.h_out), ("x_out", n.x_out), ("r2", n.rstd_pre), ("r1", n.rstd_post)):
        if got is not None:
            want[name].holds(got.reshape(want[name].value.shape), name)
    if kept:
        for k, t in ((n.f_checkpoint, a["f"]), (n.h_checkpoint, n.h_out)):
            q, s = ref.codes(t.reshape(-1, D))
            assert torch.equal(k.codes.cpu().view(-1, D), q) and torch.equal(k.scales.cpu().view(s.shape), s)
    return n


def _check_norm_grad(a, n, f, h_out, f64, h64, alpha=0.7, with_gh=True):
    D = a["f"].shape[-1]
    gh = a["gh"] if with_gh else None
    g = fadam.block_norm_backward(gh, a["gx"], f, h_out, n.rstd_post, n.rstd_pre, a["pre"],
                                  post_weight=a["post"], gate=a["gate"], residual_scale=alpha)
    gx = _d(a["gx"]).reshape(-1, D)
    want = ref.block_norm_grad(torch.zeros_like(gx) if gh is None else _d(gh).reshape(-1, D), gx, f64, h64,
                               None if n.rstd_post is None else _d(n.rstd_post).reshape(-1),
                               _d(n.rstd_pre).reshape(-1), _d(a["pre"]), _d(a["post"]), _d(a["gate"]), alpha)
    for name, got in (("h", g.h), ("f", g.f), ("pre", g.pre_weight), ("post", g.post_weight), ("gate", g.gate)):
        assert (got is not None) == (name in want)
        if got is not None:
            want[name].holds(got.reshape(want[name].value.shape), name)
    return g


NORM_TYPES = [(BF16, BF16, BF16), (BF16, F32, F32), (F16, F16, F32), (F16, F32, F16), (F32, F32, F32)]


@pytest.mark.parametrize("block,residual,params", NORM_TYPES)
@pytest.mark.parametrize("rows,D,post,gates", [
    (1, 1, True, 1), (1, 8, True, 0), (3, 40, False, 3), (6, 128, True, 2), (5, 513, True, 1),
    (12, 1000, True, 4), (9, 1005, False, 1), (700, 256, True, 1), (2500, 128, True, 5),
    (1, 4096, True, 1), (40, 4096, True, 40), (330, 4096, True, 0), (10, 5000, True, 1),
    (400, 8192, True, 1), (6, 8200, True, 2), (3, 16384, True, 1), (4, 12345, False, 1)])
def test_block_norm(rows, D, post, gates, block, residual, params):
    a = _norm_case(rows, D, block, residual, params, post, gates, seed=rows + D)
    n = _check_norm(a, kept=True)
    plain = _check_norm(a)
    for name in ("h_out", "x_out", "rstd_pre"):
        assert torch.equal(getattr(n, name), getattr(plain, name))
    _check_norm_grad(a, n, a["f"], n.h_out, a["f"].double(), n.h_out.double())
    _check_norm_grad(a, n, n.f_checkpoint, n.h_checkpoint, ref.values(*n.f_checkpoint[:2]),
                     ref.values(*n.h_checkpoint[:2]))
    g = _check_norm_grad(a, n, a["f"], n.h_checkpoint, a["f"].double(), ref.values(*n.h_checkpoint[:2]),
                         with_gh=False)
    again = fadam.block_norm_backward(None, a["gx"], a["f"], n.h_checkpoint, n.rstd_post, n.rstd_pre,
                                      a["pre"], post_weight=a["post"], gate=a["gate"], residual_scale=0.7)
    for x, y in zip(g, again):
        assert x is None and y is None or torch.equal(x, y)


def test_block_norm_strides_and_alignment():
    D = 64
    for c0, cols in ((8, 96), (3, 96), (1, 77)):
        a = _norm_case(30, D, BF16, F32, BF16, True, 3)
        for name in ("f", "h", "gh", "gx"):
            big = torch.full((40, cols), float("nan"), dtype=a[name].dtype, device="cuda")
            v = big[2:32, c0:c0 + D]
            v.copy_(a[name])
            a[name] = v
        n = _check_norm(a, kept=True)
        assert n.h_out.is_contiguous() and n.x_out.is_contiguous()
        _check_norm_grad(a, n, a["f"], n.h_out, a["f"].double(), n.h_out.double())
    w = torch.ones(D + 1, dtype=BF16, device="cuda")[1:]      # parameters off 16 bytes
    a = _norm_case(30, D, BF16, BF16, BF16, True, 1)
    a["pre"] = w
    n = _check_norm(a)
    _check_norm_grad(a, n, a["f"], n.h_out, a["f"].double(), n.h_out.double())


def test_block_norm_leading_dimensions_and_sequences():
    a = _norm_case(24, 96, BF16, BF16, BF16, True, 4)
    a3 = {k: v.view(4, 6, 96) if k in ("f", "h", "gh", "gx") else v for k, v in a.items()}
    n3, n = _check_norm(a3, kept=True), _check_norm(a, kept=True)
    assert n3.h_out.shape == (4, 6, 96) and n3.rstd_pre.shape == (4, 6)
    assert torch.equal(n3.x_out.view(24, 96), n.x_out)
    g3 = _check_norm_grad(a3, n3, a3["f"], n3.h_out, a["f"].double(), n.h_out.double())
    assert g3.f.shape == (4, 6, 96) and g3.gate.shape == (4, 96)


def test_block_norm_zero_and_non_finite_rows():
    a = _norm_case(8, 256, BF16, BF16, BF16, True, 1)
    a["f"][1], a["h"][1] = 0, 0                     # an empty row: only eps under the root
    n = _check_norm(a)
    assert (n.x_out[1] == 0).all()
    _check_norm_grad(a, n, a["f"], n.h_out, a["f"].double(), n.h_out.double())
    a["f"][3, 7], a["h"][5, 2] = float("nan"), float("inf")
    n = fadam.block_norm(a["f"], a["h"], a["pre"], post_weight=a["post"], gate=a["gate"])
    bad = torch.zeros(8, dtype=torch.bool, device="cuda")
    bad[3] = bad[5] = True
    assert torch.isfinite(n.x_out[~bad]).all() and torch.isnan(n.x_out[3]).all()
    assert torch.isnan(n.x_out[5, 2])


def test_block_norm_no_rows():
    a = _norm_case(4, 64, BF16, BF16, F32, True, 1)
    e = a["f"][:0]
    n = fadam.block_norm(e, e, a["pre"], post_weight=a["post"], gate=a["gate"], checkpoint=True)
    g = fadam.block_norm_backward(e, e, n.f_checkpoint, n.h_out, n.rstd_post, n.rstd_pre, a["pre"],
                                  post_weight=a["post"], gate=a["gate"])
    assert g.f.shape == (0, 64) and all((t == 0).all() for t in (g.pre_weight, g.post_weight, g.gate))


def test_block_norm_gradients_against_differences():
    a = _norm_case(6, 72, F32, F32, F32, True, 2, seed=3)
    n = _check_norm(a, eps=1e-3)
    g = _check_norm_grad(a, n, a["f"], n.h_out, a["f"].double(), n.h_out.double())
    d64 = {k: _d(v) for k, v in a.items()}

    def value(**kw):
        c = {k: d64[k] for k in ("f", "h", "pre", "post", "gate")} | kw
        r = ref.block_norm(c["f"], c["h"], c["pre"], c["post"], c["gate"], 0.7, 1e-3)
        return (r.h_out * d64["gh"]).sum() + (r.x_out * d64["gx"]).sum()

    gen, h = _gen(7), 1e-6
    for name, grad in (("f", g.f), ("h", g.h), ("pre", g.pre_weight), ("post", g.post_weight), ("gate", g.gate)):
        d = torch.randn(d64[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        slope = (value(**{name: d64[name] + h * d}) - value(**{name: d64[name] - h * d})) / (2 * h)
        # fp32 gradients, each within 10^-4 of its largest term
        limit = 1e-4 * (grad.double().abs() * d.abs()).sum()
        assert abs(slope - (grad.double() * d).sum()) <= limit, name


# ---- how they are called ----------------------------------------------------------------------

def _step(x, w, y, f, h, pre, k, dy):
    r = fadam.linear_cross_entropy(x, w, y)
    n = fadam.block_norm(f, h, pre, post_weight=pre, checkpoint=True)
    g = fadam.block_norm_backward(h, f, n.f_checkpoint, n.h_out, n.rstd_post, n.rstd_pre, pre, post_weight=pre)
    return [r.loss, r.grad_x, r.grad_weight, n.h_out, n.x_out, g.f, g.h, g.pre_weight, g.post_weight,
            fadam.checkpoint8_weight_grad(dy, k), fadam.checkpoint8_restore(k)]


def _step_inputs(seed):
    x, w, y = _xent_case(300, 72, 700, BF16, seed=seed)
    a = _norm_case(400, 256, BF16, BF16, BF16, False, 0, seed=seed)
    k = fadam.checkpoint8(a["f"])
    return x, w, y, a["f"], a["h"], a["pre"], k, _rand(_gen(seed + 1), 400, 64).to(BF16)


def test_side_stream_gives_the_same():
    args = _step_inputs(1)
    want = _step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _step(*args)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_replays_with_new_inputs():
    args, other = _step_inputs(2), _step_inputs(3)
    _step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(*args)
    want = [t.clone() for t in _step(*other)]
    for to, src in zip(args, other):
        if isinstance(to, fadam.Checkpoint8):
            to.codes.copy_(src.codes)
            to.scales.copy_(src.scales)
        else:
            to.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_the_first_call_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    code = """
import torch
import adamw_optimizer_step_persistent_gb300 as fadam
x = torch.randn(300, 72, device="cuda").bfloat16()
w = torch.randn(500, 72, device="cuda").bfloat16()
y = torch.randint(0, 500, (300,), device="cuda")
p = torch.ones(72, device="cuda").bfloat16()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    r = fadam.linear_cross_entropy(x, w, y)
    n = fadam.block_norm(x, x, p, post_weight=p, checkpoint=True)
    g = fadam.block_norm_backward(x, x, n.f_checkpoint, n.h_out, n.rstd_post, n.rstd_pre, p, post_weight=p)
    d = fadam.checkpoint8_weight_grad(x, n.f_checkpoint)
graph.replay()
torch.cuda.synchronize()
s = fadam.linear_cross_entropy(x, w, y)
assert torch.equal(r.loss, s.loss) and torch.equal(r.grad_weight, s.grad_weight)
assert torch.equal(d, fadam.checkpoint8_weight_grad(x, fadam.checkpoint8(x)))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=240,
                   env=dict(os.environ, PYTHONPATH=root))


# ---- offsets beyond 32 bits -----------------------------------------------------------------------

def test_xent_beyond_2_to_the_31_logits():
    T, D, V = 33000, 64, 70001
    x, w, y = _xent_case(T, D, V, BF16, seed=13, ignored=0.1)
    r = fadam.linear_cross_entropy(x, w, y, reduction="sum")
    at = torch.cat([torch.arange(0, T, 997, device="cuda"), torch.arange(T - 40, T, device="cuda")])
    b = ref.xent_bounds(x[at].double(), w.double(), y[at], BF16, mean=False)
    b["lse"].holds(r.lse[at], "lse")
    b["row_loss"].holds(r.row_loss[at], "row_loss")
    b["grad_x"].holds(r.grad_x[at], "grad_x")
    # dW of some entries of the vocabulary, over all rows
    cols = torch.cat([torch.arange(0, V, 1501, device="cuda"), torch.arange(V - 20, V, device="cuda")])
    p = (x.double() @ w[cols].double().t() - r.lse.double()[:, None]).exp()
    p -= (y[:, None] == cols).double()
    p[y == -100] = 0
    size = p.abs().t() @ x.double().abs()
    # one rounding of dz, one of the kept exponential, the logits' and the sums' in fp32
    off = size * (ref.U[BF16] + 2.0 ** -11 + 2.0 ** -14) + 2.0 ** -25 * x.double().abs().sum(0) \
        + T * ref.E32 * size
    ref.Bounded(p.t() @ x.double(), off).holds(r.grad_weight[cols], "grad_w")


def test_checkpoint_beyond_2_to_the_31_elements():
    T, D = 270000, 8192
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    x[::9001] = _rand(_gen(1), len(range(0, T, 9001)), D).to(BF16)
    x[-3:] = _rand(_gen(2), 3, D).to(BF16)
    k = fadam.checkpoint8(x)
    back = fadam.checkpoint8_restore(k)
    for at in (slice(0, T, 9001), slice(T - 4, T)):
        q, s = ref.codes(x[at])
        assert torch.equal(k.codes[at].cpu(), q) and torch.equal(k.scales[at].cpu(), s)
        assert torch.equal(back[at], ref.values(k.codes[at], k.scales[at]).float().to(BF16))


@pytest.mark.parametrize("D", [8192, 8191])
def test_block_norm_beyond_2_to_the_31_elements(D):
    T = 264000
    g = _gen(3)
    f = torch.zeros(T, D, dtype=BF16, device="cuda")
    at = torch.cat([torch.arange(0, T, 8999, device="cuda"), torch.arange(T - 3, T, device="cuda")])
    f[at] = _rand(g, len(at), D).to(BF16)
    w = (1 + 0.2 * _rand(g, D)).to(BF16)
    n = fadam.block_norm(f, f, w, post_weight=w, checkpoint=True)
    a = {"f": f[at], "h": f[at], "pre": w, "post": w, "gate": None}
    want = ref.block_norm_bounds(_d(a["f"]), _d(a["h"]), _d(w), _d(w), None, 1.0, 1e-6)
    want["h_out"].holds(n.h_out[at], "h_out")
    want["x_out"].holds(n.x_out[at], "x_out")
    q, s = ref.codes(n.h_out[at])
    assert torch.equal(n.h_checkpoint.codes[at].cpu(), q) and torch.equal(n.h_checkpoint.scales[at].cpu(), s)
    d = fadam.block_norm_backward(f, f, f, n.h_out, n.rstd_post, n.rstd_pre, w, post_weight=w)
    grad = ref.block_norm_grad(_d(f[at]), _d(f[at]), _d(f[at]), _d(n.h_out[at]), _d(n.rstd_post[at]),
                               _d(n.rstd_pre[at]), _d(w), _d(w), None, 1.0)
    grad["h"].holds(d.h[at], "h")
    grad["f"].holds(d.f[at], "f")
    # every other row is zero and adds nothing
    ref.Bounded(grad["pre"].value, grad["pre"].off * (1 + T / len(at))).holds(d.pre_weight, "pre")


def test_gradients_land_in_the_optimizer_shard():
    """The example: a model trained through all of the operators."""
    from examples import train_step
    losses = train_step.main(["--steps", "25", "--rows", "512"])
    assert losses[0] > 6.0 and losses[-1] < 0.7 * losses[0]


def test_block_norm_in_place_on_the_residual_stream():
    """h_out may be h (C ABI): the same bits as out of place."""
    import ctypes

    from adamw_optimizer_step_persistent_gb300 import _abi
    for rows, D in ((700, 256), (700, 255), (3, 256)):
        a = _norm_case(rows, D, BF16, F32, BF16, True, 1)
        n = fadam.block_norm(a["f"], a["h"], a["pre"], post_weight=a["post"], gate=a["gate"], checkpoint=True)
        h, x = a["h"].clone(), torch.empty_like(a["f"])
        r1, r2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        k = fadam.checkpoint8(a["h"])
        d = _abi.BlockNorm(f=a["f"].data_ptr(), h=h.data_ptr(), post_weight=a["post"].data_ptr(),
                           pre_weight=a["pre"].data_ptr(), gate=a["gate"].data_ptr(), h_out=h.data_ptr(),
                           x_out=x.data_ptr(), rstd_post=r1.data_ptr(), rstd_pre=r2.data_ptr(),
                           h_kept=_abi.Kept8(k.codes.data_ptr(), k.scales.data_ptr()), rows=rows, width=D,
                           gate_rows=1, f_stride=D, h_stride=D, residual_scale=1.0, eps=1e-6,
                           block_dtype=_abi.DT_BF16, residual_dtype=_abi.DT_F32, param_dtype=_abi.DT_BF16)
        stream = torch.cuda.current_stream().cuda_stream
        assert _abi.lib().fadam_block_norm_forward(ctypes.byref(d), stream) == _abi.OK
        torch.cuda.synchronize()
        assert torch.equal(h, n.h_out) and torch.equal(x, n.x_out) and torch.equal(r2, n.rstd_pre)
        assert torch.equal(k.codes, n.h_checkpoint.codes) and torch.equal(k.scales, n.h_checkpoint.scales)
