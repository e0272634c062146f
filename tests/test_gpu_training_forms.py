"""Forms of the training operators whose kernels take other turns than at the
usual sizes: more gate rows than CTAs, rows beyond 8192 columns with several to
a CTA, logits of several chunks with several tiles to a pair of CTAs, one
gradient without the other."""
import ctypes

import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from adamw_optimizer_step_persistent_gb300 import _abi
from tests import training_reference as ref
from tests.test_gpu_training import _check_norm, _check_norm_grad, _check_xent, _norm_case, _xent_case

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    assert fadam.ops_status() == 0


def _both_ways(a):
    n = _check_norm(a, kept=True)
    _check_norm_grad(a, n, a["f"], n.h_out, a["f"].double(), n.h_out.double())
    g = _check_norm_grad(a, n, n.f_checkpoint, n.h_checkpoint, ref.values(*n.f_checkpoint[:2]),
                         ref.values(*n.h_checkpoint[:2]))
    again = fadam.block_norm_backward(a["gh"], a["gx"], n.f_checkpoint, n.h_checkpoint, n.rstd_post,
                                      n.rstd_pre, a["pre"], post_weight=a["post"], gate=a["gate"],
                                      residual_scale=0.7)
    for x, y in zip(g, again):
        assert x is None and y is None or torch.equal(x, y)


@pytest.mark.parametrize("block,residual,params", [(BF16, BF16, BF16), (F16, F32, F16), (F32, F32, F32)])
@pytest.mark.parametrize("rows,D,post,gates", [
    (6000, 128, True, 2000), (3000, 128, False, 3000),     # 1216 CTAs at most
    (1400, 4096, True, 700), (700, 4096, True, 700),       # 304
    (4000, 1005, True, 2000), (2600, 520, True, 1300)])
def test_more_gate_rows_than_ctas(rows, D, post, gates, block, residual, params):
    _both_ways(_norm_case(rows, D, block, residual, params, post, gates, seed=rows))


@pytest.mark.parametrize("block,residual,params", [(BF16, BF16, BF16), (F16, F32, F16), (F32, F32, F32)])
@pytest.mark.parametrize("rows,D,post,gates", [
    (700, 8200, True, 1), (600, 16384, True, 2), (500, 12345, False, 1), (400, 10000, True, 200),
    (700, 5120, True, 1), (650, 7168, True, 5)])
def test_wide_rows_with_several_to_a_cta(rows, D, post, gates, block, residual, params):
    _both_ways(_norm_case(rows, D, block, residual, params, post, gates, seed=D))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,D,V", [(700, 2112, 20011), (1300, 4104, 7001), (300, 1600, 50021)])
def test_xent_several_chunks_and_several_tiles(T, D, V, dtype):
    x, w, y = _xent_case(T, D, V, dtype, seed=T)
    r = fadam.linear_cross_entropy(x, w, y)
    _check_xent(r, x, w, y, mean=True)
    again = fadam.linear_cross_entropy(x, w, y)
    for a, b in zip(r, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T", [1, 300])
def test_xent_logits_are_summed_in_chunks(T, dtype):
    """Products of one sign: the tensor cores' additions would lose some 10^-4 in
    2048 of them; a chunk has 64, each two units of its sum at most."""
    D, V = 32768, 600
    g = torch.Generator(device="cuda").manual_seed(T)
    x = (torch.rand(T, D, generator=g, device="cuda") + 0.5).to(dtype)
    w = (torch.rand(V, D, generator=g, device="cuda") + 0.5).to(dtype)
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    r = fadam.linear_cross_entropy(x, w, y, grads=False)
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    chunk = 1024 if T > 256 else 256
    off = (2 * chunk / 16 + D / chunk / 2 + 4) * 2.0 ** -23 * z.max()
    assert (r.lse.double() - lse).abs().max() <= off, float(((r.lse.double() - lse).abs() / off).max())


@pytest.mark.parametrize("chunk", [0, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_xent_one_gradient_without_the_other(dtype, chunk):
    T, D, V = 300, 136, 1000
    x, w, y = _xent_case(T, D, V, dtype, seed=9)
    want = fadam.linear_cross_entropy(x, w, y, reduction="sum", chunk_rows=chunk)
    code = _abi.DT_BF16 if dtype is BF16 else _abi.DT_F16
    L, stream = _abi.lib(), torch.cuda.current_stream().cuda_stream
    for wants_x in (True, False):
        loss, rows, lse = torch.empty(1, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        out = torch.empty_like(x if wants_x else w)
        d = _abi.Xent(x=x.data_ptr(), w=w.data_ptr(), targets=y.data_ptr(), loss=loss.data_ptr(),
                      row_loss=rows.data_ptr(), lse=lse.data_ptr(),
                      grad_x=out.data_ptr() if wants_x else None, grad_w=None if wants_x else out.data_ptr(),
                      rows=T, width=D, vocab=V, x_stride=D, w_stride=D, grad_x_stride=D, grad_w_stride=D,
                      ignore_index=-100, chunk_rows=chunk, loss_scale=1.0, dtype=code, grad_w_dtype=code, flags=0)
        need = ctypes.c_size_t()
        assert L.fadam_xent_workspace(d, need) == _abi.OK
        ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        assert L.fadam_xent_run(d, ws.data_ptr(), need.value, stream) == _abi.OK
        assert torch.equal(out, want.grad_x if wants_x else want.grad_weight)
        assert torch.equal(loss[0], want.loss) and torch.equal(rows, want.row_loss) and torch.equal(lse, want.lse)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,cols,c0", [(96, 128, 8), (96, 101, 3), (203, 216, 8), (520, 520, 0), (333, 333, 0)])
def test_gradients_added_to_a_view(D, cols, c0, dtype, wide):
    """The view's elements are added to, and nothing around it is touched."""
    g = torch.Generator(device="cuda").manual_seed(D)
    for N in (300, 40):
        base = torch.randn(N + 9, cols, generator=g, device="cuda").to(F32 if wide else dtype)
        x, w, y = _xent_case(150, D, N, dtype, seed=D)
        k = fadam.checkpoint8(x)
        dy = torch.randn(150, N, generator=g, device="cuda").to(dtype)
        for chunk in (0, 64, None):
            room = base.clone()
            view = room[4:4 + N, c0:c0 + D]
            old = view.clone()
            if chunk is None:
                fadam.checkpoint8_weight_grad(dy, k, out=view, accumulate=True)
                v = ref.values(*k[:2])
                want, off = dy.double().t() @ v, dy.double().abs().t() @ v.abs() * (ref.U[dtype] + 150 * ref.E32)
                ref.Bounded(want + old.double(), off + ref.E32 * old.double().abs()).holds(view, "out")
            else:
                r = fadam.linear_cross_entropy(x, w, y, grad_weight=view, accumulate=True, chunk_rows=chunk)
                _check_xent(r, x, w, y, mean=True, base=old)
            view.copy_(old)
            assert torch.equal(room, base)
