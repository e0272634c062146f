"""Checks of the training operators that need no GPU.

* the library exports what include/fadam_ops.h declares, and the ctypes
  structures lie in memory as the C ones do;
* every host-side argument check returns its status before any CUDA call and
  leaves a message; the Python face raises on what it does not take;
* the gradients' formulas against differences of the functions themselves.
"""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from adamw_optimizer_step_persistent_gb300 import _abi
from tests import training_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fadam_ops.h")
L = _abi.lib()
FAKE = 0x7F0000000000  # never dereferenced: the checks fail before any use

STRUCTS = {"fadam_xent": _abi.Xent, "fadam_checkpoint8": _abi.Kept8, "fadam_wgrad": _abi.Wgrad,
           "fadam_block_norm": _abi.BlockNorm, "fadam_block_norm_grad": _abi.BlockNormGrad}


def test_library_exports_every_declared_function():
    names = re.findall(r"^(?:fadam_status|const char\*)\s+(fadam_\w+)\(", open(HEADER).read(), re.M)
    assert len(names) == 11
    assert {n for n, _, _ in _abi.OPS_SIGNATURES} == set(names)
    assert all(hasattr(L, n) for n in names)


def test_structures_match_the_header(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "fadam_ops.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0; }\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    want = dict(l.split() for l in subprocess.run([exe], check=True, capture_output=True,
                                                  text=True).stdout.splitlines())
    for name, cls in STRUCTS.items():
        assert int(want[name]) == ctypes.sizeof(cls)
        for field, *_ in cls._fields_:
            assert int(want[f"{name}.{field}"]) == getattr(cls, field).offset, (name, field)


# ---- refusals of the C ABI -----------------------------------------------------------------

def _xent(**kw):
    d = dict(x=FAKE, w=FAKE, targets=FAKE, loss=FAKE, row_loss=FAKE, lse=FAKE, grad_x=FAKE,
             grad_w=FAKE, rows=4, width=64, vocab=100, x_stride=64, w_stride=64, grad_x_stride=64,
             grad_w_stride=64, ignore_index=-100, chunk_rows=0, loss_scale=1.0, dtype=_abi.DT_BF16,
             grad_w_dtype=_abi.DT_BF16, flags=0)
    return _abi.Xent(**(d | kw))


@pytest.mark.parametrize("change,want", [
    ({"dtype": _abi.DT_F32}, _abi.EDTYPE), ({"dtype": 7}, _abi.EDTYPE),
    ({"grad_w_dtype": _abi.DT_F16}, _abi.EDTYPE), ({"flags": 4}, _abi.EINVAL),
    ({"rows": -1}, _abi.EINVAL), ({"width": 0}, _abi.EINVAL), ({"vocab": 0}, _abi.EINVAL),
    ({"chunk_rows": -1}, _abi.EINVAL), ({"rows": 2**31}, _abi.ELIMIT),
    ({"x_stride": 63}, _abi.EINVAL), ({"w_stride": 8}, _abi.EINVAL),
    ({"grad_w_stride": 1}, _abi.EINVAL), ({"grad_x_stride": 1}, _abi.EINVAL),
    ({"x": None}, _abi.EINVAL), ({"w": None}, _abi.EINVAL), ({"targets": None}, _abi.EINVAL),
    ({"loss": None}, _abi.EINVAL), ({"lse": None}, _abi.EINVAL), ({"x": FAKE + 1}, _abi.EALIGN),
    ({"targets": FAKE + 4}, _abi.EALIGN), ({"loss": FAKE + 2}, _abi.EALIGN),
    ({"grad_w_dtype": _abi.DT_F32, "grad_w": FAKE + 2}, _abi.EALIGN),
    ({"loss_scale": float("nan")}, _abi.EINVAL), ({"loss_scale": float("inf")}, _abi.EINVAL),
])
def test_xent_refuses(change, want):
    d, size = _xent(**change), ctypes.c_size_t()
    assert L.fadam_xent_run(d, FAKE, 1 << 40, None) == want
    assert L.fadam_ops_last_error()
    assert L.fadam_xent_workspace(d, size) == want


def _wgrad(**kw):
    d = dict(dy=FAKE, x=_abi.Kept8(FAKE, FAKE), out=FAKE, rows=4, n=32, width=64, dy_stride=32,
             out_stride=64, dtype=_abi.DT_BF16, out_dtype=_abi.DT_F32, flags=0, reserved=0)
    return _abi.Wgrad(**(d | kw))


@pytest.mark.parametrize("change,want", [
    ({"dtype": _abi.DT_F32}, _abi.EDTYPE), ({"out_dtype": _abi.DT_F16}, _abi.EDTYPE),
    ({"flags": 2}, _abi.EINVAL), ({"rows": -1}, _abi.EINVAL), ({"n": 0}, _abi.EINVAL),
    ({"width": 0}, _abi.EINVAL), ({"dy_stride": 31}, _abi.EINVAL), ({"out_stride": 63}, _abi.EINVAL),
    ({"dy": None}, _abi.EINVAL), ({"out": None}, _abi.EINVAL),
    ({"x": _abi.Kept8(FAKE, None)}, _abi.EINVAL), ({"x": _abi.Kept8(FAKE, FAKE + 1)}, _abi.EALIGN),
    ({"out": FAKE + 2}, _abi.EALIGN), ({"width": 2**31, "out_stride": 2**31}, _abi.ELIMIT),
])
def test_wgrad_refuses(change, want):
    d, size = _wgrad(**change), ctypes.c_size_t()
    assert L.fadam_checkpoint8_wgrad(d, FAKE, 1 << 40, None) == want
    assert L.fadam_ops_last_error()
    assert L.fadam_checkpoint8_wgrad_workspace(d, size) == want


@pytest.mark.parametrize("args,want", [
    ((FAKE, 4, 64, 64, 9), _abi.EDTYPE), ((FAKE, -1, 64, 64, _abi.DT_F32), _abi.EINVAL),
    ((FAKE, 4, 0, 64, _abi.DT_F32), _abi.EINVAL), ((FAKE, 4, 64, 63, _abi.DT_F32), _abi.EINVAL),
    ((None, 4, 64, 64, _abi.DT_F32), _abi.EINVAL), ((FAKE + 2, 4, 64, 64, _abi.DT_F32), _abi.EALIGN),
    ((FAKE, 2**31, 64, 64, _abi.DT_F32), _abi.ELIMIT),
])
def test_checkpoint_refuses(args, want):
    x, rows, width, stride, dtype = args
    kept = _abi.Kept8(FAKE, FAKE)
    assert L.fadam_checkpoint8_pack(x, rows, width, stride, dtype, kept, None) == want
    assert L.fadam_checkpoint8_restore(kept, rows, width, x, stride, dtype, None) == want
    assert L.fadam_ops_last_error()


def test_empty_matrices_are_accepted():
    kept = _abi.Kept8(None, None)
    assert L.fadam_checkpoint8_pack(None, 0, 64, 64, _abi.DT_F32, kept, None) == _abi.OK
    assert L.fadam_checkpoint8_restore(kept, 0, 64, None, 64, _abi.DT_F32, None) == _abi.OK


def _norm(**kw):
    d = dict(f=FAKE, h=FAKE, post_weight=FAKE, pre_weight=FAKE, gate=FAKE, h_out=FAKE, x_out=FAKE,
             rstd_post=FAKE, rstd_pre=FAKE, f_kept=_abi.Kept8(), h_kept=_abi.Kept8(), rows=6,
             width=64, gate_rows=3, f_stride=64, h_stride=64, residual_scale=1.0, eps=1e-6,
             block_dtype=_abi.DT_BF16, residual_dtype=_abi.DT_F32, param_dtype=_abi.DT_BF16)
    return _abi.BlockNorm(**(d | kw))


BOTH_NORMS = [
    ({"block_dtype": 0}, _abi.EDTYPE), ({"residual_dtype": _abi.DT_F16}, _abi.EDTYPE),
    ({"param_dtype": _abi.DT_F16}, _abi.EDTYPE), ({"rows": -6}, _abi.EINVAL),
    ({"width": 0}, _abi.EINVAL), ({"width": 16385, "f_stride": 16385}, _abi.ELIMIT),
    ({"gate_rows": 4}, _abi.EINVAL), ({"gate_rows": 0}, _abi.EINVAL),
    ({"gate": None, "gate_rows": 3}, _abi.EINVAL), ({"residual_scale": float("inf")}, _abi.EINVAL),
    ({"f_stride": 63}, _abi.EINVAL), ({"pre_weight": None}, _abi.EINVAL),
    ({"rstd_post": None}, _abi.EINVAL), ({"rstd_pre": None}, _abi.EINVAL),
    ({"f": FAKE + 1}, _abi.EALIGN), ({"pre_weight": FAKE + 1}, _abi.EALIGN),
]


@pytest.mark.parametrize("change,want", BOTH_NORMS + [
    ({"eps": -1.0}, _abi.EINVAL), ({"eps": float("nan")}, _abi.EINVAL), ({"h_stride": 1}, _abi.EINVAL),
    ({"h": None}, _abi.EINVAL), ({"x_out": None}, _abi.EINVAL), ({"h": FAKE + 2}, _abi.EALIGN),
    ({"f_kept": _abi.Kept8(FAKE, None)}, _abi.EINVAL),
    ({"h_kept": _abi.Kept8(FAKE, FAKE + 2)}, _abi.EALIGN),
])
def test_block_norm_refuses(change, want):
    assert L.fadam_block_norm_forward(_norm(**change), None) == want
    assert L.fadam_ops_last_error()


def _norm_grad(**kw):
    d = dict(grad_h_out=FAKE, grad_x_out=FAKE, f=FAKE, h_out=FAKE, f_kept=_abi.Kept8(),
             h_kept=_abi.Kept8(), rstd_post=FAKE, rstd_pre=FAKE, post_weight=FAKE, pre_weight=FAKE,
             gate=FAKE, grad_f=FAKE, grad_h=FAKE, grad_post_weight=FAKE, grad_pre_weight=FAKE,
             grad_gate=FAKE, rows=6, width=64, gate_rows=3, grad_h_out_stride=64,
             grad_x_out_stride=64, f_stride=64, h_out_stride=64, residual_scale=1.0,
             block_dtype=_abi.DT_BF16, residual_dtype=_abi.DT_F32, param_dtype=_abi.DT_BF16)
    return _abi.BlockNormGrad(**(d | kw))


@pytest.mark.parametrize("change,want", BOTH_NORMS + [
    ({"grad_x_out": None}, _abi.EINVAL), ({"f": None}, _abi.EINVAL), ({"h_out": None}, _abi.EINVAL),
    ({"f": None, "f_kept": _abi.Kept8(FAKE, None)}, _abi.EINVAL),
    ({"grad_gate": None}, _abi.EINVAL), ({"grad_post_weight": None}, _abi.EINVAL),
    ({"grad_pre_weight": None}, _abi.EINVAL), ({"post_weight": None}, _abi.EINVAL),
    ({"grad_h": FAKE + 2}, _abi.EALIGN), ({"grad_h_out_stride": 2}, _abi.EINVAL),
])
def test_block_norm_backward_refuses(change, want):
    d, size = _norm_grad(**change), ctypes.c_size_t()
    assert L.fadam_block_norm_backward(d, FAKE, 1 << 40, None) == want
    assert L.fadam_ops_last_error()
    assert L.fadam_block_norm_backward_workspace(d, size) == want


# ---- refusals of the Python face -------------------------------------------------------------

def _b(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("error,call", [
    (ValueError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 8), _b(4, dtype=torch.int64))),
    (TypeError, lambda: fadam.linear_cross_entropy(_b(4, 8, dtype=torch.float32),
                                                   _b(9, 8, dtype=torch.float32),
                                                   _b(4, dtype=torch.int64))),
    (TypeError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 8, dtype=torch.float16),
                                                   _b(4, dtype=torch.int64))),
    (ValueError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 7), _b(4, dtype=torch.int64))),
    (ValueError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 8), _b(4, dtype=torch.int32))),
    (ValueError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 8), _b(3, dtype=torch.int64))),
    (ValueError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 8), _b(4, dtype=torch.int64),
                                                    reduction="none")),
    (ValueError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 8), _b(4, dtype=torch.int64),
                                                    accumulate=True)),
    (ValueError, lambda: fadam.linear_cross_entropy(_b(4, 8), _b(9, 8), _b(4, dtype=torch.int64),
                                                    grads=False, grad_weight=_b(9, 8))),
    (ValueError, lambda: fadam.checkpoint8(_b(4, 8))),
    (ValueError, lambda: fadam.checkpoint8(_b(8, 4).t())),
    (ValueError, lambda: fadam.checkpoint8_restore(fadam.Checkpoint8(
        _b(4, 8, dtype=torch.int8), _b(4, 2, dtype=torch.float32), torch.bfloat16))),
    (TypeError, lambda: fadam.checkpoint8_weight_grad(_b(4, 8, dtype=torch.float32),
                                                      fadam.Checkpoint8(
        _b(4, 8, dtype=torch.int8), _b(4, 1, dtype=torch.float32), torch.bfloat16))),
    (ValueError, lambda: fadam.checkpoint8_weight_grad(_b(3, 8), fadam.Checkpoint8(
        _b(4, 8, dtype=torch.int8), _b(4, 1, dtype=torch.float32), torch.bfloat16))),
    (ValueError, lambda: fadam.block_norm(_b(4, 8), _b(4, 8), _b(8))),
    (ValueError, lambda: fadam.block_norm(_b(4, 8), _b(5, 8), _b(8))),
    (TypeError, lambda: fadam.block_norm(_b(4, 8), _b(4, 8, dtype=torch.float16), _b(8))),
    (ValueError, lambda: fadam.block_norm(_b(4, 8), _b(4, 8), _b(7))),
    (TypeError, lambda: fadam.block_norm(_b(4, 8), _b(4, 8), _b(8, dtype=torch.float16))),
    (TypeError, lambda: fadam.block_norm(_b(4, 8), _b(4, 8), _b(8),
                                         post_weight=_b(8, dtype=torch.float32))),
    (ValueError, lambda: fadam.block_norm(_b(4, 8), _b(4, 8), _b(8), gate=_b(3, 8))),
    (ValueError, lambda: fadam.block_norm_backward(None, _b(4, 8), _b(4, 8), _b(3, 8), None,
                                                   _b(4, dtype=torch.float32), _b(8))),
    (ValueError, lambda: fadam.block_norm_backward(None, _b(4, 8), _b(4, 8), _b(4, 8), None,
                                                   _b(4, dtype=torch.float32), _b(8),
                                                   post_weight=_b(8))),
    (TypeError, lambda: fadam.block_norm_backward(None, _b(4, 8), _b(4, 8, dtype=torch.float32),
                                                  _b(4, 8), None, _b(4, dtype=torch.float32), _b(8))),
    (ValueError, lambda: fadam.block_norm_backward(None, _b(4, 8), _b(4, 8), _b(4, 8), None,
                                                   _b(4), _b(8))),
])
def test_python_face_refuses(error, call):
    with pytest.raises(error):
        call()


# ---- the formulas against differences -----------------------------------------------------------

def _slope(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_xent_formula_against_differences():
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(5, 7, generator=gen, dtype=torch.float64)
    w = torch.randn(11, 7, generator=gen, dtype=torch.float64)
    y = torch.tensor([3, -100, 0, 10, 3])
    for mean in (False, True):
        r = ref.xent(x, w, y, mean=mean)
        for at, grad, f in ((x, r.grad_x, lambda v: ref.xent(v, w, y, mean=mean).loss),
                            (w, r.grad_w, lambda v: ref.xent(x, v, y, mean=mean).loss)):
            d = torch.randn(at.shape, generator=gen, dtype=torch.float64)
            assert abs(_slope(f, at, d) - (grad * d).sum()) < 1e-8


@pytest.mark.parametrize("post,gates", [(True, 1), (True, 3), (False, 6), (True, 0), (False, 0)])
def test_block_norm_formula_against_differences(post, gates):
    gen = torch.Generator().manual_seed(2)

    def rand(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    args = {"f": rand(6, 9), "h": rand(6, 9), "pre": rand(9), "post": rand(9) if post else None,
            "gate": rand(gates, 9) if gates else None}
    gh, gx = rand(6, 9), rand(6, 9)

    def value(a):
        r = ref.block_norm(**a, alpha=0.7, eps=1e-3)
        return (r.h_out * gh).sum() + (r.x_out * gx).sum()

    r = ref.block_norm(**args, alpha=0.7, eps=1e-3)
    g = ref.block_norm_grad(gh, gx, args["f"], r.h_out, r.r1, r.r2, args["pre"], args["post"],
                            args["gate"], 0.7)
    for name, v in args.items():
        if v is not None:
            d = rand(*v.shape)
            slope = _slope(lambda z: value(args | {name: z}), v, d)
            assert abs(slope - (g[name].value * d).sum()) < 1e-6, name
