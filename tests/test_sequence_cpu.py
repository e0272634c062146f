"""Checks of the sequence operators that need no GPU: exports and structures
against include/fadam_seq.h, refusals before any CUDA call, and the gradients'
formulas against differences of the functions themselves."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import adamw_optimizer_step_persistent_gb300 as fadam
from adamw_optimizer_step_persistent_gb300 import _abi
from tests import sequence_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fadam_seq.h")
L = _abi.lib()
FAKE = 0x7F0000000000  # never dereferenced: the checks fail before any use
BF16, F16 = torch.bfloat16, torch.float16

STRUCTS = {"fadam_embed": _abi.Embed, "fadam_embed_grad": _abi.EmbedGrad,
           "fadam_attention": _abi.Attention, "fadam_attention_grad": _abi.AttentionGrad}


def test_library_exports_every_declared_function():
    names = re.findall(r"^fadam_status\s+(fadam_\w+)\(", open(HEADER).read(), re.M)
    assert len(names) == 7
    assert {n for n, _, _ in _abi.SEQ_SIGNATURES} == set(names)
    assert all(hasattr(L, n) for n in names)
    text = open(HEADER).read()
    for name, value in (("EMBED_PADDING", "1u"), ("EMBED_ACCUMULATE", "2u"), ("ATTENTION_CAUSAL", "1u"),
                        ("ATTENTION_MAX_WIDTH", "128")):
        assert re.search(rf"#define FADAM_{name} {value}\b", text)
        assert getattr(_abi, name) == int(value.rstrip("u"))


def test_structures_match_the_header(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "fadam_seq.h"\nint main(void) {\n'
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

NAN, INF = float("nan"), float("inf")


def _embed(**kw):
    d = dict(tokens=FAKE, weight=FAKE, out=FAKE, rows=4, width=64, vocab=100, weight_stride=64,
             out_stride=64, padding_index=0, scale=1.0, weight_dtype=_abi.DT_BF16,
             out_dtype=_abi.DT_F32, flags=0)
    return _abi.Embed(**(d | kw))


@pytest.mark.parametrize("change,want", [
    ({"weight_dtype": 0}, _abi.EDTYPE), ({"out_dtype": _abi.DT_F16}, _abi.EDTYPE),
    ({"flags": 2}, _abi.EINVAL), ({"rows": -1}, _abi.EINVAL), ({"width": 0}, _abi.EINVAL),
    ({"vocab": 0}, _abi.EINVAL), ({"rows": 2**31}, _abi.ELIMIT), ({"vocab": 2**31}, _abi.ELIMIT),
    ({"weight_stride": 63}, _abi.EINVAL), ({"out_stride": 63}, _abi.EINVAL), ({"scale": NAN}, _abi.EINVAL),
    ({"scale": INF}, _abi.EINVAL), ({"tokens": None}, _abi.EINVAL), ({"weight": None}, _abi.EINVAL),
    ({"out": None}, _abi.EINVAL), ({"tokens": FAKE + 4}, _abi.EALIGN), ({"weight": FAKE + 1}, _abi.EALIGN),
    ({"out": FAKE + 2}, _abi.EALIGN)])
def test_embed_refuses(change, want):
    assert L.fadam_embed_forward(_embed(**change), None) == want
    assert L.fadam_ops_last_error()


def _embed_grad(**kw):
    d = dict(tokens=FAKE, grad=FAKE, out=FAKE, rows=4, width=64, vocab=100, grad_stride=64, out_stride=64,
             padding_index=0, scale=1.0, grad_dtype=_abi.DT_BF16, out_dtype=_abi.DT_F32, flags=0)
    return _abi.EmbedGrad(**(d | kw))


@pytest.mark.parametrize("change,want", [
    ({"grad_dtype": 0}, _abi.EDTYPE), ({"out_dtype": _abi.DT_F16}, _abi.EDTYPE), ({"out_dtype": 0}, _abi.EDTYPE),
    ({"flags": 4}, _abi.EINVAL), ({"rows": -1}, _abi.EINVAL), ({"width": 0}, _abi.EINVAL),
    ({"vocab": -2}, _abi.EINVAL), ({"rows": 2**31}, _abi.ELIMIT), ({"width": 2**31}, _abi.ELIMIT),
    ({"grad_stride": 63}, _abi.EINVAL), ({"out_stride": 63}, _abi.EINVAL), ({"scale": -INF}, _abi.EINVAL),
    ({"tokens": None}, _abi.EINVAL), ({"grad": None}, _abi.EINVAL), ({"out": None}, _abi.EINVAL),
    ({"tokens": FAKE + 4}, _abi.EALIGN), ({"grad": FAKE + 1}, _abi.EALIGN), ({"out": FAKE + 2}, _abi.EALIGN)])
def test_embed_grad_refuses(change, want):
    d, size = _embed_grad(**change), ctypes.c_size_t()
    assert L.fadam_embed_grad_run(d, FAKE, 1 << 40, None) == want
    assert L.fadam_ops_last_error()
    assert L.fadam_embed_grad_workspace(d, size) == want


def test_embed_grad_workspace_and_no_rows():
    size = ctypes.c_size_t(7)
    assert L.fadam_embed_grad_workspace(_embed_grad(), size) == _abi.OK and size.value > 400
    assert L.fadam_embed_grad_workspace(_embed_grad(rows=0), size) == _abi.OK and size.value == 0
    assert L.fadam_embed_grad_workspace(_embed_grad(), None) == _abi.EINVAL
    assert L.fadam_embed_forward(_embed(rows=0, tokens=None, out=None), None) == _abi.OK
    none = _embed_grad(rows=0, tokens=None, grad=None, flags=_abi.EMBED_ACCUMULATE)
    assert L.fadam_embed_grad_run(none, None, 0, None) == _abi.OK


def _attention(**kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, slopes=None, documents=None, prefix=None, tokens=64,
             sequence=32, n_documents=0, q_stride=256, k_stride=128, v_stride=128, q_head_stride=64,
             k_head_stride=64, v_head_stride=64, heads=4, kv_heads=2, width=64, scale=0.125, softcap=0.0,
             dtype=_abi.DT_BF16, flags=_abi.ATTENTION_CAUSAL, reserved=0)
    return _abi.Attention(**(d | kw))


BAD_ATTENTION = [
    ({"dtype": _abi.DT_F32}, _abi.EDTYPE), ({"dtype": 9}, _abi.EDTYPE), ({"flags": 2}, _abi.EINVAL),
    ({"tokens": -1}, _abi.EINVAL), ({"heads": 0}, _abi.EINVAL), ({"kv_heads": 0}, _abi.EINVAL),
    ({"kv_heads": 3}, _abi.EINVAL), ({"kv_heads": -2}, _abi.EINVAL), ({"width": 0}, _abi.EINVAL),
    ({"width": 60}, _abi.EINVAL), ({"width": 136}, _abi.ELIMIT), ({"tokens": 2**25}, _abi.ELIMIT),
    ({"heads": 2**15}, _abi.ELIMIT), ({"tokens": 2**24, "heads": 2**14, "sequence": 1}, _abi.ELIMIT), ({"sequence": 0}, _abi.EINVAL), ({"sequence": 48}, _abi.EINVAL),
    ({"documents": FAKE, "n_documents": -1}, _abi.EINVAL), ({"scale": 0.0}, _abi.EINVAL),
    ({"scale": -1.0}, _abi.EINVAL), ({"scale": NAN}, _abi.EINVAL), ({"scale": INF}, _abi.EINVAL),
    ({"softcap": -1.0}, _abi.EINVAL), ({"softcap": NAN}, _abi.EINVAL), ({"softcap": INF}, _abi.EINVAL),
    ({"softcap": 1e-45}, _abi.EINVAL), ({"softcap": 1e16}, _abi.EINVAL), ({"softcap": 1e-9}, _abi.EINVAL), ({"q": None}, _abi.EINVAL), ({"k": None}, _abi.EINVAL),
    ({"v": None}, _abi.EINVAL), ({"out": None}, _abi.EINVAL), ({"lse": None}, _abi.EINVAL),
    ({"q": FAKE + 8}, _abi.EALIGN), ({"k": FAKE + 2}, _abi.EALIGN), ({"v": FAKE + 4}, _abi.EALIGN),
    ({"out": FAKE + 8}, _abi.EALIGN), ({"lse": FAKE + 2}, _abi.EALIGN), ({"slopes": FAKE + 2}, _abi.EALIGN),
    ({"documents": FAKE + 2}, _abi.EALIGN), ({"prefix": FAKE + 1}, _abi.EALIGN),
    ({"q_stride": 260}, _abi.EALIGN), ({"k_head_stride": 68}, _abi.EALIGN), ({"q_head_stride": 56}, _abi.EINVAL),
    ({"v_stride": 56}, _abi.EINVAL), ({"k_stride": 0}, _abi.EINVAL), ({"k_head_stride": 0}, _abi.EINVAL),
    ({"v_stride": 2**39}, _abi.EINVAL), ({"reserved": 1}, _abi.EINVAL)]


@pytest.mark.parametrize("change,want", BAD_ATTENTION)
def test_attention_refuses(change, want):
    d, size = _attention(**change), ctypes.c_size_t()
    assert L.fadam_attention_run(d, FAKE, 1 << 40, None) == want
    assert L.fadam_ops_last_error()
    assert L.fadam_attention_workspace(d, size) == want
    g = _abi.AttentionGrad(d, FAKE, FAKE, FAKE, FAKE, 256, 64, 256, 64)
    assert L.fadam_attention_backward(g, FAKE, 1 << 40, None) == want
    assert L.fadam_attention_backward_workspace(g, size) == want


@pytest.mark.parametrize("at,value,want", [
    (1, None, _abi.EINVAL), (2, None, _abi.EINVAL), (3, None, _abi.EINVAL), (4, None, _abi.EINVAL),
    (1, FAKE + 8, _abi.EALIGN), (2, FAKE + 8, _abi.EALIGN), (3, FAKE + 2, _abi.EALIGN), (4, FAKE + 4, _abi.EALIGN),
    (5, 260, _abi.EALIGN), (6, 56, _abi.EINVAL), (7, 0, _abi.EINVAL), (8, 68, _abi.EALIGN)])
def test_attention_backward_refuses(at, value, want):
    args = [_attention(), FAKE, FAKE, FAKE, FAKE, 256, 64, 256, 64]
    args[at] = value
    g, size = _abi.AttentionGrad(*args), ctypes.c_size_t()
    assert L.fadam_attention_backward(g, FAKE, 1 << 40, None) == want
    assert L.fadam_ops_last_error()
    assert L.fadam_attention_backward_workspace(g, size) == want


def test_attention_workspace():
    size = ctypes.c_size_t(3)
    assert L.fadam_attention_workspace(_attention(sequence=64), size) == _abi.OK and size.value == 0
    packed = _attention(documents=FAKE, n_documents=3)
    assert L.fadam_attention_workspace(packed, size) == _abi.OK and size.value >= 16 * 64
    none = _attention(tokens=0, q=None, k=None, v=None, out=None, lse=None)
    assert L.fadam_attention_run(none, None, 0, None) == _abi.OK
    # a head or token dimension of one has no stride
    assert L.fadam_attention_workspace(_attention(kv_heads=1, k_head_stride=3, v_head_stride=0), size) == _abi.OK
    one = _attention(tokens=1, sequence=1, q_stride=1, k_stride=0, v_stride=7)
    assert L.fadam_attention_workspace(one, size) == _abi.OK
    g = _abi.AttentionGrad(none, None, None, None, None, 256, 64, 256, 64)
    assert L.fadam_attention_backward(g, None, 0, None) == _abi.OK


# ---- refusals of the Python face ---------------------------------------------------------------

def _t(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def test_python_embedding_refuses():
    w, t = _t(10, 8), torch.zeros(3, dtype=torch.int64)
    for args, kw, error in (
            ((t, _t(10)), {}, ValueError), ((t.int(), w), {}, TypeError), ((t, w), {"dtype": F16}, TypeError),
            ((t, w.double()), {}, Exception), ((t, w), {}, ValueError)):        # (the last: not on a GPU)
        with pytest.raises(error):
            fadam.embedding(*args, **kw)
    g = _t(3, 8)
    for args, kw, error in (
            ((g, t.int(), 10), {}, TypeError), ((_t(4, 8), t, 10), {}, ValueError), ((g, t), {}, ValueError),
            ((g, t, 10), {"accumulate": True}, ValueError), ((g, t, 10), {}, ValueError)):
        with pytest.raises(error):
            fadam.embedding_weight_grad(*args, **kw)


def test_python_attention_refuses():
    q, k = _t(2, 6, 4, 64), _t(2, 6, 2, 64)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    for args, kw, error in (
            ((q.float(), k.float(), k.float()), {}, TypeError), ((q, k, k.half()), {}, TypeError),
            ((q[0, 0], k, k), {}, ValueError), ((q, k, k[:, :5]), {}, ValueError),
            ((q, k[:1], k[:1]), {}, ValueError), ((q, k[..., :56], k[..., :56]), {}, ValueError),
            ((q, _t(2, 6, 3, 64), _t(2, 6, 3, 64)), {}, ValueError), ((q[..., ::2], k, k), {}, ValueError),
            ((_t(2, 6, 4, 136),) * 3, {}, ValueError), ((_t(2, 6, 4, 60),) * 3, {}, ValueError),
            ((_t(6, 2, 4, 64).transpose(0, 1), k, k), {}, ValueError),     # tokens not evenly strided
            ((q, k, k), {}, ValueError)):                                    # not on a GPU
        with pytest.raises(error):
            fadam.attention(*args, **kw)
    lse = _t(2, 6, 4, dtype=torch.float32)
    with pytest.raises(ValueError):
        fadam.attention_backward(q, q, k, k, q, lse)
    del ints


# ---- the gradients' formulas ------------------------------------------------------------------------

def _small_case(**kw):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(14, h, 8, generator=g, dtype=torch.float64) for h in (4, 2, 2))
    return ref.Case(q, k, v, 0.4, **{"sequence": 14, **kw})


@pytest.mark.parametrize("kw", [
    {}, {"causal": False}, {"softcap": 1.5}, {"slopes": torch.tensor([0.5, 0.1, 0.0, -0.2])},
    {"offsets": [1, 5, 5, 12], "prefix": [2, 1, 4], "softcap": 2.0}, {"sequence": 7, "prefix": [3, 9]}])
def test_attention_gradient_formula_against_differences(kw):
    c = _small_case(**kw)
    out, lse, empty = ref.attention(c)
    go = torch.randn(14, 4, 8, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    lse = torch.where(empty[:, None], -torch.inf, lse.value)
    want = ref.attention_grad(c, go, out.value, lse)

    def loss(**at):
        return (ref.attention(c._replace(**at))[0].value * go).sum()

    for name in "qkv":
        x = getattr(c, name)
        for index in ((0, 0, 0), (4, 1, 3), (9, 1, 7), (13, 0, 2)):
            step = torch.zeros_like(x)
            step[index] = 1e-6
            slope = (loss(**{name: x + step}) - loss(**{name: x - step})) / 2e-6
            assert abs(slope - want[name].value[index]) < 1e-7, (name, index)


def test_embedding_gradient_formula():
    t = torch.tensor([0, 2, 2, 5, -1, 2])
    g = torch.randn(6, 3, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    want = ref.embedding_grad(g, t, 4, 2.0, 0).value
    assert torch.equal(want[2], 2 * (g[1] + g[2] + g[5])) and not want[[0, 1, 3]].any()
