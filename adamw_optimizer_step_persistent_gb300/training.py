"""Python face of the training operators (include/fadam_ops.h).

They stand next to the optimizer step and produce what its shards read: the
loss over a vocabulary with its gradients, the norms around a block forward
and backward, and activations kept in 8 bits.  The functions check and
marshal tensors, allocate outputs and workspace from PyTorch's caching
allocator and launch on the current stream; nothing synchronises, so calls
can be captured in a CUDA graph.

Matrices are given as tensors of any number of dimensions whose last one is
the row; the leading ones are taken together as rows and must be evenly
strided (no copy is made).

The functions stand outside autograd: they take tensors that require a
gradient like any others and return tensors that do not, so in the middle of a
module they would cut the graph.  Gradients are passed on by the caller, e.g.
``x.backward(linear_cross_entropy(x, w, y).grad_x)``, or from the ``forward``
and ``backward`` of a ``torch.autograd.Function``.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional, Union

import torch

from . import _abi
from .optimizer import _ptr, dtype_code

_16BIT = (torch.bfloat16, torch.float16)
_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else lambda i: torch.cuda.current_stream(i).cuda_stream


class LinearCrossEntropy(NamedTuple):
    """What ``linear_cross_entropy`` returns."""
    loss: torch.Tensor                    # [] fp32
    row_loss: torch.Tensor                # [rows] fp32, 0 where ignored
    lse: torch.Tensor                     # [rows] fp32
    grad_x: Optional[torch.Tensor]        # as x
    grad_weight: Optional[torch.Tensor]   # as weight, or the buffer that was given


class Checkpoint8(NamedTuple):
    """An activation kept in 8 bits: element = code * scale of its group."""
    codes: torch.Tensor     # int8, the activation's shape
    scales: torch.Tensor    # fp32, [..., ceil(width / 128)]
    dtype: torch.dtype      # of the activation


class BlockNorm(NamedTuple):
    """What ``block_norm`` returns."""
    h_out: torch.Tensor
    x_out: torch.Tensor
    rstd_post: Optional[torch.Tensor]
    rstd_pre: torch.Tensor
    f_checkpoint: Optional[Checkpoint8]
    h_checkpoint: Optional[Checkpoint8]


class BlockNormGrads(NamedTuple):
    """What ``block_norm_backward`` returns."""
    f: torch.Tensor
    h: torch.Tensor
    post_weight: Optional[torch.Tensor]
    pre_weight: torch.Tensor
    gate: Optional[torch.Tensor]


def _rows(t: torch.Tensor, what: str):
    """(rows, width, stride) of a tensor taken as a matrix."""
    if t.dim() < 1:
        raise ValueError(f"{what} has no dimension")
    width = t.size(-1)
    if t.is_contiguous():
        return (t.numel() // width if width else 0), width, width
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {what} is not contiguous")
    if t.dim() == 1:
        return 1, width, width
    m = t if t.dim() == 2 else t.view(-1, width) if _collapses(t) else None
    if m is None:
        raise ValueError(f"the leading dimensions of {what} are not evenly strided")
    stride = m.stride(0) if m.shape[0] > 1 else max(width, m.stride(0))
    if stride < width:
        raise ValueError(f"the rows of {what} overlap")
    return m.shape[0], width, stride


def _collapses(t: torch.Tensor) -> bool:
    dims = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    return all(a[1] == b[0] * b[1] for a, b in zip(dims, dims[1:]))


def _device(t: torch.Tensor, what: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{what} is on {t.device}, not on a CUDA device")
    return index


def _check_device(index: int, what: str, *tensors: Optional[torch.Tensor]) -> None:
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, {what} on cuda:{index}")


def _like(t: torch.Tensor, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """A new contiguous tensor of t's shape (empty_like is the cheapest call
    there is, but keeps the strides of what is dense in another order)."""
    if t.is_contiguous():
        return torch.empty_like(t, dtype=dtype) if dtype is not None else torch.empty_like(t)
    return torch.empty((*t.shape,), dtype=dtype or t.dtype, device=t.device)


_HERE = contextlib.nullcontext()


def _current(index: int):
    """A context in which the device is the current one (most often it is)."""
    return _HERE if torch.cuda.current_device() == index else torch.cuda.device(index)


def _workspace(size_of, desc, where: str, like: torch.Tensor):
    """(tensor or None, address, bytes) of the workspace that a call needs."""
    need = ctypes.c_size_t()
    status = size_of(desc, need)
    if status:
        _abi.check_ops(status, where)
    if not need.value:
        return None, None, 0
    ws = torch.empty(need.value, dtype=torch.uint8, device=like.device)
    return ws, ws.data_ptr(), need.value


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                         ignore_index: int = -100, reduction: str = "mean",
                         loss_scale: float = 1.0, grads: bool = True,
                         grad_weight: Optional[torch.Tensor] = None, accumulate: bool = False,
                         chunk_rows: int = 0) -> LinearCrossEntropy:
    """Softmax cross entropy of ``x @ weight.T`` against ``targets``, with the
    gradients of ``x`` and ``weight`` (``fadam_xent_run``).

    ``x`` [..., width] and ``weight`` [vocab, width] are bf16 or fp16, targets
    [...] int64.  The logits are never held: forward alone needs 8 bytes of
    scratch for 128 of them, with gradients a chunk of rows' exponentials is
    held in 16 bits (``chunk_rows``; 0: as many as fit 4 GiB).  ``reduction``
    is "mean" over the rows whose target is not ``ignore_index`` (0 when there
    is none) or "sum".  Products are cut by the sizes, so a row's last bits can
    change with the number of rows beside it.  The gradients are those of ``loss_scale * loss``: an optimizer
    shard takes it back out with its grad scale.

    ``grad_weight`` is a [vocab, width] buffer of the weight's dtype or fp32,
    such as a view of an optimizer shard's gradient; with ``accumulate`` the
    gradient is added to it (the second and later micro-batches of a step).
    ``grads=False`` computes the loss alone.  A target outside the vocabulary
    makes the loss and the gradients NaN, which the shard's screen or norm
    turns into a skipped step.
    """
    rows, width, x_stride = _rows(x, "x")
    if weight.dim() != 2 or weight.shape[1] != width:
        raise ValueError(f"weight must be [vocab, {width}], got {tuple(weight.shape)}")
    if x.dtype not in _16BIT or weight.dtype != x.dtype:
        raise TypeError(f"x and weight must both be bf16 or fp16, got {x.dtype} and {weight.dtype}")
    if targets.dtype != torch.int64 or targets.shape != x.shape[:-1]:
        raise ValueError(f"targets must be int64 of shape {tuple(x.shape[:-1])}")
    if reduction not in ("mean", "sum"):
        raise ValueError(f"reduction {reduction!r} is neither 'mean' nor 'sum'")
    if accumulate and grad_weight is None:
        raise ValueError("accumulate needs a grad_weight buffer")
    if grad_weight is not None and not grads:
        raise ValueError("a grad_weight buffer without grads")
    index = _device(x, "x")
    _check_device(index, "x", weight, targets, grad_weight)
    vocab, _, w_stride = _rows(weight, "weight")
    targets = targets.contiguous()
    code = dtype_code(x.dtype)
    grad_x, gw_stride, gw_code = None, width, code
    if grads and grad_weight is not None:
        if (grad_weight.shape != weight.shape
                or grad_weight.dtype not in (weight.dtype, torch.float32)):
            raise ValueError("grad_weight must have the weight's shape, and its dtype or fp32")
        gw_stride, gw_code = _rows(grad_weight, "grad_weight")[2], dtype_code(grad_weight.dtype)
    with _current(index):
        row_loss = torch.empty_like(targets, dtype=torch.float32)
        lse = torch.empty_like(row_loss)
        loss = torch.empty((), dtype=torch.float32, device=x.device)
        if grads:
            grad_x = _like(x)
            if grad_weight is None:
                grad_weight = _like(weight)
        flags = ((_abi.XENT_MEAN if reduction == "mean" else 0)
                 | (_abi.XENT_ACCUMULATE if accumulate else 0))
        desc = _abi.Xent(
            x.data_ptr(), weight.data_ptr(), targets.data_ptr(), loss.data_ptr(),
            row_loss.data_ptr(), lse.data_ptr(), _ptr(grad_x), _ptr(grad_weight), rows, width,
            vocab, x_stride, w_stride, width, gw_stride, int(ignore_index), int(chunk_rows),
            float(loss_scale), code, gw_code, flags)
        lib = _abi.lib()
        ws, at, size = _workspace(lib.fadam_xent_workspace, desc, "fadam_xent_workspace", x)
        status = lib.fadam_xent_run(desc, at, size, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_xent_run")
    return LinearCrossEntropy(loss, row_loss, lse, grad_x, grad_weight)


# ---- 8-bit checkpoints ---------------------------------------------------------------

def _empty_checkpoint(like: torch.Tensor) -> Checkpoint8:
    shape = like.shape
    groups = -(-shape[-1] // _abi.CHECKPOINT8_GROUP)
    return Checkpoint8(_like(like, torch.int8),
                       torch.empty((*shape[:-1], groups), dtype=torch.float32,
                                   device=like.device), like.dtype)


def _kept(c: Optional[Checkpoint8]) -> _abi.Kept8:
    return _NOT_KEPT if c is None else _abi.Kept8(c.codes.data_ptr(), c.scales.data_ptr())


_NOT_KEPT = _abi.Kept8()


def _check_checkpoint(c: Checkpoint8, what: str) -> None:
    codes, scales = c.codes, c.scales
    groups = -(-codes.shape[-1] // _abi.CHECKPOINT8_GROUP)
    if (codes.dtype != torch.int8 or scales.dtype != torch.float32
            or not codes.is_contiguous() or not scales.is_contiguous()
            or scales.shape != codes.shape[:-1] + (groups,)
            or codes.get_device() != scales.get_device()):
        raise ValueError(f"{what} is not a checkpoint: contiguous int8 codes [..., width] and fp32 "
                         "scales [..., ceil(width / 128)] on one device")


def checkpoint8(x: torch.Tensor) -> Checkpoint8:
    """An activation [..., width] (bf16, fp16 or fp32) kept in 8 bits, one fp32
    scale for each started group of 128 elements of a row: 1.03 bytes an
    element, each off by at most 1/254 of its group's largest magnitude.  A
    group that holds an infinity or a NaN is restored as NaN throughout."""
    rows, width, stride = _rows(x, "x")
    index = _device(x, "x")
    code = dtype_code(x.dtype)
    with _current(index):
        out = _empty_checkpoint(x)
        status = _abi.lib().fadam_checkpoint8_pack(x.data_ptr(), rows, width, stride, code,
                                                   _kept(out), _stream(index))
    if status:
        _abi.check_ops(status, "fadam_checkpoint8_pack")
    return out


def checkpoint8_restore(c: Checkpoint8) -> torch.Tensor:
    """The activation that ``checkpoint8`` kept, in its dtype."""
    _check_checkpoint(c, "c")
    index = _device(c.codes, "c")
    rows, width, stride = _rows(c.codes, "c")
    code = dtype_code(c.dtype)
    with _current(index):
        x = torch.empty_like(c.codes, dtype=c.dtype)
        status = _abi.lib().fadam_checkpoint8_restore(_kept(c), rows, width, x.data_ptr(), stride,
                                                      code, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_checkpoint8_restore")
    return x


def checkpoint8_weight_grad(grad_y: torch.Tensor, c: Checkpoint8, *,
                            out: Optional[torch.Tensor] = None,
                            accumulate: bool = False) -> torch.Tensor:
    """The weight gradient ``grad_y.T @ x`` [n, width] of a linear layer, from
    its output's gradient [..., n] (bf16 or fp16) and the checkpoint of its
    input [..., width], whose values are rounded to grad_y's dtype for the
    product (under fp16, those kept from bf16 or fp32 are brought into range by
    a power of two first).  ``out`` is a buffer of grad_y's dtype or fp32, such as
    a view of an optimizer shard's gradient; with ``accumulate`` the gradient
    is added to it."""
    _check_checkpoint(c, "c")
    if grad_y.dtype not in _16BIT:
        raise TypeError(f"grad_y must be bf16 or fp16, got {grad_y.dtype}")
    if grad_y.shape[:-1] != c.codes.shape[:-1]:
        raise ValueError(f"grad_y {tuple(grad_y.shape)} and the checkpoint {tuple(c.codes.shape)} "
                         "have different rows")
    if accumulate and out is None:
        raise ValueError("accumulate needs an out buffer")
    index = _device(grad_y, "grad_y")
    _check_device(index, "grad_y", c.codes, out)
    rows, n, stride = _rows(grad_y, "grad_y")
    width = c.codes.shape[-1]
    # fp16 operands end at 65504; what was kept from fp16 is below that
    wide = grad_y.dtype is torch.float16 and c.dtype is not torch.float16
    if out is not None and (out.shape != (n, width)
                            or out.dtype not in (grad_y.dtype, torch.float32)):
        raise ValueError(f"out must be [{n}, {width}] of grad_y's dtype or fp32")
    with _current(index):
        if out is None:
            out = torch.empty((n, width), dtype=grad_y.dtype, device=grad_y.device)
        desc = _abi.Wgrad(grad_y.data_ptr(), _kept(c), out.data_ptr(), rows, n, width, stride,
                          _rows(out, "out")[2], dtype_code(grad_y.dtype), dtype_code(out.dtype),
                          (_abi.WGRAD_ACCUMULATE if accumulate else 0)
                          | (_abi.WGRAD_WIDE_X if wide else 0))
        lib = _abi.lib()
        ws, at, size = _workspace(lib.fadam_checkpoint8_wgrad_workspace, desc,
                                  "fadam_checkpoint8_wgrad_workspace", grad_y)
        status = lib.fadam_checkpoint8_wgrad(desc, at, size, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_checkpoint8_wgrad")
    return out


# ---- the norms around a block ------------------------------------------------------------

def _norm_params(width: int, rows: int, block: torch.dtype, pre_weight, post_weight, gate):
    """The parameters' dtype, and how many rows the gate has."""
    dtype = pre_weight.dtype
    if dtype is not block and dtype is not torch.float32:
        raise TypeError(f"the parameters must be {block} or fp32, got {dtype}")
    for name, w in (("pre_weight", pre_weight), ("post_weight", post_weight)):
        if w is not None:
            if w.dim() != 1 or w.size(0) != width or not w.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [{width}]")
            if w.dtype is not dtype:
                raise TypeError("pre_weight, post_weight and gate must have one dtype")
    if gate is None:
        return dtype, 1
    if gate.dtype is not dtype:
        raise TypeError("pre_weight, post_weight and gate must have one dtype")
    if gate.dim() < 1 or gate.size(-1) != width or not gate.is_contiguous():
        raise ValueError(f"gate must be a contiguous [..., {width}]")
    gate_rows = gate.numel() // width if width else 0
    if gate_rows < 1 or rows % gate_rows:
        raise ValueError(f"{gate_rows} gate rows do not divide {rows} rows")
    return dtype, gate_rows


def block_norm(f: torch.Tensor, h: torch.Tensor, pre_weight: torch.Tensor, *,
               post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               residual_scale: float = 1.0, eps: float = 1e-6,
               checkpoint: bool = False) -> BlockNorm:
    """The norms around a block, in one pass (``fadam_block_norm_forward``): the
    post-norm of its output ``f`` (when ``post_weight`` is given), its gate and
    residual scale, the addition to the residual stream ``h``, and the pre-norm
    of the next block::

        n = f * rsqrt(mean(f^2) + eps) * post_weight      (or f)
        h_out = h + residual_scale * gate * n
        x_out = h_out * rsqrt(mean(h_out^2) + eps) * pre_weight

    ``f`` and ``x_out`` are of one dtype (bf16, fp16 or fp32), ``h`` and
    ``h_out`` of that dtype or fp32, the parameters of the block's dtype or
    fp32.  ``gate`` [..., width] has one row for all rows, one for each
    equally long run of rows (a sequence), or one for each row.  With
    ``checkpoint`` the same pass keeps ``f`` and ``h_out`` in 8 bits for
    ``block_norm_backward``.
    """
    rows, width, f_stride = _rows(f, "f")
    if h.shape != f.shape:
        raise ValueError(f"f {tuple(f.shape)} and h {tuple(h.shape)} differ in shape")
    if h.dtype not in (f.dtype, torch.float32):
        raise TypeError(f"h must be {f.dtype} or fp32, got {h.dtype}")
    block = dtype_code(f.dtype)
    residual = block if h.dtype is f.dtype else dtype_code(h.dtype)
    params, gate_rows = _norm_params(width, rows, f.dtype, pre_weight, post_weight, gate)
    index = _device(f, "f")
    _check_device(index, "f", h, pre_weight, post_weight, gate)
    h_stride = width if h.is_contiguous() else _rows(h, "h")[2]
    with _current(index):
        h_out = _like(h)
        x_out = _like(f)
        r2 = torch.empty((*f.shape[:-1],), dtype=torch.float32, device=f.device)
        r1 = torch.empty_like(r2) if post_weight is not None else None
        f_kept = _empty_checkpoint(f) if checkpoint else None
        h_kept = _empty_checkpoint(h) if checkpoint else None
        desc = _abi.BlockNorm(
            f.data_ptr(), h.data_ptr(), _ptr(post_weight), pre_weight.data_ptr(), _ptr(gate),
            h_out.data_ptr(), x_out.data_ptr(), _ptr(r1), r2.data_ptr(), _kept(f_kept),
            _kept(h_kept), rows, width, gate_rows, f_stride, h_stride, float(residual_scale),
            float(eps), block, residual, block if params is f.dtype else dtype_code(params))
        status = _abi.lib().fadam_block_norm_forward(desc, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_block_norm_forward")
    return BlockNorm(h_out, x_out, r1, r2, f_kept, h_kept)


def _saved(t: Union[torch.Tensor, Checkpoint8], what: str, shape: torch.Size):
    """(a tensor on its device, tensor's address or None, kept or not, stride)."""
    kept = isinstance(t, Checkpoint8)
    if kept:
        _check_checkpoint(t, what)
    data = t.codes if kept else t
    if data.shape != shape:
        raise ValueError(f"{what} {tuple(data.shape)} and grad_x_out {tuple(shape)} differ in shape")
    if kept:
        return data, None, _kept(t), shape[-1]
    return data, data.data_ptr(), _NOT_KEPT, _rows(data, what)[2]


def block_norm_backward(grad_h_out: Optional[torch.Tensor], grad_x_out: torch.Tensor,
                        f: Union[torch.Tensor, Checkpoint8],
                        h_out: Union[torch.Tensor, Checkpoint8],
                        rstd_post: Optional[torch.Tensor], rstd_pre: torch.Tensor,
                        pre_weight: torch.Tensor, *, post_weight: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None,
                        residual_scale: float = 1.0) -> BlockNormGrads:
    """The gradients of ``block_norm``, in one pass over the rows, from those of
    ``h_out`` (None: zero, the last block) and ``x_out`` and what the forward
    pass left: ``f`` and ``h_out``, each the tensor or its 8-bit checkpoint,
    and the rstds.  The parameters' gradients have the parameters' dtype."""
    rows, width, gx_stride = _rows(grad_x_out, "grad_x_out")
    block, shape = grad_x_out.dtype, grad_x_out.shape
    f_data, f_at, f_kept, f_stride = _saved(f, "f", shape)
    h_data, h_at, h_kept, h_stride = _saved(h_out, "h_out", shape)
    residual = h_out.dtype
    if f.dtype is not block or residual is not block and residual is not torch.float32:
        raise TypeError(f"f must be {block} and h_out that or fp32, got {f.dtype}, {residual}")
    gh_stride = width
    if grad_h_out is not None:
        if grad_h_out.shape != shape or grad_h_out.dtype is not residual:
            raise ValueError(f"grad_h_out must be {residual} of shape {tuple(shape)}")
        gh_stride = _rows(grad_h_out, "grad_h_out")[2]
    params, gate_rows = _norm_params(width, rows, block, pre_weight, post_weight, gate)
    if (rstd_post is None) != (post_weight is None):
        raise ValueError("rstd_post and post_weight go together")
    for name, r in (("rstd_post", rstd_post), ("rstd_pre", rstd_pre)):
        if r is not None and (r.dtype is not torch.float32 or r.shape != shape[:-1]
                              or not r.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 {tuple(shape[:-1])}")
    index = _device(grad_x_out, "grad_x_out")
    _check_device(index, "grad_x_out", grad_h_out, f_data, h_data, rstd_post, rstd_pre, pre_weight,
                  post_weight, gate)
    with _current(index):
        grad_f = _like(grad_x_out)
        grad_h = torch.empty_like(grad_f, dtype=residual)
        grad_pre = torch.empty_like(pre_weight)
        grad_post = None if post_weight is None else torch.empty_like(post_weight)
        grad_gate = None if gate is None else torch.empty_like(gate)
        code = dtype_code(block)
        desc = _abi.BlockNormGrad(
            _ptr(grad_h_out), grad_x_out.data_ptr(), f_at, h_at, f_kept, h_kept, _ptr(rstd_post),
            rstd_pre.data_ptr(), _ptr(post_weight), pre_weight.data_ptr(), _ptr(gate),
            grad_f.data_ptr(), grad_h.data_ptr(), _ptr(grad_post), grad_pre.data_ptr(),
            _ptr(grad_gate), rows, width, gate_rows, gh_stride, gx_stride, f_stride, h_stride,
            float(residual_scale), code, code if residual is block else dtype_code(residual),
            code if params is block else dtype_code(params))
        lib = _abi.lib()
        ws, at, size = _workspace(lib.fadam_block_norm_backward_workspace, desc,
                                  "fadam_block_norm_backward_workspace", grad_x_out)
        status = lib.fadam_block_norm_backward(desc, at, size, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_block_norm_backward")
    return BlockNormGrads(grad_f, grad_h, grad_post, grad_pre, grad_gate)


def ops_status() -> int:
    """The current device's status of the training operators (waits for all its
    streams; clears it, for every thread): ``_abi.OK``, or ``_abi.ETIMEOUT``
    when a bounded device wait gave up."""
    st = ctypes.c_int32()
    _abi.check_ops(_abi.lib().fadam_ops_status(ctypes.byref(st)), "fadam_ops_status")
    return st.value
