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
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Union

import torch

from . import _abi
from .optimizer import _ptr, _stream_handle, dtype_code

_16BIT = (torch.bfloat16, torch.float16)


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
    width = t.shape[-1]
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


def _same_device(device: torch.device, **tensors: Optional[torch.Tensor]) -> None:
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}, not on a CUDA device")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _workspace(size_of, desc, where: str, device: torch.device) -> Optional[torch.Tensor]:
    need = ctypes.c_size_t()
    _abi.check_ops(size_of(ctypes.byref(desc), ctypes.byref(need)), where)
    return torch.empty(need.value, dtype=torch.uint8, device=device) if need.value else None


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
    held in 16 bits (``chunk_rows``; 0 chooses).  ``reduction`` is "mean" over
    the rows whose target is not ``ignore_index`` (0 when there is none) or
    "sum".  The gradients are those of ``loss_scale * loss``: an optimizer
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
    device = x.device
    _same_device(device, weight=weight, targets=targets, grad_weight=grad_weight)
    vocab, _, w_stride = _rows(weight, "weight")
    targets = targets.contiguous()
    with torch.cuda.device(device):
        row_loss, lse = torch.empty(2, *targets.shape, dtype=torch.float32, device=device)
        loss = torch.empty((), dtype=torch.float32, device=device)
        grad_x, gw_stride = None, width
        if grads:
            grad_x = torch.empty(x.shape, dtype=x.dtype, device=device)
            if grad_weight is None:
                grad_weight = torch.empty(vocab, width, dtype=weight.dtype, device=device)
            elif (grad_weight.shape != weight.shape
                  or grad_weight.dtype not in (weight.dtype, torch.float32)):
                raise ValueError("grad_weight must have the weight's shape, and its dtype or fp32")
            gw_stride = _rows(grad_weight, "grad_weight")[2]
        flags = ((_abi.XENT_MEAN if reduction == "mean" else 0)
                 | (_abi.XENT_ACCUMULATE if accumulate else 0))
        desc = _abi.Xent(
            x=x.data_ptr(), w=weight.data_ptr(), targets=targets.data_ptr(), loss=loss.data_ptr(),
            row_loss=row_loss.data_ptr(), lse=lse.data_ptr(), grad_x=_ptr(grad_x),
            grad_w=_ptr(grad_weight), rows=rows, width=width, vocab=vocab, x_stride=x_stride,
            w_stride=w_stride, grad_x_stride=width, grad_w_stride=gw_stride,
            ignore_index=int(ignore_index), chunk_rows=int(chunk_rows),
            loss_scale=float(loss_scale), dtype=dtype_code(x.dtype),
            grad_w_dtype=dtype_code(grad_weight.dtype if grads else x.dtype), flags=flags)
        lib = _abi.lib()
        ws = _workspace(lib.fadam_xent_workspace, desc, "fadam_xent_workspace", device)
        _abi.check_ops(lib.fadam_xent_run(ctypes.byref(desc), _ptr(ws), ws.numel() if ws is not None
                                          else 0, _stream_handle(device)), "fadam_xent_run")
    return LinearCrossEntropy(loss, row_loss, lse, grad_x, grad_weight)


# ---- 8-bit checkpoints ---------------------------------------------------------------

def _empty_checkpoint(like: torch.Tensor) -> Checkpoint8:
    groups = -(-like.shape[-1] // _abi.CHECKPOINT8_GROUP)
    return Checkpoint8(torch.empty(like.shape, dtype=torch.int8, device=like.device),
                       torch.empty(*like.shape[:-1], groups, dtype=torch.float32,
                                   device=like.device), like.dtype)


def _kept(c: Optional[Checkpoint8]) -> _abi.Kept8:
    return _abi.Kept8() if c is None else _abi.Kept8(c.codes.data_ptr(), c.scales.data_ptr())


def _check_checkpoint(c: Checkpoint8, what: str) -> None:
    groups = -(-c.codes.shape[-1] // _abi.CHECKPOINT8_GROUP)
    if (c.codes.dtype != torch.int8 or c.scales.dtype != torch.float32
            or not c.codes.is_contiguous() or not c.scales.is_contiguous()
            or c.scales.shape != (*c.codes.shape[:-1], groups)
            or c.codes.device != c.scales.device):
        raise ValueError(f"{what} is not a checkpoint: contiguous int8 codes [..., width] and fp32 "
                         "scales [..., ceil(width / 128)] on one device")


def checkpoint8(x: torch.Tensor) -> Checkpoint8:
    """An activation [..., width] (bf16, fp16 or fp32) kept in 8 bits, one fp32
    scale for each started group of 128 elements of a row: 1.03 bytes an
    element, each off by at most 1/254 of its group's largest magnitude.  A
    group that holds an infinity or a NaN is restored as NaN throughout."""
    rows, width, stride = _rows(x, "x")
    _same_device(x.device)
    code = dtype_code(x.dtype)
    with torch.cuda.device(x.device):
        out = _empty_checkpoint(x)
        _abi.check_ops(_abi.lib().fadam_checkpoint8_pack(
            x.data_ptr(), rows, width, stride, code, ctypes.byref(_kept(out)),
            _stream_handle(x.device)), "fadam_checkpoint8_pack")
    return out


def checkpoint8_restore(c: Checkpoint8) -> torch.Tensor:
    """The activation that ``checkpoint8`` kept, in its dtype."""
    _check_checkpoint(c, "c")
    device = c.codes.device
    _same_device(device)
    rows, width, stride = _rows(c.codes, "c")
    with torch.cuda.device(device):
        x = torch.empty(c.codes.shape, dtype=c.dtype, device=device)
        _abi.check_ops(_abi.lib().fadam_checkpoint8_restore(
            ctypes.byref(_kept(c)), rows, width, x.data_ptr(), stride, dtype_code(c.dtype),
            _stream_handle(device)), "fadam_checkpoint8_restore")
    return x


def checkpoint8_weight_grad(grad_y: torch.Tensor, c: Checkpoint8, *,
                            out: Optional[torch.Tensor] = None,
                            accumulate: bool = False) -> torch.Tensor:
    """The weight gradient ``grad_y.T @ x`` [n, width] of a linear layer, from
    its output's gradient [..., n] (bf16 or fp16) and the checkpoint of its
    input [..., width].  ``out`` is a buffer of grad_y's dtype or fp32, such as
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
    device = grad_y.device
    _same_device(device, checkpoint=c.codes, out=out)
    rows, n, stride = _rows(grad_y, "grad_y")
    width = c.codes.shape[-1]
    with torch.cuda.device(device):
        if out is None:
            out = torch.empty(n, width, dtype=grad_y.dtype, device=device)
        elif out.shape != (n, width) or out.dtype not in (grad_y.dtype, torch.float32):
            raise ValueError(f"out must be [{n}, {width}] of grad_y's dtype or fp32")
        desc = _abi.Wgrad(dy=grad_y.data_ptr(), x=_kept(c), out=out.data_ptr(), rows=rows, n=n,
                          width=width, dy_stride=stride, out_stride=_rows(out, "out")[2],
                          dtype=dtype_code(grad_y.dtype), out_dtype=dtype_code(out.dtype),
                          flags=_abi.WGRAD_ACCUMULATE if accumulate else 0)
        lib = _abi.lib()
        ws = _workspace(lib.fadam_checkpoint8_wgrad_workspace, desc,
                        "fadam_checkpoint8_wgrad_workspace", device)
        _abi.check_ops(lib.fadam_checkpoint8_wgrad(
            ctypes.byref(desc), _ptr(ws), ws.numel() if ws is not None else 0,
            _stream_handle(device)), "fadam_checkpoint8_wgrad")
    return out


# ---- the norms around a block ------------------------------------------------------------

def _norm_params(width: int, rows: int, block: torch.dtype, pre_weight, post_weight, gate):
    """The parameters' dtype, and how many rows the gate has."""
    for name, w in (("pre_weight", pre_weight), ("post_weight", post_weight)):
        if w is not None and (w.shape != (width,) or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous [{width}]")
    dtype = pre_weight.dtype
    if any(t is not None and t.dtype != dtype for t in (post_weight, gate)):
        raise TypeError("pre_weight, post_weight and gate must have one dtype")
    if dtype not in (block, torch.float32):
        raise TypeError(f"the parameters must be {block} or fp32, got {dtype}")
    if gate is None:
        return dtype, 1
    if not gate.is_contiguous() or gate.shape[-1] != width:
        raise ValueError(f"gate must be a contiguous [..., {width}]")
    gate_rows = gate.numel() // width
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
    params, gate_rows = _norm_params(width, rows, f.dtype, pre_weight, post_weight, gate)
    device = f.device
    _same_device(device, h=h, pre_weight=pre_weight, post_weight=post_weight, gate=gate)
    with torch.cuda.device(device):
        h_out = torch.empty(h.shape, dtype=h.dtype, device=device)
        x_out = torch.empty(f.shape, dtype=f.dtype, device=device)
        r2 = torch.empty(f.shape[:-1], dtype=torch.float32, device=device)
        r1 = torch.empty_like(r2) if post_weight is not None else None
        f_kept = _empty_checkpoint(f) if checkpoint else None
        h_kept = _empty_checkpoint(h) if checkpoint else None
        desc = _abi.BlockNorm(
            f=f.data_ptr(), h=h.data_ptr(), post_weight=_ptr(post_weight),
            pre_weight=pre_weight.data_ptr(), gate=_ptr(gate), h_out=h_out.data_ptr(),
            x_out=x_out.data_ptr(), rstd_post=_ptr(r1), rstd_pre=r2.data_ptr(),
            f_kept=_kept(f_kept), h_kept=_kept(h_kept), rows=rows, width=width,
            gate_rows=gate_rows, f_stride=f_stride, h_stride=_rows(h, "h")[2],
            residual_scale=float(residual_scale), eps=float(eps), block_dtype=block,
            residual_dtype=dtype_code(h.dtype), param_dtype=dtype_code(params))
        _abi.check_ops(_abi.lib().fadam_block_norm_forward(ctypes.byref(desc),
                                                           _stream_handle(device)),
                       "fadam_block_norm_forward")
    return BlockNorm(h_out, x_out, r1, r2, f_kept, h_kept)


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
    block = grad_x_out.dtype
    saved, strides, dtypes = [], [], []
    for name, t in (("f", f), ("h_out", h_out)):
        kept = isinstance(t, Checkpoint8)
        if kept:
            _check_checkpoint(t, name)
        data = t.codes if kept else t
        if data.shape != grad_x_out.shape:
            raise ValueError(f"{name} {tuple(data.shape)} and grad_x_out "
                             f"{tuple(grad_x_out.shape)} differ in shape")
        saved.append((None, t) if kept else (t, None))
        strides.append(_rows(data, name)[2])
        dtypes.append(t.dtype)
    if dtypes[0] != block or dtypes[1] not in (block, torch.float32):
        raise TypeError(f"f must be {block} and h_out that or fp32, got {dtypes[0]}, {dtypes[1]}")
    if grad_h_out is not None and (grad_h_out.shape != grad_x_out.shape
                                   or grad_h_out.dtype != dtypes[1]):
        raise ValueError(f"grad_h_out must be {dtypes[1]} of shape {tuple(grad_x_out.shape)}")
    params, gate_rows = _norm_params(width, rows, block, pre_weight, post_weight, gate)
    if (rstd_post is None) != (post_weight is None):
        raise ValueError("rstd_post and post_weight go together")
    for name, r in (("rstd_post", rstd_post), ("rstd_pre", rstd_pre)):
        if r is not None and (r.dtype != torch.float32 or r.shape != grad_x_out.shape[:-1]
                              or not r.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 {tuple(grad_x_out.shape[:-1])}")
    device = grad_x_out.device
    _same_device(device, grad_h_out=grad_h_out, f=f[0] if isinstance(f, Checkpoint8) else f,
                 h_out=h_out[0] if isinstance(h_out, Checkpoint8) else h_out, rstd_post=rstd_post,
                 rstd_pre=rstd_pre, pre_weight=pre_weight, post_weight=post_weight, gate=gate)
    with torch.cuda.device(device):
        grad_f = torch.empty(grad_x_out.shape, dtype=block, device=device)
        grad_h = torch.empty(grad_x_out.shape, dtype=dtypes[1], device=device)
        grad_pre = torch.empty_like(pre_weight)
        grad_post = None if post_weight is None else torch.empty_like(post_weight)
        grad_gate = None if gate is None else torch.empty_like(gate)
        desc = _abi.BlockNormGrad(
            grad_h_out=_ptr(grad_h_out), grad_x_out=grad_x_out.data_ptr(), f=_ptr(saved[0][0]),
            h_out=_ptr(saved[1][0]), f_kept=_kept(saved[0][1]), h_kept=_kept(saved[1][1]),
            rstd_post=_ptr(rstd_post), rstd_pre=rstd_pre.data_ptr(),
            post_weight=_ptr(post_weight), pre_weight=pre_weight.data_ptr(), gate=_ptr(gate),
            grad_f=grad_f.data_ptr(), grad_h=grad_h.data_ptr(), grad_post_weight=_ptr(grad_post),
            grad_pre_weight=grad_pre.data_ptr(), grad_gate=_ptr(grad_gate), rows=rows, width=width,
            gate_rows=gate_rows,
            grad_h_out_stride=width if grad_h_out is None else _rows(grad_h_out, "grad_h_out")[2],
            grad_x_out_stride=gx_stride, f_stride=strides[0], h_out_stride=strides[1],
            residual_scale=float(residual_scale), block_dtype=dtype_code(block),
            residual_dtype=dtype_code(dtypes[1]), param_dtype=dtype_code(params))
        lib = _abi.lib()
        ws = _workspace(lib.fadam_block_norm_backward_workspace, desc,
                        "fadam_block_norm_backward_workspace", device)
        _abi.check_ops(lib.fadam_block_norm_backward(
            ctypes.byref(desc), _ptr(ws), ws.numel() if ws is not None else 0,
            _stream_handle(device)), "fadam_block_norm_backward")
    return BlockNormGrads(grad_f, grad_h, grad_post, grad_pre, grad_gate)


def ops_status() -> int:
    """The training operators' device status (synchronises; clears it):
    ``_abi.OK``, or ``_abi.ETIMEOUT`` when a bounded device wait gave up."""
    st = ctypes.c_int32()
    _abi.check_ops(_abi.lib().fadam_ops_status(ctypes.byref(st)), "fadam_ops_status")
    return st.value
