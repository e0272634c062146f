"""Python face of the sequence operators (include/fadam_seq.h).

They stand next to the training operators (``training.py``) and follow the same
rules: the token embedding with its weight's gradient, and attention over packed
documents, forward and backward.  Matrices are tensors whose leading dimensions
are taken together and must be evenly strided; no matrix is copied, nothing
synchronises, calls can be captured in a CUDA graph (the tensors they are given
have to live as long as it does), and the functions stand outside autograd.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _abi
from .optimizer import _ptr, dtype_code
from .training import _16BIT, _check_device, _current, _device, _rows, _stream, _workspace


class Attention(NamedTuple):
    """What ``attention`` returns."""
    out: torch.Tensor     # as q
    lse: torch.Tensor     # fp32, q's shape without the last dimension


class AttentionGrads(NamedTuple):
    """What ``attention_backward`` returns."""
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor


# ---- token embedding ---------------------------------------------------------------------

def _tokens(tokens: torch.Tensor) -> torch.Tensor:
    if tokens.dtype != torch.int64:
        raise TypeError(f"tokens must be int64, got {tokens.dtype}")
    return tokens.contiguous()


def embedding(tokens: torch.Tensor, weight: torch.Tensor, *, scale: float = 1.0,
              padding_index: Optional[int] = None,
              dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """The rows of ``weight`` [vocab, width] (bf16, fp16 or fp32) at ``tokens``
    [...] (int64), times ``scale``: [..., width] of the weight's dtype, or of
    ``dtype`` fp32 (``fadam_embed_forward``).  A token that is ``padding_index``
    gives zeros, one outside the vocabulary NaN, which reaches the loss and with
    it the shard's screen or norm."""
    if weight.dim() != 2:
        raise ValueError(f"weight must be [vocab, width], got {tuple(weight.shape)}")
    kind = weight.dtype
    code = out_code = dtype_code(kind)
    if dtype is not None and dtype is not kind:
        if dtype is not torch.float32:
            raise TypeError(f"dtype must be {kind} or fp32, got {dtype}")
        kind, out_code = dtype, _abi.DT_F32
    tokens = _tokens(tokens)
    index = _device(tokens, "tokens")
    _check_device(index, "tokens", weight)
    vocab, width, stride = _rows(weight, "weight")
    with _current(index):
        out = tokens.new_empty((*tokens.shape, width), dtype=kind)
        desc = _abi.Embed(tokens.data_ptr(), weight.data_ptr(), out.data_ptr(), tokens.numel(),
                          width, vocab, stride, width, int(padding_index or 0), float(scale), code,
                          out_code, 0 if padding_index is None else _abi.EMBED_PADDING)
        status = _abi.lib().fadam_embed_forward(desc, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_embed_forward")
    return out


def embedding_weight_grad(grad: torch.Tensor, tokens: torch.Tensor, vocab: Optional[int] = None, *,
                          scale: float = 1.0, padding_index: Optional[int] = None,
                          out: Optional[torch.Tensor] = None,
                          accumulate: bool = False) -> torch.Tensor:
    """The gradient [vocab, width] of ``embedding``'s weight, from that of its
    output [..., width] (``fadam_embed_grad_run``).  ``out`` is a buffer of
    grad's dtype or fp32 (any where grad is fp32), such as a view of an
    optimizer shard's gradient; with ``accumulate`` the gradient is added to it
    and rows of no token are not touched, else they are zero.  Padding and
    tokens outside the vocabulary have no gradient.  A token's rows are summed
    in one fixed order."""
    tokens = _tokens(tokens)
    if grad.dim() < 1 or grad.shape[:-1] != tokens.shape:
        raise ValueError(f"grad {tuple(grad.shape)} is not [..., width] over tokens {tuple(tokens.shape)}")
    if accumulate and out is None:
        raise ValueError("accumulate needs an out buffer")
    if vocab is None and out is None:
        raise ValueError("vocab or an out buffer must be given")
    code = dtype_code(grad.dtype)
    index = _device(grad, "grad")
    _check_device(index, "grad", tokens, out)
    _, width, stride = _rows(grad, "grad")
    if out is not None:
        if out.dim() != 2 or out.shape[1] != width or vocab not in (None, out.shape[0]):
            raise ValueError(f"out must be [{'vocab' if vocab is None else vocab}, {width}]")
        if out.dtype not in (grad.dtype, torch.float32) and grad.dtype is not torch.float32:
            raise TypeError(f"out must be {grad.dtype} or fp32, got {out.dtype}")
    with _current(index):
        if out is None:
            out = torch.empty((vocab, width), dtype=grad.dtype, device=grad.device)
        desc = _abi.EmbedGrad(
            tokens.data_ptr(), grad.data_ptr(), out.data_ptr(), tokens.numel(), width, out.shape[0],
            stride, _rows(out, "out")[2], int(padding_index or 0), float(scale), code,
            dtype_code(out.dtype), (_abi.EMBED_ACCUMULATE if accumulate else 0)
            | (0 if padding_index is None else _abi.EMBED_PADDING))
        lib = _abi.lib()
        ws, at, size = _workspace(lib.fadam_embed_grad_workspace, desc,
                                  "fadam_embed_grad_workspace", grad)
        status = lib.fadam_embed_grad_run(desc, at, size, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_embed_grad_run")
    return out


# ---- attention ---------------------------------------------------------------------------

def _heads(t: torch.Tensor, shape: tuple, what: str):
    """(token stride, head stride) of [..., tokens, heads, width]."""
    step, width = t.stride(), shape[-1]
    if step[-1] != 1 and width > 1:
        raise ValueError(f"the last dimension of {what} is not contiguous")
    # tokens: the dimensions before the heads, evenly strided
    token, many = step[-3], shape[-3]
    for n, s in zip(shape[-4::-1], step[-4::-1]):
        if n == 1:
            continue
        if many == 1:
            token = s
        elif s != token * many and n and many:
            raise ValueError(f"the leading dimensions of {what} are not evenly strided")
        many *= n
    return (token if many > 1 else shape[-2] * width), (step[-2] if shape[-2] > 1 else width)


def _attention(q, k, v, causal, scale, softcap, slopes, documents, prefix):
    """The descriptor but for out and lse, and the device."""
    dtype = q.dtype
    if dtype not in _16BIT or k.dtype is not dtype or v.dtype is not dtype:
        raise TypeError(f"q, k and v must all be bf16 or fp16, got {dtype}, {k.dtype} and {v.dtype}")
    of_q, of_k = tuple(q.shape), tuple(k.shape)
    if len(of_q) < 3:
        raise ValueError(f"q must be [..., tokens, heads, width], got {of_q}")
    if of_k != tuple(v.shape) or of_k[:-2] != of_q[:-2] or of_k[-1] != of_q[-1]:
        raise ValueError(f"q {of_q}, k {of_k} and v {tuple(v.shape)} do not fit")
    qs, ks, vs = _heads(q, of_q, "q"), _heads(k, of_k, "k"), _heads(v, of_k, "v")
    sequence, heads, width = of_q[-3:]
    kv_heads = of_k[-2]
    if not kv_heads or not heads or heads % kv_heads:
        raise ValueError(f"{kv_heads} heads of k and v do not divide {heads} of q")
    if width % 8 or not 0 < width <= _abi.ATTENTION_MAX_WIDTH:
        raise ValueError(f"a head's width must be a multiple of 8 up to "
                         f"{_abi.ATTENTION_MAX_WIDTH}, got {width}")
    index = _device(q, "q")
    _check_device(index, "q", k, v, slopes, documents, prefix)
    if slopes is not None and (slopes.dtype is not torch.float32 or slopes.shape != (heads,)
                               or not slopes.is_contiguous()):
        raise ValueError(f"slopes must be a contiguous fp32 [{heads}]")
    tokens = q.numel() // (heads * width)
    count = tokens // sequence if sequence else 0
    if documents is not None:
        if documents.dtype is not torch.int32 or documents.dim() != 1 or not documents.is_contiguous() \
                or documents.shape[0] < 1:
            raise ValueError("documents must be a contiguous int32 [n + 1]")
        count = documents.shape[0] - 1
    if prefix is not None:
        if not causal:
            raise ValueError("a prefix without causal: every key is seen already")
        if prefix.dtype is not torch.int32 or prefix.shape != (count,) or not prefix.is_contiguous():
            raise ValueError(f"prefix must be a contiguous int32 [{count}]")
    return index, _abi.Attention(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, _ptr(slopes), _ptr(documents),
        _ptr(prefix), tokens, max(sequence, 1), count, qs[0], ks[0], vs[0], qs[1], ks[1], vs[1],
        heads, kv_heads, width, float(width ** -0.5 if scale is None else scale), float(softcap),
        dtype_code(dtype), _abi.ATTENTION_CAUSAL if causal else 0, 0)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = True,
              scale: Optional[float] = None, softcap: float = 0.0,
              slopes: Optional[torch.Tensor] = None, documents: Optional[torch.Tensor] = None,
              prefix: Optional[torch.Tensor] = None) -> Attention:
    """Softmax attention within documents (``fadam_attention_run``).

    ``q`` [..., tokens, heads, width], ``k`` and ``v`` [..., tokens, kv_heads,
    width] are bf16 or fp16, ``kv_heads`` divides ``heads`` (query heads next to
    each other share one), the width is a multiple of 8 up to 128; views of one
    projection's output are taken as they are, where they start on 16 bytes and
    their strides are multiples of 8.  Each run of ``tokens`` is one
    document, or (``documents``, int32 [n + 1] on the device) all tokens
    together are cut into documents at these offsets, and tokens outside them
    see nothing: their rows are 0 and their lse -infinity.

    The score of query i and key j is ``scale * q_i . k_j`` (scale: width^-0.5),
    with ``softcap`` > 0 put through ``softcap * tanh(s / softcap)``, then with
    ``slopes`` (fp32 [heads]) lowered by ``slopes[h] * |i - j|``.  With
    ``causal`` i sees j <= i and, with ``prefix`` (int32, one number for each
    document or run), the first ``prefix`` tokens of its document too.
    """
    index, desc = _attention(q, k, v, causal, scale, softcap, slopes, documents, prefix)
    with _current(index):
        shape = q.shape
        out = q.new_empty(shape)
        lse = q.new_empty(shape[:-1], dtype=torch.float32)
        desc.out, desc.lse = out.data_ptr(), lse.data_ptr()
        lib = _abi.lib()
        ws, at, size = _workspace(lib.fadam_attention_workspace, desc, "fadam_attention_workspace", q)
        status = lib.fadam_attention_run(desc, at, size, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_attention_run")
    return Attention(out, lse)


def attention_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       out: torch.Tensor, lse: torch.Tensor, *, causal: bool = True,
                       scale: Optional[float] = None, softcap: float = 0.0,
                       slopes: Optional[torch.Tensor] = None,
                       documents: Optional[torch.Tensor] = None,
                       prefix: Optional[torch.Tensor] = None) -> AttentionGrads:
    """The gradients of ``attention`` with respect to q, k and v, from that of
    ``out`` and from what the forward pass left (``fadam_attention_backward``);
    the other arguments are those of the forward call.  The slopes are constants.
    The gradients of k and v are sums over the query heads that share them, in
    one fixed order."""
    index, desc = _attention(q, k, v, causal, scale, softcap, slopes, documents, prefix)
    shape = tuple(q.shape)
    for name, t in (("out", out), ("grad_out", grad_out)):
        if tuple(t.shape) != shape or t.dtype is not q.dtype:
            raise ValueError(f"{name} must be {q.dtype} of shape {shape}")
    if tuple(lse.shape) != shape[:-1] or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous fp32 {shape[:-1]}")
    strides = *_heads(out, shape, "out"), *_heads(grad_out, shape, "grad_out")
    _check_device(index, "q", grad_out, out, lse)
    with _current(index):
        grads = AttentionGrads(*(t.new_empty(t.shape) for t in (q, k, v)))
        desc.out, desc.lse = out.data_ptr(), lse.data_ptr()
        desc = _abi.AttentionGrad(desc, grad_out.data_ptr(), *(t.data_ptr() for t in grads), *strides)
        lib = _abi.lib()
        ws, at, size = _workspace(lib.fadam_attention_backward_workspace, desc,
                                  "fadam_attention_backward_workspace", q)
        status = lib.fadam_attention_backward(desc, at, size, _stream(index))
    if status:
        _abi.check_ops(status, "fadam_attention_backward")
    return grads
