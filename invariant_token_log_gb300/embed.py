"""PyTorch front end of the embedding: argument marshalling only.

    y_i = round(scale * weight[id_i]),   dweight[v] = scale * sum of dy_i over the i with id_i = v

The gradient sums each token's rows in a fixed order (its places sorted, no atomics
on floating-point numbers), so its bits are reproducible.

Tokens are [*lead] int64 (narrower integers are widened); the table [V, H] is
float32, bfloat16 or float16 with unit column stride.  A token outside the table
gives a NaN row and no gradient; one equal to ``padding_idx`` gives its row and no
gradient.  Outputs whose H is no multiple of 16 bytes are views of rows that are
padded to one.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from .logp import _DEVICE_OBJECTS, _NARROW_INTS, _code, _device_object, _first_derivative, _need_cuda, _stream_handle
from .norm import _call, _padded, _rows


def _tokens(ids: torch.Tensor, index: int) -> torch.Tensor:
    if ids.dtype is not torch.int64:
        if ids.dtype not in _NARROW_INTS:
            raise TypeError("ids must be an integer tensor")
        ids = ids.to(torch.int64)
    if ids.get_device() != index:
        raise ValueError("ids must be on the rows' device")
    return ids if ids.dim() == 1 and ids.is_contiguous() else ids.reshape(-1).contiguous()


def embedding_fwd(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """The tokens' rows of the table times ``scale``: [*lead, H] in the table's type."""
    index = weight.get_device()
    if index < 0 or ids.get_device() < 0:
        _need_cuda(ids, weight)
    if weight.dim() != 2 or weight.shape[0] < 1 or weight.shape[1] < 1:
        raise ValueError("weight must be [V, H]")
    code = _code(weight.dtype)
    t = _tokens(ids, index)
    w2, ld_w = _rows(weight, "weight")
    vocab, width = w2.shape
    y, ld_y = _padded(t.shape[0], width, 4 if code == _lib.F32 else 8, w2.dtype,
                      _DEVICE_OBJECTS.get(index) or _device_object(index))
    _call("bil_embedding_fwd", index, t.data_ptr(), t.shape[0], w2.data_ptr(), code, vocab, width, ld_w, float(scale),
          y.data_ptr(), ld_y, _stream_handle(index))
    return y if ids.dim() == 1 else y.reshape(*ids.shape, width)


@functools.lru_cache(maxsize=256)
def bwd_workspace_bytes(n_tokens: int, width: int) -> int:
    """Device scratch bytes ``embedding_bwd`` needs: the sorted places and the sums of tokens in several segments."""
    out = ctypes.c_int64(0)
    _lib.check("bil_embedding_bwd_workspace_bytes",
               _lib.load().bil_embedding_bwd_workspace_bytes(n_tokens, width, ctypes.byref(out)))
    return out.value


def embedding_bwd(dy: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0, padding_idx: int | None = None,
                  out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None, accumulate: bool = False,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The table's gradient [vocab, H], every row of it, in ``out_dtype`` (dy's type, the
    default, or float32) from dy [*lead, H].  ``out`` receives it; with ``accumulate``
    it is added to what ``out`` holds (a tied LM head's gradient, or the last
    microbatch's), and rows without a token are not touched."""
    index = dy.get_device()
    if index < 0 or ids.get_device() < 0 or (out is not None and out.get_device() < 0):
        _need_cuda(dy, ids, out)
    if dy.dim() < 1 or tuple(dy.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"dy {tuple(dy.shape)} must have ids' shape {tuple(ids.shape)} and a last dimension")
    vocab = int(vocab)
    if vocab < 1 or dy.shape[-1] < 1:
        raise ValueError("the table needs at least one row and one column")
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError(f"padding_idx {padding_idx} outside [0, {vocab})")
    code = _code(dy.dtype)
    t = _tokens(ids, index)
    d2, ld_dy = _rows(dy, "dy")
    n, width = d2.shape
    dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
    if out is None:
        if accumulate:
            raise ValueError("accumulate adds to out: give it")
        out_dtype = dy.dtype if out_dtype is None else out_dtype
        if out_dtype not in (dy.dtype, torch.float32):
            raise TypeError("out_dtype must be float32 or dy's type")
        out, ld_out = _padded(vocab, width, 4 if out_dtype == torch.float32 else 8, out_dtype, dev)
    else:
        if out_dtype is not None and out_dtype != out.dtype:
            raise TypeError("out_dtype is not out's type")
        if tuple(out.shape) != (vocab, width) or out.get_device() != index or out.dtype not in (dy.dtype, torch.float32):
            raise ValueError(f"out must be [{vocab}, {width}] of dy's type or float32 on dy's device")
        if (width > 1 and out.stride(1) != 1) or (vocab > 1 and out.stride(0) < width):
            raise ValueError("out must have rows of unit column stride that do not overlap")
        ld_out = out.stride(0) if vocab > 1 else max(out.stride(0), width)
    need = bwd_workspace_bytes(n, width)
    if workspace is None:
        workspace, have = torch.empty(need or 16, dtype=torch.uint8, device=dev), need
    else:
        _need_cuda(workspace)
        have = workspace.numel() * workspace.element_size()
        if have < need or not workspace.is_contiguous():
            raise ValueError(f"workspace holds {have} bytes, needs {need}")
    _call("bil_embedding_bwd", index, d2.data_ptr(), code, n, width, ld_dy, t.data_ptr(), vocab, float(scale),
          -1 if padding_idx is None else int(padding_idx), out.data_ptr(), _code(out.dtype), ld_out,
          1 if accumulate else 0, workspace.data_ptr(), have, _stream_handle(index))
    return out


class Embedding(torch.autograd.Function):
    """y = Embedding.apply(ids, weight, scale, padding_idx)"""

    @staticmethod
    def forward(ctx, ids, weight, scale, padding_idx):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale, ctx.padding_idx = weight.shape[0], scale, padding_idx
        return embedding_fwd(ids, weight, scale)

    @staticmethod
    def backward(ctx, grad):
        (ids,) = ctx.saved_tensors
        dw = embedding_bwd(grad, ids, ctx.vocab, ctx.scale, ctx.padding_idx)
        return None, _first_derivative(dw, grad), None, None


def embedding(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0, padding_idx: int | None = None) -> torch.Tensor:
    """Differentiable ``embedding_fwd``: the table's gradient is dense."""
    if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
        raise ValueError(f"padding_idx {padding_idx} outside [0, {weight.shape[0]})")
    return Embedding.apply(ids, weight, scale, padding_idx)
