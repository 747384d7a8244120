"""PyTorch front end of the LM head's cross entropy: argument marshalling only.

    z = hidden . weight^T
    loss_r = lse_r - (1 - e) z_rt - (e / V) sum_c z_rc + f lse_r^2      (e: label_smoothing, f: z_loss)

and the gradients of hidden and weight, without the logits: the forward keeps what a
row needs of each 128 columns, the backward goes over the vocabulary in pieces.  Rows
whose target is ``ignore_index`` take no part: their loss and gradient are 0, their
hidden states are not read.  A target outside the vocabulary gives a NaN loss.

``reduction``: "mean" over the rows that are not ignored (over none: 0), "sum", or "none".

Layouts as ``linear_logp``'s: hidden [*lead, H] and weight [V, H], both bfloat16 or both
float16, rows 16-byte aligned.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from .linear import _IN_DTYPES, _in_code, _ld, _matrix, _pad8
from .logp import (
    _DEVICE_OBJECTS,
    IGNORE_INDEX,
    _device_object,
    _first_derivative,
    _need_cuda,
    _stream_handle,
    _targets1d,
)
from .norm import _call, _padded

_REDUCTIONS = {"none": 0, "mean": 1, "sum": 2}


def _operands(hidden, weight, target_ids, label_smoothing, reduction):
    index = hidden.get_device()
    lead, dtype = target_ids.shape, hidden.dtype
    if (index >= 0 and target_ids.dtype is torch.int64 and len(lead) == 1 and dtype in _IN_DTYPES and
            weight.dtype is dtype and target_ids.get_device() == index and weight.get_device() == index):
        # The common call, row-major matrices and int64 [N], without the general path's conversions.
        h_shape, w_shape = hidden.shape, weight.shape
        if (len(h_shape) == 2 and len(w_shape) == 2 and h_shape[0] == lead[0] and h_shape[1] == w_shape[1] and
                w_shape[0] and w_shape[1] and w_shape[1] % 8 == 0 and hidden.is_contiguous() and weight.is_contiguous() and
                target_ids.is_contiguous() and hidden.data_ptr() % 16 == 0 and weight.data_ptr() % 16 == 0 and
                0.0 <= label_smoothing <= 1.0 and reduction in _REDUCTIONS):
            return (index, _DEVICE_OBJECTS.get(index) or _device_object(index), _IN_DTYPES[dtype], lead, hidden, weight,
                    target_ids, w_shape[1], w_shape[1])
    if index < 0 or weight.get_device() < 0 or target_ids.get_device() < 0:
        _need_cuda(hidden, weight, target_ids)
    if hidden.dim() < 1 or weight.dim() != 2:
        raise ValueError("hidden is [*lead, H], weight [V, H]")
    if hidden.dtype != weight.dtype:
        raise TypeError("hidden and weight must have the same element type")
    if hidden.shape[-1] != weight.shape[1] or weight.shape[0] < 1 or weight.shape[1] < 1:
        raise ValueError(f"hidden size {hidden.shape[-1]} != weight's {weight.shape[1]}, or an empty weight")
    if weight.get_device() != index:
        raise ValueError("hidden and weight must be on one device")
    if not 0.0 <= label_smoothing <= 1.0:
        raise ValueError(f"label_smoothing {label_smoothing} outside [0, 1]")
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction {reduction!r}: it is one of {', '.join(_REDUCTIONS)}")
    code = _in_code(hidden.dtype)
    lead = hidden.shape[:-1]
    dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
    t = _targets1d(target_ids, lead, dev)
    h2 = hidden if hidden.dim() == 2 else hidden.reshape(t.shape[0], hidden.shape[-1])
    h2, w2 = _matrix(h2, "hidden"), _matrix(weight, "weight")
    if h2.shape[0] > 1 and h2.stride(0) < h2.shape[1]:
        h2 = h2.contiguous()  # an expanded tensor
    if w2.shape[0] > 1 and w2.stride(0) < w2.shape[1]:
        w2 = w2.contiguous()
    return index, dev, code, lead, h2, w2, t, _ld(h2), _ld(w2)


def _scratch(workspace: torch.Tensor | None, need: int, dev: torch.device) -> tuple[torch.Tensor, int]:
    if workspace is None:
        return torch.empty(need or 16, dtype=torch.uint8, device=dev), need
    _need_cuda(workspace)
    have = workspace.numel() * workspace.element_size()
    if have < need or not workspace.is_contiguous():
        raise ValueError(f"workspace holds {have} bytes, needs {need}")
    return workspace, have


@functools.lru_cache(maxsize=256)
def fwd_workspace_bytes(n_rows: int, hidden_size: int, vocab: int, smoothing: bool = False) -> int:
    """Device scratch bytes of ``linear_cross_entropy_fwd``."""
    out = ctypes.c_int64(0)
    _lib.check("bil_linear_cross_entropy_fwd_workspace_bytes", _lib.load().bil_linear_cross_entropy_fwd_workspace_bytes(
        n_rows, hidden_size, vocab, 1 if smoothing else 0, ctypes.byref(out)))
    return out.value


@functools.lru_cache(maxsize=256)
def _bwd_workspace_bytes(n_rows: int, hidden_size: int, vocab: int, piece: int, index: int) -> int:
    out = ctypes.c_int64(0)
    _call("bil_linear_cross_entropy_bwd_workspace_bytes", index, n_rows, hidden_size, vocab, piece, ctypes.byref(out))
    return out.value


def bwd_workspace_bytes(n_rows: int, hidden_size: int, vocab: int, device: torch.device, piece: int = 0) -> int:
    """Device scratch bytes of ``linear_cross_entropy_bwd`` on a device."""
    return _bwd_workspace_bytes(n_rows, hidden_size, vocab, piece, device.index)


def linear_cross_entropy_fwd(hidden: torch.Tensor, weight: torch.Tensor, target_ids: torch.Tensor,
                             ignore_index: int = IGNORE_INDEX, label_smoothing: float = 0.0, z_loss: float = 0.0,
                             reduction: str = "mean", validate: bool = False, workspace: torch.Tensor | None = None):
    """(loss, lse): the float32 loss, one number or with reduction "none" [*lead], and the rows'
    lse [*lead] that ``linear_cross_entropy_bwd`` takes."""
    index, dev, code, lead, h2, w2, t, ld_h, ld_w = _operands(hidden, weight, target_ids, label_smoothing, reduction)
    n, hs = h2.shape
    vocab = w2.shape[0]
    loss = torch.empty(lead if reduction == "none" else (), dtype=torch.float32, device=dev)
    lse = torch.empty(lead, dtype=torch.float32, device=dev)
    workspace, have = _scratch(workspace, fwd_workspace_bytes(n, hs, vocab, label_smoothing > 0.0) if n else 0, dev)
    _call("bil_linear_cross_entropy_fwd", index, h2.data_ptr(), w2.data_ptr(), code, n, hs, ld_h, vocab, ld_w,
          t.data_ptr(), int(ignore_index), float(label_smoothing), float(z_loss), _REDUCTIONS[reduction],
          loss.data_ptr(), lse.data_ptr(), workspace.data_ptr(), have, 1 if validate else 0, _stream_handle(index))
    return loss, lse


def linear_cross_entropy_bwd(hidden: torch.Tensor, weight: torch.Tensor, target_ids: torch.Tensor, lse: torch.Tensor,
                             grad_loss: torch.Tensor, ignore_index: int = IGNORE_INDEX, label_smoothing: float = 0.0,
                             z_loss: float = 0.0, reduction: str = "mean", out_dtype: torch.dtype | None = None,
                             piece: int | None = None, need_hidden: bool = True, need_weight: bool = True,
                             workspace: torch.Tensor | None = None):
    """(dhidden [*lead, H], dweight [V, H]) for the gradient ``grad_loss`` of the loss (one
    number, or with reduction "none" [*lead]), in ``out_dtype``: the inputs' type (the
    default) or float32.  ``piece``: the columns of the vocabulary whose gradient is held
    at a time, 2 bytes for each of them and row.  One that is not needed is None."""
    index, dev, code, lead, h2, w2, t, ld_h, ld_w = _operands(hidden, weight, target_ids, label_smoothing, reduction)
    n, hs = h2.shape
    vocab = w2.shape[0]
    if not (need_hidden or need_weight):
        return None, None
    out_dtype = h2.dtype if out_dtype is None else out_dtype
    if out_dtype not in (torch.float32, h2.dtype):
        raise TypeError("out_dtype must be float32 or the inputs' type")
    if piece is not None and piece < 1:
        raise ValueError(f"a piece of {piece} columns")
    want = n if reduction == "none" else 1
    for x, what, count in ((lse, "lse", n), (grad_loss, "grad_loss", want)):
        if x.get_device() != index or x.numel() != count or not x.dtype.is_floating_point:
            raise ValueError(f"{what} must hold {count} numbers on hidden's device")
    lse, grad_loss = (x if x.dtype is torch.float32 and x.is_contiguous() else x.to(torch.float32).contiguous()
                      for x in (lse, grad_loss))
    oc = _lib.F32 if out_dtype == torch.float32 else code
    dh = dw = None
    if need_hidden:
        dh, _ = _padded(n, hs, 8, out_dtype, dev)
    if need_weight:
        dw, _ = _padded(vocab, hs, 8, out_dtype, dev)
    piece = 0 if piece is None else int(piece)
    workspace, have = _scratch(workspace, _bwd_workspace_bytes(n, hs, vocab, piece, index) if n else 0, dev)
    _call("bil_linear_cross_entropy_bwd", index, h2.data_ptr(), w2.data_ptr(), code, n, hs, ld_h, vocab, ld_w,
          t.data_ptr(), int(ignore_index), float(label_smoothing), float(z_loss), _REDUCTIONS[reduction],
          lse.data_ptr(), grad_loss.data_ptr(), piece, None if dh is None else dh.data_ptr(), oc,
          0 if dh is None else _pad8(hs), None if dw is None else dw.data_ptr(), oc, 0 if dw is None else _pad8(hs),
          workspace.data_ptr(), have, _stream_handle(index))
    return (dh if dh is None or len(lead) == 1 else dh.reshape(*lead, hs)), dw


class LinearCrossEntropy(torch.autograd.Function):
    """loss = LinearCrossEntropy.apply(hidden, weight, target_ids, ignore_index, label_smoothing, z_loss, reduction,
    piece): the forward keeps the rows' lse, the backward computes the logits again."""

    @staticmethod
    def forward(ctx, hidden, weight, target_ids, ignore_index, label_smoothing, z_loss, reduction, piece):
        loss, lse = linear_cross_entropy_fwd(hidden, weight, target_ids, ignore_index, label_smoothing, z_loss, reduction)
        ctx.save_for_backward(hidden, weight, target_ids, lse)
        ctx.how = (ignore_index, label_smoothing, z_loss, reduction)
        ctx.piece = piece
        return loss

    @staticmethod
    def backward(ctx, grad):
        hidden, weight, target_ids, lse = ctx.saved_tensors
        need_h, need_w = ctx.needs_input_grad[:2]
        dh, dw = linear_cross_entropy_bwd(hidden, weight, target_ids, lse, grad, *ctx.how, piece=ctx.piece,
                                          need_hidden=need_h, need_weight=need_w)
        dh, dw = (None if d is None else _first_derivative(d, grad, hidden, weight) for d in (dh, dw))
        return dh, dw, None, None, None, None, None, None


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, target_ids: torch.Tensor,
                         ignore_index: int = IGNORE_INDEX, label_smoothing: float = 0.0, z_loss: float = 0.0,
                         reduction: str = "mean", piece: int | None = None) -> torch.Tensor:
    """Differentiable loss of the LM head on hidden states: see ``linear_cross_entropy_fwd`` and ``_bwd``."""
    return LinearCrossEntropy.apply(hidden, weight, target_ids, ignore_index, label_smoothing, z_loss, reduction, piece)
