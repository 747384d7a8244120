"""PyTorch front end of the selected-token log-probability with the row's largest
alternatives: argument marshalling only.

``logp_topk`` gives what ``logp_fwd`` gives (the same bits) and the k most likely
columns of every row with their log-probabilities, in one pass over the logits;
``logp_topk_bwd`` is the gradient of all of it.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from .logp import (
    _DEVICE_OBJECTS,
    DEFAULT_TILE_V,
    IGNORE_INDEX,
    _code,
    _device_object,
    _f32_1d,
    _first_derivative,
    _get_device,
    _need_cuda,
    _on_device,
    _ptr,
    _row_stride,
    _rows2d,
    _stream_handle,
    _targets1d,
)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(dtype: int, n_rows: int, vocab: int, tile_v: int, k: int, entropy: bool) -> int:
    out = ctypes.c_int64(0)
    st = _lib.load().bil_logp_topk_workspace_bytes(dtype, n_rows, vocab, tile_v, k, int(entropy), ctypes.byref(out))
    if st:
        _lib.check("bil_logp_topk_workspace_bytes", st)
    return out.value


def workspace_bytes(dtype: torch.dtype, n_rows: int, vocab: int, k: int, tile_v: int = DEFAULT_TILE_V,
                    entropy: bool = False) -> int:
    """Device scratch bytes ``logp_topk`` needs (host arithmetic)."""
    return _workspace_bytes(_code(dtype), n_rows, vocab, tile_v, k, entropy)


def _logits2d(logits: torch.Tensor, vocab: int | None) -> tuple[torch.Tensor, int]:
    x2 = _rows2d(logits)
    if x2.shape[0] > 1 and x2.stride(0) < x2.shape[1]:
        x2 = x2.contiguous()  # an expanded tensor
    v = x2.shape[1] if vocab is None else int(vocab)
    if not 1 <= v <= x2.shape[1]:
        raise ValueError(f"vocab {v} outside [1, {x2.shape[1]}]")
    return x2, v


def logp_topk(logits: torch.Tensor, target_ids: torch.Tensor, k: int, ignore_index: int = IGNORE_INDEX,
              tile_v: int = DEFAULT_TILE_V, validate: bool = False, vocab: int | None = None,
              temperature: float = 1.0, return_entropy: bool = False, workspace: torch.Tensor | None = None):
    """(logp, lse[, entropy], top_ids, top_logp): ``logp_fwd``'s results and, per row, the k
    columns with the largest logits (int64 [*lead, k], best first, equal logits by the lowest
    column, NaN last) and their float32 log-probabilities.  Ignored rows give -1 and 0.

    1 <= k <= min(vocab, 128).  Other arguments as for ``logp_fwd``."""
    index = logits.get_device()
    if index < 0 or target_ids.get_device() < 0:
        _need_cuda(logits, target_ids)
    lead = logits.shape[:-1]
    x2, v = _logits2d(logits, vocab)
    n, width = x2.shape
    k = int(k)
    if not 1 <= k <= min(v, _lib.MAX_TOPK):
        raise ValueError(f"k {k} outside [1, {min(v, _lib.MAX_TOPK)}]")
    dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
    t1 = _targets1d(target_ids, lead, dev)
    code = _code(x2.dtype)
    # one allocation a result: on small batches the host's time is what counts, and a view costs more
    logp = torch.empty(n, dtype=torch.float32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev)
    entropy = torch.empty(n, dtype=torch.float32, device=dev) if return_entropy else None
    top_ids = torch.empty((n, k), dtype=torch.int64, device=dev)
    top_logp = torch.empty((n, k), dtype=torch.float32, device=dev)
    need = _workspace_bytes(code, n, v, tile_v, k, return_entropy)
    if workspace is None:
        have = need
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_cuda(workspace)
        have = workspace.numel() * workspace.element_size()
        if have < need or not workspace.is_contiguous():
            raise ValueError(f"workspace holds {have} bytes, needs {need}")
    fn = _lib.load().bil_logp_topk_fwd
    args = (x2.data_ptr(), code, n, v, x2.stride(0) if n > 1 else width, t1.data_ptr(), int(ignore_index), tile_v,
            float(temperature), k, logp.data_ptr(), lse.data_ptr(), entropy.data_ptr() if return_entropy else None,
            top_ids.data_ptr(), top_logp.data_ptr(), workspace.data_ptr() if have else None, have, 1 if validate else 0,
            _stream_handle(index))
    st = fn(*args) if _get_device() == index else _on_device(index, fn, *args)
    if st:
        _lib.check("bil_logp_topk_fwd", st)
    if len(lead) != 1:
        logp, lse = logp.reshape(lead), lse.reshape(lead)
        top_ids, top_logp = top_ids.reshape(*lead, k), top_logp.reshape(*lead, k)
        if return_entropy:
            entropy = entropy.reshape(lead)
    return (logp, lse, entropy, top_ids, top_logp) if return_entropy else (logp, lse, top_ids, top_logp)


def logp_topk_bwd(logits: torch.Tensor, target_ids: torch.Tensor, top_ids: torch.Tensor, lse: torch.Tensor,
                  grad_logp: torch.Tensor, grad_top: torch.Tensor, ignore_index: int = IGNORE_INDEX,
                  dlogits_dtype: torch.dtype | None = None, vocab: int | None = None,
                  out: torch.Tensor | None = None, temperature: float = 1.0, entropy: torch.Tensor | None = None,
                  grad_entropy: torch.Tensor | None = None) -> torch.Tensor:
    """dlogits of g * logp + sum_j gk_j * top_logp_j (+ gh * entropy) from the saved LSE (and entropy).

    ``top_ids`` and ``grad_top`` [*lead, k]: the forward's columns, or any others, and
    the gradients of their log-probabilities.  ``out`` must not be the logits.  Other
    arguments as for ``logp_bwd``."""
    _need_cuda(logits, target_ids, top_ids, lse, grad_logp, grad_top, out, entropy, grad_entropy)
    if (entropy is None) != (grad_entropy is None):
        raise ValueError("entropy and grad_entropy go together")
    lead = logits.shape[:-1]
    x2, v = _logits2d(logits, vocab)
    n, width = x2.shape
    dev = x2.device
    t1 = _targets1d(target_ids, lead, dev)
    if top_ids.dtype != torch.int64:
        raise TypeError("top_ids must be int64")
    k = top_ids.shape[-1] if top_ids.dim() else 0
    if tuple(top_ids.shape) != (*lead, k) or top_ids.shape != grad_top.shape:
        raise ValueError("top_ids and grad_top must have the targets' shape and k columns")
    if not 1 <= k <= min(v, _lib.MAX_TOPK):
        raise ValueError(f"k {k} outside [1, {min(v, _lib.MAX_TOPK)}]")
    ids = top_ids.reshape(n, k).contiguous()
    gk = grad_top.reshape(n, k).to(torch.float32).contiguous()
    per_row = [None if x is None else _f32_1d(x) for x in (lse, grad_logp, entropy, grad_entropy)]
    for x in (*per_row, ids, gk):
        if x is not None and (x.shape[0] != n or x.device != dev):
            raise ValueError("lse, the gradients and the entropy must have the targets' shape and device")
    odt = logits.dtype if dlogits_dtype is None else dlogits_dtype
    if out is None:
        out = torch.empty((n, width), dtype=odt, device=dev)
    if n == 0:
        return out.reshape(logits.shape) if out.numel() == 0 else out
    o2 = out if out.dim() == 2 else out.reshape(n, -1)
    if o2.shape[0] != n or o2.stride(-1) != 1 or o2.shape[1] < width:
        raise ValueError("out must be row-major with at least the logits' columns")
    sums = torch.empty(n, dtype=torch.float32, device=dev)
    st = _on_device(dev.index, _lib.load().bil_logp_topk_bwd, x2.data_ptr(), _code(x2.dtype), n, v, _row_stride(x2),
                    t1.data_ptr(), int(ignore_index), float(temperature), ids.data_ptr(), k, _ptr(per_row[0]),
                    _ptr(per_row[1]), gk.data_ptr(), _ptr(per_row[2]), _ptr(per_row[3]), o2.data_ptr(),
                    _code(o2.dtype), _row_stride(o2), width, sums.data_ptr(), _stream_handle(dev.index))
    if st:
        _lib.check("bil_logp_topk_bwd", st)
    return out.reshape(logits.shape) if out.numel() == logits.numel() else out


class BatchInvariantLogpTopk(torch.autograd.Function):
    """(logp, entropy, top_ids, top_logp) = BatchInvariantLogpTopk.apply(logits, target_ids, k,
    ignore_index, tile_v, validate, temperature): all but top_ids differentiable with
    respect to the logits (the choice of the columns is taken as fixed)."""

    @staticmethod
    def forward(ctx, logits, target_ids, k, ignore_index=IGNORE_INDEX, tile_v=DEFAULT_TILE_V, validate=False,
                temperature=1.0):
        logp, lse, ent, ids, top = logp_topk(logits, target_ids, k, ignore_index, tile_v, validate,
                                             temperature=temperature, return_entropy=True)
        ctx.save_for_backward(logits, target_ids, ids, lse, ent)
        ctx.ignore_index, ctx.temperature = ignore_index, temperature
        ctx.mark_non_differentiable(ids)
        ctx.set_materialize_grads(False)
        return logp, ent, ids, top

    @staticmethod
    def backward(ctx, grad_logp, grad_ent, grad_ids, grad_top):
        logits, target_ids, ids, lse, ent = ctx.saved_tensors
        if grad_logp is None:
            grad_logp = torch.zeros_like(lse)
        if grad_top is None:
            grad_top = torch.zeros_like(ids, dtype=torch.float32)
        d = logp_topk_bwd(logits, target_ids, ids, lse, grad_logp, grad_top, ctx.ignore_index,
                          temperature=ctx.temperature, entropy=None if grad_ent is None else ent,
                          grad_entropy=grad_ent)
        return _first_derivative(d, logits), None, None, None, None, None, None


def batch_invariant_logp_topk(logits: torch.Tensor, target_ids: torch.Tensor, k: int,
                              ignore_index: int = IGNORE_INDEX, validate: bool = False,
                              tile_v: int = DEFAULT_TILE_V, temperature: float = 1.0):
    """Differentiable (logp, entropy, top_ids, top_logp) of the target and the k largest alternatives."""
    return BatchInvariantLogpTopk.apply(logits, target_ids, k, ignore_index, tile_v, validate, temperature)
