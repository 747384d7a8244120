"""PyTorch front end of layer norm: argument marshalling only.

The norm of a residual stream with dropout of what joins it and the residual's
addition in one pass, and its backward with the gradients of the weight and the bias:

    h = round(drop(x) + residual),  u = (h - mean) / sqrt(var + eps),  y = u * weight + bias

``p``, ``seed`` and ``offset`` are those of ``dropout_fwd`` (p = 0: no dropout).
Rows are [*lead, H] float32, bfloat16 or float16 with unit column stride (any
row stride), H up to 16384; weight and bias [H] have the rows' type or float32;
outputs whose H is no multiple of 16 bytes are views of rows that are padded to one.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from .drop import _random, dropout_bwd
from .logp import _DEVICE_OBJECTS, _code, _device_object, _first_derivative, _need_cuda, _stream_handle
from .norm import _call, _check_width, _padded, _rows, _rows_like, _weight

EPS = 1e-5


def _vector(w: torch.Tensor, x: torch.Tensor, width: int, index: int) -> torch.Tensor:
    if w.get_device() == index and w.shape == (width,) and w.dtype == x.dtype and w.is_contiguous() and w.data_ptr() % 16 == 0:
        return w
    _need_cuda(w)
    return _weight(w, x, width)


def _plain(x, weight, bias, residual, index) -> bool:
    """Whether a call needs no copy, no padded output and no conversion."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2 or not x.is_contiguous() or shape[1] % 8 or not 0 < shape[1] <= _lib.MAX_NORM_WIDTH:
        return False
    for v in (weight, bias):
        if v is not None and (v.dtype != dtype or v.shape != shape[1:] or v.get_device() != index or not v.is_contiguous() or
                              v.data_ptr() % 16):
            return False
    return residual is None or (residual.shape == shape and residual.dtype == dtype and residual.get_device() == index and
                                residual.is_contiguous())


def _check_stats(t: torch.Tensor, what: str, n: int, index: int) -> torch.Tensor:
    if t.dtype != torch.float32 or t.numel() != n or t.get_device() != index:
        raise ValueError(f"{what} must be float32, one per row ({n})")
    return t if t.dim() == 1 and t.is_contiguous() else t.reshape(-1).contiguous()


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                   residual: torch.Tensor | None = None, eps: float = EPS, p: float = 0.0,
                   seed: int | torch.Tensor = 0, offset: int = 0):
    """(y, h, mean, rstd): the norm of h = drop(x) + residual in the rows' type, h itself
    (the stream that goes on; None without a residual and dropout, where it is x) and
    the float32 mean and rstd [*lead] that ``layer_norm_bwd`` takes."""
    index = x.get_device()
    if not p and index >= 0 and _plain(x, weight, bias, residual, index):
        # The common call, row-major [N, H] of whole 16-byte units and vectors of its type, without the general path's
        # checks: the per-call host time is what bounds a few rows.
        n, width = x.shape
        code = _code(x.dtype)
        y = torch.empty_like(x)
        h, h_ptr, r_ptr = None, None, None
        if residual is not None:
            h = torch.empty_like(x)
            h_ptr, r_ptr = h.data_ptr(), residual.data_ptr()
        dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
        mean = torch.empty(n, dtype=torch.float32, device=dev)
        rstd = torch.empty(n, dtype=torch.float32, device=dev)
        _call("bil_layer_norm_fwd", index, x.data_ptr(), r_ptr, weight.data_ptr(), None if bias is None else bias.data_ptr(),
              code, code, n, width, width, width, float(eps), 0.0, 0, 0, None, y.data_ptr(), width, h_ptr, width,
              mean.data_ptr(), rstd.data_ptr(), _stream_handle(index))
        return y, h, mean, rstd
    if index < 0 or weight.get_device() < 0:
        _need_cuda(x, weight, bias, residual)
    p, word, step, rng = _random(p, seed, offset, index) if p else (0.0, 0, 0, None)
    x2, ld_x = _rows(x, "x")
    n, width = x2.shape
    _check_width(width)
    code = _code(x2.dtype)
    w = _vector(weight, x2, width, index)
    b_ptr = None
    if bias is not None:
        b = _vector(bias, x2, width, index)
        if b.dtype != w.dtype:
            raise TypeError("bias must have weight's type")
        b_ptr = b.data_ptr()
    dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
    per = 4 if code == _lib.F32 else 8
    r2, ld_r, r_ptr, h, ld_h, h_ptr = None, 0, None, None, 0, None
    if residual is not None:
        _need_cuda(residual)
        r2, ld_r = _rows_like(residual, "residual", x)
        r_ptr = r2.data_ptr()
    if residual is not None or p > 0.0:
        h, ld_h = _padded(n, width, per, x2.dtype, dev)
        h_ptr = h.data_ptr()
    y, ld_y = _padded(n, width, per, x2.dtype, dev)
    mean = torch.empty(n, dtype=torch.float32, device=dev)
    rstd = torch.empty(n, dtype=torch.float32, device=dev)
    _call("bil_layer_norm_fwd", index, x2.data_ptr(), r_ptr, w.data_ptr(), b_ptr, code, _code(w.dtype), n, width, ld_x,
          ld_r, float(eps), p, word, step, rng, y.data_ptr(), ld_y, h_ptr, ld_h, mean.data_ptr(), rstd.data_ptr(),
          _stream_handle(index))
    if x.dim() != 2:
        y, mean, rstd = y.reshape(x.shape), mean.reshape(x.shape[:-1]), rstd.reshape(x.shape[:-1])
        h = None if h is None else h.reshape(x.shape)
    return y, h, mean, rstd


@functools.lru_cache(maxsize=256)
def _bwd_workspace_bytes(n_rows: int, width: int, need_bias: bool, index: int) -> int:
    out = ctypes.c_int64(0)
    _call("bil_layer_norm_bwd_workspace_bytes", index, n_rows, width, 1 if need_bias else 0, ctypes.byref(out))
    return out.value


def bwd_workspace_bytes(n_rows: int, width: int, device: torch.device, need_bias: bool = True) -> int:
    """Device scratch bytes ``layer_norm_bwd`` needs on a device: the rows' partial sums for dweight and dbias."""
    return _bwd_workspace_bytes(n_rows, width, bool(need_bias), device.index)


def layer_norm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                   grad_h: torch.Tensor | None = None, p: float = 0.0, seed: int | torch.Tensor = 0, offset: int = 0,
                   need_bias: bool = True, need_residual: bool = True, workspace: torch.Tensor | None = None):
    """(dx, dresidual, dweight, dbias) of ``layer_norm_fwd``: dx and dresidual [*lead, H] in
    the rows' type, dweight and dbias [H] float32.  Without dropout dresidual is dx
    itself; with ``need_bias`` or ``need_residual`` false the one not needed is None.
    ``h`` is the forward's (x where it had none), ``grad_h`` the gradient of h as an
    output of its own; p, seed and offset are the forward's."""
    index = h.get_device()
    if index < 0 or dy.get_device() < 0 or weight.get_device() < 0 or mean.get_device() < 0 or rstd.get_device() < 0:
        _need_cuda(dy, h, weight, mean, rstd)
    p, word, step, rng = _random(p, seed, offset, index) if p else (0.0, 0, 0, None)
    h2, ld_h = _rows(h, "h")
    n, width = h2.shape
    _check_width(width)
    d2, ld_dy = _rows_like(dy, "dy", h)
    code = _code(h2.dtype)
    w = _vector(weight, h2, width, index)
    mean, rstd = _check_stats(mean, "mean", n, index), _check_stats(rstd, "rstd", n, index)
    g2, ld_g, g_ptr = None, 0, None
    if grad_h is not None:
        _need_cuda(grad_h)
        g2, ld_g = _rows_like(grad_h, "grad_h", h)
        g_ptr = g2.data_ptr()
    dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
    per = 4 if code == _lib.F32 else 8
    dx, ld_dx = _padded(n, width, per, h2.dtype, dev)
    dr, ld_dr, dr_ptr = None, 0, None
    if need_residual and p > 0.0:
        dr, ld_dr = _padded(n, width, per, h2.dtype, dev)
        dr_ptr = dr.data_ptr()
    dw = torch.empty(width, dtype=torch.float32, device=dev)
    db = torch.empty(width, dtype=torch.float32, device=dev) if need_bias else None
    need = _bwd_workspace_bytes(n, width, bool(need_bias), index)
    if workspace is None:
        workspace, have = torch.empty(need or 16, dtype=torch.uint8, device=dev), need
    else:
        _need_cuda(workspace)
        have = workspace.numel() * workspace.element_size()
        if have < need or not workspace.is_contiguous():
            raise ValueError(f"workspace holds {have} bytes, needs {need}")
    _call("bil_layer_norm_bwd", index, d2.data_ptr(), h2.data_ptr(), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
          g_ptr, code, _code(w.dtype), n, width, ld_dy, ld_h, ld_g, p, word, step, rng, dx.data_ptr(), ld_dx, dr_ptr,
          ld_dr, dw.data_ptr(), None if db is None else db.data_ptr(), workspace.data_ptr(), have,
          _stream_handle(index))
    if h.dim() != 2:
        dx = dx.reshape(h.shape)
        dr = None if dr is None else dr.reshape(h.shape)
    if need_residual and p == 0.0:
        dr = dx
    return dx, dr, dw, db


class LayerNorm(torch.autograd.Function):
    """y[, h] = LayerNorm.apply(x, weight, bias, residual, eps, p, seed, offset): h only with a residual."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps, p, seed, offset):
        y, h, mean, rstd = layer_norm_fwd(x, weight, bias, residual, eps, p, seed, offset)
        ctx.p, ctx.offset, ctx.seed = float(p), offset, seed
        saved = [x if h is None else h, weight, mean, rstd]
        if isinstance(seed, torch.Tensor):  # saved, so that a step written too early is an error
            saved.append(seed)
            ctx.seed = None
        ctx.save_for_backward(*saved)
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, h)

    @staticmethod
    def backward(ctx, grad_y, grad_h=None):
        h, weight, mean, rstd, *words = ctx.saved_tensors
        seed = words[0] if ctx.seed is None else ctx.seed
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        nones = (None,) * 4
        if grad_y is None:  # only the stream was used: it passes through
            dx = None
            if need_x and grad_h is not None:
                dx = grad_h
                if ctx.p > 0.0:
                    dx = _first_derivative(dropout_bwd(grad_h, ctx.p, seed, ctx.offset), grad_h)
            return (dx, None, None, grad_h if need_r else None) + nones
        grads = layer_norm_bwd(grad_y, h, weight, mean, rstd, grad_h, ctx.p, seed, ctx.offset, need_bias=need_b,
                               need_residual=need_r)
        dx, dr, dw, db = (None if d is None else _first_derivative(d, grad_y, h, weight) for d in grads)
        return (dx if need_x else None, dw.to(weight.dtype) if need_w else None,
                None if db is None else db.to(weight.dtype), dr) + nones


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               residual: torch.Tensor | None = None, eps: float = EPS, p: float = 0.0, seed: int | torch.Tensor = 0,
               offset: int = 0):
    """Differentiable norm: y, or with a residual (y, h)."""
    return LayerNorm.apply(x, weight, bias, residual, eps, p, seed, offset)
