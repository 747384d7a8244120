"""PyTorch front end of the root-mean-square norm: argument marshalling only.

What stands between the last layer and the LM head: the residual's addition
and the norm in one pass, with an output in the stream's type (and its
backward), or in 8 bits with a scale per row for ``linear_logp_fp8``.

    h = round(x + residual),  rstd = 1 / sqrt(mean h^2 + eps),  y = h * rstd * weight

Rows are [*lead, H] float32, bfloat16 or float16 with unit column stride (any
row stride); outputs whose H is no multiple of 16 bytes are views of rows that
are padded to one.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .logp import _code, _need_cuda, _on_device, _ptr, _stream_handle

EPS = 1e-6


def _rows(x: torch.Tensor, what: str, like: torch.Tensor | None = None) -> tuple[torch.Tensor, int]:
    """(x as [N, H] with unit column stride, its row stride); a copy only where no such view exists."""
    if x.dim() == 0:
        raise ValueError(f"{what} must have a last dimension")
    if like is not None and (x.shape != like.shape or x.dtype != like.dtype or x.device != like.device):
        raise ValueError(f"{what} must have the rows' shape, type and device")
    width = x.shape[-1]
    x2 = x if x.dim() == 2 else x.reshape(x.numel() // max(width, 1), width)
    n = x2.shape[0]
    if n and ((width > 1 and x2.stride(1) != 1) or (n > 1 and x2.stride(0) < width)):
        x2 = x2.contiguous()  # a transposed or an expanded tensor
    return x2, x2.stride(0) if n > 1 else max(x2.stride(0), width)


def _padded(n: int, width: int, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """[n, width] whose rows start on 16-byte boundaries."""
    per = 16 // dtype.itemsize
    if width % per == 0:
        return torch.empty((n, width), dtype=dtype, device=device)
    return torch.empty((n, -(-width // per) * per), dtype=dtype, device=device)[:, :width]


def _weight(weight: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
    if weight.dim() != 1 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight must be [{x.shape[-1]}]")
    if weight.device != x.device:
        raise ValueError("weight must be on the rows' device")
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise TypeError("weight must have the rows' type or float32")
    return weight.contiguous()


def _check_width(width: int) -> None:
    if not 1 <= width <= _lib.MAX_NORM_WIDTH:
        raise ValueError(f"rows of {width} elements; the norm takes 1 to {_lib.MAX_NORM_WIDTH}")


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = EPS):
    """(y, h, rstd): the norm of h = x + residual in the rows' type, h itself (the stream
    that goes on; None without a residual, where it is x) and the float32 rstd [*lead]
    that ``rms_norm_bwd`` takes.  ``weight`` [H] has the rows' type or float32."""
    _need_cuda(x, weight, residual)
    x2, ld_x = _rows(x, "x")
    n, width = x2.shape
    _check_width(width)
    w = _weight(weight, x2)
    dev = x2.device
    r2, ld_r, h = None, 0, None
    if residual is not None:
        r2, ld_r = _rows(residual, "residual", x)
        h = _padded(n, width, x2.dtype, dev)
    y = _padded(n, width, x2.dtype, dev)
    rstd = torch.empty(n, dtype=torch.float32, device=dev)
    st = _on_device(dev.index, _lib.load().bil_rms_norm_fwd, _ptr(x2), _ptr(r2), _ptr(w), _code(x2.dtype),
                    _code(w.dtype), n, width, ld_x, ld_r, float(eps), _ptr(y), y.stride(0), _ptr(h),
                    0 if h is None else h.stride(0), _ptr(rstd), _stream_handle(dev.index))
    if st:
        _lib.check("bil_rms_norm_fwd", st)
    lead = x.shape[:-1]
    return y.reshape(x.shape), None if h is None else h.reshape(x.shape), rstd.reshape(lead)


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = EPS):
    """(q, scale, h): the norm in 8 bits, float8_e4m3fn q [*lead, H] (rows on 16-byte
    boundaries, as ``linear_logp_fp8`` reads them) and the float32 scale [*lead] with
    q * scale standing for y; h as in ``rms_norm_fwd``.  For serving: no backward."""
    _need_cuda(x, weight, residual)
    x2, ld_x = _rows(x, "x")
    n, width = x2.shape
    _check_width(width)
    w = _weight(weight, x2)
    dev = x2.device
    r2, ld_r, h = None, 0, None
    if residual is not None:
        r2, ld_r = _rows(residual, "residual", x)
        h = _padded(n, width, x2.dtype, dev)
    q = _padded(n, width, torch.float8_e4m3fn, dev)
    scale = torch.empty(n, dtype=torch.float32, device=dev)
    st = _on_device(dev.index, _lib.load().bil_rms_norm_quant, _ptr(x2), _ptr(r2), _ptr(w), _code(x2.dtype),
                    _code(w.dtype), n, width, ld_x, ld_r, float(eps), _ptr(q), q.stride(0), _ptr(scale), _ptr(h),
                    0 if h is None else h.stride(0), _stream_handle(dev.index))
    if st:
        _lib.check("bil_rms_norm_quant", st)
    lead = x.shape[:-1]
    return q.reshape(x.shape), scale.reshape(lead), None if h is None else h.reshape(x.shape)


def quantize_rows(x: torch.Tensor):
    """(q, scale) of the rows as they are: float8_e4m3fn q [*lead, H] and float32 scale
    [*lead] with scale = max |x| / 448 of the row.  A weight [V, H] is laid out so once
    for ``linear_logp_fp8``."""
    _need_cuda(x)
    x2, ld_x = _rows(x, "x")
    n, width = x2.shape
    _check_width(width)
    dev = x2.device
    q = _padded(n, width, torch.float8_e4m3fn, dev)
    scale = torch.empty(n, dtype=torch.float32, device=dev)
    st = _on_device(dev.index, _lib.load().bil_quantize_rows, _ptr(x2), _code(x2.dtype), n, width, ld_x, _ptr(q),
                    q.stride(0), _ptr(scale), _stream_handle(dev.index))
    if st:
        _lib.check("bil_quantize_rows", st)
    return q.reshape(x.shape), scale.reshape(x.shape[:-1])


def rms_norm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                 grad_h: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(dx, dweight) of ``rms_norm_fwd``: dx [*lead, H] in the rows' type is the gradient
    of x and of the residual alike, dweight [H] is float32.  ``h`` is the forward's
    (x where it had no residual), ``grad_h`` the gradient of h as an output of its own."""
    _need_cuda(dy, h, weight, rstd, grad_h, workspace)
    h2, ld_h = _rows(h, "h")
    n, width = h2.shape
    _check_width(width)
    d2, ld_dy = _rows(dy, "dy", h)
    w = _weight(weight, h2)
    dev = h2.device
    if rstd.dtype != torch.float32 or rstd.numel() != n or rstd.device != dev:
        raise ValueError(f"rstd must be float32, one per row ({n})")
    rstd = rstd.reshape(-1).contiguous()
    g2, ld_g = (None, 0) if grad_h is None else _rows(grad_h, "grad_h", h)
    dx = _padded(n, width, h2.dtype, dev)
    dw = torch.empty(width, dtype=torch.float32, device=dev)
    need = bwd_workspace_bytes(n, width, dev)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    elif workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, needs {need}")
    st = _on_device(dev.index, _lib.load().bil_rms_norm_bwd, _ptr(d2), _ptr(h2), _ptr(w), _ptr(rstd), _ptr(g2),
                    _code(h2.dtype), _code(w.dtype), n, width, ld_dy, ld_h, ld_g, _ptr(dx), dx.stride(0), _ptr(dw),
                    _ptr(workspace), workspace.numel() * workspace.element_size(), _stream_handle(dev.index))
    if st:
        _lib.check("bil_rms_norm_bwd", st)
    return dx.reshape(h.shape), dw


def bwd_workspace_bytes(n_rows: int, width: int, device: torch.device) -> int:
    """Device scratch bytes ``rms_norm_bwd`` needs: the rows' partial sums for dweight."""
    out = ctypes.c_int64(0)
    st = _on_device(device.index, _lib.load().bil_rms_norm_bwd_workspace_bytes, n_rows, width, ctypes.byref(out))
    if st:
        _lib.check("bil_rms_norm_bwd_workspace_bytes", st)
    return out.value


class RMSNorm(torch.autograd.Function):
    """y[, h] = RMSNorm.apply(x, weight, residual, eps): h only with a residual."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = rms_norm_fwd(x, weight, residual, eps)
        ctx.save_for_backward(x if h is None else h, weight, rstd)
        ctx.set_materialize_grads(False)
        return y if h is None else (y, h)

    @staticmethod
    def backward(ctx, grad_y, grad_h=None):
        h, weight, rstd = ctx.saved_tensors
        if grad_y is None:  # only the stream was used: it passes through
            return grad_h, None, grad_h, None
        dx, dw = rms_norm_bwd(grad_y, h, weight, rstd, grad_h)
        return dx, dw.to(weight.dtype), dx if ctx.needs_input_grad[2] else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = EPS):
    """Differentiable norm: y, or with a residual (y, h)."""
    return RMSNorm.apply(x, weight, residual, eps)
