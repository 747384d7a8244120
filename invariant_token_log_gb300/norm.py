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
import functools

import torch

from . import _lib
from .logp import (
    _DEVICE_OBJECTS,
    _code,
    _device_object,
    _first_derivative,
    _get_device,
    _need_cuda,
    _on_device,
    _stream_handle,
)

EPS = 1e-6


def _rows(x: torch.Tensor, what: str) -> tuple[torch.Tensor, int]:
    """(x as [N, H] with unit column stride, its row stride); a copy only where no such view exists."""
    if x.dim() != 2:
        if x.dim() == 0:
            raise ValueError(f"{what} must have a last dimension")
        x = x.reshape(x.numel() // max(x.shape[-1], 1), x.shape[-1])
    n, width = x.shape
    ld, unit = x.stride()
    if n and ((width > 1 and unit != 1) or (n > 1 and ld < width)):
        x = x.contiguous()  # a transposed or an expanded tensor
        ld = width
    return x, ld if n > 1 else max(ld, width)


def _rows_like(x: torch.Tensor, what: str, like: torch.Tensor) -> tuple[torch.Tensor, int]:
    if x.shape != like.shape or x.dtype != like.dtype or x.get_device() != like.get_device():
        raise ValueError(f"{what} must have the rows' shape, type and device")
    return _rows(x, what)


def _padded(n: int, width: int, per: int, dtype: torch.dtype, device: torch.device) -> tuple[torch.Tensor, int]:
    """[n, width] whose rows start on 16-byte boundaries (`per` elements), and its row stride."""
    ld = -(-width // per) * per
    if ld == width:
        return torch.empty((n, width), dtype=dtype, device=device), ld
    return torch.empty_strided((n, width), (ld, 1), dtype=dtype, device=device), ld


def _weight(weight: torch.Tensor, x: torch.Tensor, width: int) -> torch.Tensor:
    if weight.dim() != 1 or weight.shape[0] != width:
        raise ValueError(f"weight must be [{width}]")
    if weight.get_device() != x.get_device():
        raise ValueError("weight must be on the rows' device")
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise TypeError("weight must have the rows' type or float32")
    weight = weight.contiguous()
    return weight if weight.data_ptr() % 16 == 0 else weight.clone()


def _check_width(width: int) -> None:
    if not 1 <= width <= _lib.MAX_NORM_WIDTH:
        raise ValueError(f"rows of {width} elements; the norm takes 1 to {_lib.MAX_NORM_WIDTH}")


def _call(name: str, index: int, *args) -> None:
    fn = getattr(_lib.load(), name)
    st = fn(*args) if _get_device() == index else _on_device(index, fn, *args)
    if st:
        _lib.check(name, st)


def _norm(x, weight, residual, eps, quant):
    """The forward, in the rows' type or in 8 bits: (y or q, h or None, rstd or scale)."""
    index = x.get_device()
    if index < 0 or weight.get_device() < 0 or (residual is not None and residual.get_device() < 0):
        _need_cuda(x, weight, residual)
    x2, ld_x = _rows(x, "x")
    n, width = x2.shape
    _check_width(width)
    dtype = x2.dtype
    code = _code(dtype)
    w = _weight(weight, x2, width)
    dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
    per = 4 if code == _lib.F32 else 8
    r2, ld_r, h, ld_h, h_ptr, r_ptr = None, 0, None, 0, None, None
    if residual is not None:
        r2, ld_r = _rows_like(residual, "residual", x)
        h, ld_h = _padded(n, width, per, dtype, dev)
        h_ptr, r_ptr = h.data_ptr(), r2.data_ptr()
    y, ld_y = _padded(n, width, 16, torch.float8_e4m3fn, dev) if quant else _padded(n, width, per, dtype, dev)
    stat = torch.empty(n, dtype=torch.float32, device=dev)
    if quant:
        _call("bil_rms_norm_quant", index, x2.data_ptr(), r_ptr, w.data_ptr(), code, _code(w.dtype), n, width, ld_x,
              ld_r, float(eps), y.data_ptr(), ld_y, stat.data_ptr(), h_ptr, ld_h, _stream_handle(index))
    else:
        _call("bil_rms_norm_fwd", index, x2.data_ptr(), r_ptr, w.data_ptr(), code, _code(w.dtype), n, width, ld_x,
              ld_r, float(eps), y.data_ptr(), ld_y, h_ptr, ld_h, stat.data_ptr(), _stream_handle(index))
    if x.dim() != 2:
        y, stat = y.reshape(x.shape), stat.reshape(x.shape[:-1])
        h = None if h is None else h.reshape(x.shape)
    return y, h, stat


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = EPS):
    """(y, h, rstd): the norm of h = x + residual in the rows' type, h itself (the stream
    that goes on; None without a residual, where it is x) and the float32 rstd [*lead]
    that ``rms_norm_bwd`` takes.  ``weight`` [H] has the rows' type or float32."""
    return _norm(x, weight, residual, eps, False)


def rms_norm_quant(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = EPS):
    """(q, scale, h): the norm in 8 bits, float8_e4m3fn q [*lead, H] (rows on 16-byte
    boundaries, as ``linear_logp_fp8`` reads them) and the float32 scale [*lead] with
    q * scale standing for y; h as in ``rms_norm_fwd``.  For serving: no backward."""
    q, h, scale = _norm(x, weight, residual, eps, True)
    return q, scale, h


def quantize_rows(x: torch.Tensor):
    """(q, scale) of the rows as they are: float8_e4m3fn q [*lead, H] and float32 scale
    [*lead] with scale = max |x| / 448 of the row.  A weight [V, H] is laid out so once
    for ``linear_logp_fp8``."""
    _need_cuda(x)
    index = x.get_device()
    x2, ld_x = _rows(x, "x")
    n, width = x2.shape
    _check_width(width)
    dev = x2.device
    q, ld_q = _padded(n, width, 16, torch.float8_e4m3fn, dev)
    scale = torch.empty(n, dtype=torch.float32, device=dev)
    _call("bil_quantize_rows", index, x2.data_ptr(), _code(x2.dtype), n, width, ld_x, q.data_ptr(), ld_q,
          scale.data_ptr(), _stream_handle(index))
    return q.reshape(x.shape), scale.reshape(x.shape[:-1])


def rms_norm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                 grad_h: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(dx, dweight) of ``rms_norm_fwd``: dx [*lead, H] in the rows' type is the gradient
    of x and of the residual alike, dweight [H] is float32.  ``h`` is the forward's
    (x where it had no residual), ``grad_h`` the gradient of h as an output of its own."""
    index = h.get_device()
    if index < 0 or dy.get_device() < 0 or weight.get_device() < 0 or rstd.get_device() < 0:
        _need_cuda(dy, h, weight, rstd)
    h2, ld_h = _rows(h, "h")
    n, width = h2.shape
    _check_width(width)
    d2, ld_dy = _rows_like(dy, "dy", h)
    code = _code(h2.dtype)
    w = _weight(weight, h2, width)
    if rstd.dtype != torch.float32 or rstd.numel() != n or rstd.get_device() != index:
        raise ValueError(f"rstd must be float32, one per row ({n})")
    if rstd.dim() != 1 or not rstd.is_contiguous():
        rstd = rstd.reshape(-1).contiguous()
    g2, ld_g, g_ptr = None, 0, None
    if grad_h is not None:
        _need_cuda(grad_h)
        g2, ld_g = _rows_like(grad_h, "grad_h", h)
        g_ptr = g2.data_ptr()
    dev = _DEVICE_OBJECTS.get(index) or _device_object(index)
    dx, ld_dx = _padded(n, width, 4 if code == _lib.F32 else 8, h2.dtype, dev)
    dw = torch.empty(width, dtype=torch.float32, device=dev)
    need = _bwd_workspace_bytes(n, width, index)
    if workspace is None:
        workspace, have = torch.empty(need or 16, dtype=torch.uint8, device=dev), need
    else:
        _need_cuda(workspace)
        have = workspace.numel() * workspace.element_size()
        if have < need or not workspace.is_contiguous():
            raise ValueError(f"workspace holds {have} bytes, needs {need}")
    _call("bil_rms_norm_bwd", index, d2.data_ptr(), h2.data_ptr(), w.data_ptr(), rstd.data_ptr(), g_ptr, code,
          _code(w.dtype), n, width, ld_dy, ld_h, ld_g, dx.data_ptr(), ld_dx, dw.data_ptr(), workspace.data_ptr(), have,
          _stream_handle(index))
    return dx if h.dim() == 2 else dx.reshape(h.shape), dw


@functools.lru_cache(maxsize=256)
def _bwd_workspace_bytes(n_rows: int, width: int, index: int) -> int:
    out = ctypes.c_int64(0)
    _call("bil_rms_norm_bwd_workspace_bytes", index, n_rows, width, ctypes.byref(out))
    return out.value


def bwd_workspace_bytes(n_rows: int, width: int, device: torch.device) -> int:
    """Device scratch bytes ``rms_norm_bwd`` needs on a device: the rows' partial sums for dweight."""
    return _bwd_workspace_bytes(n_rows, width, device.index)


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
        dx, dw = (_first_derivative(d, grad_y, h, weight) for d in rms_norm_bwd(grad_y, h, weight, rstd, grad_h))
        return dx, dw.to(weight.dtype), dx if ctx.needs_input_grad[2] else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = EPS):
    """Differentiable norm: y, or with a residual (y, h)."""
    return RMSNorm.apply(x, weight, residual, eps)
