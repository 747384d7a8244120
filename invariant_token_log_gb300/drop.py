"""PyTorch front end of dropout from a counter-based generator: argument marshalling only.

    y = round(x * f + residual),  f = 0 where an element is dropped, else 65536 / (65536 - border)

border is p * 65536 rounded to nearest even.  The mask is a function of a seed, a
step and an element's place in [N, H] (Philox4x32-10; include/bil.h has the
counters), so it is never stored: the backward pass makes it again.

``seed`` is an integer, or an int64 CUDA tensor of two elements, the seed and a step,
which the kernels read when they run: a training step captured in a CUDA graph gets
new masks by writing the tensor between replays (after the backward pass).  ``offset``
is added to the step (0 with an integer seed): give each dropout of a model its own.

Rows are [*lead, H] float32, bfloat16 or float16 with unit column stride (any row
stride); outputs whose H is no multiple of 16 bytes are views of rows that are
padded to one.
"""
from __future__ import annotations

import torch

from . import _lib
from .logp import _DEVICE_OBJECTS, _code, _device_object, _first_derivative, _need_cuda, _stream_handle
from .norm import _call, _padded, _rows, _rows_like

_WORD = (1 << 64) - 1


def _random(p: float, seed: int | torch.Tensor, offset: int, index: int) -> tuple[float, int, int, int | None]:
    """(p, seed, step, pointer to the device's words or None) as the C ABI takes them."""
    p = float(p)
    if not 0.0 <= p < 1.0 or round(p * 65536) >= 65536:
        raise ValueError(f"the share to drop, {p}, must be in [0, 1) and below 1 - 2^-17")
    if not isinstance(offset, int):
        raise TypeError("offset must be an integer")
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 2 or not seed.is_contiguous():
            raise ValueError("a seed tensor holds two int64 elements: the seed and the step")
        if seed.get_device() != index:
            raise ValueError("the seed tensor must be on the rows' device")
        return p, 0, offset & _WORD, seed.data_ptr()
    if not isinstance(seed, int):
        raise TypeError("seed must be an integer or an int64 tensor of two elements")
    return p, seed & _WORD, offset & _WORD, None


def dropout_fwd(x: torch.Tensor, p: float, seed: int | torch.Tensor, offset: int = 0,
                residual: torch.Tensor | None = None) -> torch.Tensor:
    """y [*lead, H]: x with a share p of its elements dropped and the others scaled, plus
    the residual (of x's shape) where there is one, rounded once to x's type."""
    index = x.get_device()
    if index < 0 or (residual is not None and residual.get_device() < 0):
        _need_cuda(x, residual)
    p, word, step, rng = _random(p, seed, offset, index)
    code = _code(x.dtype)
    x2, ld_x = _rows(x, "x")
    n, width = x2.shape
    if width < 1:
        raise ValueError("rows need at least one element")
    r2, ld_r, r_ptr = None, 0, None
    if residual is not None:
        r2, ld_r = _rows_like(residual, "residual", x)
        r_ptr = r2.data_ptr()
    y, ld_y = _padded(n, width, 4 if code == _lib.F32 else 8, x2.dtype,
                      _DEVICE_OBJECTS.get(index) or _device_object(index))
    _call("bil_dropout", index, x2.data_ptr(), r_ptr, code, n, width, ld_x, ld_r, p, word, step, rng, y.data_ptr(), ld_y,
          _stream_handle(index))
    return y if x.dim() == 2 else y.reshape(x.shape)


def dropout_bwd(dy: torch.Tensor, p: float, seed: int | torch.Tensor, offset: int = 0) -> torch.Tensor:
    """The gradient of x: ``dropout_fwd`` of dy under the same mask.  The residual's is dy."""
    return dropout_fwd(dy, p, seed, offset)


class Dropout(torch.autograd.Function):
    """y = Dropout.apply(x, p, seed, offset, residual)"""

    @staticmethod
    def forward(ctx, x, p, seed, offset, residual):
        ctx.p, ctx.offset, ctx.seed = p, offset, seed
        if isinstance(seed, torch.Tensor):  # saved, so that a step written too early is an error
            ctx.save_for_backward(seed)
            ctx.seed = None
        return dropout_fwd(x, p, seed, offset, residual)

    @staticmethod
    def backward(ctx, grad):
        seed = ctx.saved_tensors[0] if ctx.seed is None else ctx.seed
        dx = None
        if ctx.needs_input_grad[0]:
            dx = _first_derivative(dropout_bwd(grad, ctx.p, seed, ctx.offset), grad)
        return dx, None, None, None, grad if ctx.needs_input_grad[4] else None


def dropout(x: torch.Tensor, p: float, seed: int | torch.Tensor, offset: int = 0,
            residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable ``dropout_fwd``."""
    return Dropout.apply(x, p, seed, offset, residual)
