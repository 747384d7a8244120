"""Rows whose ring of stages comes close to all of an SM's shared memory.
Formulas and tolerances are test_gpu_norm's."""
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import check_watchdog
from test_gpu_norm import EPS_R, TINY, U, check_backward, check_quant, forward64, gen, rows, same, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


# widths at which two to four stages of one to three operands take between 226 and 226.5 KB, and their neighbours
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("dtype,width", [
    (torch.float32, 4816), (torch.float32, 4824), (torch.float32, 6432), (torch.float32, 7232), (torch.float32, 7241),
    (torch.float32, 9636), (torch.float32, 9640), (torch.float32, 9661), (torch.float32, 14464), (torch.float32, 14493),
    (torch.bfloat16, 9640), (torch.bfloat16, 12856), (torch.bfloat16, 14472), (torch.float16, 9633),
])
def test_backward_at_the_limit(dtype, width, stream):
    g = gen(width)
    n = 21
    h, dy = rows(n, width, dtype, g, 2.0), rows(n, width, dtype, g)
    dh = rows(n, width, dtype, g) if stream else None
    w = (1 + 0.1 * torch.randn(width, generator=g, device="cuda")).to(dtype)
    dx, dw = bil.rms_norm_bwd(dy, h, w, bil.rms_norm_fwd(h, w)[2], dh)
    check_backward(dx, dw, dy, h, w, dh, 1e-6)


@pytest.mark.parametrize("width,pad", [(9641, 0), (9640, 1), (14465, 0), (14464, 3)])
def test_forward_at_the_limit(width, pad):
    g = gen(width)
    x, r = rows(5, width, torch.float32, g, pad=pad), rows(5, width, torch.float32, g, 4.0, pad=pad)
    w = 1 + 0.1 * torch.randn(width, generator=g, device="cuda")
    y, h, rstd = bil.rms_norm_fwd(x, w, r)
    rh, rrstd, ry = forward64(x, w, r, 1e-6)
    assert same(h, rh)
    within(rstd, rrstd, EPS_R * rrstd, "rstd")
    within(y, ry, (U[torch.float32] + EPS_R) * ry.abs() + TINY[torch.float32], "y")
    q, scale, h8 = bil.rms_norm_quant(x, w, r)
    assert same(h8, rh)
    check_quant(q, scale, ry, "q")
