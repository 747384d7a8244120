"""Dropout against its formula in 64 bits under masks from the tests' own generator.

The factor 65536 / (65536 - border) is rounded once to float32, the product and the
sum once each: with u = 2^-24
    |dy| <= u_T |y| + 4 u (|x f| + |r|)   (+ 2^-25 for float16, whose small values have steps of 2^-24)
A dropped element is the residual's bits (without one: zero).
"""
import pytest
import torch

import invariant_token_log_gb300 as bil
from philox import border_of, keep_mask

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}
TYPES = list(U)
IDS = ["f32", "bf16", "f16"]
SEED, OFFSET = 0x1234567890ABCDEF, 5


def rows(n, width, dtype, seed, scale=1.0, pad=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((n * (width + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    view = buf[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    view.copy_(scale * torch.randn(n, width, generator=g, device="cuda"))
    return view


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def check(y, x, r, p, seed, step):
    n, width = x.shape
    keep = torch.from_numpy(keep_mask(n, width, p, seed, step)).cuda()
    f = keep.double() * (65536 / (65536 - border_of(p)))
    r64 = torch.zeros_like(x, dtype=torch.float64) if r is None else r.double()
    ref = torch.where(keep, x.double() * f, 0.0) + r64
    bound = U[x.dtype] * ref.abs() + 4 * 2.0 ** -24 * ((x.double() * f).abs() + r64.abs()) + TINY[x.dtype]
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    dropped = torch.zeros_like(x) if r is None else r
    assert torch.equal(bits(y)[~keep], bits(dropped + 0.0)[~keep])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n,width,pad,shift", [(1, 1, 0, 0), (3, 7, 0, 0), (5, 8, 0, 0), (129, 64, 0, 0), (1000, 1104, 0, 0),
                                               (33, 4097, 0, 0), (17, 4096, 7, 3), (64, 2048, 64, 0), (2, 20000, 0, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_and_backward(dtype, n, width, pad, shift, residual):
    x = rows(n, width, dtype, 1, pad=pad, shift=shift)
    r = rows(n, width, dtype, 2, 4.0, pad=pad, shift=shift) if residual else None
    y = bil.dropout_fwd(x, 0.3, SEED, OFFSET, residual=r)
    check(y, x, r, 0.3, SEED, OFFSET)
    dy = rows(n, width, dtype, 3, pad=pad)
    check(bil.dropout_bwd(dy, 0.3, SEED, OFFSET), dy, None, 0.3, SEED, OFFSET)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 2.0 ** -16, 0.1, 0.5, 0.999, 1 - 2.0 ** -16])
def test_shares(p):
    x = rows(64, 512, torch.float32, 4)
    check(bil.dropout_fwd(x, p, 9), x, None, p, 9, 0)
    if border_of(p) == 0:
        assert torch.equal(bil.dropout_fwd(x, p, 9), x)


@pytest.mark.parametrize("seed,step,offset", [(0, 0, 0), (2 ** 63 - 1, 2 ** 62, 3), (-1, -1, 0), (5, 2 ** 63 - 1, 1)])
def test_seed_tensor(seed, step, offset):
    x = rows(40, 264, torch.bfloat16, 5)
    words = torch.tensor([seed, step], device="cuda")
    y = bil.dropout_fwd(x, 0.25, words, offset)
    check(y, x, None, 0.25, seed, step + offset)
    assert torch.equal(bits(y), bits(bil.dropout_fwd(x, 0.25, seed, step + offset)))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_dropped_elements_add_nothing(dtype):
    x = rows(50, 80, dtype, 6)
    keep = torch.from_numpy(keep_mask(50, 80, 0.4, 11)).cuda()
    bad = x.clone()
    bad[~keep] = float("inf")
    bad[0][~keep[0]] = float("nan")
    assert torch.equal(bits(bil.dropout_fwd(bad, 0.4, 11)), bits(bil.dropout_fwd(x, 0.4, 11)))


def test_layout_and_batch_do_not_matter():
    """The mask goes by the row's number and the column: the same for another type, pitch or shape."""
    x = rows(96, 72, torch.float32, 7)
    y = bil.dropout_fwd(x, 0.5, 3)
    assert torch.equal(bil.dropout_fwd(x[:31], 0.5, 3), y[:31])
    assert torch.equal(bil.dropout_fwd(x.view(4, 24, 72), 0.5, 3).view(96, 72), y)
    assert torch.equal(bil.dropout_fwd(x.t().contiguous().t(), 0.5, 3), y)
    one = torch.ones(1, 72, dtype=torch.bfloat16, device="cuda").expand(96, 72)
    assert torch.equal(bil.dropout_fwd(one, 0.5, 3) != 0, y != 0)
    assert bil.dropout_fwd(x[:0], 0.5, 3).shape == (0, 72)


def test_autograd():
    x, r = (rows(20, 100, torch.float32, s).clone().requires_grad_() for s in (8, 9))
    dy = rows(20, 100, torch.float32, 10)
    words = torch.tensor([77, 1], device="cuda")
    y = bil.dropout(x, 0.2, words, 4, residual=r)
    dx, dr = torch.autograd.grad(y, (x, r), dy, retain_graph=True)
    check(dx, dy, None, 0.2, 77, 5)
    assert torch.equal(dr, dy)
    words[1] += 1  # the step moved on before the backward pass: an error, not another mask
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, x, dy)


def test_captured_calls_get_new_masks():
    x = rows(64, 256, torch.bfloat16, 11)
    words = torch.tensor([5, 0], device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        bil.dropout_fwd(x, 0.5, words)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = bil.dropout_fwd(x, 0.5, words)
    for step in (0, 1, 9):
        words[1] = step
        graph.replay()
        torch.cuda.synchronize()
        check(y, x, None, 0.5, 5, step)
