"""The root-mean-square norm, forward, 8-bit and backward, against its formula in 64 bits.

Tolerances.  u_T is the type's unit roundoff (2^-24, 2^-8, 2^-11); float16
values below 2^-14 round to steps of 2^-24.  A row's sum runs over at most 32
elements of a thread in order, five butterfly steps and five more across the
warps: 42 additions of positive terms, relative error 42 * 2^-24 plus the
squares' own; the division, square root and reciprocal add four roundings and
halve it: rstd is within 24 * 2^-24 < 2^-19, and EPS_R = 2^-18 allows twice
that.
    y:  |dy| <= (u_T + EPS_R) |y| (+ 2^-25 for float16)
    scale: EPS_R relative;  q * scale: half a step of e4m3 (2^-4 relative, 2^-10
    of the scale among its subnormals) plus 2 EPS_R |y|
    dx = rstd (v - u c) + dh: c's sum has terms of both signs, so its error is
    2^-19 of mean |v u|; with the products' roundings
        2^-17 rstd (|v| + |u| mean |v u|) + 2^-23 |dh| + u_T |dx|
    dw: N terms in an order of at most N + 64 additions: (N + 64) 2^-24 sum |dy u|
        + EPS_R sum |dy u|.
"""
import numpy as np
import pytest
import torch

import invariant_token_log_gb300 as bil
from invariant_token_log_gb300 import norm as norm_mod

pytestmark = pytest.mark.gpu

EPS_R = 2.0 ** -18
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}
TYPES = list(U)
IDS = ["f32", "bf16", "f16"]

# every layout of a row over threads: one to four groups a lane of a warp, two to sixteen warps, and the
# widths at and around the steps between them
WIDTHS = [1, 7, 8, 9, 256, 257, 1000, 1024, 1025, 2049, 4096, 5001, 8192, 8193, 16383, 16384]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(n, width, dtype, g, scale=1.0, pad=0, shift=0):
    """[n, width] of `dtype`, rows `pad` elements apart, the first `shift` elements into its storage;
    the elements around the rows are NaN."""
    buf = torch.full((n * (width + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    view = buf[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    view.copy_(scale * torch.randn(n, width, generator=g, device="cuda"))
    return view


def bits(t):
    t = t.contiguous()
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.uint8 if t.itemsize == 1 else torch.int16)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).max()))


def forward64(x, w, r, eps):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h64 = h.double()
    rstd = 1 / torch.sqrt(h64.square().mean(dim=-1) + eps)
    return h, rstd, h64 * rstd[..., None] * w.double()


def check_quant(q, scale, y, what):
    within(scale, y.abs().amax(dim=-1) / 448, 2 * EPS_R * y.abs().amax(dim=-1) / 448 + 1e-45, what + " scale")
    back = q.double() * scale.double()[:, None]
    within(back, y, (2.0 ** -4 + 2 * EPS_R) * y.abs() + 2.0 ** -10 * scale.double()[:, None], what)
    assert bool((q.double().abs().amax(dim=-1) == 448).all()), what


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward_and_quant(width, residual, dtype):
    g = gen(width)
    n = 5
    x = rows(n, width, dtype, g)
    r = rows(n, width, dtype, g, 4.0) if residual else None
    w = (1 + 0.1 * torch.randn(width, generator=g, device="cuda")).to(dtype)
    y, h, rstd = bil.rms_norm_fwd(x, w, r, eps=1e-5)
    rh, rrstd, ry = forward64(x, w, r, 1e-5)
    assert (h is None) == (r is None)
    if residual:
        assert same(h, rh)
    within(rstd, rrstd, EPS_R * rrstd, "rstd")
    within(y, ry, (U[dtype] + EPS_R) * ry.abs() + TINY[dtype], "y")
    q, scale, h8 = bil.rms_norm_quant(x, w, r, eps=1e-5)
    assert q.dtype == torch.float8_e4m3fn and q.stride(0) % 16 == 0
    if residual:
        assert same(h8, rh)
    check_quant(q, scale, ry, "q")
    q, scale = bil.quantize_rows(x)
    check_quant(q, scale, x.double(), "quantize_rows")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("width", WIDTHS)
def test_backward(width, stream, dtype):
    g = gen(width + 1)
    n = 37
    h, dy = rows(n, width, dtype, g, 2.0), rows(n, width, dtype, g)
    dh = rows(n, width, dtype, g) if stream else None
    w = (1 + 0.1 * torch.randn(width, generator=g, device="cuda")).to(dtype)
    rstd = bil.rms_norm_fwd(h, w)[2]
    dx, dw = bil.rms_norm_bwd(dy, h, w, rstd, dh)
    check_backward(dx, dw, dy, h, w, dh, 1e-6)


def check_backward(dx, dw, dy, h, w, dh, eps):
    dtype, n = h.dtype, h.shape[0]
    h64, d64 = h.double(), dy.double()
    r = 1 / torch.sqrt(h64.square().mean(dim=-1, keepdim=True) + eps)
    u, v = h64 * r, d64 * w.double()
    ref = r * (v - u * (v * u).mean(dim=-1, keepdim=True))
    bound = 2.0 ** -17 * r * (v.abs() + u.abs() * (v * u).abs().mean(dim=-1, keepdim=True))
    if dh is not None:
        ref = ref + dh.double()
        bound = bound + 2.0 ** -23 * dh.double().abs()
    within(dx, ref, bound + U[dtype] * (ref.abs() + bound) + TINY[dtype], "dx")
    s = (d64 * u).abs().sum(dim=0)
    within(dw, (d64 * u).sum(dim=0), ((n + 64) * 2.0 ** -24 + EPS_R) * s + 1e-45, "dw")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("width", [37, 1024, 1999, 4100])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (8, 4), (16, 0)])
def test_rows_off_boundaries_give_the_same_bits(width, pad, shift, dtype):
    g = gen(3)
    n = 11
    x, r, dy, dh = (rows(n, width, dtype, g, pad=pad, shift=shift) for _ in range(4))
    w = torch.randn(width + 1, generator=g, device="cuda").to(dtype)[1:]
    a = [t.clone(memory_format=torch.contiguous_format) for t in (x, r, dy, dh)]
    padded = []
    for t in a:
        per = 16 // t.itemsize
        buf = torch.zeros(n, -(-width // per) * per, dtype=dtype, device="cuda")
        buf[:, :width] = t
        padded.append(buf[:, :width])
    wa = torch.zeros(width, dtype=dtype, device="cuda").copy_(w)
    for got, ref in zip(bil.rms_norm_fwd(x, w, r), bil.rms_norm_fwd(padded[0], wa, padded[1])):
        assert same(got, ref)
    for got, ref in zip(bil.rms_norm_quant(x, w, r), bil.rms_norm_quant(padded[0], wa, padded[1])):
        assert same(got, ref)
    for got, ref in zip(bil.quantize_rows(x), bil.quantize_rows(padded[0])):
        assert same(got, ref)
    _, h, rstd = bil.rms_norm_fwd(padded[0], wa, padded[1])
    odd = rows(n, width, dtype, g, pad=pad, shift=shift)
    odd.copy_(h)
    for got, ref in zip(bil.rms_norm_bwd(dy, odd, w, rstd, dh), bil.rms_norm_bwd(padded[2], h, wa, rstd, padded[3])):
        assert same(got, ref)


@pytest.mark.parametrize("width", [200, 1024, 4096, 10000])
def test_rows_bitwise_across_batches(width):
    g = gen(4)
    n = 300
    x, r, dy, dh = (rows(n, width, torch.bfloat16, g) for _ in range(4))
    w = torch.randn(width, generator=g, device="cuda")
    y, h, rstd = bil.rms_norm_fwd(x, w, r)
    q, scale, _ = bil.rms_norm_quant(x, w, r)
    dx, _ = bil.rms_norm_bwd(dy, h, w, rstd, dh)
    for size in (1, 2, 7, 129):
        idx = torch.randperm(n, generator=g, device="cuda")[:size]
        y1, h1, rstd1 = bil.rms_norm_fwd(x[idx], w, r[idx])
        q1, scale1, _ = bil.rms_norm_quant(x[idx], w, r[idx])
        dx1, _ = bil.rms_norm_bwd(dy[idx], h1, w, rstd1, dh[idx])
        for got, ref in ((y1, y), (h1, h), (rstd1, rstd), (scale1, scale), (dx1, dx)):
            assert same(got, ref[idx]), size
        assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)[idx])


@pytest.mark.parametrize("n", [1, 2, 607, 608, 609, 3000])
@pytest.mark.parametrize("width", [96, 1100])
def test_dweight_over_row_counts(n, width):
    """One row, and row counts around what one round of blocks takes; twice the same bits."""
    g = gen(5)
    h, dy = rows(n, width, torch.float32, g), rows(n, width, torch.float32, g)
    w = torch.randn(width, generator=g, device="cuda")
    rstd = bil.rms_norm_fwd(h, w)[2]
    dx, dw = bil.rms_norm_bwd(dy, h, w, rstd)
    check_backward(dx, dw, dy, h, w, None, 1e-6)
    assert same(bil.rms_norm_bwd(dy, h, w, rstd)[1], dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_float32_weight(dtype):
    g = gen(6)
    x, dy = rows(9, 520, dtype, g), rows(9, 520, dtype, g)
    w = torch.randn(520, generator=g, device="cuda")
    y, _, rstd = bil.rms_norm_fwd(x, w)
    ry = forward64(x, w, None, 1e-6)[2]
    within(y, ry, (U[dtype] + EPS_R) * ry.abs() + TINY[dtype], "y")
    check_backward(*bil.rms_norm_bwd(dy, x, w, rstd), dy, x, w, None, 1e-6)


def test_gradient_against_differences():
    """Central differences of the float32 forward along random directions.  L = sum dy y + sum dh h over
    3 x 64 elements: |L| terms are of order 1, their rounding 2^-23 each, so a difference over 2 eps =
    2^-6 carries about sqrt(192) 2^-23 2^6 = 1e-4; the third derivative's eps^2 / 6 = 1e-5.  2e-3 of the
    gradient's norm (about 14) is fifteen times both."""
    g = gen(7)
    n, width, eps = 3, 64, 2.0 ** -7
    x, r = rows(n, width, torch.float32, g), rows(n, width, torch.float32, g)
    w = 1 + 0.1 * torch.randn(width, generator=g, device="cuda")
    dy, dh = rows(n, width, torch.float32, g), rows(n, width, torch.float32, g)

    def loss(x, r, w):
        y, h, _ = bil.rms_norm_fwd(x, w, r)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())

    _, h, rstd = bil.rms_norm_fwd(x, w, r)
    dx, dw = bil.rms_norm_bwd(dy, h, w, rstd, dh)
    for _ in range(4):
        d = torch.randn(n, width, generator=g, device="cuda")
        num = (loss(x + eps * d, r, w) - loss(x - eps * d, r, w)) / (2 * eps)
        assert abs(num - float((dx.double() * d.double()).sum())) <= 2e-3 * float(dx.norm())
        num = (loss(x, r + eps * d, w) - loss(x, r - eps * d, w)) / (2 * eps)
        assert abs(num - float((dx.double() * d.double()).sum())) <= 2e-3 * float(dx.norm())
        dwd = torch.randn(width, generator=g, device="cuda")
        num = (loss(x, r, w + eps * dwd) - loss(x, r, w - eps * dwd)) / (2 * eps)
        assert abs(num - float((dw.double() * dwd.double()).sum())) <= 2e-3 * float(dw.norm())


@pytest.mark.parametrize("residual", [False, True])
def test_autograd(residual):
    """Through autograd, with an expanded gradient (a sum's) and with only one of the outputs used."""
    g = gen(8)
    x = rows(6, 40, torch.float32, g).reshape(2, 3, 40).contiguous().requires_grad_()
    r = rows(6, 40, torch.float32, g).reshape(2, 3, 40).contiguous().requires_grad_() if residual else None
    w = torch.randn(40, generator=g, device="cuda").requires_grad_()

    def plain(x, w, r):
        h = x if r is None else x + r
        return h * torch.rsqrt(h.square().mean(dim=-1, keepdim=True) + 1e-6) * w, h

    leaves = [x, w] + ([r] if residual else [])
    if residual:
        got = torch.autograd.grad(sum(t.sum() for t in bil.rms_norm(x, w, r)), leaves)
        ref = torch.autograd.grad(sum(t.sum() for t in plain(x, w, r)), leaves)
        only = torch.autograd.grad(bil.rms_norm(x, w, r)[1].sum(), [x, r])
        assert all(bool((t == 1).all()) for t in only)
    else:
        got = torch.autograd.grad(bil.rms_norm(x, w).sum(), leaves)
        ref = torch.autograd.grad(plain(x, w, None)[0].sum(), leaves)
    for a, b in zip(got, ref):
        assert a.shape == b.shape and a.dtype == b.dtype
        assert float((a - b).abs().max()) <= 1e-5 * (1 + float(b.abs().max()))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_special_rows(dtype):
    """Zero rows (eps keeps them finite; their scale stays positive), a NaN and an infinity, in a row's last,
    partial group: no other row changes."""
    g = gen(9)
    width = 1029
    x = rows(6, width, dtype, g)
    w = torch.ones(width, dtype=dtype, device="cuda")
    ref = bil.rms_norm_quant(x, w)
    x[1] = 0
    x[2, 1028] = float("nan")
    x[3, 1028] = float("inf")
    y, _, rstd = bil.rms_norm_fwd(x, w, eps=1e-6)
    assert bool((y[1] == 0).all()) and abs(float(rstd[1]) - 1e3) < 1
    assert bool(y[2].isnan().all()) and bool(y[3, 1028].isnan()) and bool((y[3, :1028] == 0).all())
    for q, scale in (bil.rms_norm_quant(x, w)[:2], bil.quantize_rows(x)):
        assert float(scale[1]) > 0 and bool((q[1].float() == 0).all())
        back = q.float() * scale[:, None]
        assert bool(back[2].isnan().all()) and bool(back[3].isnan().all())
        assert bool(back[[0, 4, 5]].isfinite().all())
    q, scale, _ = bil.rms_norm_quant(x, w)
    for i in (0, 4, 5):
        assert torch.equal(q.view(torch.uint8)[i], ref[0].view(torch.uint8)[i]) and same(scale[i:i + 1], ref[1][i:i + 1])
    y, _, rstd = bil.rms_norm_fwd(x[1:2], w, eps=0.0)  # the formula's own 0 * inf
    assert bool(y.isnan().all()) and bool(rstd.isinf().all())


def test_extremes_of_the_8_bits():
    """Values at e4m3's rounding points: ties to even, subnormals of 2^-9, the largest 448."""
    v = torch.tensor([448.0, 432.0, 433.0, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 2.0 ** -10 * 1.01, 3 * 2.0 ** -10, -448.0, 0.0,
                      -0.0, 240.0, 0.0156, 1.0625, 1.1875], device="cuda")[None]
    q, scale = bil.quantize_rows(v)
    assert float(scale[0]) == 1.0
    assert torch.equal(q.view(torch.uint8), v.to(torch.float8_e4m3fn).view(torch.uint8))


def test_tiny_and_huge_rows():
    x = torch.tensor([[1e-38, -3e-39, 1e-45, 0.0], [3e38, -1e38, 1.0, 0.0]], device="cuda")
    q, scale = bil.quantize_rows(x)
    back = q.double() * scale.double()[:, None]
    # below 2^-100 the scale stays at 2^-100 / 448: such rows come out as zero
    assert bool((q[0].float() == 0).all()) and float(scale[0]) > 0
    assert float((back[1] - x[1].double()).abs().max()) <= 2.0 ** -4 * 3e38


def test_in_place_stream_and_leading_shape():
    """The C calls may write h over the residual and dx over dy; here through the ABI."""
    from invariant_token_log_gb300 import _lib
    from invariant_token_log_gb300.logp import _stream_handle
    g = gen(10)
    x, r = rows(7, 512, torch.bfloat16, g), rows(7, 512, torch.bfloat16, g)
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = bil.rms_norm_fwd(x, w, r)
    buf, y2 = r.clone(), torch.empty_like(y)
    assert _lib.load().bil_rms_norm_fwd(x.data_ptr(), buf.data_ptr(), w.data_ptr(), _lib.BF16, _lib.BF16, 7, 512, 512,
                                        512, 1e-6, y2.data_ptr(), 512, buf.data_ptr(), 512, None,
                                        _stream_handle(0)) == _lib.OK
    assert same(buf, h) and same(y2, y)
    lead = bil.rms_norm_fwd(x[:6].reshape(2, 3, 512), w, r[:6].reshape(2, 3, 512))
    assert lead[0].shape == (2, 3, 512) and lead[2].shape == (2, 3)
    assert same(lead[0].reshape(6, 512), y[:6]) and same(lead[2].reshape(6), rstd[:6])


def test_strided_expanded_and_transposed_inputs():
    g = gen(11)
    base = torch.randn(64, 10, generator=g, device="cuda")
    w = torch.ones(64, device="cuda")
    assert same(bil.rms_norm_fwd(base.t(), w)[0], bil.rms_norm_fwd(base.t().contiguous(), w)[0])
    one = torch.randn(64, generator=g, device="cuda").expand(5, 64)
    assert same(bil.rms_norm_fwd(one, w)[0], bil.rms_norm_fwd(one.contiguous(), w)[0])
    every = torch.randn(10, 64, generator=g, device="cuda")[::2]
    assert same(bil.rms_norm_fwd(every, w)[0], bil.rms_norm_fwd(every.contiguous(), w)[0])


def test_another_stream():
    g = gen(12)
    x = rows(400, 4096, torch.bfloat16, g)
    w = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    ref = bil.rms_norm_fwd(x, w)
    dref = bil.rms_norm_bwd(x, x, w, ref[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y, _, rstd = bil.rms_norm_fwd(x, w)
        d = bil.rms_norm_bwd(x, x, w, rstd)
    s.synchronize()
    assert same(y, ref[0]) and same(d[0], dref[0]) and same(d[1], dref[1])


def test_empty_and_refusals():
    g = gen(13)
    x = rows(4, 64, torch.bfloat16, g)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = bil.rms_norm_fwd(x[:0], w, x[:0])
    assert y.shape == (0, 64) and h.shape == (0, 64) and rstd.shape == (0,)
    q, scale, _ = bil.rms_norm_quant(x[:0], w)
    assert q.shape == (0, 64) and scale.shape == (0,)
    dx, dw = bil.rms_norm_bwd(x[:0], x[:0], w, rstd)
    assert dx.shape == (0, 64) and bool((dw == 0).all())
    with pytest.raises(ValueError, match="no CPU path"):
        bil.rms_norm_fwd(x.cpu(), w)
    with pytest.raises(TypeError):
        bil.rms_norm_fwd(x.double(), w.double())
    with pytest.raises(TypeError):
        bil.rms_norm_fwd(x, w.to(torch.float16))
    for bad_w in (w[:63], w[None]):
        with pytest.raises(ValueError):
            bil.rms_norm_fwd(x, bad_w)
    for bad_r in (x[:3], x.float(), x[:, :32]):
        with pytest.raises(ValueError):
            bil.rms_norm_fwd(x, w, bad_r)
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(bil.BilError):
            bil.rms_norm_fwd(x, w, eps=eps)
    wide = torch.zeros(2, norm_mod._lib.MAX_NORM_WIDTH + 8, device="cuda")
    with pytest.raises(ValueError):
        bil.quantize_rows(wide)
    with pytest.raises(ValueError):
        bil.quantize_rows(x[:, :0])
    good = bil.rms_norm_fwd(x, w)[2]
    with pytest.raises(ValueError):
        bil.rms_norm_bwd(x, x, w, good[:3])
    with pytest.raises(ValueError):
        bil.rms_norm_bwd(x[:3], x, w, good)
    with pytest.raises(ValueError):
        bil.rms_norm_bwd(x, x, w, good, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
