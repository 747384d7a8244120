"""Layer norm, forward and backward, with dropout and without, against its formula in 64 bits.

Tolerances, with u = 2^-24, u_T the type's unit roundoff and A = mean |h| of the row.  A
row's sum runs over at most 32 elements of a thread in order, five butterfly steps and
five more across the warps, 42 additions:
    mean:  D = 2^-18 A
    a centred element is off by D and one rounding; in the squares D enters squared (the
    centred row's sum is zero), so rstd is within EPS_R = 2^-18 (see the root-mean-square
    norm's tests) plus (D rstd)^2, and with Q = EPS_R + (D rstd)^2 an element of the
    normed row U is within
    E = (Q + 2^-22) |U| + D rstd
    y:   |w| E + 2^-22 (|w U| + |b|) + u_T |y|
    c1 = mean v within 2^-18 mean |v|, c2 = mean v U within 2^-18 mean |v U| + mean |v| E
    d:   rstd (2^-20 |v| + err c1 + |U| err c2 + |c2| E) + (Q + 2^-20) |rstd (v - c1 - U c2)| + 2^-22 |dh| + u_T |d|
    dx:  the same times the factor, and 3 u |dx| more
    dw:  (N + 64) u sum |dy U| + sum |dy| E;   db: (N + 64) u sum |dy|
(and half a step of 2^-24 for float16's small values).
"""
import pytest
import torch

import invariant_token_log_gb300 as bil
from philox import border_of, keep_mask

pytestmark = pytest.mark.gpu

EPS_R, EPS = 2.0 ** -18, 1e-5
U24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}
TYPES = list(U)
IDS = ["f32", "bf16", "f16"]
# every layout of a row over threads, and the widths at and around the steps between them
WIDTHS = [1, 7, 8, 9, 256, 257, 1000, 1024, 1025, 2049, 4096, 5001, 8192, 8193, 16383, 16384]
SEED = 0xABCDEF0123


def rows(n, width, dtype, seed, scale=1.0, pad=0, shift=0, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((n * (width + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    view = buf[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    view.copy_(scale * torch.randn(n, width, generator=g, device="cuda") + offset)
    return view


def vector(width, dtype, seed, about=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (about + 0.3 * torch.randn(width, generator=g, device="cuda")).to(dtype)


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), (what, float((err / bound).nan_to_num(nan=float("inf")).max()))


class Reference:
    """The formula in 64 bits from the stored h, and the bounds above."""

    def __init__(self, h, w, eps):
        self.h, self.w, self.dtype = h.double(), w.double(), h.dtype
        self.mean = self.h.mean(dim=1, keepdim=True)
        centred = self.h - self.mean
        self.rstd = 1 / torch.sqrt(centred.square().mean(dim=1, keepdim=True) + eps)
        self.u = centred * self.rstd
        self.d = 2.0 ** -18 * self.h.abs().mean(dim=1, keepdim=True) + 2.0 ** -140
        self.q = EPS_R + (self.d * self.rstd) ** 2
        self.e = (self.q + 2.0 ** -22) * self.u.abs() + self.d * self.rstd

    def check_forward(self, y, b, mean, rstd):
        b = torch.zeros_like(self.w) if b is None else b.double()
        ref = self.u * self.w + b
        within(mean, self.mean[:, 0], self.d[:, 0], "mean")
        within(rstd, self.rstd[:, 0], (self.q * self.rstd)[:, 0], "rstd")
        bound = self.w.abs() * self.e + 2.0 ** -22 * ((self.w * self.u).abs() + b.abs()) + U[self.dtype] * ref.abs()
        within(y, ref, bound + TINY[self.dtype], "y")

    def check_backward(self, dx, dr, dw, db, dy, dh, factor):
        n = len(self.h)
        dy = dy.double()
        dh = torch.zeros_like(dy) if dh is None else dh.double()
        v = dy * self.w
        c1, c2 = v.mean(dim=1, keepdim=True), (v * self.u).mean(dim=1, keepdim=True)
        e1 = 2.0 ** -18 * v.abs().mean(dim=1, keepdim=True)
        e2 = 2.0 ** -18 * (v * self.u).abs().mean(dim=1, keepdim=True) + (v.abs() * self.e).mean(dim=1, keepdim=True)
        inner = self.rstd * (v - c1 - self.u * c2)
        d = inner + dh
        bound = (self.rstd * (2.0 ** -20 * v.abs() + e1 + self.u.abs() * e2 + c2.abs() * self.e) +
                 (self.q + 2.0 ** -20) * inner.abs() + 2.0 ** -22 * dh.abs())
        rounded = U[self.dtype] * d.abs() + TINY[self.dtype]
        if factor is None:
            within(dx, d, bound + rounded, "dx")
            assert dr is None or dr is dx
        else:
            within(dx, d * factor, factor * (bound + rounded + 3 * U24 * d.abs()) + TINY[self.dtype], "dx")
            assert bool((dx[factor == 0] == 0).all())
            if dr is not None:
                within(dr, d, bound + rounded, "dr")
        within(dw, (dy * self.u).sum(dim=0), (n + 64) * U24 * (dy * self.u).abs().sum(dim=0) +
               (dy.abs() * self.e).sum(dim=0) + 1e-40, "dw")
        if db is not None:
            within(db, dy.sum(dim=0), (n + 64) * U24 * dy.abs().sum(dim=0) + 1e-40, "db")


def run(n, width, dtype, wtype, residual=True, bias=True, p=0.0, pad=0, shift=0, offset=0.0, eps=EPS):
    x = rows(n, width, dtype, 1, 1.0, pad, shift, offset)
    r = rows(n, width, dtype, 2, 4.0, pad, shift) if residual else None
    w, b = vector(width, wtype, 3, 1.0), vector(width, wtype, 4) if bias else None
    y, h, mean, rstd = bil.layer_norm_fwd(x, w, b, residual=r, eps=eps, p=p, seed=SEED, offset=2)
    factor = None
    if p:
        keep = torch.from_numpy(keep_mask(n, width, p, SEED, 2)).cuda()
        factor = keep.double() * (65536 / (65536 - border_of(p)))
    if h is None:
        assert r is None and not p
        h = x
    else:
        r64 = 0.0 if r is None else r.double()
        exact = (x.double() if factor is None else x.double() * factor) + r64
        slack = 4 * U24 * ((x.double() * (1.0 if factor is None else factor)).abs() + (0.0 if r is None else r64.abs()))
        within(h, exact, U[dtype] * exact.abs() + slack + TINY[dtype], "h")
    ref = Reference(h, w, eps)
    ref.check_forward(y, b, mean, rstd)
    dy = rows(n, width, dtype, 5, pad=pad, shift=shift)
    dh = rows(n, width, dtype, 6, pad=pad, shift=shift) if residual else None
    dx, dr, dw, db = bil.layer_norm_bwd(dy, h, w, mean, rstd, grad_h=dh, p=p, seed=SEED, offset=2, need_bias=bias,
                                        need_residual=residual)
    assert (db is None) == (not bias) and (dr is None) == (not residual)
    ref.check_backward(dx, dr, dw, db, dy, dh, factor)
    torch.cuda.synchronize()
    assert bil.watchdog_status() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    run(37, width, dtype, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("width", [1, 9, 257, 1000, 4096, 5001, 8192, 16383])
def test_widths_with_dropout(width, dtype):
    run(37, width, dtype, dtype, p=0.3)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("residual,bias,p", [(False, False, 0.0), (False, True, 0.0), (True, False, 0.0), (False, True, 0.2),
                                             (False, False, 0.2), (True, False, 0.2)])
@pytest.mark.parametrize("width,pad,shift", [(1104, 0, 0), (1104, 7, 3), (520, 64, 0)])
def test_forms(dtype, residual, bias, p, width, pad, shift):
    run(65, width, dtype, dtype, residual, bias, p, pad, shift)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("n,width,p,shift", [(50, 2048, 0.0, 0), (50, 2048, 0.1, 0), (50, 2047, 0.0, 1), (9, 100, 0.1, 0)])
def test_float32_weight(dtype, n, width, p, shift):
    run(n, width, dtype, torch.float32, p=p, shift=shift)


@pytest.mark.parametrize("n", [1, 2, 151, 153, 3000])
@pytest.mark.parametrize("width", [64, 768, 4096])
def test_row_counts(n, width):
    run(n, width, torch.bfloat16, torch.bfloat16, p=0.1)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("offset", [30.0, -500.0])
def test_rows_far_from_zero(dtype, offset):
    run(40, 1000, dtype, dtype, residual=False, offset=offset)


def test_constant_rows():
    """No variance: the normed row is zero (eps keeps rstd finite) and y is the bias."""
    x = torch.full((5, 512), 3.25, dtype=torch.bfloat16, device="cuda")
    w, b = vector(512, torch.bfloat16, 3, 1.0), vector(512, torch.bfloat16, 4)
    y, h, mean, rstd = bil.layer_norm_fwd(x, w, b)
    assert h is None and torch.equal(y, b.expand(5, 512)) and bool((mean == 3.25).all())
    assert bool(((rstd.double() * EPS ** 0.5 - 1).abs() < EPS_R).all())


def test_bad_values_stay_in_their_rows():
    x = rows(6, 300, torch.float32, 1)
    w, b = vector(300, torch.float32, 3, 1.0), vector(300, torch.float32, 4)
    good = bil.layer_norm_fwd(x, w, b)[0]
    x[1, 7], x[4, 0] = float("nan"), float("inf")
    y = bil.layer_norm_fwd(x, w, b)[0]
    assert bool(y[[1, 4]].isnan().all())
    assert torch.equal(y[[0, 2, 3, 5]], good[[0, 2, 3, 5]])


def test_rows_do_not_depend_on_the_batch():
    x, r = rows(300, 1104, torch.bfloat16, 1), rows(300, 1104, torch.bfloat16, 2)
    w, b = vector(1104, torch.bfloat16, 3, 1.0), vector(1104, torch.bfloat16, 4)
    whole = bil.layer_norm_fwd(x, w, b, residual=r)
    dx = bil.layer_norm_bwd(r, whole[1], w, whole[2], whole[3])[0]
    for a, e in ((0, 1), (7, 19), (150, 300)):
        part = bil.layer_norm_fwd(x[a:e], w, b, residual=r[a:e])
        for p, q in zip(part, whole):
            assert torch.equal(p, q[a:e])
        assert torch.equal(bil.layer_norm_bwd(r[a:e], part[1], w, part[2], part[3])[0], dx[a:e])


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, h, mean, rstd = bil.layer_norm_fwd(x, w, w, residual=x)
    assert y.shape == h.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    dx, dr, dw, db = bil.layer_norm_bwd(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_lead_dimensions_and_strides():
    x = rows(24, 264, torch.float16, 1)
    w, b = vector(264, torch.float16, 3, 1.0), vector(264, torch.float16, 4)
    y, _, mean, rstd = bil.layer_norm_fwd(x, w, b)
    y3, _, m3, s3 = bil.layer_norm_fwd(x.view(2, 3, 4, 264), w, b)
    assert y3.shape == (2, 3, 4, 264) and m3.shape == s3.shape == (2, 3, 4)
    assert torch.equal(y3.reshape(24, 264), y) and torch.equal(m3.reshape(-1), mean)
    assert torch.equal(bil.layer_norm_fwd(x.t().contiguous().t(), w, b)[0], y)
    one = x[:1].expand(24, 264)  # broadcast rows
    assert torch.equal(bil.layer_norm_fwd(one, w, b)[0], y[:1].expand(24, 264))
    d = bil.layer_norm_bwd(y[:1].expand(24, 264), x, w, mean, rstd)
    e = bil.layer_norm_bwd(y[:1].repeat(24, 1), x, w, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(d, e))


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_autograd_against_differences(p):
    """The gradient of a weighted sum of y and h along random directions, by central differences in 64 bits of the
    formula (under the kernel's mask), within a thousandth: the step's error is about 1e-6 of the value, the float32
    gradient's 1e-5 of the terms'."""
    n, width = 6, 40
    g = torch.Generator(device="cuda").manual_seed(9)
    x, r = (torch.randn(n, width, generator=g, device="cuda").requires_grad_() for _ in range(2))
    w, b = ((1 + 0.3 * torch.randn(width, generator=g, device="cuda")).requires_grad_() for _ in range(2))
    cy, ch = (torch.randn(n, width, generator=g, device="cuda") for _ in range(2))
    y, h = bil.layer_norm(x, w, b, residual=r, p=p, seed=SEED, offset=1)
    grads = torch.autograd.grad((y * cy + h * ch).sum(), (x, w, b, r))
    f = torch.from_numpy(keep_mask(n, width, p, SEED, 1)).cuda().double() * (65536 / (65536 - border_of(p)))

    def value(x, w, b, r):
        h = x * f + r
        c = h - h.mean(dim=1, keepdim=True)
        u = c / (c.square().mean(dim=1, keepdim=True) + EPS).sqrt()
        return ((u * w + b) * cy.double() + h * ch.double()).sum()

    at = [t.detach().double() for t in (x, w, b, r)]
    for i in range(4):
        way = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-5 * way, at[i] - 1e-5 * way
        slope = float(value(*up) - value(*down)) / 2e-5
        terms = float((grads[i].double() * way).abs().sum())
        assert abs(float((grads[i].double() * way).sum()) - slope) <= 1e-3 * terms


def test_autograd_partial_uses():
    x, r = (rows(8, 72, torch.float32, s).clone().requires_grad_() for s in (1, 2))
    w, b = (vector(72, torch.float32, s, 1.0).requires_grad_() for s in (3, 4))
    d = rows(8, 72, torch.float32, 5)
    y, h = bil.layer_norm(x, w, b, residual=r, p=0.5, seed=4)
    dx, dr = torch.autograd.grad(h, (x, r), d, retain_graph=True)  # the stream alone
    assert torch.equal(dr, d) and torch.equal(dx, bil.dropout_bwd(d, 0.5, 4))
    dx, dw = torch.autograd.grad(y, (x, w), d, retain_graph=True)  # y alone
    _, h2, mean, rstd = bil.layer_norm_fwd(x, w, b, residual=r, p=0.5, seed=4)
    ex, er, ew, eb = bil.layer_norm_bwd(d, h2, w, mean, rstd, p=0.5, seed=4)
    assert torch.equal(dx, ex) and torch.equal(dw, ew)
    frozen = bil.layer_norm(x.detach(), w.detach(), b, p=0.0)
    (db,) = torch.autograd.grad(frozen, b, d)
    assert torch.equal(db, eb)
    (gx,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(gx.sum(), x)  # a second derivative is an error
