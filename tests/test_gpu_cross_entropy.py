"""The LM head's cross entropy and its gradients against the formula in 64 bits.

Tolerances, with u = 2^-24 and u_T the 16-bit type's unit roundoff.
  Z:    a logit is accumulated in float32 in steps of 16 products; with P the largest
        prefix sum and C the largest sum of a step's |products|, E_z = (H / 16 + 1) 2^-23 (P + C).
  lse:  a term 2^((z - m) log2 e) is within |t| 2^-23 + 2^-22 relative, |t| < 2^5 where a term
        counts, its sums are at most 16 + 3 + V / 4096 + 34 additions deep: 2^-17 covers both for
        V < 2^18, and E_lse = E_z + 2^-17 + 2^-22 |lse|.
  loss: 2 E_z + 2^-16 + 2^-21 (|lse| + |z_t| + mean |z| + f lse^2) + 2 f |lse| E_lse; added up over N
        rows: (N / 1024 + 16) u sum |loss| more.
  dz:   with a = g (1 + 2 f lse), b = g (1 - e), c = g e / V and D = a p + b [c = t] + c in magnitudes,
        (E_z + E_lse + 2 f E_lse + 2^-18) D, and its rounding u_T |dz|; in float16 the largest a or b is brought
        to 2^12, so that half a step of 2^-24 below 2^-14 is 2^-36 of the largest D or less.
  products: K / 16 + 16 accumulation steps of 2^-23 of sum |dz| |w| (or |x|) at most, and the result's rounding.
"""
import pytest
import torch

import invariant_token_log_gb300 as bil
from invariant_token_log_gb300.cross_entropy import bwd_workspace_bytes, fwd_workspace_bytes

pytestmark = pytest.mark.gpu

IGNORE = -100
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}
TYPES = [torch.bfloat16, torch.float16]
IDS = ["bf16", "f16"]
SIZES = [(1, 1, 8), (1, 300, 64), (5, 257, 72), (64, 1000, 128), (130, 129, 264), (257, 5000, 72), (300, 2049, 1104),
         (1000, 700, 136), (33, 40000, 64), (513, 256, 4096)]


def make(n, vocab, width, dtype, seed=1, ignored=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, width, generator=g, device="cuda").to(dtype)
    w = (torch.randn(vocab, width, generator=g, device="cuda") * (3 / width ** 0.5)).to(dtype)
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    t[torch.rand(n, generator=g, device="cuda") < ignored] = IGNORE
    return x, w, t


class Reference:
    def __init__(self, x, w, t, smoothing=0.0, z_loss=0.0, reduction="mean"):
        self.dtype, self.e, self.f, self.reduction = x.dtype, smoothing, z_loss, reduction
        self.act = t != IGNORE
        self.x, self.w = torch.where(self.act[:, None], x.double(), 0.0), w.double()
        n, width = x.shape
        self.n, self.vocab = n, w.shape[0]
        z = torch.zeros(n, self.vocab, dtype=torch.float64, device="cuda")
        prefix = step = 0.0
        for k in range(0, width, 16):
            z += self.x[:, k:k + 16] @ self.w[:, k:k + 16].t()
            prefix = max(prefix, float(z.abs().max()))
            step = max(step, float((self.x[:, k:k + 16].abs() @ self.w[:, k:k + 16].abs().t()).max()))
        self.z, self.ez = z, (width / 16 + 1) * 2.0 ** -23 * (prefix + step)
        self.lse = torch.where(self.act, z.logsumexp(dim=1), 0.0)
        self.elose = self.ez + 2.0 ** -17 + 2.0 ** -22 * self.lse.abs()
        self.at = t.clamp(0, self.vocab - 1)[:, None]
        zt = z.gather(1, self.at)[:, 0]
        rows = self.lse - (1 - smoothing) * zt - smoothing * z.mean(dim=1) + z_loss * self.lse ** 2
        self.rows = torch.where(self.act, rows, 0.0)
        self.erows = torch.where(self.act, 2 * self.ez + 2.0 ** -16 + 2.0 ** -21 *
                                 (self.lse.abs() + zt.abs() + z.abs().mean(dim=1) + abs(z_loss) * self.lse ** 2) +
                                 2 * abs(z_loss) * self.lse.abs() * self.elose, 0.0)
        self.count = max(1, int(self.act.sum()))

    def check_loss(self, loss, lse):
        assert loss.dtype == lse.dtype == torch.float32
        assert bool(((lse.double() - self.lse).abs() <= self.elose * self.act).all())
        if self.reduction == "none":
            err, bound = (loss.double() - self.rows).abs(), self.erows
        else:
            by = self.count if self.reduction == "mean" else 1
            err = (loss.double() - self.rows.sum() / by).abs()
            bound = (self.erows.sum() + (self.n / 1024 + 16) * 2.0 ** -24 * self.rows.abs().sum()) / by + 1e-30
        assert bool((err <= bound).all()), float((err / bound).max())

    def check_grads(self, dh, dw, g):
        g = torch.where(self.act, g.double().expand(self.n), 0.0)
        if self.reduction == "mean":
            g = g / self.count
        p = (self.z - self.lse[:, None]).exp()
        a, b, c = g * (1 + 2 * self.f * self.lse), g * (1 - self.e), g * self.e / self.vocab
        dz = a[:, None] * p - c[:, None]
        dz.scatter_add_(1, self.at, -b[:, None])
        size = a.abs()[:, None] * p + c.abs()[:, None]
        size.scatter_add_(1, self.at, b.abs()[:, None])
        slack = self.ez + (1 + 2 * abs(self.f)) * self.elose[:, None] + 2.0 ** -18
        err = slack * size + U[self.dtype] * dz.abs()
        if self.dtype == torch.float16:
            err = err + 2.0 ** -36 * float(torch.maximum(a.abs(), b.abs()).max()) * self.act[:, None]
        for got, left, right, terms, what in ((dh, (dz, err), self.w, self.vocab, "dhidden"),
                                              (dw, (dz.t(), err.t()), self.x, self.n, "dweight")):
            if got is None:
                continue
            ref = left[0] @ right
            bound = left[1] @ right.abs() + (terms / 16 + 16) * 2.0 ** -23 * (left[0].abs() @ right.abs())
            bound = bound * 1.01 + U[got.dtype] * ref.abs() + TINY[got.dtype]
            off = (got.double() - ref).abs()
            assert bool((off <= bound).all()), (what, float((off / bound).nan_to_num(nan=float("inf")).max()))
        if dh is not None:
            assert bool((dh[~self.act] == 0).all())


def run(x, w, t, g=None, piece=None, out_dtype=None, **how):
    reduction = how.get("reduction", "mean")
    if g is None:
        gen = torch.Generator(device="cuda").manual_seed(5)
        g = torch.randn(x.shape[0], generator=gen, device="cuda") if reduction == "none" else torch.tensor(0.7, device="cuda")
    ref = Reference(x, w, t, how.get("label_smoothing", 0.0), how.get("z_loss", 0.0), reduction)
    loss, lse = bil.linear_cross_entropy_fwd(x, w, t, **how)
    ref.check_loss(loss, lse)
    dh, dw = bil.linear_cross_entropy_bwd(x, w, t, lse, g, piece=piece, out_dtype=out_dtype, **how)
    assert dh.dtype == dw.dtype == (out_dtype or x.dtype) and dh.shape == x.shape and dw.shape == w.shape
    ref.check_grads(dh, dw, g)
    assert bil.watchdog_status() == 0
    return loss, lse, dh, dw


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n,vocab,width", SIZES)
def test_mean(n, vocab, width, dtype):
    run(*make(n, vocab, width, dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n,vocab,width", [(1, 300, 64), (130, 129, 264), (257, 5000, 72), (300, 2049, 1104)])
@pytest.mark.parametrize("reduction,smoothing,z_loss", [("sum", 0.1, 0.0), ("none", 0.0, 1e-3), ("mean", 1.0, 0.0),
                                                        ("none", 0.3, 1e-2)])
def test_forms(n, vocab, width, dtype, reduction, smoothing, z_loss):
    run(*make(n, vocab, width, dtype), reduction=reduction, label_smoothing=smoothing, z_loss=z_loss)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n,vocab,width,piece", [(300, 2049, 136, 256), (300, 2049, 136, 700), (64, 5000, 72, 1024),
                                                 (600, 1024, 520, 512), (20, 300, 64, 10 ** 12)])
def test_pieces(n, vocab, width, piece, dtype):
    x, w, t = make(n, vocab, width, dtype)
    _, lse, dh, dw = run(x, w, t, piece=piece, z_loss=1e-4)
    whole = bil.linear_cross_entropy_bwd(x, w, t, lse, torch.tensor(0.7, device="cuda"), z_loss=1e-4)
    assert torch.equal(dw, whole[1])  # a row of it lies in one piece


@pytest.mark.parametrize("which", ["none", "all", "one", "first", "last", "alternate", "blocks"])
@pytest.mark.parametrize("n", [1, 63, 300, 700])
def test_ignored_rows(n, which):
    """What an ignored row holds reaches nothing: NaN and infinities there, the others' bits as without them."""
    x, w, t = make(n, 700, 72, torch.bfloat16, ignored=0.0)
    i = torch.arange(n, device="cuda")
    ignored = {"none": i < 0, "all": i >= 0, "one": i != n // 2, "first": i < 130, "last": i >= n - 130, "alternate": i % 2 == 0,
               "blocks": i // 256 % 2 == 1}[which]
    t[ignored] = IGNORE
    loss, lse, dh, dw = run(x, w, t, z_loss=1e-4)
    bad = x.clone()
    bad[ignored] = float("nan")
    bad[ignored, ::2] = float("inf")
    l2, s2 = bil.linear_cross_entropy_fwd(bad, w, t, z_loss=1e-4)
    h2, w2 = bil.linear_cross_entropy_bwd(bad, w, t, lse, torch.tensor(0.7, device="cuda"), z_loss=1e-4)
    assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(h2, dh) and torch.equal(w2, dw)
    if bool(ignored.all()):
        assert float(loss) == 0 and not dw.any() and not dh.any()
    else:  # and the rows that count alone give the same bits
        kept = ~ignored
        l3, s3 = bil.linear_cross_entropy_fwd(x[kept], w, t[kept], z_loss=1e-4)
        h3, w3 = bil.linear_cross_entropy_bwd(x[kept], w, t[kept], s3, torch.tensor(0.7, device="cuda"), z_loss=1e-4)
        assert torch.equal(l3, loss) and torch.equal(s3, lse[kept]) and torch.equal(w3, dw)


@pytest.mark.parametrize("scale", [1e-12, 1e-6, 1.0, 65536.0, 1e20])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gradient_scales(scale, dtype):
    """The loss's gradient at any size: float32 results, where float16 ones would overflow."""
    x, w, t = make(200, 3000, 72, dtype)
    run(x, w, t, g=torch.tensor(scale, device="cuda"), out_dtype=torch.float32)
    g = scale * torch.linspace(-1, 1, 200, device="cuda")
    run(x, w, t, g=g, out_dtype=torch.float32, reduction="none")


def test_zero_gradient():
    x, w, t = make(100, 500, 64, torch.float16)
    _, lse = bil.linear_cross_entropy_fwd(x, w, t)
    dh, dw = bil.linear_cross_entropy_bwd(x, w, t, lse, torch.tensor(0.0, device="cuda"))
    assert not dh.any() and not dw.any()


def test_targets_outside_the_vocabulary():
    x, w, t = make(40, 300, 64, torch.bfloat16, ignored=0.0)
    t[3], t[17], t[20] = 300, -1, 2 ** 40
    loss, lse = bil.linear_cross_entropy_fwd(x, w, t, reduction="none")
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 17, 20]] = True
    assert bool(loss[bad].isnan().all()) and not loss[~bad].isnan().any() and not lse.isnan().any()
    dh, dw = bil.linear_cross_entropy_bwd(x, w, t, lse, torch.ones(40, device="cuda"), reduction="none")
    assert bool(dh[bad].isnan().all()) and not dh[~bad].isnan().any() and bool(dw.isnan().all())
    with pytest.raises(bil.BilError):
        bil.linear_cross_entropy_fwd(x, w, t, validate=True)


def test_a_nan_row_stays_a_row():
    x, w, t = make(40, 300, 64, torch.bfloat16, ignored=0.0)
    good = bil.linear_cross_entropy_fwd(x, w, t, reduction="none")[0]
    x[5, 3] = float("nan")
    loss = bil.linear_cross_entropy_fwd(x, w, t, reduction="none")[0]
    keep = torch.arange(40, device="cuda") != 5
    assert bool(loss[5].isnan()) and torch.equal(loss[keep], good[keep])


def test_lse_does_not_depend_on_the_batch():
    x, w, t = make(700, 3000, 264, torch.bfloat16)
    lse = bil.linear_cross_entropy_fwd(x, w, t)[1]
    for a, b in ((0, 1), (3, 140), (256, 700)):
        assert torch.equal(bil.linear_cross_entropy_fwd(x[a:b], w, t[a:b])[1], lse[a:b])


def test_the_same_bits_every_time():
    x, w, t = make(900, 3000, 520, torch.bfloat16)
    g = torch.tensor(1.0, device="cuda")
    first = None
    for _ in range(4):
        loss, lse = bil.linear_cross_entropy_fwd(x, w, t, label_smoothing=0.1)
        now = (loss, lse, *bil.linear_cross_entropy_bwd(x, w, t, lse, g, label_smoothing=0.1, piece=512))
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_layouts():
    x, w, t = make(60, 500, 72, torch.bfloat16)
    loss, lse, dh, dw = run(x, w, t)
    wide = torch.full((60, 96), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, 8:80] = x
    tall = torch.full((500, 88), float("nan"), dtype=x.dtype, device="cuda")
    tall[:, :72] = w
    for xx, ww in ((wide[:, 8:80], tall[:, :72]), (x.t().contiguous().t(), w.t().contiguous().t()), (wide[:, 8:80], w)):
        l2, s2 = bil.linear_cross_entropy_fwd(xx, ww, t)
        h2, w2 = bil.linear_cross_entropy_bwd(xx, ww, t, s2, torch.tensor(0.7, device="cuda"))
        assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(h2, dh) and torch.equal(w2, dw)
    l3, s3 = bil.linear_cross_entropy_fwd(x.view(3, 20, 72), w, t.view(3, 20), reduction="none")
    assert l3.shape == s3.shape == (3, 20)
    h3, w3 = bil.linear_cross_entropy_bwd(x.view(3, 20, 72), w, t.view(3, 20).to(torch.int32), lse,
                                          torch.tensor(0.7, device="cuda"))
    assert h3.shape == (3, 20, 72) and torch.equal(h3.view(60, 72), dh) and torch.equal(w3, dw)
    one, ones = x[:1].expand(60, 72), t.clamp_min(0)  # one row's hidden states for every target
    run(one.contiguous(), w, ones)
    assert torch.equal(bil.linear_cross_entropy_fwd(one, w, ones)[0], bil.linear_cross_entropy_fwd(one.contiguous(), w, ones)[0])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_hidden_sizes_off_eight_elements(dtype):
    """Rows of a padded buffer, a hidden size of no whole 16 bytes: what lies behind a row is not read."""
    for width in (1, 7, 65, 135):
        x, w, t = make(50, 300, width, dtype)
        ld = -(-width // 8) * 8 + 8
        xx, ww = (torch.full((m.shape[0], ld), float("nan"), dtype=dtype, device="cuda") for m in (x, w))
        xx[:, :width], ww[:, :width] = x, w
        run(xx[:, :width], ww[:, :width], t)


def test_one_of_the_gradients():
    x, w, t = make(300, 1500, 136, torch.bfloat16)
    g = torch.tensor(1.0, device="cuda")
    lse = bil.linear_cross_entropy_fwd(x, w, t)[1]
    dh, dw = bil.linear_cross_entropy_bwd(x, w, t, lse, g, piece=512)
    a, b = bil.linear_cross_entropy_bwd(x, w, t, lse, g, piece=512, need_weight=False)
    assert b is None and torch.equal(a, dh)
    a, b = bil.linear_cross_entropy_bwd(x, w, t, lse, g, piece=512, need_hidden=False)
    assert a is None and torch.equal(b, dw)


def test_no_rows():
    x, w, t = make(0, 300, 64, torch.bfloat16)
    loss, lse = bil.linear_cross_entropy_fwd(x, w, t)
    assert float(loss) == 0 and lse.shape == (0,)
    dh, dw = bil.linear_cross_entropy_bwd(x, w, t, lse, torch.tensor(1.0, device="cuda"))
    assert dh.shape == (0, 64) and not dw.any()
    assert bil.linear_cross_entropy_fwd(x, w, t, reduction="none")[0].shape == (0,)


def test_given_workspaces():
    x, w, t = make(70, 900, 72, torch.bfloat16)
    dev = x.device
    f = torch.empty(fwd_workspace_bytes(70, 72, 900, True), dtype=torch.uint8, device=dev)
    b = torch.empty(bwd_workspace_bytes(70, 72, 900, dev, 256), dtype=torch.uint8, device=dev)
    loss, lse = bil.linear_cross_entropy_fwd(x, w, t, label_smoothing=0.2, workspace=f)
    got = bil.linear_cross_entropy_bwd(x, w, t, lse, torch.tensor(1.0, device=dev), label_smoothing=0.2, piece=256, workspace=b)
    ref = Reference(x, w, t, 0.2)
    ref.check_loss(loss, lse)
    ref.check_grads(*got, torch.tensor(1.0, device=dev))
    with pytest.raises(ValueError, match="workspace"):
        bil.linear_cross_entropy_fwd(x, w, t, label_smoothing=0.2, workspace=f[:-1])


@pytest.mark.parametrize("smoothing,z_loss", [(0.0, 0.0), (0.1, 1e-2)])
def test_autograd_against_differences(smoothing, z_loss):
    """Along random directions, by central differences of the formula in 64 bits: the 16-bit gradients are within
    u_T of their terms three times over (dz, the sum, the result), 2^-6 of them for bfloat16."""
    x, w, t = make(24, 200, 64, torch.bfloat16)
    x, w = x.requires_grad_(), w.requires_grad_()
    loss = bil.linear_cross_entropy(x, w, t, label_smoothing=smoothing, z_loss=z_loss)
    grads = torch.autograd.grad(loss, (x, w))

    def value(x, w):
        z = x @ w.t()
        lse = z.logsumexp(dim=1)
        rows = lse - (1 - smoothing) * z.gather(1, t.clamp_min(0)[:, None])[:, 0] - smoothing * z.mean(dim=1) + z_loss * lse ** 2
        return (rows * (t != IGNORE)).sum() / (t != IGNORE).sum()

    at = [x.detach().double(), w.detach().double()]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for i in range(2):
        way = torch.randn(at[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-5 * way, at[i] - 1e-5 * way
        slope = float(value(*up) - value(*down)) / 2e-5
        terms = float((grads[i].double() * way).abs().sum())
        assert abs(float((grads[i].double() * way).sum()) - slope) <= 2.0 ** -6 * terms
    with pytest.raises(RuntimeError):  # a second derivative is an error
        (gx,) = torch.autograd.grad(bil.linear_cross_entropy(x, w, t), x, create_graph=True)
        torch.autograd.grad(gx.sum(), x)


def test_first_call_of_a_thread():
    """A thread whose first CUDA call is the library's (a backward pass's thread)."""
    import threading
    x, w, t = make(50, 300, 64, torch.bfloat16)
    loss, lse = bil.linear_cross_entropy_fwd(x, w, t)
    g = torch.tensor(1.0, device="cuda")
    want = bil.linear_cross_entropy_bwd(x, w, t, lse, g)
    torch.cuda.synchronize()
    got = []
    thread = threading.Thread(target=lambda: got.append(bil.linear_cross_entropy_bwd(x, w, t, lse, g)))
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert len(got) == 1 and torch.equal(got[0][0], want[0]) and torch.equal(got[0][1], want[1])
