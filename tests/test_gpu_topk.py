"""The selected-token log-probability with the row's largest alternatives.

logp, lse and the entropy have to be logp_fwd's bits; the columns are exact
(compared with a sort); an alternative's log-probability is z - lse rounded
once, so it is compared bit for bit with that, and with 64 bits within the
logits path's 1e-4.

Gradient tolerance (float32 gradients).  Per element, with the forward's lse
and H in the kernel: entropy_grad_tol of gpu_helpers with G = g + sum gk in the
place of g (1e-6 + rcp (|G| rho p + |gh| ...)).  G is a float32 sum of k + 1
terms, off by at most 2^-19 sum |gk| for k <= 128 (k / 32 + 6 additions): times
p.  A named column's W is such a sum too: (k + 2) 2^-24 sum of its |terms|.
"""
import math

import numpy as np
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import LOGP_ATOL, assert_close_elementwise, check_watchdog, entropy_grad_tol, f32_bits
from invariant_token_log_gb300 import _lib
from invariant_token_log_gb300 import topk as topk_mod

pytestmark = pytest.mark.gpu
IGNORE = bil.IGNORE_INDEX
NAN, INF = math.nan, math.inf
TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(n, vocab, dtype, seed, pad=0, shift=0, scale=3.0):
    """[n, vocab] logits in rows `pad` elements further apart, `shift` elements into their storage; what
    lies around them is +inf, which would win every comparison it got into."""
    buf = torch.full((n * (vocab + pad) + shift + 8,), INF, dtype=dtype, device="cuda")
    view = buf[shift:shift + n * (vocab + pad)].view(n, vocab + pad)[:, :vocab]
    view.copy_(scale * torch.randn(n, vocab, generator=gen(seed), device="cuda"))
    return view


def targets(n, vocab, seed, ignore_every=0):
    t = torch.randint(0, vocab, (n,), generator=gen(seed + 1), device="cuda")
    if ignore_every:
        t[::ignore_every] = IGNORE
    return t


def sorted_columns(x, k):
    """The first k columns by (value descending, column ascending, NaN last), from a stable sort on the host."""
    v = x.detach().double().cpu().numpy()
    key = np.where(np.isnan(v), 1, 0), np.where(np.isnan(v), 0.0, -v)
    return np.lexsort((key[1], key[0]), axis=-1)[:, :k]  # lexsort is stable


def rcp_of(temperature):
    return np.float32(1.0) / np.float32(temperature)


def check(x, t, k, tile_v=4096, temperature=1.0, **kw):
    """Every output of logp_topk against logp_fwd, the sort and the subtraction."""
    logp, lse, ent, ids, top = bil.logp_topk(x, t, k, tile_v=tile_v, temperature=temperature, return_entropy=True, **kw)
    rlogp, rlse, rent = bil.logp_fwd(x, t, tile_v=tile_v, temperature=temperature, return_entropy=True)
    for name, a, b in (("logp", logp, rlogp), ("lse", lse, rlse), ("entropy", ent, rent)):
        a, b = f32_bits(a), f32_bits(b)
        both_nan = np.isnan(a.view(np.float32)) & np.isnan(b.view(np.float32))
        assert np.array_equal(np.where(both_nan, 0, a), np.where(both_nan, 0, b)), name
    act = (t != IGNORE).cpu().numpy()
    want = np.where(act[:, None], sorted_columns(x, k), -1)
    assert np.array_equal(ids.cpu().numpy(), want)
    z = x.float().gather(1, ids.clamp_min(0)) + 0.0
    if temperature != 1.0:
        z = z * float(rcp_of(temperature))
    want = torch.where((t != IGNORE)[:, None], z - lse[:, None], torch.zeros((), device="cuda"))
    assert torch.equal(top.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
    # without the entropy: the same bits
    plain = bil.logp_topk(x, t, k, tile_v=tile_v, temperature=temperature, **kw)
    for a, b in zip(plain, (logp, lse, ids, top)):
        assert torch.equal(a.nan_to_num(nan=7.0) if a.is_floating_point() else a,
                           b.nan_to_num(nan=7.0) if b.is_floating_point() else b)
    return logp, lse, ent, ids, top


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [1, 7, 8, 9, 33, 255, 4095, 4096, 4097, 20000])
def test_vocabularies(vocab, dtype):
    x = rows(6, vocab, dtype, vocab, pad=-vocab % 8)
    t = targets(6, vocab, vocab, ignore_every=4)
    for k in sorted({1, min(5, vocab), min(20, vocab), min(128, vocab)}):
        check(x, t, k)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 64, 65, 127, 128])
def test_counts(k, dtype):
    x = rows(9, 5003, dtype, k, pad=5)
    check(x, targets(9, 5003, k), k, temperature=0.7)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n", [1, 2, 3, 17, 64, 300])
def test_batches_of_the_benchmark_vocabulary(n, dtype):
    """From a row cut into many units to a row a warp."""
    x = rows(n, 151936, dtype, n)
    logp, lse, ent, ids, top = check(x, targets(n, 151936, n), 20)
    ref = torch.log_softmax(x.double(), dim=1).gather(1, ids)
    assert float((top.double() - ref).abs().max()) <= LOGP_ATOL


@pytest.mark.parametrize("n", [2127, 2128, 2129, 5000])
def test_more_rows_than_warps(n):
    x = rows(n, 9000, torch.bfloat16, n)
    check(x, targets(n, 9000, n, ignore_every=7), 10)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (0, 1), (3, 5), (8, 7), (7, 3)])
def test_rows_off_boundaries(pad, shift, dtype):
    for vocab, k in ((5001, 20), (12345, 50)):
        x = rows(5, vocab, dtype, 3, pad=pad, shift=shift)
        check(x, targets(5, vocab, 3), k)
        check(x, targets(5, vocab, 3), k, temperature=1.7)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("tile_v", [8, 512, 2048, 4096, 8192, 16384])
@pytest.mark.parametrize("pad", [0, 3])
def test_tile_widths(tile_v, pad, dtype):
    """Tiles of one group up to a stage of 64 KB, held in registers or not; the alternatives are the same."""
    vocab = 12000 if tile_v >= 512 else 3000
    x = rows(4, vocab, dtype, tile_v, pad=pad)
    t = targets(4, vocab, tile_v)
    for k in (3, 40):
        check(x, t, k, tile_v=tile_v)


def test_largest_tile_of_16_bits():
    x = rows(3, 70000, torch.bfloat16, 1)
    check(x, targets(3, 70000, 1), 33, tile_v=32768)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("k", [1, 20, 128])
def test_ties_and_orders(k, dtype):
    """Rows of one value, of two, of a few, ascending (every column enters the list) and descending, both
    zeros, infinities."""
    vocab = 9000
    ramp = torch.arange(vocab, device="cuda", dtype=torch.float32) / 64 - 70
    x = torch.zeros(9, vocab, device="cuda")
    x[1] = -2.5
    x[2] = torch.randint(0, 2, (vocab,), generator=gen(1), device="cuda").float()
    x[3] = torch.randint(0, 5, (vocab,), generator=gen(2), device="cuda").float()
    x[4] = ramp
    x[5] = -ramp
    x[6, ::2] = -0.0
    x[7] = ramp
    x[7, 5000:5200] = INF
    x[8] = torch.where(torch.arange(vocab, device="cuda") % 100 == 99, 1.0, -1.0)
    check(x.to(dtype), targets(9, vocab, 5), k)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("k", [1, 20, 100])
@pytest.mark.parametrize("hole", ["-inf", "lowest"])
def test_masks(k, hole, dtype):
    """Masks that leave nothing, one column, fewer than k, the last column, all but one; masked columns hold
    -inf or the type's lowest value."""
    vocab = 10007
    low = -INF if hole == "-inf" else torch.finfo(dtype).min
    x = torch.full((7, vocab), low, dtype=dtype, device="cuda")
    src = rows(7, vocab, dtype, 9)
    x[1, 777] = src[1, 777]
    x[2, 5000:5010] = src[2, 5000:5010]
    x[3, vocab - 1] = src[3, vocab - 1]
    x[4] = src[4]
    x[4, 123] = low
    x[5, ::997] = src[5, ::997]
    x[6, 4096:] = src[6, 4096:]
    check(x, targets(7, vocab, 9), k)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("k", [1, 20, 64])
def test_nan(k, dtype):
    """A NaN makes the row's statistics NaN and comes last among its columns, even after -inf."""
    vocab = 6000
    x = rows(6, vocab, dtype, 11)
    x[0, 17] = NAN
    x[1] = NAN
    x[2] = NAN
    x[2, 3000:3005] = -INF
    x[3, :4096] = NAN
    x[4] = -INF
    x[4, ::2] = NAN
    check(x, targets(6, vocab, 11), k)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("k", [1, 20, 33, 128])
def test_concentrated_columns(k, dtype):
    """Thousands of large logits where few lanes of few tiles hold them, distinct, few-valued and equal: the
    columns above any bound taken over lanes are many."""
    vocab = 40000
    x = rows(6, vocab, dtype, 12, scale=1.0)
    c = torch.arange(vocab, device="cuda")
    lane, tile = c // 8 % 32, c // 4096
    noise = torch.rand(vocab, generator=gen(13), device="cuda")
    for r, (lanes, tiles) in enumerate(((10, 1), (10, 10), (1, 10), (32, 1))):
        where = (lane < lanes) & (tile < tiles)
        x[r] = torch.where(where, 50 + 100 * noise, x[r].float()).to(dtype)
    x[4] = torch.where(lane < 5, 60 + (4 * noise).floor(), x[4].float()).to(dtype)
    x[5] = torch.where((lane == 7) & (tile > 4), torch.full_like(noise, 40.0), x[5].float()).to(dtype)
    check(x, targets(6, vocab, 12), k)


@pytest.mark.parametrize("n", [3, 200, 3000])
def test_rows_bitwise_across_batches(n):
    """A row's results do not depend on how the batch is cut."""
    bank = rows(3000, 8200, torch.bfloat16, 21)[:n]
    t = targets(n, 8200, 21)
    ref = bil.logp_topk(bank, t, 20, return_entropy=True)
    for size in (1, 2, min(n, 150)):
        idx = torch.randperm(n, generator=gen(size), device="cuda")[:size]
        for a, b in zip(bil.logp_topk(bank[idx], t[idx], 20, return_entropy=True), ref):
            assert torch.equal(a, b[idx])


def test_vocab_argument_leading_shape_and_targets():
    x = rows(12, 3000, torch.bfloat16, 22)
    x[:, 2900:] = INF  # pad columns past `vocab` take no part
    t = targets(12, 2900, 22)
    ref = bil.logp_topk(x[:, :2900].contiguous(), t, 7, return_entropy=True)
    got = bil.logp_topk(x, t, 7, vocab=2900, return_entropy=True)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    got = bil.logp_topk(x.reshape(3, 4, 3000), t.to(torch.int32).reshape(3, 4), 7, vocab=2900, return_entropy=True)
    assert got[0].shape == (3, 4) and got[3].shape == (3, 4, 7)
    for a, b in zip(got, ref):
        assert torch.equal(a.reshape(b.shape), b)
    t[3], t[5] = 2900, -7
    logp, lse, ids, top = bil.logp_topk(x, t, 7, vocab=2900)
    assert bool(logp[3].isnan() & logp[5].isnan())
    assert torch.equal(lse, ref[1]) and torch.equal(ids, ref[3]) and torch.equal(top, ref[4])


def test_the_target_among_the_alternatives_has_the_same_bits():
    x = rows(50, 4000, torch.float32, 23)
    t = x.argmax(dim=1)
    logp, _, ids, top = bil.logp_topk(x, t, 3, temperature=0.9)
    assert torch.equal(ids[:, 0], t) and torch.equal(top[:, 0], logp)


def test_offsets_past_32_bits():
    """More than 2^32 logits: the last rows are those of a small batch."""
    n, vocab = 28500, 151936
    assert n * vocab > 2 ** 32
    x = torch.zeros(n, vocab, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rows(3, vocab, torch.bfloat16, 24)
    t = targets(n, vocab, 24)
    got = bil.logp_topk(x, t, 5)
    ref = bil.logp_topk(x[-3:].clone(), t[-3:], 5)
    for a, b in zip(got, ref):
        assert torch.equal(a[-3:], b)
    assert torch.equal(got[2][0], torch.arange(5, device="cuda"))
    g, gk = torch.ones(n, device="cuda"), torch.ones(n, 5, device="cuda")
    d = bil.logp_topk_bwd(x, t, got[2], got[1], g, gk)
    dref = bil.logp_topk_bwd(x[-3:].clone(), t[-3:], ref[2], ref[1], g[-3:], gk[-3:])
    assert torch.equal(d[-3:], dref)


def test_another_stream_and_a_kept_workspace():
    x, t = rows(40, 151936, torch.bfloat16, 25), targets(40, 151936, 25)
    ref = bil.logp_topk(x, t, 20, return_entropy=True)
    torch.cuda.synchronize()
    space = torch.empty(topk_mod.workspace_bytes(x.dtype, 40, 151936, 20, entropy=True), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [bil.logp_topk(x, t, 20, return_entropy=True, workspace=space) for _ in range(3)]
    s.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, ref))


# ---------------------------------------------------------------------------
# Backward.
# ---------------------------------------------------------------------------

def gradient64(x, t, ids, lse, g, gk, ent, gh, temperature):
    """(d, p, a + H) in 64 bits from the forward's lse and entropy."""
    v = x.shape[1]
    z = x.double() / temperature
    a = z - torch.logsumexp(z, dim=1, keepdim=True)
    p = a.exp()
    H = -(torch.where(p > 0, p * a, p)).sum(dim=1, keepdim=True)
    w = torch.zeros_like(z)
    w.scatter_add_(1, t.clamp(0, v - 1)[:, None], g.double()[:, None])
    ok = (ids >= 0) & (ids < v)
    w.scatter_add_(1, ids.clamp(0, v - 1), torch.where(ok, gk.double(), torch.zeros((), dtype=torch.float64, device="cuda")))
    G = g.double() + gk.double().sum(dim=1)
    d = w - G[:, None] * p
    if gh is not None:
        d = d - gh.double()[:, None] * torch.where(p > 0, p * (a + H), p)
    d = d / temperature
    return torch.where((t != IGNORE)[:, None], d, torch.zeros((), dtype=torch.float64, device="cuda")), p, a + H, G


def check_gradient(d, x, t, ids, lse, g, gk, ent, gh, temperature):
    ref, p, ah, G = gradient64(x, t, ids, lse, g, gk, ent, gh, temperature)
    np_ = lambda v: v.double().cpu().numpy()  # noqa: E731
    tol = entropy_grad_tol(np_(p), np_(ah), np_(G), np.zeros(len(t)) if gh is None else np_(gh), 1 / temperature)
    k = gk.shape[1]
    tol = tol + (2.0 ** -19 * np_(gk.abs().sum(dim=1))[:, None] * np_(p)
                 + (k + 2) * 2.0 ** -24 * (np_(gk.abs().sum(dim=1)) + np_(g.abs()))[:, None]) / temperature
    assert_close_elementwise(d.float().cpu().numpy(), np_(ref), tol, "dlogits")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("k,temperature", [(1, 1.0), (20, 0.7), (128, 1.3)])
def test_backward_against_64_bits(k, temperature, entropy, dtype):
    n, vocab = 12, 3001
    x = rows(n, vocab, dtype, k, pad=7)
    t = targets(n, vocab, k, ignore_every=5)
    logp, lse, ent, ids, top = bil.logp_topk(x, t, k, temperature=temperature, return_entropy=True)
    t[1] = ids[1, 0] if t[1] != IGNORE else t[1]  # the target among the alternatives
    g = torch.randn(n, generator=gen(1), device="cuda")
    gk = torch.randn(n, k, generator=gen(2), device="cuda")
    gh = torch.randn(n, generator=gen(3), device="cuda") if entropy else None
    d = bil.logp_topk_bwd(x, t, ids, lse, g, gk, dlogits_dtype=torch.float32, temperature=temperature,
                          entropy=ent if entropy else None, grad_entropy=gh)
    check_gradient(d, x, t, ids, lse, g, gk, ent, gh, temperature)
    # elsewhere the bits are logp_bwd's for the summed gradient; in the logits' type they are these, rounded
    own = bil.logp_topk_bwd(x, t, ids, lse, g, gk, temperature=temperature, entropy=ent if entropy else None,
                            grad_entropy=gh)
    assert own.dtype == dtype and torch.equal(own, d.to(dtype))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_backward_of_any_columns(dtype):
    """Columns of the caller's choice: named twice, the target named, out of range (they count in G alone)."""
    n, vocab, k = 6, 2000, 9
    x, t = rows(n, vocab, dtype, 31), targets(n, vocab, 31)
    lse = bil.logp_fwd(x, t)[1]
    ids = torch.randint(0, vocab, (n, k), generator=gen(4), device="cuda")
    ids[0, 3] = ids[0, 5]
    ids[1, 2] = t[1]
    ids[2, :] = t[2]
    ids[3, 1], ids[3, 4] = -1, vocab
    g, gk = torch.randn(n, generator=gen(5), device="cuda"), torch.randn(n, k, generator=gen(6), device="cuda")
    d = bil.logp_topk_bwd(x, t, ids, lse, g, gk, dlogits_dtype=torch.float32)
    check_gradient(d, x, t, ids, lse, g, gk, None, None, 1.0)


def test_backward_leaves_other_columns_and_special_rows():
    n, vocab, k = 5, 1500, 4
    x, t = rows(n, vocab + 20, torch.float32, 32), targets(n, vocab, 32)
    t[1], t[2] = IGNORE, vocab + 3
    logp, lse, ids, top = bil.logp_topk(x, t, k, vocab=vocab)
    g, gk = torch.randn(n, generator=gen(7), device="cuda"), torch.randn(n, k, generator=gen(8), device="cuda")
    d = bil.logp_topk_bwd(x, t, ids, lse, g, gk, vocab=vocab)
    assert bool((d[:, vocab:] == 0).all()) and bool((d[1] == 0).all()) and bool(d[2, :vocab].isnan().all())
    G = g.clone()
    for j in range(k):  # 4 terms: lanes 0 to 3, butterfly (g0 + g2) + (g1 + g3)
        pass
    G = g + ((gk[:, 0] + gk[:, 2]) + (gk[:, 1] + gk[:, 3]))
    full = bil.logp_bwd(x, t, lse, G, vocab=vocab)
    named = torch.zeros_like(d, dtype=torch.bool)
    for r in (0, 3, 4):
        named[r, ids[r]] = True
        named[r, t[r]] = True
        assert torch.equal(d[r][~named[r]], full[r][~named[r]])


def test_gradient_against_differences():
    """Central differences of logp + sum w top_logp + H in 64 bits from the float32 forward.  Its outputs
    are off by about 1e-6 each; over 2 eps = 0.1 and k + 2 = 7 of them 7e-5; the truncation eps^2 / 6 times a
    third derivative of order 1 is 4e-4.  2e-3 is four times both."""
    n, vocab, k, eps = 4, 60, 5, 0.05
    x = rows(n, vocab, torch.float32, 33, scale=1.0)
    x = x + torch.arange(vocab, device="cuda") * 0.25  # the order of the columns holds under the steps
    t = targets(n, vocab, 33)
    w = torch.randn(n, k, generator=gen(9), device="cuda")
    logp, lse, ent, ids, top = bil.logp_topk(x, t, k, return_entropy=True)
    one = torch.ones(n, device="cuda")
    d = bil.logp_topk_bwd(x, t, ids, lse, one, w, entropy=ent, grad_entropy=one)

    def loss(x):
        lp, ls, h = bil.logp_fwd(x, t, return_entropy=True)
        z = x.double().gather(1, ids) - ls.double()[:, None]
        return (lp.double() + h.double() + (w.double() * z).sum(dim=1)).cpu().numpy()

    for _ in range(5):
        step = torch.randn(n, vocab, generator=gen(40 + _), device="cuda")
        step = step / step.norm(dim=1, keepdim=True)
        num = (loss(x + eps * step) - loss(x - eps * step)) / (2 * eps)
        ana = (d.double() * step.double()).sum(dim=1).cpu().numpy()
        assert np.all(np.abs(num - ana) <= 2e-3 * (1 + np.abs(w.cpu().numpy()).sum(axis=1)))


def test_autograd():
    n, vocab, k = 6, 500, 3
    x0, t = rows(n, vocab, torch.float32, 34), targets(n, vocab, 34)
    x = x0.clone().reshape(2, 3, vocab).requires_grad_()
    logp, ent, ids, top = bil.batch_invariant_logp_topk(x, t.reshape(2, 3), k, temperature=0.8)
    assert not ids.requires_grad and top.shape == (2, 3, k)
    (logp.sum() + 0.5 * ent.sum() + top.sum()).backward()
    y = x0.clone().double().requires_grad_()
    ls = torch.log_softmax(y / 0.8, dim=1)
    (ls.gather(1, t[:, None]).sum() - 0.5 * (ls.exp() * ls).sum() + ls.gather(1, ids.reshape(n, k)).sum()).backward()
    assert float((x.grad.reshape(n, vocab).double() - y.grad).abs().max()) <= 2e-5
    x = x0.clone().requires_grad_()
    bil.batch_invariant_logp_topk(x, t, k)[3][:, 1].sum().backward()  # one output, an expanded gradient
    y = x0.clone().double().requires_grad_()
    torch.log_softmax(y, dim=1).gather(1, ids.reshape(n, k))[:, 1].sum().backward()
    assert float((x.grad.double() - y.grad).abs().max()) <= 2e-5


def test_empty_and_refusals():
    x, t = rows(4, 100, torch.bfloat16, 35), targets(4, 100, 35)
    logp, lse, ids, top = bil.logp_topk(x[:0], t[:0], 5)
    assert logp.shape == (0,) and ids.shape == (0, 5) and top.shape == (0, 5)
    d = bil.logp_topk_bwd(x[:0], t[:0], ids, lse, logp, top)
    assert d.shape == (0, 100)
    for k in (0, -1, 101, 129):
        with pytest.raises(ValueError):
            bil.logp_topk(x, t, k)
    with pytest.raises(ValueError, match="no CPU path"):
        bil.logp_topk(x.cpu(), t.cpu(), 5)
    with pytest.raises(TypeError):
        bil.logp_topk(x.double(), t, 5)
    with pytest.raises(ValueError):
        bil.logp_topk(x, t[:3], 5)
    with pytest.raises(ValueError):
        bil.logp_topk(x, t, 5, vocab=101)
    with pytest.raises(ValueError):
        bil.logp_topk(x, t, 5, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    for kw in (dict(tile_v=12), dict(tile_v=0), dict(temperature=0.0), dict(temperature=NAN)):
        with pytest.raises(bil.BilError):
            bil.logp_topk(x, t, 5, **kw)
    bad = t.clone()
    bad[2] = 100
    with pytest.raises(bil.BilError) as e:
        bil.logp_topk(x, bad, 5, validate=True)
    assert e.value.status == _lib.E_TARGET_RANGE
    logp, lse, ids, top = bil.logp_topk(x, t, 5)
    with pytest.raises(TypeError):
        bil.logp_topk_bwd(x, t, ids.to(torch.int32), lse, logp, top)
    with pytest.raises(ValueError):
        bil.logp_topk_bwd(x, t, ids, lse, logp, top[:, :4])
    with pytest.raises(ValueError):
        bil.logp_topk_bwd(x, t, ids, lse[:3], logp, top)
    with pytest.raises(ValueError):
        bil.logp_topk_bwd(x, t, ids, lse, logp, top, entropy=lse)


@pytest.mark.parametrize("dtype", TYPES[1:], ids=IDS[1:])
@pytest.mark.parametrize("tile_v", [512, 4096])
@pytest.mark.parametrize("vocab,pad", [(33000, 0), (40007, 0), (40008, 5)])
@pytest.mark.parametrize("k", [1, 20, 128])
def test_few_rows_and_many_give_the_same_bits(vocab, pad, tile_v, k, dtype):
    """Rows that need every way of the choice, few (a cluster a row) and among many (two kernels)."""
    n = 9
    x = rows(n, vocab, dtype, 41, pad=pad)
    noise = torch.randn(vocab, generator=gen(42), device="cuda")
    x[1] = 2.0                                            # all equal
    x[2] = (2 * noise).round().to(dtype)                  # crowded
    x[3] = -INF
    x[3, vocab - 1] = 1.0                                 # one column left
    x[4] = NAN                                            # none at all
    x[5, 7::3] = NAN
    x[6] = torch.finfo(dtype).min
    x[7] = -INF                                           # nothing left
    x[8, 100] = INF
    t = targets(n, vocab, 41)
    t[0] = IGNORE
    check(x, t, k, tile_v=tile_v)
    few = bil.logp_topk(x, t, k, tile_v=tile_v, return_entropy=True)
    many = bil.logp_topk(x.repeat(20, 1), t.repeat(20), k, tile_v=tile_v, return_entropy=True)
    for a, b in zip(few, many):
        b = b.reshape(20, *a.shape)
        for c in (b[0], b[11], b[19]):
            assert torch.equal(a.nan_to_num(nan=7.0) if a.is_floating_point() else a,
                               c.nan_to_num(nan=7.0) if c.is_floating_point() else c)


def test_workspace_of_few_rows():
    assert topk_mod.workspace_bytes(torch.bfloat16, 40, 151936, 20) == 0
    assert topk_mod.workspace_bytes(torch.bfloat16, 1000, 151936, 20) > 0
    assert topk_mod.workspace_bytes(torch.float32, 40, 151936, 20) > 0   # a 16-bit type's alone
    assert topk_mod.workspace_bytes(torch.bfloat16, 40, 7 * 4096, 20) > 0  # eight tiles or more
    assert topk_mod.workspace_bytes(torch.bfloat16, 1, 300 * 4096, 20) > 0  # and 256 at most
