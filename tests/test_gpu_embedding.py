"""The embedding's lookup, bit for bit, and its gradient against the sums in 64 bits.

A row of the gradient is a float32 sum of k rows in some fixed order, at most k - 1
roundings deep, times the scale, rounded to the type: with u = 2^-24
    |error| <= scale (k + 2) u sum |dy| + u_T |ref|  (+ 2^-25 for float16's small values)
Accumulating into an output adds one rounding of it: u (|old| + |ref|) more.
"""
import pytest
import torch

import invariant_token_log_gb300 as bil

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}
TYPES = list(U)
IDS = ["f32", "bf16", "f16"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(n, width, dtype, seed, scale=1.0, pad=0, shift=0):
    buf = torch.full((n * (width + pad) + shift + 8,), float("nan"), dtype=dtype, device="cuda")
    view = buf[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    view.copy_(scale * torch.randn(n, width, generator=gen(seed), device="cuda"))
    return view


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def skewed(n, vocab, seed):
    u = torch.rand(n, generator=gen(seed), device="cuda", dtype=torch.float64)
    return ((vocab + 1.0) ** u).long().sub_(1).clamp_(0, vocab - 1)


def check_gradient(got, dy, ids, vocab, scale, padding=None, old=None):
    kept = (ids >= 0) & (ids < vocab)
    if padding is not None:
        kept &= ids != padding
    t, d = ids[kept], dy[kept].double()
    width = dy.shape[1]
    count = torch.bincount(t, minlength=vocab).double()[:, None]
    ref = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, t, d) * scale
    size = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, t, d.abs()) * abs(scale)
    bound = (count + 2) * 2.0 ** -24 * size
    if old is not None:
        ref = ref + old.double()
        bound = bound + 2.0 ** -24 * (size + old.double().abs()) * (count > 0)
    bound = bound + (U[got.dtype] * ref.abs() + TINY[got.dtype]) * (count > 0)
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp_min(1e-300)).max())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n,vocab,width,pad,shift", [(1, 1, 1, 0, 0), (3, 10, 7, 0, 0), (64, 1000, 64, 0, 0), (65, 5000, 1105, 7, 3),
                                                     (300, 2000, 4096, 0, 0), (17, 300, 5000, 64, 0)])
@pytest.mark.parametrize("scale", [1.0, 0.3])
def test_lookup(dtype, n, vocab, width, pad, shift, scale):
    w = rows(vocab, width, dtype, 1, pad=pad, shift=shift)
    ids = torch.randint(0, vocab, (n,), generator=gen(2), device="cuda")
    y = bil.embedding_fwd(ids, w, scale)
    assert torch.equal(bits(y), bits((w[ids].float() * scale).to(dtype)))


def test_lookup_shapes_types_and_bad_tokens():
    w = rows(50, 40, torch.bfloat16, 1)
    ids = torch.randint(0, 50, (4, 3), generator=gen(2), device="cuda")
    y = bil.embedding_fwd(ids, w)
    assert y.shape == (4, 3, 40) and torch.equal(y, w[ids])
    for t in (torch.int32, torch.int16, torch.uint8):
        assert torch.equal(bil.embedding_fwd(ids.to(t), w), y)
    assert torch.equal(bil.embedding_fwd(ids.t(), w), w[ids.t()])
    assert torch.equal(bil.embedding_fwd(ids, w.t().contiguous().t()), y)
    assert torch.equal(bil.embedding_fwd(ids[0, 0], w), w[ids[0, 0]])
    assert bil.embedding_fwd(ids[:0], w).shape == (0, 3, 40)
    bad = torch.tensor([0, -1, 50, 2 ** 40, -2 ** 62, 49], device="cuda")
    y = bil.embedding_fwd(bad, w)
    assert bool(y[1:5].isnan().all()) and torch.equal(y[[0, 5]], w[[0, 49]])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n,vocab,width,pad,shift", [(1, 1, 1, 0, 0), (31, 3, 9, 0, 0), (33, 511, 64, 0, 0), (64, 512, 100, 0, 0),
                                                     (1000, 700, 1104, 0, 0), (4096, 20000, 264, 0, 0), (5003, 32003, 1105, 7, 3),
                                                     (4097, 300, 4097, 0, 0), (70000, 5000, 72, 0, 0), (20000, 700000, 72, 0, 0)])
def test_gradient(dtype, n, vocab, width, pad, shift):
    ids = skewed(n, vocab, 3)
    dy = rows(n, width, dtype, 4, pad=pad, shift=shift)
    check_gradient(bil.embedding_bwd(dy, ids, vocab, 0.5), dy, ids, vocab, 0.5)
    if dtype != torch.float32:
        check_gradient(bil.embedding_bwd(dy, ids, vocab, out_dtype=torch.float32), dy, ids, vocab, 1.0)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 65, 1023, 1024, 1025, 4097, 8193, 16384, 16385, 65536, 65537, 70001])
@pytest.mark.parametrize("pattern", ["one", "two", "each", "blocks"])
def test_runs_of_tokens(n, pattern):
    """Tokens whose places end inside, at and behind the segments; one token for all places."""
    i = torch.arange(n, device="cuda")
    vocab = max(n, 8)
    ids = {"one": torch.full_like(i, 5), "two": i % 2 * (vocab - 1), "each": i.flip(0), "blocks": i // 48}[pattern]
    dy = rows(n, 40, torch.float32, 5)
    check_gradient(bil.embedding_bwd(dy, ids, vocab), dy, ids, vocab, 1.0)


@pytest.mark.parametrize("vocab", [1, 2, 511, 512, 513, 2 ** 18 - 1, 2 ** 18, 2 ** 18 + 1, 3000000])
def test_vocabularies(vocab):
    """One, two and three digits of the sort; the last row and tokens behind it."""
    n = 3000
    ids = torch.randint(0, vocab, (n,), generator=gen(6), device="cuda")
    ids[::7], ids[1::11], ids[2::13] = vocab - 1, vocab, -1
    dy = rows(n, 8, torch.float32, 7)
    check_gradient(bil.embedding_bwd(dy, ids, vocab), dy, ids, vocab, 1.0)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_padding_and_accumulation(dtype):
    n, vocab, width = 2000, 90, 136
    ids = skewed(n, vocab, 8)
    dy = rows(n, width, dtype, 9)
    got = bil.embedding_bwd(dy, ids, vocab, 2.0, padding_idx=0)
    check_gradient(got, dy, ids, vocab, 2.0, padding=0)
    assert not got[0].any()
    for out_dtype in {dtype, torch.float32}:
        buf = rows(vocab, width, out_dtype, 10, pad=8)
        old = buf.clone()
        out = bil.embedding_bwd(dy[:50], ids[:50], vocab, out=buf, accumulate=True)
        assert out is buf
        check_gradient(buf, dy[:50], ids[:50], vocab, 1.0, old=old)
        untouched = torch.ones(vocab, dtype=torch.bool, device="cuda")
        untouched[ids[:50]] = False
        assert bool(untouched.any()) and torch.equal(bits(buf[untouched]), bits(old[untouched]))
    none = torch.full((40,), 3, device="cuda")
    assert not bil.embedding_bwd(dy[:40], none, vocab, padding_idx=3).any()


def test_the_gap_between_rows_is_left_alone():
    ids = skewed(500, 64, 11)
    dy = rows(500, 30, torch.float32, 12)
    whole = torch.full((64, 37), 7.0, device="cuda")
    bil.embedding_bwd(dy, ids, 64, out=whole[:, :30])
    check_gradient(whole[:, :30], dy, ids, 64, 1.0)
    assert bool((whole[:, 30:] == 7).all())


def test_the_same_bits_every_time_and_for_any_layout():
    ids = skewed(9000, 400, 13)
    dy = rows(9000, 264, torch.bfloat16, 14)
    first = bil.embedding_bwd(dy, ids, 400, out_dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(bil.embedding_bwd(dy, ids, 400, out_dtype=torch.float32), first)
    wide = torch.empty(9000, 271, dtype=torch.bfloat16, device="cuda")[:, 3:267]
    wide.copy_(dy)
    assert torch.equal(bil.embedding_bwd(wide, ids, 400, out_dtype=torch.float32), first)
    part = bil.embedding_bwd(dy[:, :100], ids, 400, out_dtype=torch.float32)  # columns do not mix
    assert torch.equal(part, first[:, :100])


def test_no_tokens():
    dy = torch.empty(0, 16, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    assert not bil.embedding_bwd(dy, ids, 9).any()
    out = torch.ones(9, 16, device="cuda")
    bil.embedding_bwd(dy, ids, 9, out=out, accumulate=True)
    assert bool((out == 1).all())


def test_autograd():
    ids = skewed(60, 30, 15).view(6, 10)
    w = rows(30, 24, torch.float32, 16).clone().requires_grad_()
    dy = rows(60, 24, torch.float32, 17).view(6, 10, 24)
    y = bil.embedding(ids, w, 3.0, padding_idx=1)
    (dw,) = torch.autograd.grad(y, w, dy, retain_graph=True)
    check_gradient(dw, dy.reshape(60, 24), ids.reshape(-1), 30, 3.0, padding=1)
    (dw,) = torch.autograd.grad(y.sum(), w)  # a broadcast gradient
    check_gradient(dw, torch.ones(60, 24, device="cuda"), ids.reshape(-1), 30, 3.0, padding=1)
