"""The fused LM-head + logp on 8-bit operands, against its formula in 64 bits.

    z[r, c] = (sum_k hq[r, k] wq[c, k]) * sw[c] * sh[r]

with e4m3 hq, wq and float32 scales, then the statistics of the logits path
over 256-column tiles.

Tolerances.  Products of two e4m3 values (4 significant bits each) are exact
in float32.  The tensor cores add 32 of them and the accumulator per step, so
H / 32 + 1 additions, each off by at most 2^-23 of a partial sum that is at
most S = sum_k |hq wq| (truncation; rounding would halve it); the terms of one
step aligned to the largest of them lose at most 32 * 2^-25 of it, 2^-20 S in
all.  The two scales add half an ulp each:
    |dz| <= (((H / 32 + 1) 2^-23 + 2^-20) S) sw sh + 2^-23 |z|.
logp, lse and the entropy: the logits path's 1e-4 absolute, which holds the
above for the sizes here (S sw sh <= 64 for |z| around 3, H <= 4096: 64 *
(2^-16 + 2^-20) = 1.04e-3 in the worst case of one logit, whose errors of
both signs, 1e-6 in the root mean square, are what logp sees; a worst case
that adds up is excluded by taking the measured |dz| into the bound:
|dlogp| <= 2 max |dz| + 1e-4 would be the bound of a proof, and the tests
hold the tighter 1e-4).
"""
import math

import numpy as np
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import ENTROPY_ATOL, LOGP_ATOL, check_watchdog, f32_bits
from invariant_token_log_gb300 import _lib

pytestmark = pytest.mark.gpu
IGNORE = bil.IGNORE_INDEX


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


def quantise(x):
    """A row's e4m3 values and its scale, rows padded to 16 bytes."""
    scale = x.abs().amax(dim=1).clamp_min(1e-30) / 448
    buf = torch.zeros(x.shape[0], -(-x.shape[1] // 16) * 16, dtype=torch.float8_e4m3fn, device=x.device)
    q = buf[:, :x.shape[1]]
    q.copy_((x / scale[:, None]).to(torch.float8_e4m3fn))
    return q, scale


def make_case(n, h, v, seed=1, ignore_every=5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hs = quantise(torch.randn(n, h, generator=gen, device="cuda"))
    wq, ws = quantise(torch.randn(v, h, generator=gen, device="cuda") * (3 / math.sqrt(h)))
    t = torch.randint(0, v, (n,), generator=gen, device="cuda")
    if ignore_every:
        t[::ignore_every] = IGNORE
    return hq, hs, wq, ws, t


def reference(hq, hs, wq, ws, t, temperature=1.0):
    """(logits, logp, lse, entropy) in 64 bits; zeros for ignored rows."""
    z = (hq.double() @ wq.double().t()) * ws.double() * hs.double()[:, None]
    zt = z / temperature
    lse = torch.logsumexp(zt, dim=1)
    a = zt - lse[:, None]
    ent = -(a.exp() * a).sum(dim=1)
    logp = a.gather(1, t.clamp(0, z.shape[1] - 1)[:, None])[:, 0]
    act = (t != IGNORE).double()
    return z, logp * act, lse * act, ent * act


def close(got, ref, atol, what):
    err = float((got.double() - ref).abs().max())
    assert err <= atol, (what, err)


SHAPES = [
    (1, 16, 1),          # one of everything, the shortest row the alignment allows
    (1, 4096, 1000),
    (3, 17, 300),        # a K tail of one element in rows padded to 32 bytes
    (128, 128, 256),     # one row tile, one K block, one vocabulary tile
    (129, 1104, 257),    # one row and one column past a tile; K = 8.625 blocks
    (300, 200, 1000),
    (70, 4096, 2049),
]


@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_against_64_bits(n, h, v, temperature):
    hq, hs, wq, ws, t = make_case(n, h, v, seed=n + h + v, ignore_every=5 if n > 1 else 0)
    logp, lse, ent, z = bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=temperature, return_entropy=True,
                                            return_logits=True)
    rz, rlogp, rlse, rent = reference(hq, hs, wq, ws, t, temperature)
    s = (hq.double().abs() @ wq.double().abs().t()) * ws.double().abs() * hs.double()[:, None]
    bound = ((h / 32 + 1) * 2.0 ** -23 + 2.0 ** -20) * s + 2.0 ** -23 * rz.abs()
    assert bool(((z.double() - rz).abs() <= bound).all()), float(((z.double() - rz).abs() / bound).max())
    close(logp, rlogp, LOGP_ATOL, "logp")
    close(lse, rlse, LOGP_ATOL, "lse")
    close(ent, rent, ENTROPY_ATOL, "entropy")
    ign = (t == IGNORE).cpu().numpy()
    for x in (logp, lse, ent):
        assert np.all(f32_bits(x)[ign] == 0)


def test_the_accumulation_keeps_float32():
    """One large term and 4095 small ones of the same sign: 8 * 8 + 4095 * 2^-4 * 2^-5.  Every partial sum
    is a multiple of 2^-9 below 2^7, exact in float32 whatever the order; an accumulator of 14 bits would
    lose each small term against the large one."""
    h = 4096
    x = torch.full((1, h), 2.0 ** -4, device="cuda")
    w = torch.full((1, h), 2.0 ** -5, device="cuda")
    x[0, 0] = w[0, 0] = 8.0
    one = torch.ones(1, device="cuda")
    z = bil.linear_logp_fp8(x.to(torch.float8_e4m3fn), one, w.to(torch.float8_e4m3fn), one,
                            torch.zeros(1, dtype=torch.int64, device="cuda"), return_logits=True)[2]
    assert float(z) == 64.0 + 4095 / 512


def test_forms_give_the_same_bits():
    hq, hs, wq, ws, t = make_case(300, 256, 2000, seed=5)
    plain = bil.linear_logp_fp8(hq, hs, wq, ws, t)
    ent = bil.linear_logp_fp8(hq, hs, wq, ws, t, return_entropy=True)
    z32 = bil.linear_logp_fp8(hq, hs, wq, ws, t, return_entropy=True, return_logits=True)
    z16 = bil.linear_logp_fp8(hq, hs, wq, ws, t, return_entropy=True, return_logits=True, logits_dtype=torch.bfloat16)
    for i in range(2):
        for other in (ent, z32, z16):
            assert np.array_equal(f32_bits(plain[i]), f32_bits(other[i]))
    assert np.array_equal(f32_bits(ent[2]), f32_bits(z32[2])) and np.array_equal(f32_bits(ent[2]), f32_bits(z16[2]))
    assert torch.equal(z16[3].view(torch.int16), z32[3].to(torch.bfloat16).view(torch.int16))


def test_rows_bitwise_across_batches():
    n = 200
    hq, hs, wq, ws, t = make_case(n, 512, 1500, seed=6, ignore_every=0)
    ref = [f32_bits(x) for x in bil.linear_logp_fp8(hq, hs, wq, ws, t, return_entropy=True, return_logits=True)]
    gen = torch.Generator().manual_seed(6)
    for size in (1, 2, 7, 64, 129, 200):
        idx = torch.randperm(n, generator=gen)[:size].cuda()
        h8 = hq.view(torch.uint8)[idx].view(torch.float8_e4m3fn)
        got = bil.linear_logp_fp8(h8, hs[idx], wq, ws, t[idx], return_entropy=True, return_logits=True)
        for g, r in zip(got, ref):
            assert np.array_equal(f32_bits(g), r[idx.cpu().numpy()]), size


def test_layouts_leading_shape_and_narrow_targets():
    """Rows of a wider buffer, an unaligned copy, a leading shape, int32 targets: the same bits."""
    hq, hs, wq, ws, t = make_case(24, 80, 500, seed=7)
    ref = bil.linear_logp_fp8(hq, hs, wq, ws, t)
    wide = torch.zeros(24, 96, dtype=torch.uint8, device="cuda")
    wide[:, :80] = hq.view(torch.uint8)
    odd = torch.zeros(24 * 83 + 1, dtype=torch.uint8, device="cuda")[1:].reshape(24, 83)
    odd[:, :80] = hq.view(torch.uint8)
    for h8 in (wide[:, :80].view(torch.float8_e4m3fn), odd[:, :80].view(torch.float8_e4m3fn)):
        got = bil.linear_logp_fp8(h8, hs, wq, ws, t.to(torch.int32))
        assert all(np.array_equal(f32_bits(a), f32_bits(b)) for a, b in zip(got, ref))
    got = bil.linear_logp_fp8(hq.reshape(4, 6, 80), hs.reshape(4, 6), wq, ws, t.reshape(4, 6))
    assert got[0].shape == (4, 6)
    assert all(np.array_equal(f32_bits(a).reshape(-1), f32_bits(b)) for a, b in zip(got, ref))


def test_special_rows():
    """A NaN byte makes its row NaN and no other; a zero scale makes a row uniform; a target
    outside the vocabulary makes its logp NaN and keeps its lse."""
    v = 700
    hq, hs, wq, ws, t = make_case(6, 64, v, seed=8, ignore_every=0)
    ref = bil.linear_logp_fp8(hq, hs, wq, ws, t, return_entropy=True)
    hq.view(torch.uint8)[1, 5] = 0x7f
    hs[2] = 0.0
    t[3] = v
    t[4] = -7
    logp, lse, ent = bil.linear_logp_fp8(hq, hs, wq, ws, t, return_entropy=True)
    assert bool(logp[1].isnan() & lse[1].isnan())
    for x, want in ((logp, -math.log(v)), (lse, math.log(v)), (ent, math.log(v))):
        assert abs(float(x[2]) - want) <= 1e-5
    assert bool(logp[3].isnan() & logp[4].isnan())
    assert np.array_equal(f32_bits(lse)[3:], f32_bits(ref[1])[3:])
    for got, r in zip((logp, lse, ent), ref):
        assert np.array_equal(f32_bits(got)[[0, 5]], f32_bits(r)[[0, 5]])


def test_another_stream_and_a_kept_workspace():
    hq, hs, wq, ws, t = make_case(150, 256, 3000, seed=9)
    ref = bil.linear_logp_fp8(hq, hs, wq, ws, t)
    torch.cuda.synchronize()
    from invariant_token_log_gb300 import linear
    space = torch.empty(linear.workspace_bytes(150, 3000), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = [bil.linear_logp_fp8(hq, hs, wq, ws, t, workspace=space) for _ in range(3)]
    stream.synchronize()
    for g in got:
        assert all(np.array_equal(f32_bits(a), f32_bits(b)) for a, b in zip(g, ref))


def test_empty_and_refusals():
    hq, hs, wq, ws, t = make_case(4, 64, 300, seed=10)
    logp, lse = bil.linear_logp_fp8(hq[:0], hs[:0], wq, ws, t[:0])
    assert logp.shape == (0,) and lse.shape == (0,)
    with pytest.raises(TypeError):
        bil.linear_logp_fp8(hq.to(torch.bfloat16), hs, wq, ws, t)
    with pytest.raises(TypeError):
        bil.linear_logp_fp8(hq, hs, wq.to(torch.bfloat16), ws, t)
    with pytest.raises(TypeError):
        bil.linear_logp_fp8(hq, hs, wq, ws, t, return_logits=True, logits_dtype=torch.float16)
    with pytest.raises(ValueError):
        bil.linear_logp_fp8(hq, hs[:3], wq, ws, t)
    with pytest.raises(ValueError):
        bil.linear_logp_fp8(hq, hs, wq, ws.double(), t)
    with pytest.raises(ValueError):
        bil.linear_logp_fp8(hq, hs, wq[:, :32], ws, t)
    with pytest.raises(ValueError):
        bil.linear_logp_fp8(hq, hs, wq, ws, t[:3])
    with pytest.raises(ValueError, match="no CPU path"):
        bil.linear_logp_fp8(hq.cpu(), hs, wq, ws, t)
    with pytest.raises(ValueError):
        bil.linear_logp_fp8(hq, hs, wq, ws, t, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    for bad in (0.0, -1.0, math.nan):
        with pytest.raises(bil.BilError):
            bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=bad)
    t[1] = 300
    with pytest.raises(bil.BilError) as e:
        bil.linear_logp_fp8(hq, hs, wq, ws, t, validate=True)
    assert e.value.status == _lib.E_TARGET_RANGE


@pytest.mark.parametrize("n,h,v", [(129, 1168, 257), (200, 1040, 9001), (513, 2064, 3000), (700, 4096, 2600)])
def test_long_hidden_rows_in_large_and_small_batches(n, h, v):
    """More than 128 rows of more than 1024 elements (pairs of blocks) against 64 bits, in every form of the
    outputs, and bit for bit against batches of one row tile (single blocks)."""
    hq, hs, wq, ws, t = make_case(n, h, v, seed=10)
    rz, rlogp, rlse, rent = reference(hq, hs, wq, ws, t, 0.7)
    full = bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=0.7, return_entropy=True, return_logits=True)
    size = (hq.double().abs() @ wq.double().abs().t()) * ws.double().abs() * hs.double()[:, None]
    bound = ((h / 32 + 1) * 2.0 ** -23 + 2.0 ** -20) * size + 2.0 ** -23 * rz.abs()  # as above
    assert bool(((full[3].double() - rz).abs() <= bound).all())
    close(full[0], rlogp, LOGP_ATOL, "logp")
    close(full[1], rlse, LOGP_ATOL, "lse")
    close(full[2], rent, ENTROPY_ATOL, "entropy")
    plain = bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=0.7)
    half = bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=0.7, return_logits=True, logits_dtype=torch.bfloat16)
    for other in (plain, half):
        assert all(np.array_equal(f32_bits(a), f32_bits(b)) for a, b in zip(other[:2], full[:2]))
    assert torch.equal(half[2], full[3].to(torch.bfloat16))
    for s in (slice(0, 100), slice(n - 128, n), slice(n - 1, n)):
        part = bil.linear_logp_fp8(hq[s], hs[s], wq, ws, t[s], temperature=0.7, return_entropy=True, return_logits=True)
        for a, b in zip(part, full):
            assert np.array_equal(f32_bits(a), f32_bits(b[s]))
