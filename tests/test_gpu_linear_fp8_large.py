"""The 8-bit LM head on logits of some hundreds.

Small integers as e4m3 values make every accumulator an exact integer, so that
what is left are the epilogue's roundings.  u = 2^-24, M = a row's largest |z|:
a logit takes three (two scales, the temperature), 3 u M; in the sums each
column's difference from the tile's maximum has the rounding of either operand
and of itself, at most 3 u M and weighted by the softmax; the merge's differences
of the tiles' maxima (3 u M each side, their own 1) cancel all but 1 u M against
the maxima's own error; adding the logarithm and subtracting round once each, at
most u (M + log V).  Together 12 u M; the exponentials (2 ulps, relative) and the
logarithm stay within 2e-6:
    |d lse|, |d logp| <= 12 u M + 2e-6
The entropy is a difference of such sums, -sum p (z - lse): 1e-4 of the logits
path for its own arithmetic, and 12 u M times the size of the softmax's weights' move:
    |dH| <= 1e-4 + 12 u M * sum p |z - lse + H|.
"""
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import ENTROPY_ATOL, check_watchdog
from test_gpu_linear_fp8 import reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


def integers(n, h, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-12, 13, (n, h), generator=g, device="cuda").float().to(torch.float8_e4m3fn)


def scales(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 0.5 + torch.rand(n, generator=g, device="cuda")


# K past and below where pairs of blocks begin; the standard deviation is that of the products' sum, 49 sqrt(H), times
# the scales' size
@pytest.mark.parametrize("n,h,v,std", [(70, 128, 3001, 50.0), (300, 2048, 2000, 50.0), (300, 256, 2000, 200.0),
                                       (1, 128, 1, 300.0)])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_large_logits_against_64_bits(n, h, v, std, temperature):
    hq, wq = integers(n, h, n + h), integers(v, h, v)
    hs, ws = scales(n, 1) * (std / (52 * h ** 0.5)), scales(v, 2)
    t = torch.randint(0, v, (n,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    logp, lse, ent = bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=temperature, return_entropy=True)
    z, rlogp, rlse, rent = reference(hq, hs, wq, ws, t, temperature)
    m = z.abs().amax(dim=1) / temperature
    bound = 12 * U * m + 2e-6
    assert bool(((lse.double() - rlse).abs() <= bound).all())
    assert bool(((logp.double() - rlogp).abs() <= bound).all())
    a = z / temperature - rlse[:, None]
    spread = (a.exp() * (a + rent[:, None]).abs()).sum(dim=1)
    assert bool(((ent.double() - rent).abs() <= ENTROPY_ATOL + 12 * U * m * spread).all())


@pytest.mark.parametrize("h,n", [(256, 3), (256, 200), (2048, 200)])  # one block a tile, and pairs
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_a_column_far_above_the_others_has_all_of_the_probability(n, h, temperature):
    """One column at some hundreds, the others over 150 below it: e^-150 is nothing to 1, so lse is that column's
    logit bit for bit, logp and the entropy are zero."""
    v, col = 700, 300
    hq = torch.ones(n, h, device="cuda").to(torch.float8_e4m3fn)
    wq = torch.zeros(v, h, device="cuda").to(torch.float8_e4m3fn)
    wq[col] = 1.0
    hs = (200 + 300 * torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")) / h
    ws = torch.full((v,), 1.01, device="cuda")
    t = torch.full((n,), col, device="cuda")
    logp, lse, ent, z = bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=temperature, return_entropy=True,
                                            return_logits=True)
    want = z[:, col] * (1.0 if temperature == 1.0 else torch.tensor(1.0 / temperature, dtype=torch.float64).float().cuda())
    assert torch.equal(lse, want) and bool((logp == 0).all()) and bool((ent == 0).all())
