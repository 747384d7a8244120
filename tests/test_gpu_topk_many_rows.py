"""The alternatives where one warp takes a row (from four rows an SM on), on the
rows that need every way of the choice, and a workspace of the caller's on another
stream.  The reference of a row is the same row in a small batch, which test_gpu_topk's
check compares with logp_fwd and a sort."""
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import check_watchdog
from invariant_token_log_gb300 import topk as topk_mod
from test_gpu_topk import IDS, IGNORE, INF, NAN, TYPES, check, gen, rows, targets

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


def same(a, b):
    return torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0)) if a.is_floating_point() else torch.equal(a, b)


def special_rows(vocab, dtype, pad):
    x = rows(17, vocab, dtype, 51, pad=pad)
    c = torch.arange(vocab, device="cuda")
    noise = torch.randn(vocab, generator=gen(52), device="cuda")
    ramp = c.float() / 64 - 70
    low = torch.finfo(dtype).min
    x[1] = 2.0                                                    # all equal
    x[2] = (2 * noise).round().to(dtype)                          # crowded
    x[3] = -INF
    x[3, vocab - 1] = 1.0                                         # one column left
    x[4] = -INF                                                   # none
    x[5] = NAN
    x[6, 7::3] = NAN
    x[7] = low                                                    # the type's lowest value everywhere
    x[8] = torch.where(c % 997 == 3, x[8].float(), float(low)).to(dtype)
    x[9] = ramp.to(dtype)                                         # every column enters any list
    x[10] = -ramp.to(dtype)
    x[11] = torch.where(c // 8 % 32 < 5, 60 + (4 * noise).floor(), noise).to(dtype)  # large ones in a few lanes
    x[12] = torch.where(c < 2000, 50 + 9 * noise, noise).to(dtype)                   # and at the row's start
    x[13, 100] = INF
    x[14] = torch.where(c % 2 == 0, -0.0, 0.0).to(dtype)          # zeros of both signs
    x[15] = -INF
    x[15, 5:5 + 30] = 1.5                                         # 30 equal columns, then -inf
    x[16, ::2] = -INF
    return x


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("vocab,pad", [(3001, 0), (9000, 0), (20011, 5)])
@pytest.mark.parametrize("k", [1, 20, 33, 128])
def test_a_warp_a_row(vocab, pad, k, dtype):
    bank = special_rows(vocab, dtype, pad)
    t = targets(len(bank), vocab, 53)
    t[0] = IGNORE
    few = check(bank, t, k)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    times = 4 * sms // len(bank) + 1
    assert times * len(bank) >= 4 * sms > len(bank)
    many = torch.empty(times * len(bank), vocab + pad, dtype=dtype, device="cuda")[:, :vocab]
    many.copy_(bank.repeat(times, 1))
    got = bil.logp_topk(many, t.repeat(times), k, return_entropy=True)
    plain = bil.logp_topk(many, t.repeat(times), k)
    for want, a in zip(few, got):
        a = a.reshape(times, *want.shape)
        assert all(same(a[i], want) for i in range(times))
    for a, b in zip(plain, (got[0], got[1], got[3], got[4])):
        assert same(a, b)


@pytest.mark.parametrize("n,vocab,dtype", [(64, 151936, torch.bfloat16), (40, 32003, torch.float32),
                                           (900, 8200, torch.float16)])
def test_a_kept_workspace_on_another_stream(n, vocab, dtype):
    """Batch after batch in one workspace, which each call finds as the one before left it."""
    need = topk_mod.workspace_bytes(dtype, n, vocab, 20, entropy=True)
    assert need > 0
    batches = [(rows(n, vocab, dtype, seed, scale=3.0 + seed), targets(n, vocab, seed, ignore_every=5)) for seed in range(3)]
    want = [bil.logp_topk(x, t, 20, return_entropy=True) for x, t in batches]
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [bil.logp_topk(x, t, 20, return_entropy=True, workspace=space) for x, t in batches + batches[::-1]]
    s.synchronize()
    for g, w in zip(got, want + want[::-1]):
        assert all(same(a, b) for a, b in zip(g, w))
    for short in (need - 1, 0):
        with pytest.raises(ValueError, match="workspace"):
            bil.logp_topk(*batches[0], 20, return_entropy=True, workspace=space[:short])
