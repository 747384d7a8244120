"""The 8-bit LM head picks single blocks or pairs of blocks by the sizes and by
whether rows lie on 128-byte lines: the same bits either way."""
import numpy as np
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import check_watchdog, f32_bits
from test_gpu_linear_fp8 import make_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


@pytest.mark.parametrize("n,h,v", [(300, 1280, 1000), (700, 1664, 2600)])  # single blocks on lines, pairs off them
def test_rows_on_and_off_lines(n, h, v):
    hq, hs, wq, ws, t = make_case(n, h, v, seed=n)
    want = bil.linear_logp_fp8(hq, hs, wq, ws, t, temperature=0.7, return_entropy=True, return_logits=True)
    apart = torch.zeros(v, h + 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :h]
    apart.copy_(wq)
    got = bil.linear_logp_fp8(hq, hs, apart, ws, t, temperature=0.7, return_entropy=True, return_logits=True)
    for a, b in zip(got, want):
        assert np.array_equal(f32_bits(a), f32_bits(b))
