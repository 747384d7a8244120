"""Tile widths whose stages come close to all of an SM's shared memory, with enough
rows for every warp to have one: logp_fwd's bits, and the columns of a sort."""
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import check_watchdog
from test_gpu_topk import rows, targets

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


# widths at which 4 to 7 warps' stages take between 226 and 227 KB, and a neighbour on either side
@pytest.mark.parametrize("dtype,tile_v", [
    (torch.bfloat16, 16496), (torch.bfloat16, 16560), (torch.bfloat16, 16584), (torch.float16, 19304),
    (torch.bfloat16, 23160), (torch.bfloat16, 28960), (torch.float32, 8272), (torch.float32, 9648),
    (torch.float32, 11584), (torch.float32, 14480),
])
@pytest.mark.parametrize("pad", [0, 3])
def test_tiles_at_the_limit(dtype, tile_v, pad):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, vocab, k = 7 * sms - 1, 2 * tile_v - 24, 5  # two tiles a row: a unit for each of seven warps an SM
    x, t = rows(n, vocab, dtype, tile_v, pad=pad), targets(n, vocab, tile_v)
    logp, lse, ids, top = bil.logp_topk(x, t, k, tile_v=tile_v)
    rlogp, rlse = bil.logp_fwd(x, t, tile_v=tile_v)
    assert torch.equal(logp, rlogp) and torch.equal(lse, rlse)
    want, order = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(ids, order[:, :k]) and torch.equal(top, want[:, :k] - lse[:, None])
