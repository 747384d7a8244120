"""The norm's backward writing dx over one of its operands, as the header allows: a
warp a row, the ring of stages, and rows wider than the ring."""
import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import check_watchdog
from invariant_token_log_gb300 import _lib
from invariant_token_log_gb300 import norm as norm_mod
from invariant_token_log_gb300.logp import _code, _stream_handle
from test_gpu_norm import IDS, TYPES, gen, rows, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


@pytest.mark.parametrize("over", ["dy", "dh"])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("n,width,pad", [(333, 512, 0), (333, 301, 0), (700, 4096, 0), (700, 4097, 0), (333, 1000, 7),
                                         (170, 9664, 0), (170, 9665, 0)])
def test_dx_over_an_operand(n, width, pad, dtype, over):
    g = gen(width)
    h, dy, dh = (rows(n, width, dtype, g, pad=pad) for _ in range(3))
    w = (1 + 0.1 * torch.randn(width, generator=g, device="cuda")).to(dtype)
    rstd = bil.rms_norm_fwd(h, w)[2]
    dx, dw = bil.rms_norm_bwd(dy, h, w, rstd, dh)
    buf = {"dy": dy, "dh": dh}[over]
    dw2 = torch.empty_like(dw)
    need = norm_mod.bwd_workspace_bytes(n, width, h.device)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    ld = width + pad
    assert _lib.load().bil_rms_norm_bwd(dy.data_ptr(), h.data_ptr(), w.data_ptr(), rstd.data_ptr(), dh.data_ptr(),
                                        _code(dtype), _code(dtype), n, width, ld, ld, ld, buf.data_ptr(), ld,
                                        dw2.data_ptr(), space.data_ptr(), need, _stream_handle(0)) == _lib.OK
    assert same(buf, dx) and same(dw2, dw)
