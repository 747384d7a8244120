"""The gradient of the alternatives reads the logits of the named columns after it has written the others:
into the logits' own buffer it is refused."""
import ctypes

import pytest
import torch

import invariant_token_log_gb300 as bil
from invariant_token_log_gb300 import _lib
from invariant_token_log_gb300 import build as lib_build
from test_operators_host import TOPK_BWD


def test_refused_on_the_host():
    lib_build.build()
    call = _lib.load().bil_logp_topk_bwd
    same = ctypes.c_void_p(0x40000)  # never dereferenced: the call is refused
    assert call(*{**TOPK_BWD, "logits": same, "d": same}.values()) == _lib.E_INVALID_ARG


@pytest.mark.gpu
def test_refused_from_python():
    x = torch.randn(4, 300, device="cuda")
    t = torch.arange(4, device="cuda")
    _, lse, ids, top = bil.logp_topk(x, t, 5)
    before = x.clone()
    with pytest.raises(bil.BilError):
        bil.logp_topk_bwd(x, t, ids, lse, lse, top, out=x)
    assert torch.equal(x, before)
