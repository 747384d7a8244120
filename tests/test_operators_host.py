"""The C entry points of the top-k, norm and 8-bit calls without a GPU: bad arguments are refused on the host,
before anything touches CUDA, and the limits the header states are the binding's."""
import ctypes
import os
import re

import pytest
import torch

import invariant_token_log_gb300 as bil
from invariant_token_log_gb300 import _lib
from invariant_token_log_gb300 import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x10000)       # never dereferenced: the call is refused
P8 = ctypes.c_void_p(0x10008)      # 8-byte aligned
ODD = ctypes.c_void_p(0x10001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return _lib.load()


def test_limits_match_the_header():
    text = open(os.path.join(ROOT, "include", "bil.h")).read()
    consts = dict(re.findall(r"#define (BIL_MAX_[A-Z_]+) ([0-9]+)\n", text))
    assert int(consts["BIL_MAX_TOPK"]) == _lib.MAX_TOPK
    assert int(consts["BIL_MAX_NORM_WIDTH"]) == _lib.MAX_NORM_WIDTH


TOPK = dict(logits=P, dtype=_lib.BF16, n=4, vocab=300, ld=300, tgt=P, ign=-100, tile=4096, temp=1.0, k=5, logp=P, lse=P,
            ent=None, ids=P, top=P, ws=P, bytes=1 << 40, validate=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), _lib.OK),
    (dict(n=0, logits=None, tgt=None, logp=None, ids=None, top=None, ws=None), _lib.OK),
    (dict(n=-1), _lib.E_INVALID_ARG),
    (dict(vocab=0), _lib.E_INVALID_ARG),
    (dict(ld=299), _lib.E_INVALID_ARG),
    (dict(k=0), _lib.E_INVALID_ARG),
    (dict(k=301), _lib.E_INVALID_ARG),
    (dict(k=129), _lib.E_UNSUPPORTED),
    (dict(dtype=9), _lib.E_DTYPE),
    (dict(tile=12), _lib.E_INVALID_ARG),
    (dict(tile=65536), _lib.E_UNSUPPORTED),
    (dict(vocab=8 * 2049, ld=8 * 2049, tile=8), _lib.E_UNSUPPORTED),
    (dict(vocab=2 ** 31, ld=2 ** 31, tile=32768), _lib.E_UNSUPPORTED),
    (dict(n=2 ** 40), _lib.E_UNSUPPORTED),
    (dict(n=2 ** 20, ld=2 ** 28), _lib.E_UNSUPPORTED),
    (dict(temp=0.0), _lib.E_INVALID_ARG),
    (dict(temp=NAN), _lib.E_INVALID_ARG),
    (dict(logits=None), _lib.E_INVALID_ARG),
    (dict(tgt=None), _lib.E_INVALID_ARG),
    (dict(logp=None), _lib.E_INVALID_ARG),
    (dict(ids=None), _lib.E_INVALID_ARG),
    (dict(top=None), _lib.E_INVALID_ARG),
    (dict(ws=None), _lib.E_INVALID_ARG),
    (dict(bytes=10), _lib.E_INVALID_ARG),
    (dict(logits=ODD), _lib.E_ALIGN),
    (dict(ids=ctypes.c_void_p(0x10004)), _lib.E_ALIGN),
    (dict(ent=ODD), _lib.E_ALIGN),
    (dict(ws=P8), _lib.E_ALIGN),
])
def test_topk_fwd(lib, kw, status):
    assert lib.bil_logp_topk_fwd(*{**TOPK, **kw}.values()) == status


def test_topk_workspace(lib):
    out = ctypes.c_int64(0)
    ws = lib.bil_logp_topk_workspace_bytes
    assert ws(_lib.BF16, 3, 10000, 4096, 20, 0, ctypes.byref(out)) == _lib.OK
    # 3 tiles of 64 chunks in 2 bytes each, rows on 16 bytes; two [3, 3] float32 partials; blocks of 256 bytes
    assert out.value == -(-3 * 3 * 64 * 2 // 256) * 256 + 2 * 256
    assert ws(_lib.F32, 3, 10000, 4096, 20, 1, ctypes.byref(out)) == _lib.OK
    assert out.value == -(-3 * 3 * 64 * 4 // 256) * 256 + 3 * 256
    assert ws(_lib.BF16, 3, 10000, 4096, 20, 0, None) == _lib.E_INVALID_ARG
    assert ws(_lib.BF16, 3, 10, 4096, 20, 0, ctypes.byref(out)) == _lib.E_INVALID_ARG


TOPK_BWD = dict(logits=P, dtype=_lib.BF16, n=4, vocab=300, ld=300, tgt=P, ign=-100, temp=1.0, ids=P, k=5, lse=P, g=P, gk=P,
                ent=None, gent=None, d=P, odt=_lib.BF16, ldo=300, cols=300, ws=P, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), _lib.OK),
    (dict(n=-1), _lib.E_INVALID_ARG),
    (dict(k=0), _lib.E_INVALID_ARG),
    (dict(k=301), _lib.E_INVALID_ARG),
    (dict(k=129), _lib.E_UNSUPPORTED),
    (dict(dtype=9), _lib.E_DTYPE),
    (dict(odt=9), _lib.E_DTYPE),
    (dict(ldo=299, cols=299), _lib.E_INVALID_ARG),
    (dict(cols=301), _lib.E_INVALID_ARG),
    (dict(temp=-1.0), _lib.E_INVALID_ARG),
    (dict(ent=P), _lib.E_INVALID_ARG),
    (dict(logits=None), _lib.E_INVALID_ARG),
    (dict(lse=None), _lib.E_INVALID_ARG),
    (dict(ids=None), _lib.E_INVALID_ARG),
    (dict(gk=None), _lib.E_INVALID_ARG),
    (dict(g=None), _lib.E_INVALID_ARG),
    (dict(d=None), _lib.E_INVALID_ARG),
    (dict(ws=None), _lib.E_INVALID_ARG),
    (dict(d=ODD), _lib.E_ALIGN),
    (dict(ids=ctypes.c_void_p(0x10004)), _lib.E_ALIGN),
    (dict(ent=ODD, gent=P), _lib.E_ALIGN),
    (dict(n=2 ** 40), _lib.E_UNSUPPORTED),
    (dict(n=2 ** 20, ldo=2 ** 28), _lib.E_UNSUPPORTED),
])
def test_topk_bwd(lib, kw, status):
    assert lib.bil_logp_topk_bwd(*{**TOPK_BWD, **kw}.values()) == status


NORM = dict(x=P, res=P, w=P, dtype=_lib.BF16, wdtype=_lib.BF16, n=4, width=64, ldx=64, ldr=64, eps=1e-6, y=P, ldy=64, h=P,
            ldh=64, rstd=P, stream=None)
QUANT = dict(x=P, res=P, w=P, dtype=_lib.BF16, wdtype=_lib.F32, n=4, width=64, ldx=64, ldr=64, eps=1e-6, q=P, ldq=64,
             scale=P, h=P, ldh=64, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), _lib.OK),
    (dict(n=-1), _lib.E_INVALID_ARG),
    (dict(width=0), _lib.E_INVALID_ARG),
    (dict(width=16385, ldx=16385, ldr=16385, ldy=16385, ldh=16385, ldq=16385), _lib.E_UNSUPPORTED),
    (dict(dtype=9), _lib.E_DTYPE),
    (dict(wdtype=_lib.F16), _lib.E_DTYPE),
    (dict(eps=-1.0), _lib.E_INVALID_ARG),
    (dict(eps=NAN), _lib.E_INVALID_ARG),
    (dict(eps=INF), _lib.E_INVALID_ARG),
    (dict(ldx=63), _lib.E_INVALID_ARG),
    (dict(ldr=63), _lib.E_INVALID_ARG),
    (dict(ldh=63), _lib.E_INVALID_ARG),
    (dict(ldy=63, ldq=63), _lib.E_INVALID_ARG),
    (dict(x=None), _lib.E_INVALID_ARG),
    (dict(w=None), _lib.E_INVALID_ARG),
    (dict(y=None, q=None), _lib.E_INVALID_ARG),
    (dict(h=None), _lib.E_INVALID_ARG),              # a residual without its sum
    (dict(res=None), _lib.E_INVALID_ARG),            # and the other way round
    (dict(x=ODD), _lib.E_ALIGN),
    (dict(w=P8), _lib.E_ALIGN),
    (dict(n=2 ** 40), _lib.E_UNSUPPORTED),
    (dict(n=2 ** 30, ldr=2 ** 20), _lib.E_UNSUPPORTED),
])
def test_norm_forward_and_quant(lib, kw, status):
    for fn, base in ((lib.bil_rms_norm_fwd, NORM), (lib.bil_rms_norm_quant, QUANT)):
        args = {**base, **{k: v for k, v in kw.items() if k in base}}
        if kw.get("wdtype") == _lib.F16:
            args["wdtype"] = _lib.F16
        assert fn(*args.values()) == status, fn.__name__
    assert lib.bil_rms_norm_quant(*{**QUANT, "scale": None}.values()) == _lib.E_INVALID_ARG
    assert lib.bil_rms_norm_quant(*{**QUANT, "scale": ODD}.values()) == _lib.E_ALIGN
    assert lib.bil_rms_norm_fwd(*{**NORM, "rstd": ODD}.values()) == _lib.E_ALIGN


def test_quantize_rows(lib):
    f = lib.bil_quantize_rows
    #        x  dtype      n  width ldx q  ldq scale stream
    assert f(P, _lib.F32, 0, 64, 64, P, 64, P, None) == _lib.OK
    assert f(P, 9, 4, 64, 64, P, 64, P, None) == _lib.E_DTYPE
    assert f(P, _lib.F32, 4, 64, 63, P, 64, P, None) == _lib.E_INVALID_ARG
    assert f(P, _lib.F32, 4, 64, 64, P, 63, P, None) == _lib.E_INVALID_ARG
    assert f(P, _lib.F32, 4, 64, 64, P, 64, None, None) == _lib.E_INVALID_ARG
    assert f(ODD, _lib.F32, 4, 64, 64, P, 64, P, None) == _lib.E_ALIGN
    assert f(P, _lib.F32, 4, 16385, 16385, P, 16385, P, None) == _lib.E_UNSUPPORTED


NORM_BWD = dict(dy=P, h=P, w=P, rstd=P, dh=None, dtype=_lib.BF16, wdtype=_lib.BF16, n=4, width=64, lddy=64, ldh=64, lddh=0,
                dx=P, lddx=64, dw=P, ws=P, bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), _lib.E_INVALID_ARG),
    (dict(dtype=9), _lib.E_DTYPE),
    (dict(wdtype=_lib.F16), _lib.E_DTYPE),
    (dict(width=16385, lddy=16385, ldh=16385, lddx=16385), _lib.E_UNSUPPORTED),
    (dict(lddy=63), _lib.E_INVALID_ARG),
    (dict(ldh=63), _lib.E_INVALID_ARG),
    (dict(lddx=63), _lib.E_INVALID_ARG),
    (dict(dh=P, lddh=63), _lib.E_INVALID_ARG),
    (dict(dy=None), _lib.E_INVALID_ARG),
    (dict(dw=None), _lib.E_INVALID_ARG),
    (dict(rstd=None), _lib.E_INVALID_ARG),
    (dict(ws=None), _lib.E_INVALID_ARG),
    (dict(dx=ODD), _lib.E_ALIGN),
    (dict(ws=P8), _lib.E_ALIGN),
    (dict(n=2 ** 42), _lib.E_UNSUPPORTED),           # rows of 128 bytes: 2^49
])
def test_norm_bwd(lib, kw, status):
    assert lib.bil_rms_norm_bwd(*{**NORM_BWD, **kw}.values()) == status


HEAD8 = dict(h=P, hs=P, w=P, ws=P, n=4, hidden=64, ldh=64, vocab=1000, ldw=64, temp=1.0, tgt=P, ign=-100, logp=P, lse=P,
             ent=None, logits=None, ldt=_lib.F32, ldl=0, work=P, bytes=1 << 40, validate=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), _lib.OK),
    (dict(n=-1), _lib.E_INVALID_ARG),
    (dict(hidden=0), _lib.E_INVALID_ARG),
    (dict(vocab=0), _lib.E_INVALID_ARG),
    (dict(ldh=63), _lib.E_INVALID_ARG),
    (dict(ldw=63), _lib.E_INVALID_ARG),
    (dict(temp=0.0), _lib.E_INVALID_ARG),
    (dict(h=None), _lib.E_INVALID_ARG),
    (dict(hs=None), _lib.E_INVALID_ARG),
    (dict(w=None), _lib.E_INVALID_ARG),
    (dict(ws=None), _lib.E_INVALID_ARG),
    (dict(tgt=None), _lib.E_INVALID_ARG),
    (dict(logp=None), _lib.E_INVALID_ARG),
    (dict(work=None), _lib.E_INVALID_ARG),
    (dict(bytes=8), _lib.E_INVALID_ARG),
    (dict(logits=P, ldl=999), _lib.E_INVALID_ARG),
    (dict(logits=P, ldl=1000, ldt=_lib.F16), _lib.E_DTYPE),
    (dict(logits=P, ldl=1001), _lib.E_ALIGN),
    (dict(h=P8), _lib.E_ALIGN),                      # TMA: 16-byte base ...
    (dict(ldw=72), _lib.E_ALIGN),                    # ... and row stride
    (dict(hs=ODD), _lib.E_ALIGN),
    (dict(work=P8), _lib.E_ALIGN),
    (dict(n=2 ** 40), _lib.E_UNSUPPORTED),
    (dict(ldw=2 ** 40), _lib.E_UNSUPPORTED),
    (dict(vocab=2 ** 63 - 1), _lib.E_UNSUPPORTED),
])
def test_head8(lib, kw, status):
    assert lib.bil_linear_logp_fp8_fwd(*{**HEAD8, **kw}.values()) == status


def test_cpu_tensors_are_refused():
    x, t = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    w, f = torch.ones(16, dtype=torch.bfloat16), torch.zeros(2)
    q = x.to(torch.float8_e4m3fn)
    calls = [lambda: bil.logp_topk(x, t, 3),
             lambda: bil.logp_topk_bwd(x, t, torch.zeros(2, 3, dtype=torch.int64), f, f, torch.zeros(2, 3)),
             lambda: bil.rms_norm_fwd(x, w), lambda: bil.rms_norm_quant(x, w), lambda: bil.quantize_rows(x),
             lambda: bil.rms_norm_bwd(x, x, w, f), lambda: bil.linear_logp_fp8(q, f, q, f, t)]
    for call in calls:
        with pytest.raises(ValueError, match="no CPU path"):
            call()
