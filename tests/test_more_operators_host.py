"""The C entry points of layer norm, dropout, the embedding and the cross entropy without a GPU: bad arguments are
refused on the host, before anything touches CUDA, and CPU tensors are refused by the binding."""
import ctypes

import pytest
import torch

import invariant_token_log_gb300 as bil
from invariant_token_log_gb300 import _lib
from invariant_token_log_gb300 import build as lib_build
from invariant_token_log_gb300.cross_entropy import fwd_workspace_bytes
from invariant_token_log_gb300.drop import _random
from invariant_token_log_gb300.embed import bwd_workspace_bytes as embed_bytes

P = ctypes.c_void_p(0x10000)  # never dereferenced: the call is refused
P2 = ctypes.c_void_p(0x20000)
P8 = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10001)
NAN, INF = float("nan"), float("inf")
INVALID, DTYPE, ALIGN, UNSUPPORTED, OK = _lib.E_INVALID_ARG, _lib.E_DTYPE, _lib.E_ALIGN, _lib.E_UNSUPPORTED, _lib.OK


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return _lib.load()


LN = dict(x=P, res=P, w=P, b=P, dtype=_lib.BF16, wdtype=_lib.BF16, n=4, width=64, ldx=64, ldr=64, eps=1e-5, p=0.1, seed=1,
          step=2, rng=None, y=P, ldy=64, h=P2, ldh=64, mean=P, rstd=P, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK),
    (dict(n=0, x=None, res=None, y=None, h=None, mean=None, rstd=None), OK),
    (dict(n=-1), INVALID),
    (dict(width=0), INVALID),
    (dict(width=16385, ldx=16385, ldr=16385, ldy=16385, ldh=16385), UNSUPPORTED),
    (dict(dtype=9), DTYPE),
    (dict(wdtype=_lib.F16), DTYPE),
    (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID),
    (dict(p=1.0), INVALID),
    (dict(p=-0.1), INVALID),
    (dict(p=NAN), INVALID),
    (dict(p=1 - 2.0 ** -18), INVALID),
    (dict(ldx=63), INVALID),
    (dict(ldr=63), INVALID),
    (dict(ldy=63), INVALID),
    (dict(ldh=63), INVALID),
    (dict(x=None), INVALID),
    (dict(w=None), INVALID),
    (dict(y=None), INVALID),
    (dict(h=None), INVALID),                    # dropout or a residual without the sum
    (dict(p=0.0, h=None), INVALID),
    (dict(res=None, h=None), INVALID),
    (dict(p=0.0, res=None), INVALID),           # and the other way round
    (dict(x=ODD), ALIGN),
    (dict(w=P8), ALIGN),
    (dict(b=P8), ALIGN),
    (dict(rng=ctypes.c_void_p(0x10004)), ALIGN),
    (dict(mean=ODD), ALIGN),
    (dict(rstd=ODD), ALIGN),
    (dict(n=2 ** 40), UNSUPPORTED),
    (dict(n=2 ** 30, ldr=2 ** 20), UNSUPPORTED),
])
def test_layer_norm_fwd(lib, kw, status):
    assert lib.bil_layer_norm_fwd(*{**LN, **kw}.values()) == status


LN_BWD = dict(dy=P, h=P, w=P, mean=P, rstd=P, dh=None, dtype=_lib.BF16, wdtype=_lib.BF16, n=4, width=64, lddy=64, ldh=64,
              lddh=0, p=0.1, seed=1, step=2, rng=None, dx=P, lddx=64, dr=P2, lddr=64, dw=P, db=P, ws=P, bytes=1 << 40,
              stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID),
    (dict(dtype=9), DTYPE),
    (dict(wdtype=_lib.F16), DTYPE),
    (dict(width=16385, lddy=16385, ldh=16385, lddx=16385, lddr=16385), UNSUPPORTED),
    (dict(p=1.5), INVALID),
    (dict(p=0.0), INVALID),                     # without dropout the residual's gradient is dx
    (dict(dr=P), INVALID),                      # two outputs in one buffer
    (dict(lddy=63), INVALID),
    (dict(ldh=63), INVALID),
    (dict(lddx=63), INVALID),
    (dict(lddr=63), INVALID),
    (dict(dh=P, lddh=63), INVALID),
    (dict(dy=None), INVALID),
    (dict(dx=None), INVALID),
    (dict(dw=None), INVALID),
    (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID),
    (dict(ws=None), INVALID),
    (dict(dx=ODD), ALIGN),
    (dict(db=ODD), ALIGN),
    (dict(ws=P8), ALIGN),
    (dict(n=2 ** 42), UNSUPPORTED),
])
def test_layer_norm_bwd(lib, kw, status):
    assert lib.bil_layer_norm_bwd(*{**LN_BWD, **kw}.values()) == status


DROP = dict(x=P, res=P, dtype=_lib.BF16, n=4, width=64, ldx=64, ldr=64, p=0.1, seed=1, step=2, rng=None, y=P, ldy=64, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK),
    (dict(n=-1), INVALID),
    (dict(width=0), INVALID),
    (dict(dtype=9), DTYPE),
    (dict(p=1.0), INVALID),
    (dict(p=-1e-9), INVALID),
    (dict(p=NAN), INVALID),
    (dict(p=1 - 2.0 ** -18), INVALID),
    (dict(ldx=63), INVALID),
    (dict(ldr=63), INVALID),
    (dict(ldy=63), INVALID),
    (dict(x=None), INVALID),
    (dict(y=None), INVALID),
    (dict(x=ODD), ALIGN),
    (dict(res=ODD), ALIGN),
    (dict(y=ODD), ALIGN),
    (dict(rng=ctypes.c_void_p(0x10004)), ALIGN),
    (dict(n=2 ** 42), UNSUPPORTED),
    (dict(width=2 ** 31, ldx=2 ** 31, ldr=2 ** 31, ldy=2 ** 31), UNSUPPORTED),
])
def test_dropout(lib, kw, status):
    assert lib.bil_dropout(*{**DROP, **kw}.values()) == status


EMBED = dict(ids=P, n=4, w=P, dtype=_lib.BF16, vocab=100, width=64, ldw=64, scale=1.0, out=P, ldo=64, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK),
    (dict(n=-1), INVALID),
    (dict(vocab=0), INVALID),
    (dict(width=0), INVALID),
    (dict(dtype=9), DTYPE),
    (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID),
    (dict(ldw=63), INVALID),
    (dict(ldo=63), INVALID),
    (dict(ids=None), INVALID),
    (dict(w=None), INVALID),
    (dict(out=None), INVALID),
    (dict(ids=ctypes.c_void_p(0x10004)), ALIGN),
    (dict(w=ODD), ALIGN),
    (dict(out=ODD), ALIGN),
    (dict(n=2 ** 31), UNSUPPORTED),
    (dict(vocab=2 ** 31), UNSUPPORTED),
    (dict(ldw=2 ** 42), UNSUPPORTED),
])
def test_embedding_fwd(lib, kw, status):
    assert lib.bil_embedding_fwd(*{**EMBED, **kw}.values()) == status


EMBED_BWD = dict(dy=P, dtype=_lib.BF16, n=4, width=64, lddy=64, ids=P, vocab=100, scale=1.0, pad=-1, dw=P2, dwt=_lib.BF16,
                 lddw=64, acc=0, ws=P, bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0, acc=1), OK),
    (dict(n=-1), INVALID),
    (dict(vocab=0), INVALID),
    (dict(width=0), INVALID),
    (dict(dtype=9), DTYPE),
    (dict(dwt=_lib.F16), DTYPE),
    (dict(dtype=_lib.F32, dwt=_lib.BF16), DTYPE),
    (dict(dw=P), INVALID),                      # the output over dy
    (dict(scale=INF), INVALID),
    (dict(lddy=63), INVALID),
    (dict(lddw=63), INVALID),
    (dict(ids=None), INVALID),
    (dict(dy=None), INVALID),
    (dict(dw=None), INVALID),
    (dict(ws=None), INVALID),
    (dict(bytes=100), INVALID),
    (dict(ids=ODD), ALIGN),
    (dict(ws=P8), ALIGN),
    (dict(n=2 ** 31), UNSUPPORTED),
    (dict(vocab=2 ** 31), UNSUPPORTED),
    (dict(lddw=2 ** 42), UNSUPPORTED),
])
def test_embedding_bwd(lib, kw, status):
    assert lib.bil_embedding_bwd(*{**EMBED_BWD, **kw}.values()) == status


XENT = dict(h=P, w=P, dtype=_lib.BF16, n=4, hidden=64, ldh=64, vocab=1000, ldw=64, tgt=P, ign=-100, smooth=0.1, z=1e-4, red=1,
            loss=P, lse=P, ws=P, bytes=1 << 40, validate=0, stream=None)
COMMON = [
    (dict(n=-1), INVALID),
    (dict(hidden=0), INVALID),
    (dict(vocab=0), INVALID),
    (dict(dtype=_lib.F32), DTYPE),
    (dict(dtype=9), DTYPE),
    (dict(ldh=63), INVALID),
    (dict(ldw=63), INVALID),
    (dict(smooth=-0.1), INVALID),
    (dict(smooth=1.1), INVALID),
    (dict(smooth=NAN), INVALID),
    (dict(z=INF), INVALID),
    (dict(red=3), INVALID),
    (dict(red=-1), INVALID),
    (dict(h=None), INVALID),
    (dict(w=None), INVALID),
    (dict(tgt=None), INVALID),
    (dict(lse=ODD), ALIGN),
    (dict(h=P8), ALIGN),
    (dict(w=P8), ALIGN),
    (dict(ldh=68), ALIGN),
    (dict(ldw=68), ALIGN),
    (dict(tgt=ctypes.c_void_p(0x10004)), ALIGN),
    (dict(ws=None), INVALID),
    (dict(ws=P8), ALIGN),
    (dict(n=2 ** 31), UNSUPPORTED),
    (dict(vocab=2 ** 31), UNSUPPORTED),
    (dict(hidden=2 ** 25, ldh=2 ** 25, ldw=2 ** 25), UNSUPPORTED),
    (dict(ldw=2 ** 40), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(n=0, red=0), OK),
    (dict(n=0, red=0, h=None, tgt=None, loss=None, lse=None, ws=None), OK),
    (dict(n=0, loss=None), INVALID),
    (dict(loss=None), INVALID),
    (dict(loss=ODD), ALIGN),
    (dict(bytes=1000), INVALID),
])
def test_cross_entropy_fwd(lib, kw, status):
    assert lib.bil_linear_cross_entropy_fwd(*{**XENT, **kw}.values()) == status


XENT_BWD = dict(h=P, w=P, dtype=_lib.BF16, n=4, hidden=64, ldh=64, vocab=1000, ldw=64, tgt=P, ign=-100, smooth=0.1, z=1e-4,
                red=1, lse=P, g=P, piece=0, dh=P, dht=_lib.BF16, lddh=64, dw=P2, dwt=_lib.BF16, lddw=64, ws=P, bytes=1 << 40,
                stream=None)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(n=0, dw=None), OK),
    (dict(piece=-1), INVALID),
    (dict(dh=None, dw=None), INVALID),
    (dict(dw=P), INVALID),                      # the gradient over the weight
    (dict(dht=_lib.F16), DTYPE),
    (dict(dwt=_lib.F16), DTYPE),
    (dict(lddh=63), INVALID),
    (dict(lddw=63), INVALID),
    (dict(lddh=68), ALIGN),
    (dict(dw=P8), ALIGN),
    (dict(lse=None), INVALID),
    (dict(g=None), INVALID),
    (dict(g=ODD), ALIGN),
    (dict(lddw=2 ** 40), UNSUPPORTED),
])
def test_cross_entropy_bwd(lib, kw, status):
    assert lib.bil_linear_cross_entropy_bwd(*{**XENT_BWD, **kw}.values()) == status


def test_workspaces(lib):
    out = ctypes.c_int64(0)
    assert lib.bil_embedding_bwd_workspace_bytes(10, 64, None) == INVALID
    assert lib.bil_embedding_bwd_workspace_bytes(-1, 64, ctypes.byref(out)) == INVALID
    assert lib.bil_layer_norm_bwd_workspace_bytes(4, 16385, 1, ctypes.byref(out)) == UNSUPPORTED
    assert lib.bil_layer_norm_bwd_workspace_bytes(4, 64, 1, None) == INVALID
    assert lib.bil_linear_cross_entropy_fwd_workspace_bytes(4, 64, 1000, 0, None) == INVALID
    assert lib.bil_linear_cross_entropy_bwd_workspace_bytes(4, 64, 1000, -1, ctypes.byref(out)) == INVALID
    # a row count more takes no less, and the smoothing's sums a third of the parts more
    sizes = [embed_bytes(n, 64) for n in (0, 1, 1000, 4096, 20000, 70000, 10 ** 6)]
    assert sizes == sorted(sizes)
    plain, smooth = fwd_workspace_bytes(300, 64, 1000, False), fwd_workspace_bytes(300, 64, 1000, True)
    assert smooth - plain == 8 * 512 * 4  # eight 128-column parts for 512 (two units of) rows


def test_seeds():
    assert _random(0.5, -1, 0, 0)[1] == 2 ** 64 - 1 and _random(0.5, 3, -1, 0)[2] == 2 ** 64 - 1
    for p in (1.0, -0.5, NAN, 1 - 2.0 ** -18):
        with pytest.raises(ValueError):
            _random(p, 0, 0, 0)
    with pytest.raises(TypeError):
        _random(0.5, 1.0, 0, 0)
    with pytest.raises(TypeError):
        _random(0.5, 1, 0.0, 0)
    for bad in (torch.zeros(2), torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError):
            _random(0.5, bad, 0, 0)


def test_cpu_tensors_are_refused():
    x, t = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
    w, f = torch.ones(16, dtype=torch.bfloat16), torch.zeros(2)
    for call in (lambda: bil.layer_norm_fwd(x, w), lambda: bil.layer_norm_bwd(x, x, w, f, f), lambda: bil.layer_norm(x, w),
                 lambda: bil.dropout_fwd(x, 0.5, 1), lambda: bil.dropout_bwd(x, 0.5, 1), lambda: bil.dropout(x, 0.5, 1),
                 lambda: bil.embedding_fwd(t, x), lambda: bil.embedding_bwd(x, t, 4), lambda: bil.embedding(t, x),
                 lambda: bil.linear_cross_entropy_fwd(x, x, t), lambda: bil.linear_cross_entropy_bwd(x, x, t, f, f[:1]),
                 lambda: bil.linear_cross_entropy(x, x, t)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
