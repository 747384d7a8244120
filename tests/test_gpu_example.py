"""The example's two paths, each through several of the operators, against plain torch.

Tolerances.  score: the plain form starts from the same e4m3 values and scales (rms_norm_quant's, checked
elsewhere), so what is left is the head's accumulation and the statistics: 1e-4, as everywhere.
train_step: y and the logits are bfloat16, the weight's gradient a bfloat16 product: 2^-8 of each value,
and 2^-7 of the gradient's norm over all (the roundings of y, the logits, dlogits and the product are
independent, about 2^-9 each in the root mean square)."""
import importlib.util
import os

import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import check_watchdog

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("lm_head", os.path.join(ROOT, "examples", "lm_head.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def data(n, hidden, vocab):
    g = torch.Generator(device="cuda").manual_seed(5)
    x, r = (torch.randn(n, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).bfloat16()
    weight = (torch.randn(vocab, hidden, generator=g, device="cuda") * (3 / hidden ** 0.5)).bfloat16()
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    return x, r, w, weight, t


def test_score(example):
    x, r, w, weight, t = data(300, 384, 5000)
    wq, ws = bil.quantize_rows(weight)
    logp, entropy, ids, top, stream = example.score(x, r, w, wq, ws, t, k=7, temperature=0.8, rows=128)
    assert torch.equal(stream, (x.float() + r.float()).bfloat16())
    q, scale, _ = bil.rms_norm_quant(x, w, residual=r)
    z = (q.double() @ wq.double().t()) * ws.double() * scale.double()[:, None] / 0.8
    a = torch.log_softmax(z, dim=1)
    assert float((logp.double() - a.gather(1, t[:, None])[:, 0]).abs().max()) <= 1e-4
    assert float((entropy.double() + (a.exp() * a).sum(dim=1)).abs().max()) <= 1e-4
    assert float((top.double() - a.gather(1, ids)).abs().max()) <= 1e-4
    assert float((top.double() - a.topk(7, dim=1)[0]).abs().max()) <= 1e-4
    # in one piece: the same bits
    whole = example.score(x, r, w, wq, ws, t, k=7, temperature=0.8)
    for a, b in zip((logp, entropy, ids, top, stream), whole):
        assert torch.equal(a, b)
    check_watchdog()


def test_train_step(example):
    x, r, w, weight, t = data(200, 256, 3000)
    adv = torch.randn(200, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    leaves = [v.clone().requires_grad_() for v in (x, r, w, weight)]
    loss, _ = example.train_step(*leaves, t, adv)
    ref = [v.clone().double().requires_grad_() for v in (x, r, w, weight)]
    h = ref[0] + ref[1]
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-6) * ref[2]
    a = torch.log_softmax(y @ ref[3].t(), dim=1)
    lp = a.gather(1, t[:, None])[:, 0]
    top = a.topk(8, dim=1)[0]
    rloss = -(adv.double() * lp).mean() + 0.01 * (a.exp() * a).sum(dim=1).mean() + 0.1 * top.exp().sum(dim=1).mean()
    rloss.backward()
    assert abs(float(loss) - float(rloss.detach())) <= 2.0 ** -8 * (1 + abs(float(rloss.detach())))
    for got, want in zip(leaves, ref):
        assert got.grad.dtype == got.dtype
        assert float((got.grad.double() - want.grad).norm()) <= 2.0 ** -7 * float(want.grad.norm())
    check_watchdog()


def test_main_runs(example, capsys):
    example.main()
    assert "alternatives" in capsys.readouterr().out
