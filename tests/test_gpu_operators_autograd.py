"""The norm and the alternatives have first derivatives only: a second one is an
error and not the derivative of a constant."""
import pytest
import torch

import invariant_token_log_gb300 as bil

pytestmark = pytest.mark.gpu


def leaf(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").requires_grad_()


def refuses(grad, *leaves):
    """A loss with `grad` in it, and something else that can be differentiated."""
    with pytest.raises(RuntimeError, match="no second derivative"):
        (grad.square().sum() + sum(x.sum() for x in leaves)).backward(retain_graph=True)


@pytest.mark.parametrize("residual", [False, True])
def test_norm(residual):
    x, w, r = leaf(1, 5, 64), leaf(2, 64), leaf(3, 5, 64)
    leaves = (x, w, r) if residual else (x, w)

    def out():
        return bil.rms_norm(x, w, r)[0] if residual else bil.rms_norm(x, w)

    want = torch.autograd.grad(out().sum(), leaves)
    got = torch.autograd.grad(out().sum(), leaves, create_graph=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
        refuses(a, *leaves)
    for g in torch.autograd.grad(out().square().sum(), leaves, create_graph=True):
        refuses(g, *leaves)


@pytest.mark.parametrize("part", ["logp", "entropy", "top"])
def test_alternatives(part):
    x, t = leaf(4, 4, 300), torch.arange(4, device="cuda")

    def out():
        logp, ent, _, top = bil.batch_invariant_logp_topk(x, t, 3)
        return {"logp": logp, "entropy": ent, "top": top}[part]

    want, = torch.autograd.grad(out().sum(), x)
    got, = torch.autograd.grad(out().sum(), x, create_graph=True)
    assert torch.equal(got, want)
    refuses(got, x)
    refuses(torch.autograd.grad(out().square().sum(), x, create_graph=True)[0], x)
