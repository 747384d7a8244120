"""Both ends of a language model's training step around a table that embeds the tokens and
is the LM head's weight too, with a block in between.

    python examples/tied_step.py          # random weights, a few tokens, on one GPU

``loss`` is the differentiable form: embedding, dropout, layer norm, a product, layer
norm with dropout and the residual's addition, cross entropy.  ``step`` is the same with
its gradients as a sequence of calls without autograd, which a CUDA graph can hold:
the seed and the step of the masks are a tensor that the program writes between
replays, and the table's two gradients are added up in one buffer.  (A program that captures
the autograd form has to drop its eager graphs of the same leaves first.)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import invariant_token_log_gb300 as bil  # noqa: E402


def parameters(vocab, hidden, dtype=torch.bfloat16, device="cuda"):
    def normal(*shape, scale):
        return (scale * torch.randn(*shape, device=device)).to(dtype)
    return {"table": normal(vocab, hidden, scale=hidden ** -0.5), "block": normal(hidden, hidden, scale=hidden ** -0.5),
            "w1": torch.ones(hidden, dtype=dtype, device=device), "b1": torch.zeros(hidden, dtype=dtype, device=device),
            "w2": torch.ones(hidden, dtype=dtype, device=device), "b2": torch.zeros(hidden, dtype=dtype, device=device)}


def loss(params, ids, targets, rng, p=0.1, scale=1.0, label_smoothing=0.0, z_loss=0.0):
    """The mean loss of predicting ``targets`` [N] from ``ids`` [N]."""
    e = bil.embedding(ids, params["table"], scale)
    x = bil.dropout(e, p, rng, 0)
    y = bil.layer_norm(x, params["w1"], params["b1"])
    z, _ = bil.layer_norm(y @ params["block"].t(), params["w2"], params["b2"], residual=x, p=p, seed=rng, offset=1)
    return bil.linear_cross_entropy(z, params["table"], targets, label_smoothing=label_smoothing, z_loss=z_loss)


def step(params, ids, targets, rng, grad, p=0.1, scale=1.0, label_smoothing=0.0, z_loss=0.0):
    """(loss, gradients by name): ``loss`` and what its backward gives, for a gradient ``grad`` of the loss."""
    how = {"label_smoothing": label_smoothing, "z_loss": z_loss}
    table, block = params["table"], params["block"]
    x = bil.dropout_fwd(bil.embedding_fwd(ids, table, scale), p, rng, 0)
    y, _, m1, s1 = bil.layer_norm_fwd(x, params["w1"], params["b1"])
    z, h, m2, s2 = bil.layer_norm_fwd(y @ block.t(), params["w2"], params["b2"], residual=x, p=p, seed=rng, offset=1)
    value, lse = bil.linear_cross_entropy_fwd(z, table, targets, **how)
    dz, dtable = bil.linear_cross_entropy_bwd(z, table, targets, lse, grad, **how)
    da, dx, dw2, db2 = bil.layer_norm_bwd(dz, h, params["w2"], m2, s2, p=p, seed=rng, offset=1)
    dn, _, dw1, db1 = bil.layer_norm_bwd(da @ block, x, params["w1"], m1, s1, grad_h=dx)
    bil.embedding_bwd(bil.dropout_bwd(dn, p, rng, 0), ids, table.shape[0], scale, out=dtable, accumulate=True)
    return value, {"table": dtable, "block": da.t() @ y, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}


def main():
    torch.manual_seed(0)
    vocab, hidden, n = 32000, 1024, 2048
    params = parameters(vocab, hidden)
    ids, targets = (torch.randint(0, vocab, (n,), device="cuda") for _ in range(2))
    rng, grad = torch.tensor([1234, 0], device="cuda"), torch.ones((), device="cuda")
    step(params, ids, targets, rng, grad)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        value, grads = step(params, ids, targets, rng, grad)
    for i in range(5):
        rng[1] = 2 * i  # a step has two dropouts
        graph.replay()
        for name, g in grads.items():
            params[name] -= (0.1 * g).to(params[name].dtype)
        print(f"step {i}: loss {float(value):.4f}")


if __name__ == "__main__":
    main()
