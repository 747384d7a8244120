"""What stands around the LM head, together: scoring with 8 bits, and a training step.

    python examples/lm_head.py            # random weights, a few rows, on one GPU

``score`` takes the last layer's output and the residual stream to what a server
reports of its tokens: the norm with the residual's addition and an 8-bit
output, the 8-bit LM head (log-probability and entropy of the given tokens), and
from its logits the most likely alternatives.  ``train_step`` goes the other
way: the norm and its backward around a 16-bit head, with gradients through the
chosen tokens, the alternatives and the entropy.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import invariant_token_log_gb300 as bil  # noqa: E402


def score(x, residual, norm_weight, weight_q, weight_scale, targets, k=20, eps=1e-6, temperature=1.0, rows=4096):
    """(logp, entropy, top_ids, top_logp, stream) of the tokens ``targets`` [N].

    ``x``, ``residual`` [N, H]: the last layer's output and the stream it is added to
    (the sum comes back as ``stream``); ``weight_q``, ``weight_scale``: the LM head's
    rows as ``quantize_rows`` gives them, once per weight.  ``rows`` at a time, so
    that rows x vocabulary float32 logits are all that is kept of the head."""
    parts = []
    for i in range(0, max(x.shape[0], 1), rows):  # no rows are one empty part
        s = slice(i, i + rows)
        q, scale, stream = bil.rms_norm_quant(x[s], norm_weight, residual=residual[s], eps=eps)
        logp, _, entropy, logits = bil.linear_logp_fp8(q, scale, weight_q, weight_scale, targets[s],
                                                       temperature=temperature, return_entropy=True, return_logits=True)
        _, _, ids, top = bil.logp_topk(logits, targets[s], k, temperature=temperature)
        parts.append((logp, entropy, ids, top, stream))
    return tuple(torch.cat(p) for p in zip(*parts))


def train_step(x, residual, norm_weight, weight, targets, advantage, k=8, eps=1e-6, entropy_bonus=0.01, top_weight=0.1):
    """(loss, stream): a policy step's loss on the tokens, with an entropy bonus and a penalty on the mass of
    the k most likely tokens, already propagated to the leaves' ``.grad``."""
    y, stream = bil.rms_norm(x, norm_weight, residual, eps)
    logits = y @ weight.t()
    logp, entropy, _, top = bil.batch_invariant_logp_topk(logits, targets, k)
    loss = -(advantage * logp).mean() - entropy_bonus * entropy.mean() + top_weight * top.exp().sum(dim=1).mean()
    loss.backward()
    return loss.detach(), stream.detach()


def main():
    torch.manual_seed(0)
    n, hidden, vocab = 512, 1024, 32000
    x, residual = (torch.randn(n, hidden, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    norm_weight = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
    weight = torch.randn(vocab, hidden, device="cuda", dtype=torch.bfloat16) * (3 / hidden ** 0.5)
    targets = torch.randint(0, vocab, (n,), device="cuda")
    logp, entropy, ids, top, _ = score(x, residual, norm_weight, *bil.quantize_rows(weight), targets, k=5)
    print(f"logp {logp.mean():.3f}  entropy {entropy.mean():.3f}  row 0: token {int(targets[0])} {float(logp[0]):.3f}, "
          f"alternatives {ids[0].tolist()} {[round(v, 3) for v in top[0].tolist()]}")
    leaves = [t.requires_grad_() for t in (x, residual, norm_weight, weight)]
    loss, _ = train_step(*leaves, targets, torch.randn(n, device="cuda"))
    print(f"loss {float(loss):.4f}  gradient norms {[round(float(t.grad.float().norm()), 4) for t in leaves]}")


if __name__ == "__main__":
    main()
