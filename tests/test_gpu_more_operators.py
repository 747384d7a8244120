"""Layer norm, dropout, embedding and cross entropy together and under the conditions a program
brings: CUDA graphs, threads on their own streams, outputs over inputs, two graphs with one workspace, buffers past
2^31 elements, refusals of the binding.

Tolerances of the chain (test_tied_step): every stored tensor is bfloat16, one rounding of 2^-9 in the root mean
square each, some ten of them on the way to any gradient, which the block's product mixes: 2^-5 of a gradient's norm
leaves a factor of three over sqrt(10) 2^-9 times two, for the residual's two paths."""
import importlib.util
import os
import threading

import numpy as np
import pytest
import torch

import invariant_token_log_gb300 as bil
from invariant_token_log_gb300 import _lib
from invariant_token_log_gb300.cross_entropy import bwd_workspace_bytes as xent_bwd_bytes
from invariant_token_log_gb300.cross_entropy import fwd_workspace_bytes as xent_fwd_bytes
from invariant_token_log_gb300.embed import bwd_workspace_bytes as embed_bytes
from invariant_token_log_gb300.layernorm import bwd_workspace_bytes as ln_bytes
from invariant_token_log_gb300.logp import _code, _stream_handle
from philox import border_of, keep_mask, philox

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bits(x):
    x = x.detach().contiguous()
    return x if x.dtype == torch.int64 else x.view({2: torch.int16, 4: torch.int32}[x.itemsize])


def same(a, b):
    return torch.equal(bits(a), bits(b))


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")).to(dtype)


def tokens(seed, n, vocab):
    u = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=torch.float64)
    return ((vocab + 1.0) ** u).long().sub_(1).clamp_(0, vocab - 1)


class LayerNorm:
    def __init__(self, n, width, dtype, p):
        self.n, self.width, self.dtype, self.p = n, width, dtype, p

    def inputs(self, seed):
        return tuple(normal(seed + i, self.n, self.width, dtype=self.dtype) for i in range(4)) + (
            normal(seed + 4, self.width, dtype=self.dtype), normal(seed + 5, self.width, dtype=self.dtype),
            torch.tensor([seed, seed + 1], device="cuda"))

    def run(self, x, r, dy, dh, w, b, rng):
        y, h, mean, rstd = bil.layer_norm_fwd(x, w, b, residual=r, p=self.p, seed=rng)
        return (y, h, mean, rstd) + bil.layer_norm_bwd(dy, h, w, mean, rstd, grad_h=dh, p=self.p, seed=rng)


class Embedding:
    def __init__(self, n, vocab, width, dtype):
        self.n, self.vocab, self.width, self.dtype = n, vocab, width, dtype

    def inputs(self, seed):
        return (tokens(seed, self.n, self.vocab), normal(seed, self.vocab, self.width, dtype=self.dtype),
                normal(seed + 1, self.n, self.width, dtype=self.dtype))

    def run(self, ids, w, dy):
        return bil.embedding_fwd(ids, w, 2.0), bil.embedding_bwd(dy, ids, self.vocab, 2.0)


class CrossEntropy:
    def __init__(self, n, vocab, width, dtype, piece=None, reduction="mean"):
        self.n, self.vocab, self.width, self.dtype, self.piece, self.reduction = n, vocab, width, dtype, piece, reduction

    def inputs(self, seed):
        t = tokens(seed, self.n, self.vocab)
        t[torch.rand(self.n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") < 0.2] = bil.IGNORE_INDEX
        g = normal(seed + 2, self.n, dtype=torch.float32) if self.reduction == "none" else torch.tensor(1.0 + seed, device="cuda")
        return (normal(seed, self.n, self.width, dtype=self.dtype),
                normal(seed + 1, self.vocab, self.width, dtype=self.dtype, scale=3 * self.width ** -0.5), t, g)

    def run(self, x, w, t, g):
        how = {"label_smoothing": 0.1, "z_loss": 1e-4, "reduction": self.reduction}
        loss, lse = bil.linear_cross_entropy_fwd(x, w, t, **how)
        return (loss, lse) + bil.linear_cross_entropy_bwd(x, w, t, lse, g, piece=self.piece, **how)


class Dropout:
    def inputs(self, seed):
        return normal(seed, 100, 333), normal(seed + 1, 100, 333), torch.tensor([seed, 7], device="cuda")

    def run(self, x, r, rng):
        return bil.dropout_fwd(x, 0.3, rng, 1, residual=r), bil.dropout_bwd(r, 0.3, rng, 1)


CALLS = {
    "layer norm": LayerNorm(300, 4096, torch.bfloat16, 0.0),
    "layer norm with dropout": LayerNorm(300, 4096, torch.bfloat16, 0.2),
    "layer norm, off boundaries": LayerNorm(40, 1001, torch.float32, 0.2),
    "layer norm, a warp a row": LayerNorm(1000, 256, torch.float16, 0.0),
    "dropout": Dropout(),
    "embedding": Embedding(3000, 5000, 264, torch.bfloat16),
    "embedding, many tokens": Embedding(70000, 1000, 24, torch.float32),
    "cross entropy": CrossEntropy(200, 3000, 136, torch.bfloat16),
    "cross entropy in pieces": CrossEntropy(600, 2000, 264, torch.float16, 512, "none"),
    "cross entropy, many rows": CrossEntropy(9000, 500, 64, torch.bfloat16),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_captured_into_a_graph(call):
    """Captured once, replayed on other inputs in the same buffers: other numbers of rows that count, tokens, masks."""
    static = call.inputs(1)
    call.run(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call.run(*static)
    for seed in (1, 7, 13, 7):
        for buf, new in zip(static, call.inputs(seed)):
            buf.copy_(new)
        want = call.run(*static)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, want)):
            assert same(a, b), (seed, i)


def test_threads_on_their_own_streams():
    calls = list(CALLS.values())
    inputs = [c.inputs(20 + i) for i, c in enumerate(calls)]
    want = [c.run(*x) for c, x in zip(calls, inputs)]
    torch.cuda.synchronize()
    results, errors = [[] for _ in calls], []
    start = threading.Barrier(len(calls))

    def work(i):
        try:
            s = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(s):
                for _ in range(5):
                    results[i].append(calls[i].run(*inputs[i]))
            s.synchronize()
        except Exception as e:  # reported below, in the main thread
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    assert not errors, errors
    assert not any(th.is_alive() for th in threads)
    torch.cuda.synchronize()
    for i, rounds in enumerate(results):
        assert len(rounds) == 5
        for out in rounds:
            assert all(same(a, b) for a, b in zip(out, want[i])), i


def test_two_graphs_share_a_workspace():
    """Replayed one after the other on one stream, each leaves nothing in it that the other trusts."""
    dev = torch.device("cuda", 0)
    a, b = CrossEntropy(200, 3000, 136, torch.bfloat16).inputs(3), CrossEntropy(77, 900, 264, torch.bfloat16).inputs(4)
    space = torch.empty(max(f(n, h, v, *more) for n, v, h in ((200, 3000, 136), (77, 900, 264))
                            for f, more in ((xent_fwd_bytes, ()), (xent_bwd_bytes, (dev,)))), dtype=torch.uint8, device=dev)
    dy, ids = normal(5, 500, 136), tokens(6, 500, 3000)
    x, w = normal(7, 300, 1104), normal(8, 1104)
    need = max(embed_bytes(500, 136), ln_bytes(300, 1104, dev))
    assert space.numel() >= need

    def step(x_, w_, t_, g_):
        loss, lse = bil.linear_cross_entropy_fwd(x_, w_, t_, workspace=space)
        out = (loss, lse) + bil.linear_cross_entropy_bwd(x_, w_, t_, lse, g_, workspace=space)
        _, _, mean, rstd = bil.layer_norm_fwd(x, w)
        ln = bil.layer_norm_bwd(x, x, w, mean, rstd, workspace=space)
        return out + (bil.embedding_bwd(dy, ids, 3000, workspace=space), ln[0], ln[2], ln[3])

    want = [step(*a), step(*b)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for args in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(*args))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(same(p, q) for p, q in zip(outs[i], want[i])), i


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,width,pad", [(333, 512, 0), (333, 301, 0), (700, 4096, 0), (700, 4097, 0), (333, 1000, 7), (100, 9665, 0)])
def test_outputs_over_inputs(n, width, pad, dtype):
    """As the header allows: y over x and h over the residual, dx over dy and dresidual over dh, dropout over either."""
    lib, ld, code, s = _lib.load(), width + pad, _code(dtype), _stream_handle(0)
    x, r, dy, dh = (torch.empty(n, ld, dtype=dtype, device="cuda")[:, :width].copy_(normal(i, n, width, dtype=dtype))
                    for i in range(4))
    w, b = normal(5, width, dtype=dtype), normal(6, width, dtype=dtype)
    y, h, mean, rstd = bil.layer_norm_fwd(x, w, b, residual=r, p=0.2, seed=9)
    dx, dr, dw, db = bil.layer_norm_bwd(dy, h, w, mean, rstd, grad_h=dh, p=0.2, seed=9)
    d = bil.dropout_fwd(x, 0.2, 9, residual=r)
    for over in (x, r):
        xx, rr = (torch.empty(n, ld, dtype=dtype, device="cuda")[:, :width].copy_(t) for t in (x, r))
        out = xx if over is x else rr
        assert lib.bil_dropout(xx.data_ptr(), rr.data_ptr(), code, n, width, ld, ld, 0.2, 9, 0, None, out.data_ptr(), ld, s) == _lib.OK
        assert same(out, d)
    m2, s2, dw2, db2 = (torch.empty_like(t) for t in (mean, rstd, dw, db))
    hold = h.clone()
    assert lib.bil_layer_norm_fwd(x.data_ptr(), r.data_ptr(), w.data_ptr(), b.data_ptr(), code, code, n, width, ld, ld, 1e-5, 0.2,
                                  9, 0, None, x.data_ptr(), ld, r.data_ptr(), ld, m2.data_ptr(), s2.data_ptr(), s) == _lib.OK
    assert same(x, y) and same(r, hold) and same(m2, mean) and same(s2, rstd)
    need = ln_bytes(n, width, h.device)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert lib.bil_layer_norm_bwd(dy.data_ptr(), r.data_ptr(), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), dh.data_ptr(),
                                  code, code, n, width, ld, ld, ld, 0.2, 9, 0, None, dy.data_ptr(), ld, dh.data_ptr(), ld,
                                  dw2.data_ptr(), db2.data_ptr(), space.data_ptr(), need, s) == _lib.OK
    assert same(dy, dx) and same(dh, dr) and same(dw2, dw) and same(db2, db)


def test_rows_past_2_to_31_elements():
    """Offsets past 32 bits: the last rows of a large buffer are those of a small call."""
    n, width = 140000, 16000
    x = torch.empty(n, width, dtype=torch.bfloat16, device="cuda")
    x[:-50] = 1.0
    x[-50:] = normal(1, 50, width)
    w, b = normal(2, width), normal(3, width)
    y, _, mean, rstd = bil.layer_norm_fwd(x, w, b)
    want = bil.layer_norm_fwd(x[-50:], w, b)
    assert same(y[-50:], want[0]) and same(mean[-50:], want[2]) and same(rstd[-50:], want[3])
    dx = bil.layer_norm_bwd(x, x, w, mean, rstd)[0]
    assert same(dx[-50:], bil.layer_norm_bwd(x[-50:], x[-50:], w, want[2], want[3])[0])
    del dx, y
    d = bil.dropout_fwd(x, 0.5, 3)
    first = (n - 1) * ((width + 7) // 8)  # the last row's first group
    words = philox(np.array([[first % 2 ** 32, first // 2 ** 32, 0, 0]], dtype=np.uint64), (3, 0)).astype("<u4").view("<u2")[0]
    assert (d[-1, :8] != 0).tolist() == [bool(v >= border_of(0.5)) for v in words]


def test_a_table_past_2_to_31_elements():
    vocab, width = 600000, 4096
    w = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 3, vocab - 2, vocab - 1, 599000], device="cuda")
    w[ids] = normal(1, 5, width)
    y = bil.embedding_fwd(ids, w)
    assert same(y, w[ids])
    dy = normal(2, 5, width)
    dw = bil.embedding_bwd(dy, ids, vocab)
    assert same(dw[599000], dy[4]) and same(dw[vocab - 1], (dy[0].float() + dy[3].float()).bfloat16())
    assert int((dw != 0).any(dim=1).sum()) == 4
    # the LM head on it: its last rows are targets
    x = normal(3, 40, width)
    w[-1000:] = normal(4, 1000, width, scale=3 / 64)
    t = torch.randint(vocab - 1000, vocab, (40,), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    loss, lse = bil.linear_cross_entropy_fwd(x, w, t, reduction="none")
    # In 64 bits, the rows that are not zero and a logit of 0 for each of the others.  A logit's error by the bound of
    # the cross entropy's tests, (H / 16 + 1) 2^-23 (P + C) with prefix sums P and sums of 16 |products| C, twice for
    # lse and target (these logits reach 80: linear_logp, one accumulation, is 4e-4 off itself).
    used = torch.cat([ids[[1, 4]], torch.arange(vocab - 1000, vocab, device="cuda")])
    parts = torch.stack([x[:, k:k + 16].double() @ w[used, k:k + 16].double().t() for k in range(0, width, 16)])
    sizes = max(float((x[:, k:k + 16].double().abs() @ w[used, k:k + 16].double().abs().t()).max()) for k in range(0, width, 16))
    z = parts.sum(dim=0)
    bound = 2 * (width / 16 + 1) * 2.0 ** -23 * (float(parts.cumsum(dim=0).abs().max()) + sizes)
    lse64 = torch.cat([z, torch.full((40, 1), float(torch.tensor(vocab - len(used)).log()), device="cuda", dtype=torch.float64)],
                      dim=1).logsumexp(dim=1)
    want = lse64 - z.gather(1, (t - (vocab - 1000) + 2)[:, None])[:, 0]
    assert float((loss.double() - want).abs().max()) <= bound + 2.0 ** -16
    dh, dwt = bil.linear_cross_entropy_bwd(x, w, t, lse, torch.ones(40, device="cuda"), reduction="none")
    old_h, old_w = bil.linear_logp_bwd(x, w, t, lse, -torch.ones(40, device="cuda"))
    assert float((dh.double() - old_h.double()).norm() / old_h.double().norm()) <= 2.0 ** -7
    assert float((dwt[-1000:].double() - old_w[-1000:].double()).norm() / old_w.double().norm()) <= 2.0 ** -7


def test_refusals():
    x, w, t = normal(1, 6, 64), normal(2, 100, 64), tokens(3, 6, 100)
    v = normal(4, 64)
    g = torch.tensor(1.0, device="cuda")
    lse = torch.zeros(6, device="cuda")
    bad = [
        (ValueError, lambda: bil.layer_norm_fwd(x, v[:-1])),
        (TypeError, lambda: bil.layer_norm_fwd(x, v.half())),
        (TypeError, lambda: bil.layer_norm_fwd(x, v, v.float())),
        (ValueError, lambda: bil.layer_norm_fwd(x, v, v, residual=x[:3])),
        (ValueError, lambda: bil.layer_norm_fwd(x, v, v, residual=x.float())),
        (ValueError, lambda: bil.layer_norm_fwd(x, v, v, p=1.0)),
        (ValueError, lambda: bil.layer_norm_bwd(x, x, v, lse[:3], lse)),
        (ValueError, lambda: bil.layer_norm_bwd(x, x, v, lse, lse, grad_h=x[:3])),
        (TypeError, lambda: bil.layer_norm_fwd(x.long(), v)),
        (ValueError, lambda: bil.dropout_fwd(x, 0.5, torch.zeros(2, dtype=torch.int64))),
        (ValueError, lambda: bil.dropout_fwd(x, 0.5, torch.zeros(2, device="cuda"))),
        (TypeError, lambda: bil.dropout_fwd(x, 0.5, 1.5)),
        (TypeError, lambda: bil.dropout_fwd(x.to(torch.float64), 0.5, 1)),
        (TypeError, lambda: bil.embedding_fwd(t.float(), w)),
        (ValueError, lambda: bil.embedding_fwd(t, w[0])),
        (ValueError, lambda: bil.embedding(t, w, padding_idx=100)),
        (ValueError, lambda: bil.embedding_bwd(x, t[:3], 100)),
        (ValueError, lambda: bil.embedding_bwd(x, t, 100, padding_idx=-1)),
        (ValueError, lambda: bil.embedding_bwd(x, t, 100, accumulate=True)),
        (TypeError, lambda: bil.embedding_bwd(x, t, 100, out_dtype=torch.float16)),
        (ValueError, lambda: bil.embedding_bwd(x, t, 100, out=w[:50])),
        (ValueError, lambda: bil.embedding_bwd(x, t, 64, out=w[:64, :64].t())),
        (ValueError, lambda: bil.embedding_bwd(x, t, 100, out=w[:1].expand(100, 64))),
        (TypeError, lambda: bil.linear_cross_entropy_fwd(x.float(), w.float(), t)),
        (TypeError, lambda: bil.linear_cross_entropy_fwd(x, w.half(), t)),
        (ValueError, lambda: bil.linear_cross_entropy_fwd(x, w[:, :32], t)),
        (ValueError, lambda: bil.linear_cross_entropy_fwd(x, w, t[:3])),
        (TypeError, lambda: bil.linear_cross_entropy_fwd(x, w, t.float())),
        (ValueError, lambda: bil.linear_cross_entropy_fwd(x, w, t, reduction="max")),
        (ValueError, lambda: bil.linear_cross_entropy_fwd(x, w, t, label_smoothing=1.5)),
        (ValueError, lambda: bil.linear_cross_entropy_fwd(x[:, :63].contiguous(), w[:, :63].contiguous(), t)),
        (TypeError, lambda: bil.linear_cross_entropy_bwd(x, w, t, lse, g, out_dtype=torch.float16)),
        (ValueError, lambda: bil.linear_cross_entropy_bwd(x, w, t, lse[:3], g)),
        (ValueError, lambda: bil.linear_cross_entropy_bwd(x, w, t, lse, lse)),
        (ValueError, lambda: bil.linear_cross_entropy_bwd(x, w, t, lse, g, piece=0)),
        (ValueError, lambda: bil.linear_cross_entropy_bwd(x, w, t, lse, g, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            raise AssertionError(f"call {i} was not refused")


# ---------------------------------------------------------------------------
# The operators in a row, as a training step uses them.
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tied_step", os.path.join(ROOT, "examples", "tied_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_loss(params, ids, targets, rng, p, scale, smoothing, z_loss):
    """The chain in 64 bits under the tests' own masks."""
    n, hidden = len(ids), params["table"].shape[1]

    def mask(step):
        keep = torch.from_numpy(keep_mask(n, hidden, p, rng[0], rng[1] + step)).cuda()
        return keep.double() * (65536 / (65536 - border_of(p)))

    def norm(x, w, b):
        c = x - x.mean(dim=1, keepdim=True)
        return c / (c.square().mean(dim=1, keepdim=True) + 1e-5).sqrt() * w + b

    x = params["table"][ids] * scale * mask(0)
    y = norm(x, params["w1"], params["b1"])
    z = norm((y @ params["block"].t()) * mask(1) + x, params["w2"], params["b2"]) @ params["table"].t()
    lse = z.logsumexp(dim=1)
    act = targets != bil.IGNORE_INDEX
    rows = lse - (1 - smoothing) * z.gather(1, targets.clamp_min(0)[:, None])[:, 0] - smoothing * z.mean(dim=1) + z_loss * lse ** 2
    return (rows * act).sum() / act.sum()


@pytest.mark.parametrize("n,vocab,hidden", [(300, 2000, 256), (97, 1003, 136)])
def test_tied_step(example, n, vocab, hidden):
    torch.manual_seed(3)
    params = example.parameters(vocab, hidden)
    ids, targets = tokens(1, n, vocab), tokens(2, n, vocab)
    targets[::9] = bil.IGNORE_INDEX
    rng = torch.tensor([99, 4], device="cuda")
    how = {"p": 0.2, "scale": 8.0, "label_smoothing": 0.1, "z_loss": 1e-3}
    value, grads = example.step(params, ids, targets, rng, torch.ones((), device="cuda"), **how)
    ref = {k: v.double().requires_grad_() for k, v in params.items()}
    want = plain_loss(ref, ids, targets, (99, 4), 0.2, 8.0, 0.1, 1e-3)
    want_grads = dict(zip(ref, torch.autograd.grad(want, list(ref.values()))))
    assert abs(float(value) - float(want.detach())) <= 2.0 ** -6
    for k, g in grads.items():
        assert float((g.double() - want_grads[k]).norm()) <= 2.0 ** -5 * float(want_grads[k].norm()), k
    # autograd gives the same calls in the same order, but for the order of the table's two gradients
    leaves = {k: v.clone().requires_grad_() for k, v in params.items()}
    loss = example.loss(leaves, ids, targets, rng, **how)
    assert same(loss, value)
    auto = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    for k, g in auto.items():
        assert float((g.double() - grads[k].double()).norm()) <= 2.0 ** -7 * float(grads[k].double().norm()), k


def test_main_runs(example, capsys):
    example.main()
    assert capsys.readouterr().out.count("loss") == 5
