"""The calls around the LM head in CUDA graphs and on several host threads' streams:
the bits of eager calls, one after the other."""
import threading

import pytest
import torch

import invariant_token_log_gb300 as bil
from gpu_helpers import check_watchdog

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    yield
    check_watchdog()


def bits(x):
    x = x.detach().contiguous()
    return x if x.dtype == torch.int64 else x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.itemsize])


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")).to(dtype)


def ids(seed, n, vocab):
    t = torch.randint(0, vocab, (n,), generator=torch.Generator(device="cuda").manual_seed(seed + 1000), device="cuda")
    t[::6] = bil.IGNORE_INDEX
    return t


class Alternatives:
    """Forward and backward: few rows (a cluster a row) or more (two kernels and a workspace)."""
    def __init__(self, n, vocab, dtype, k=20):
        self.n, self.vocab, self.dtype, self.k = n, vocab, dtype, k

    def inputs(self, seed):
        return (normal(seed, self.n, self.vocab, dtype=self.dtype, scale=3.0), ids(seed, self.n, self.vocab),
                normal(seed + 1, self.n, dtype=torch.float32), normal(seed + 2, self.n, self.k, dtype=torch.float32))

    def run(self, x, t, g, gk):
        logp, lse, ent, top_ids, top = bil.logp_topk(x, t, self.k, temperature=0.9, return_entropy=True)
        d = bil.logp_topk_bwd(x, t, top_ids, lse, g, gk, temperature=0.9, entropy=ent, grad_entropy=g)
        return logp, lse, ent, top_ids, top, d


class Norm:
    """Forward, backward and both 8-bit forms, of rows of whole 16-byte units and of others."""
    def __init__(self, n, width, dtype):
        self.n, self.width, self.dtype = n, width, dtype

    def inputs(self, seed):
        return tuple(normal(seed + i, self.n, self.width, dtype=self.dtype) for i in range(4)) + (
            normal(seed + 4, self.width, dtype=self.dtype),)

    def run(self, x, r, dy, dh, w):
        y, h, rstd = bil.rms_norm_fwd(x, w, r)
        dx, dw = bil.rms_norm_bwd(dy, h, w, rstd, dh)
        q, scale, h8 = bil.rms_norm_quant(x, w, r)
        q2, scale2 = bil.quantize_rows(x)
        return y, h, rstd, dx, dw, q, scale, h8, q2, scale2


class Head8:
    """Single blocks a tile, or pairs."""
    def __init__(self, n, width, vocab):
        self.n, self.width, self.vocab = n, width, vocab

    def inputs(self, seed):
        hq, hs = bil.quantize_rows(normal(seed, self.n, self.width))
        wq, ws = bil.quantize_rows(normal(seed + 1, self.vocab, self.width, scale=3.0 * self.width ** -0.5))
        return hq, hs, wq, ws, ids(seed, self.n, self.vocab)

    def run(self, *operands):
        return bil.linear_logp_fp8(*operands, return_entropy=True, return_logits=True)


CALLS = {
    "alternatives, few rows": Alternatives(5, 40000, torch.bfloat16),
    "alternatives, more rows": Alternatives(100, 9001, torch.float16),
    "alternatives, float32": Alternatives(12, 33000, torch.float32),
    "norm": Norm(300, 4096, torch.bfloat16),
    "norm, off boundaries": Norm(40, 1001, torch.float32),
    "norm, a warp a row": Norm(1000, 256, torch.float16),
    "8-bit head": Head8(70, 512, 3000),
    "8-bit head, pairs": Head8(300, 2048, 2000),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_captured_into_a_graph(call):
    """Captured once, replayed on other inputs in the same buffers."""
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
            assert torch.equal(bits(a), bits(b)), (seed, i)


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
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, want[i])), i
