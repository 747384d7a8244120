"""Cases of the operators around the selected-token log-probability, for measurement.

Three operators, each in its forms:

  topk   logp, lse, entropy and the k largest alternatives of each row of
         logits ("fwd"), and the same followed by the gradient of all of them
         ("step");
  norm   root-mean-square norm of a residual stream with the residual's
         addition: an 8-bit output with a scale per row ("quant"), or an output
         in the inputs' type followed by the backward pass ("step");
  head   the LM head on 8-bit (e4m3) hidden states and weight with a scale per
         row of each: logp, lse and entropy, and the logits where asked.

``run`` computes the plain form, or with ``own`` the framework's kernels.
"""
import math

import torch

own = False

IGNORE = -100
V, V_PADDED, H = 151936, 155648, 4096  # the benchmark's vocabulary, its padded row and the LM head's hidden size
EPS = 1e-6
E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -100  # an all-zero row keeps a positive scale

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # One sequence being decoded: a single row of the full vocabulary. Latency.
        _topk("topk_decode_1", 1, V, V, "bf16", k=20),
        # Constrained decoding of a batch: a grammar's mask leaves from no column to all of
        # them, rows padded to the tile, sampling temperature.
        _topk("topk_decode_64", 64, V, V_PADDED, "bf16", k=5, temperature=0.7, masked=True),
        # Scoring a prompt with the alternatives a server reports, some rows ignored.
        _topk("topk_score", 4096, V, V_PADDED, "bf16", k=20),
        # A distillation step on a small odd vocabulary, float32 logits, many alternatives.
        _topk("topk_step_odd", 515, 32003, 32003, "f32", k=100, temperature=1.3, step=True),
        # A training step with gradients through the alternatives.
        _topk("topk_step", 4096, V, V, "bf16", k=8, step=True),
        # The norm before the LM head for a few decoded tokens. Latency.
        _norm("norm_quant_decode", 8, H, "bf16", form="quant"),
        # The same for a whole prefill batch.
        _norm("norm_quant_prefill", 16384, H, "bf16", form="quant"),
        # A training step over a whole batch.
        _norm("norm_step", 16384, H, "bf16", form="step"),
        # Odd width, rows of a wider buffer, no residual.
        _norm("norm_step_odd", 1023, 5001, "f16", form="step", residual=False, pad=7),
        # One decoded token against the whole 8-bit weight. Bound by reading it.
        _head("head_decode_1", 1, V, H),
        # Scoring a prompt: bound by the matrix product.
        _head("head_score", 4096, V, H),
        # Odd sizes, temperature, logits kept for a later pass.
        _head("head_ragged", 333, 32003, 1104, temperature=0.7, logits=True),
    ]


def _topk(name, n, vocab, ld, dtype, k, temperature=1.0, masked=False, step=False):
    return {"name": name, "op": "topk", "n": n, "vocab": vocab, "ld": ld, "dtype": dtype, "k": k,
            "temperature": temperature, "masked": masked, "step": step}


def _norm(name, n, width, dtype, form, residual=True, pad=0):
    return {"name": name, "op": "norm", "n": n, "width": width, "dtype": dtype, "form": form, "residual": residual,
            "pad": pad}


def _head(name, n, vocab, width, temperature=1.0, logits=False):
    return {"name": name, "op": "head", "n": n, "vocab": vocab, "width": width, "temperature": temperature,
            "logits": logits}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["topk", "topk", "norm", "norm", "head"])
    if op == "topk":
        vocab = _log_int(rng, 1000, V)
        c = _topk("", _log_int(rng, 1, 4096), vocab, vocab + rng.choice([0, 0, 1, 5, 64, 3712]),
                  rng.choice(["bf16", "bf16", "f16", "f32"]), _log_int(rng, 1, 128),
                  rng.choice([1.0, 1.0, 0.7, 1.3]), rng.random() < 0.3, rng.random() < 0.5)
    elif op == "norm":
        form = rng.choice(["quant", "step"])
        c = _norm("", _log_int(rng, 1, 16384), _log_int(rng, 64, 8192 if form == "quant" else 4096),
                  rng.choice(["bf16", "bf16", "f16", "f32"]), form, rng.random() < 0.7, rng.choice([0, 0, 7, 64]))
        if c["n"] * c["width"] > 16384 * H:
            c["n"] = 16384 * H // c["width"]
        if c["dtype"] == "f32":
            c["n"] = max(1, c["n"] // 2)
    else:
        c = _head("", _log_int(rng, 1, 4096), _log_int(rng, 1000, V), 16 * _log_int(rng, 4, H // 16),
                  rng.choice([1.0, 0.7, 1.3]), rng.random() < 0.3)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _targets(n, vocab, gen):
    t = torch.randint(0, vocab, (n,), generator=gen, device="cuda")
    if n >= 20:  # 5% of the rows are ignored
        t[torch.randperm(n, generator=gen, device="cuda")[:n // 20]] = IGNORE
    return t


def _quantise(x):
    """A row's e4m3 values and its scale, as a user's loader lays out a weight once."""
    scale = x.abs().amax(dim=1).clamp_min(MIN_AMAX) / E4M3_MAX
    q = torch.empty(x.shape[0], -(-x.shape[1] // 16) * 16, dtype=torch.float8_e4m3fn, device=x.device)
    q = q[:, :x.shape[1]]  # rows on 16-byte boundaries
    q.copy_((x / scale[:, None]).to(torch.float8_e4m3fn))
    return q, scale


def prepare(case, seed):
    gen = _generator(seed)
    n, state = case["n"], {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "topk":
        vocab, dtype = case["vocab"], _TYPES[case["dtype"]]
        x = torch.full((n, case["ld"]), -math.inf, dtype=dtype, device="cuda")  # pad columns hold -inf
        for i in range(0, n, 512):  # logits of standard deviation 3, as the benchmark's
            x[i:i + 512, :vocab] = 3 * normal(min(512, n - i), vocab)
        if case["masked"]:
            # the share of allowed columns differs from row to row; one row in 32 has none
            allowed = 10 ** (-5 * torch.rand(n, 1, generator=gen, device="cuda"))
            allowed[::32] = 0
            u = torch.rand(n, vocab, generator=gen, device="cuda")
            x[:, :vocab].masked_fill_(u >= allowed, -math.inf)
        t = _targets(n, vocab, gen)
        state |= {"x": x, "targets": t}
        if case["step"]:
            state |= {"g": normal(n), "gh": 0.1 * normal(n), "gk": normal(n, case["k"])}
    elif case["op"] == "norm":
        dtype, width = _TYPES[case["dtype"]], case["width"]

        def rows(scale=1.0):
            buf = torch.empty(n, width + case["pad"], dtype=dtype, device="cuda")
            buf[:, :width] = scale * normal(n, width)
            return buf[:, :width]

        state |= {"x": rows(), "r": rows(4.0) if case["residual"] else None,
                  "w": (1 + 0.1 * normal(width)).to(dtype)}
        if case["form"] == "step":
            state |= {"dy": rows(), "dh": rows() if case["residual"] else None}
    else:
        width = case["width"]
        hq, hs = _quantise(normal(n, width))
        wq, ws = _quantise(normal(case["vocab"], width) * (3 / math.sqrt(width)))
        state |= {"hq": hq, "hs": hs, "wq": wq, "ws": ws, "targets": _targets(n, case["vocab"], gen)}
    return state


# ---------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------

def _row_statistics(z, targets):
    """lse, entropy, logp of float32 rows z; zeros for ignored rows."""
    m = z.amax(dim=1)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    lse = m + (z - m[:, None]).exp().sum(dim=1).log()
    a = z - lse[:, None]
    p = a.exp()
    entropy = -torch.where(p > 0, p * a, p).sum(dim=1)
    active = targets != IGNORE
    logp = z.gather(1, targets.clamp_min(0)[:, None])[:, 0] - lse
    zero = torch.zeros_like(lse)
    return torch.where(active, logp, zero), torch.where(active, lse, zero), torch.where(active, entropy, zero)


def _plain_topk(s):
    c, x, t = s["case"], s["x"], s["targets"]
    vocab, k = c["vocab"], c["k"]
    x = x[:, :vocab].float()
    z = x / c["temperature"]
    logp, lse, entropy = _row_statistics(z, t)
    active = (t != IGNORE)[:, None]
    # whole numbers in the order of (value, lowest column first): no two are equal
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    columns = torch.arange(vocab, device=x.device)
    ids = torch.topk((order << 32) + (vocab - 1 - columns), k, dim=1)[1]
    top = torch.where(active, z.gather(1, ids) - lse[:, None], torch.zeros((), device=x.device))
    out = {"logp": logp, "lse": lse, "entropy": entropy, "ids": torch.where(active, ids, -1), "top": top}
    if c["step"]:
        g, gh, gk = s["g"], s["gh"], s["gk"]
        a = z - lse[:, None]
        p = a.exp()
        d = -(g + gk.sum(dim=1))[:, None] * p
        d -= gh[:, None] * torch.where(p > 0, p * (a + entropy[:, None]), p)
        d.scatter_add_(1, t.clamp_min(0)[:, None], g[:, None])
        d.scatter_add_(1, ids, gk)
        d = torch.where(active, d / c["temperature"], torch.zeros((), device=x.device))
        full = torch.zeros(s["x"].shape, dtype=s["x"].dtype, device=x.device)
        full[:, :vocab] = d.to(full.dtype)
        out["dlogits"] = full
    return out


def _plain_norm(s):
    c, x, r, w = s["case"], s["x"], s["r"], s["w"].float()
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    hf = h.float()
    rstd = 1 / torch.sqrt((hf * hf).mean(dim=1) + EPS)
    y = hf * rstd[:, None] * w
    out = {} if r is None else {"h": h}
    if c["form"] == "quant":
        scale = y.abs().amax(dim=1).clamp_min(MIN_AMAX) / E4M3_MAX
        return out | {"q": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale}
    dy = s["dy"].float()
    xhat = hf * rstd[:, None]
    wdy = dy * w
    dx = rstd[:, None] * (wdy - xhat * (wdy * xhat).mean(dim=1)[:, None])
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return out | {"y": y.to(x.dtype), "rstd": rstd, "dx": dx.to(x.dtype), "dw": (dy * xhat).sum(dim=0)}


def _plain_head(s):
    c = s["case"]
    logits = (s["hq"].float() @ s["wq"].float().t()) * s["hs"][:, None] * s["ws"]
    out = dict(zip(("logp", "lse", "entropy"), _row_statistics(logits / c["temperature"], s["targets"])))
    if c["logits"]:
        out["logits"] = logits
    return out


# ---------------------------------------------------------------------------
# The framework's kernels.
# ---------------------------------------------------------------------------

def _own_topk(s):
    import invariant_token_log_gb300 as bil
    c = s["case"]
    logp, lse, entropy, ids, top = bil.logp_topk(s["x"], s["targets"], c["k"], vocab=c["vocab"],
                                                 temperature=c["temperature"], return_entropy=True)
    out = {"logp": logp, "lse": lse, "entropy": entropy, "ids": ids, "top": top}
    if c["step"]:
        out["dlogits"] = bil.logp_topk_bwd(s["x"], s["targets"], ids, lse, s["g"], s["gk"], vocab=c["vocab"],
                                           temperature=c["temperature"], entropy=entropy, grad_entropy=s["gh"])
    return out


def _own_norm(s):
    import invariant_token_log_gb300 as bil
    x, r, w = s["x"], s["r"], s["w"]
    if s["case"]["form"] == "quant":
        q, scale, h = bil.rms_norm_quant(x, w, residual=r, eps=EPS)
        return {"q": q, "scale": scale} | ({} if r is None else {"h": h})
    y, h, rstd = bil.rms_norm_fwd(x, w, residual=r, eps=EPS)
    dx, dw = bil.rms_norm_bwd(s["dy"], x if r is None else h, w, rstd, grad_h=s["dh"])
    return {"y": y, "rstd": rstd, "dx": dx, "dw": dw} | ({} if r is None else {"h": h})


def _own_head(s):
    import invariant_token_log_gb300 as bil
    c = s["case"]
    got = bil.linear_logp_fp8(s["hq"], s["hs"], s["wq"], s["ws"], s["targets"], temperature=c["temperature"],
                              return_entropy=True, return_logits=c["logits"])
    return dict(zip(("logp", "lse", "entropy", "logits"), got))


def run(state):
    op = state["case"]["op"]
    if own:
        return {"topk": _own_topk, "norm": _own_norm, "head": _own_head}[op](state)
    return {"topk": _plain_topk, "norm": _plain_norm, "head": _plain_head}[op](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------

def _exact_softmax(z, targets):
    """log p in 64 bits by the library-free definition, with the rows' lse, entropy and logp."""
    top = z.max(dim=1, keepdim=True)[0].nan_to_num(neginf=0.0)
    lse = (z - top).exp().sum(dim=1, keepdim=True).log() + top
    logs = z - lse
    terms = logs.exp() * logs.clamp_min(-1e300)
    rows = torch.arange(len(z), device=z.device)
    kept = targets >= 0
    stats = {"logp": logs[rows, targets.clamp_min(0)], "lse": lse[:, 0], "entropy": -terms.sum(dim=1)}
    stats = {name: v.masked_fill(~kept, 0.0) for name, v in stats.items()}
    return logs, stats


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "topk":
        if case["n"] * case["vocab"] > 2 ** 30:
            return None
        t, vocab, k = s["targets"], case["vocab"], case["k"]
        z = s["x"][:, :vocab].double() / case["temperature"]
        logs, out = _exact_softmax(z, t)
        order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
        kept = (t >= 0)[:, None]
        out["top"] = logs.gather(1, order).masked_fill(~kept, 0.0)
        out["ids"] = order.masked_fill(~kept, -1)
        if case["step"]:
            # the gradient of the weighted sum, one log-probability at a time
            weight = torch.zeros_like(z).scatter_add_(1, order, s["gk"].double())
            weight.scatter_add_(1, t.clamp_min(0)[:, None], s["g"].double()[:, None])
            p = logs.exp()
            d = weight - p * weight.sum(dim=1, keepdim=True)
            d -= s["gh"].double()[:, None] * p * (logs.clamp_min(-1e300) + out["entropy"][:, None])
            d = (d / case["temperature"]).masked_fill(~kept, 0.0)
            out["dlogits"] = torch.nn.functional.pad(d, (0, case["ld"] - vocab))
        return out
    if case["op"] == "norm":
        x, w = s["x"].double(), s["w"].double()
        out = {}
        if s["r"] is not None:  # the stream is kept in the inputs' type: that rounding is part of the definition
            x = (s["x"].float() + s["r"].float()).to(s["x"].dtype).double()
            out["h"] = x
        size = (x.square().sum(dim=1, keepdim=True) / x.shape[1] + EPS).sqrt()
        unit = x / size
        if case["form"] == "quant":
            peak = (unit * w).abs().max(dim=1, keepdim=True)[0].clamp_min(MIN_AMAX)
            return out | {"q": unit * w * (E4M3_MAX / peak), "scale": peak[:, 0] / E4M3_MAX}
        dy = s["dy"].double()
        along = (dy * w * unit).sum(dim=1, keepdim=True) / x.shape[1]
        dx = (dy * w - unit * along) / size + (0.0 if s["dh"] is None else s["dh"].double())
        return out | {"y": unit * w, "rstd": 1 / size[:, 0], "dx": dx, "dw": (dy * unit).sum(dim=0)}
    z = (s["hq"].double() * s["hs"].double()[:, None]) @ (s["wq"].double() * s["ws"].double()[:, None]).t()
    out = _exact_softmax(z / case["temperature"], s["targets"])[1]
    if case["logits"]:
        out["logits"] = z
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------

def work(case):
    n = case["n"]
    if case["op"] == "topk":
        e = 4 if case["dtype"] == "f32" else 2
        k, elements = case["k"], n * case["vocab"]
        by = elements * e + n * 8 + n * (12 + 12 * k)
        flops = 5 * elements  # maximum, difference, exponential, two sums
        if case["step"]:  # the gradient needs the whole row's sums first: the logits again, and the gradient out
            by += elements * e + n * case["ld"] * e + n * (8 + 4 * k)
            flops += 5 * elements
        return {"bytes": by, "flops": flops}
    if case["op"] == "norm":
        e = 4 if case["dtype"] == "f32" else 2
        elements, width = n * case["width"], case["width"]
        streams = 3 if case["residual"] else 1  # x, residual in, stream out
        if case["form"] == "quant":
            return {"bytes": elements * (streams * e + 1) + 4 * n + width * e, "flops": 8 * elements}
        streams += 1 + 3 + (1 if case["residual"] else 0)  # y; dy, the stream again, dx; the stream's own gradient
        return {"bytes": elements * streams * e + 8 * n + width * (2 * e + 4), "flops": 16 * elements}
    v, width = case["vocab"], case["width"]
    by = n * width + v * width + 4 * (n + v) + n * (8 + 12) + (4 * n * v if case["logits"] else 0)
    return {"bytes": by, "flops": 2 * n * v * width + 5 * n * v}
