"""Cases of the operators at the two ends of a language model's training step, for measurement.

Four operators, each in its forms:

  embed  rows of an embedding table by token with a scale ("fwd"), and the same
         followed by the table's gradient, dense, every row of it ("step");
  norm   layer norm of a residual stream, with dropout of what joins the stream
         and the residual's addition ("fwd"), and the same followed by the
         gradients of the rows, the weight and the bias ("step");
  drop   dropout from a counter-based generator, with a residual or without,
         and its gradient ("step": the mask is made twice and never stored);
  xent   the LM head's projection and softmax cross entropy with label smoothing
         and a penalty on lse^2 ("loss"), and the same followed by the gradients
         of the hidden states and the weight ("step"), without the logits.

``run`` computes the plain form, or with ``own`` the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100
V, H = 151936, 4096  # the benchmark's vocabulary and the LM head's hidden size
EPS = 1e-5

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # The tokens of a decoding batch. Latency.
        _embed("embed_decode", 64, V, H, "bf16", scale=64.0),
        # A training batch: the lookup, and the gradient of the whole table.
        _embed("embed_step", 16384, V, H, "bf16", step=True),
        # A small odd vocabulary in float32, padding tokens, rows of a wider buffer.
        _embed("embed_step_odd", 5003, 32003, 1105, "f32", scale=0.5, step=True, padding=0, pad=7),
        # The norm of a few decoded tokens. Latency.
        _norm("norm_decode", 8, H, "bf16"),
        # A training step over a whole batch.
        _norm("norm_step", 16384, H, "bf16", step=True),
        # The same with dropout of the branch that joins the stream.
        _norm("norm_drop_step", 16384, H, "bf16", step=True, p=0.1),
        # Odd width, rows of a wider buffer, no residual, no bias.
        _norm("norm_step_odd", 1023, 5001, "f16", step=True, residual=False, bias=False, pad=7),
        # Dropout of embedded tokens, a small batch.
        _drop("drop_small", 128, 1104, "bf16", p=0.1),
        # Dropout of a branch of a training batch with the residual's addition, and back.
        _drop("drop_step", 16384, H, "bf16", p=0.1, residual=True),
        # The loss of a small batch over a small vocabulary, and its gradients.
        _xent("xent_step_small", 64, 32003, 1104, "bf16"),
        # Odd sizes, label smoothing, the penalty on lse^2, half precision with a scaled loss.
        _xent("xent_step_ragged", 333, 32003, 1104, "f16", smoothing=0.1, z_loss=1e-4, reduction="sum", grad=64.0),
        # The loss of the benchmark's training batch and its gradients. Bound by the matrix products.
        _xent("xent_step", 16384, V, H, "bf16", z_loss=1e-4),
    ]


def _embed(name, n, vocab, width, dtype, scale=1.0, step=False, padding=-1, pad=0):
    return {"name": name, "op": "embed", "n": n, "vocab": vocab, "width": width, "dtype": dtype, "scale": scale,
            "step": step, "padding": padding, "pad": pad}


def _norm(name, n, width, dtype, step=False, residual=True, bias=True, p=0.0, pad=0):
    return {"name": name, "op": "norm", "n": n, "width": width, "dtype": dtype, "step": step, "residual": residual,
            "bias": bias, "p": p, "pad": pad}


def _drop(name, n, width, dtype, p, residual=False, pad=0):
    return {"name": name, "op": "drop", "n": n, "width": width, "dtype": dtype, "p": p, "residual": residual, "pad": pad}


def _xent(name, n, vocab, width, dtype, step=True, smoothing=0.0, z_loss=0.0, reduction="mean", grad=1.0):
    return {"name": name, "op": "xent", "n": n, "vocab": vocab, "width": width, "dtype": dtype, "step": step,
            "smoothing": smoothing, "z_loss": z_loss, "reduction": reduction, "grad": grad}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["embed", "norm", "drop", "xent"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    pad = rng.choice([0, 0, 7, 64])
    p = rng.choice([0.05, 0.1, 0.3, 0.5])
    if op == "embed":
        c = _embed("", _log_int(rng, 1, 16384), _log_int(rng, 1000, V), _log_int(rng, 64, H), dtype,
                   rng.choice([1.0, 0.5, 64.0]), rng.random() < 0.7, rng.choice([-1, -1, 0, 3]), pad)
        if dtype == "f32":
            c["vocab"] = max(1000, c["vocab"] // 2)
    elif op == "norm":
        c = _norm("", _log_int(rng, 1, 16384), _log_int(rng, 64, 8192), dtype, rng.random() < 0.7, rng.random() < 0.7,
                  rng.random() < 0.7, rng.choice([0.0, p]), pad)
    elif op == "drop":
        c = _drop("", _log_int(rng, 1, 16384), _log_int(rng, 64, 8192), dtype, p, rng.random() < 0.5, pad)
    else:
        n = _log_int(rng, 1, 4096)
        c = _xent("", n, _log_int(rng, 1000, V), 8 * _log_int(rng, 8, H // 8), rng.choice(["bf16", "f16"]),
                  rng.random() < 0.8, rng.choice([0.0, 0.0, 0.1]), rng.choice([0.0, 1e-4]),
                  rng.choice(["mean", "sum", "none"]))
        if c["dtype"] == "f16":  # a scaled loss keeps the gradients of a mean inside the type's range
            c["grad"] = 64.0 * n if c["reduction"] == "mean" else 64.0
    if op in ("norm", "drop") and c["n"] * c["width"] > 16384 * H // (2 if dtype == "f32" else 1):
        c["n"] = 16384 * H // (2 if dtype == "f32" else 1) // c["width"]
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, width, dtype = case["n"], case["width"], _TYPES[case["dtype"]]
    state = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rows(count=n, scale=1.0):
        buf = torch.empty(count, width + case.get("pad", 0), dtype=dtype, device="cuda")
        buf[:, :width] = scale * normal(count, width)
        return buf[:, :width]

    # what a program draws its masks from: a seed, and the step that it is at
    state["rng"] = torch.randint(0, 2 ** 40, (2,), generator=gen, device="cuda")
    if case["op"] == "embed":
        # a token's frequency falls with its number, as a vocabulary is laid out
        u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(case["vocab"] + 1)).long() - 1).clamp_(0, case["vocab"] - 1)
        state |= {"ids": ids, "weight": rows(case["vocab"], 0.02)}
        if case["step"]:
            state["dy"] = rows()
    elif case["op"] == "norm":
        state |= {"x": rows(), "r": rows(scale=4.0) if case["residual"] else None,
                  "w": (1 + 0.1 * normal(width)).to(dtype), "b": (0.1 * normal(width)).to(dtype) if case["bias"] else None}
        if case["step"]:
            state |= {"dy": rows(), "dh": rows() if case["residual"] else None}
    elif case["op"] == "drop":
        state |= {"x": rows(), "r": rows(scale=4.0) if case["residual"] else None, "dy": rows()}
    else:
        t = torch.randint(0, case["vocab"], (n,), generator=gen, device="cuda")
        if n >= 20:  # 5% of the rows are ignored
            t[torch.randperm(n, generator=gen, device="cuda")[:n // 20]] = IGNORE
        state |= {"x": normal(n, width).to(dtype), "w": (normal(case["vocab"], width) * (3 / math.sqrt(width))).to(dtype),
                  "targets": t}
        g = torch.tensor(float(case["grad"]), device="cuda")
        state["g"] = g * normal(n) if case["reduction"] == "none" else g
    return state


# ---------------------------------------------------------------------------
# The plain forms.
# ---------------------------------------------------------------------------

def _mul_high_low(a, b):
    """The two 32-bit halves of the 64-bit products of a constant and whole numbers below 2^32."""
    part = a * (b & 0xffff)
    upper = a * (b >> 16) + (part >> 16)
    return upper >> 16, ((upper & 0xffff) << 16) | (part & 0xffff)


def _philox_round(c, k):
    h0, l0 = _mul_high_low(0xD2511F53, c[0])
    h1, l1 = _mul_high_low(0xCD9E8D57, c[2])
    return [h1 ^ c[1] ^ k[0], l1, h0 ^ c[3] ^ k[1], l0], [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]


def _keep(rng, n, width, p):
    """Which elements of [n, width] stay, and what those are multiplied by.

    Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) with the seed as its key.
    Elements 8j to 8j + 7 of a row are the eight 16-bit parts of the four words for
    the counter (j, row, step): row ceil(width / 8) + j in its lower 64 bits, the
    step in its upper. An element stays where its 16 bits are at least p 2^16."""
    groups = -(-width // 8)
    at = torch.arange(n * groups, device=rng.device)
    low, high = rng & 0xffffffff, (rng >> 32) & 0xffffffff
    c, k = [at & 0xffffffff, at >> 32, low[1], high[1]], [low[0], high[0]]
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    c, k = _philox_round(c, k)
    words = torch.stack(c, dim=1)
    parts = torch.stack((words & 0xffff, words >> 16), dim=2).view(n, groups * 8)[:, :width]
    border = round(p * 65536)
    return parts >= border, 65536 / (65536 - border)


def _dropped(x, rng, p):
    keep, times = _keep(rng, *x.shape, p)
    return torch.where(keep, x.float() * times, torch.zeros((), device=x.device))


def _plain_embed(s):
    c, ids, w = s["case"], s["ids"], s["weight"]
    out = {"y": (w[ids].float() * c["scale"]).to(w.dtype)}
    if c["step"]:
        g = torch.where((ids != c["padding"])[:, None], s["dy"].float(), torch.zeros((), device=w.device))
        table = torch.zeros(w.shape, dtype=torch.float32, device=w.device).index_add_(0, ids, g)
        out["dweight"] = (table * c["scale"]).to(w.dtype)
    return out


def _plain_norm(s):
    c, x, r, w = s["case"], s["x"], s["r"], s["w"].float()
    p, out = c["p"], {}
    hf = _dropped(x, s["rng"], p) if p else x.float()
    if r is not None:
        hf = hf + r.float()
    if p or r is not None:  # the stream goes on in its own type
        out["h"] = hf.to(x.dtype)
        hf = out["h"].float()
    mean = hf.mean(dim=1, keepdim=True)
    centred = hf - mean
    rstd = 1 / torch.sqrt((centred * centred).mean(dim=1, keepdim=True) + EPS)
    u = centred * rstd
    y = u * w
    if s["b"] is not None:
        y = y + s["b"].float()
    out |= {"y": y.to(x.dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if c["step"]:
        dy = s["dy"].float()
        v = dy * w
        d = rstd * (v - v.mean(dim=1, keepdim=True) - u * (v * u).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            d = d + s["dh"].float()
        out |= {"dx": (_dropped(d, s["rng"], p) if p else d).to(x.dtype), "dw": (dy * u).sum(dim=0)}
        if p and r is not None:
            out["dr"] = d.to(x.dtype)
        if s["b"] is not None:
            out["db"] = dy.sum(dim=0)
    return out


def _plain_drop(s):
    x, r, p = s["x"], s["r"], s["case"]["p"]
    y = _dropped(x, s["rng"], p)
    if r is not None:
        y = y + r.float()
    return {"y": y.to(x.dtype), "dx": _dropped(s["dy"], s["rng"], p).to(x.dtype)}


def _plain_xent(s):
    c, x, w, t = s["case"], s["x"], s["w"], s["targets"]
    eps, vocab = c["smoothing"], c["vocab"]
    zero = torch.zeros((), device=x.device)
    z = x.float() @ w.float().t()
    m = z.amax(dim=1)
    lse = m + (z - m[:, None]).exp().sum(dim=1).log()
    active = t != IGNORE
    at = t.clamp_min(0)[:, None]
    loss = lse - (1 - eps) * z.gather(1, at)[:, 0] + c["z_loss"] * lse * lse
    if eps:
        loss = loss - eps * z.mean(dim=1, dtype=torch.float64).float()
    loss = torch.where(active, loss, zero)
    g = torch.where(active, s["g"], zero)
    if c["reduction"] != "none":
        loss = loss.sum()
        if c["reduction"] == "mean":
            count = active.sum().clamp_min(1)
            loss, g = loss / count, g / count
    out = {"loss": loss}
    if c["step"]:
        d = z.sub_(lse[:, None]).exp_().mul_((g * (1 + 2 * c["z_loss"] * lse))[:, None])
        if eps:
            d -= (g * (eps / vocab))[:, None]
        d.scatter_add_(1, at, -(1 - eps) * g[:, None])
        out |= {"dx": (d @ w.float()).to(x.dtype), "dw": (d.t() @ x.float()).to(w.dtype)}
    return out


# ---------------------------------------------------------------------------
# The framework's kernels.
# ---------------------------------------------------------------------------

def _own_embed(s):
    import invariant_token_log_gb300 as bil
    c = s["case"]
    out = {"y": bil.embedding_fwd(s["ids"], s["weight"], scale=c["scale"])}
    if c["step"]:
        out["dweight"] = bil.embedding_bwd(s["dy"], s["ids"], c["vocab"], scale=c["scale"],
                                           padding_idx=None if c["padding"] < 0 else c["padding"])
    return out


def _own_norm(s):
    import invariant_token_log_gb300 as bil
    c, x = s["case"], s["x"]
    p = c["p"]
    y, h, mean, rstd = bil.layer_norm_fwd(x, s["w"], s["b"], residual=s["r"], eps=EPS, p=p, seed=s["rng"] if p else 0)
    out = {} if h is None else {"h": h}
    out |= {"y": y, "mean": mean, "rstd": rstd}
    if c["step"]:
        dx, dr, dw, db = bil.layer_norm_bwd(s["dy"], x if h is None else h, s["w"], mean, rstd, grad_h=s["dh"],
                                            p=p, seed=s["rng"] if p else 0, need_bias=s["b"] is not None,
                                            need_residual=s["r"] is not None)
        out |= {"dx": dx, "dw": dw}
        if p and s["r"] is not None:
            out["dr"] = dr
        if db is not None:
            out["db"] = db
    return out


def _own_drop(s):
    import invariant_token_log_gb300 as bil
    p = s["case"]["p"]
    return {"y": bil.dropout_fwd(s["x"], p, s["rng"], residual=s["r"]), "dx": bil.dropout_bwd(s["dy"], p, s["rng"])}


def _own_xent(s):
    import invariant_token_log_gb300 as bil
    c = s["case"]
    how = {"ignore_index": IGNORE, "label_smoothing": c["smoothing"], "z_loss": c["z_loss"], "reduction": c["reduction"]}
    loss, lse = bil.linear_cross_entropy_fwd(s["x"], s["w"], s["targets"], **how)
    out = {"loss": loss}
    if c["step"]:
        out["dx"], out["dw"] = bil.linear_cross_entropy_bwd(s["x"], s["w"], s["targets"], lse, s["g"], **how)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"embed": _own_embed, "norm": _own_norm, "drop": _own_drop, "xent": _own_xent}[op](state)
    return {"embed": _plain_embed, "norm": _plain_norm, "drop": _plain_drop, "xent": _plain_xent}[op](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------

def _exact_factor(rng, n, width, p):
    """Of each element of [n, width]: 0, or what dropout multiplies it by."""
    seed, step = (int(v) for v in rng.cpu())
    u64, mask = np.uint64, np.uint64(0xffffffff)
    lanes = np.arange(n * ((width + 7) // 8), dtype=u64)
    x = [lanes & mask, lanes >> u64(32), np.full_like(lanes, step & 0xffffffff), np.full_like(lanes, (step >> 32) & 0xffffffff)]
    key = [seed & 0xffffffff, (seed >> 32) & 0xffffffff]
    for _ in range(10):
        first, second = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
        x = [(second >> u64(32)) ^ x[1] ^ u64(key[0]), second & mask, (first >> u64(32)) ^ x[3] ^ u64(key[1]), first & mask]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.stack(x, axis=1).astype("<u4").view("<u2").reshape(n, -1)[:, :width]
    border = round(p * 65536)
    factor = np.where(bits < border, 0.0, 65536 / (65536 - border))
    return torch.from_numpy(np.ascontiguousarray(factor)).cuda()


def _exact_norm(s):
    c, x, w, b = s["case"], s["x"].double(), s["w"].double(), s["b"]
    factor = _exact_factor(s["rng"], *x.shape, c["p"]) if c["p"] else None
    out = {}
    if factor is not None:
        x = x * factor
    if s["r"] is not None:
        x = x + s["r"].double()
    if factor is not None or s["r"] is not None:
        # the stream is kept in the inputs' type: that rounding (of the float32 sum) is part of the definition
        out["h"] = x.float().to(s["x"].dtype).double()
        x = out["h"]
    std, mu = torch.std_mean(x, dim=1, correction=0, keepdim=True)
    size = torch.hypot(std, torch.full_like(std, math.sqrt(EPS)))
    unit = (x - mu) / size
    out |= {"y": unit * w + (0.0 if b is None else b.double()), "mean": mu[:, 0], "rstd": 1 / size[:, 0]}
    if c["step"]:
        dy = s["dy"].double()
        along = dy * w
        along = along - along.mean(dim=1, keepdim=True)  # orthogonal to the ones, then to the unit rows
        d = (along - unit * (along * unit).sum(dim=1, keepdim=True) / x.shape[1]) / size
        d = d + (0.0 if s["dh"] is None else s["dh"].double())
        out |= {"dx": d if factor is None else d * factor, "dw": torch.einsum("nc,nc->c", dy, unit)}
        if factor is not None and s["r"] is not None:
            out["dr"] = d
        if b is not None:
            out["db"] = dy.sum(dim=0)
    return out


def _exact_xent(s):
    c, x, w, t = s["case"], s["x"].double(), s["w"].double(), s["targets"]
    if 6 * x.shape[0] * w.shape[0] * x.shape[1] > 1e13:
        return None
    kept = (t >= 0).double()
    logits = x @ w.T
    lse = torch.logsumexp(logits, dim=1)
    # the target distribution: what the smoothing leaves on the target, the rest spread evenly
    q = torch.full_like(logits, c["smoothing"] / c["vocab"])
    rows = torch.arange(len(t), device=t.device)
    q[rows, t.clamp_min(0)] += 1 - c["smoothing"]
    loss = kept * (-(q * (logits - lse[:, None])).sum(dim=1) + c["z_loss"] * lse ** 2)
    weight = kept * s["g"].double()
    if c["reduction"] == "mean":
        loss, weight = loss / max(1.0, float(kept.sum())), weight / max(1.0, float(kept.sum()))
    out = {"loss": loss if c["reduction"] == "none" else loss.sum()}
    if c["step"]:
        d = weight[:, None] * (torch.softmax(logits, dim=1) * (1 + 2 * c["z_loss"] * lse[:, None]) - q)
        out |= {"dx": d @ w, "dw": d.T @ x}
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = {"y": torch.nn.functional.embedding(s["ids"], s["weight"].double()) * case["scale"]}
        if case["step"]:
            counted = s["ids"] != case["padding"]
            out["dweight"] = torch.zeros(s["weight"].shape, dtype=torch.float64, device="cuda")
            out["dweight"].index_put_((s["ids"][counted],), s["dy"].double()[counted] * case["scale"], accumulate=True)
        return out
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "drop":
        factor = _exact_factor(s["rng"], *s["x"].shape, case["p"])
        y = s["x"].double() * factor
        return {"y": y if s["r"] is None else y + s["r"].double(), "dx": s["dy"].double() * factor}
    return _exact_xent(s)


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------

def work(case):
    n, width, e = case["n"], case["width"], 4 if case["dtype"] == "f32" else 2
    elements = n * width
    if case["op"] == "embed":
        # the distinct rows that n tokens name, on average
        ranks = np.arange(1, case["vocab"] + 1)
        share = np.log1p(1 / ranks) / math.log(case["vocab"] + 1)
        distinct = float(np.sum(-np.expm1(n * np.log1p(-share))))
        by, flops = 8 * n + distinct * width * e + elements * e, elements
        if case["step"]:
            by += elements * e + case["vocab"] * width * e
            flops += 2 * elements
        return {"bytes": by, "flops": flops}
    if case["op"] == "norm":
        stored = case["residual"] or case["p"] > 0  # the stream
        streams = 2 + (1 if case["residual"] else 0) + (1 if stored else 0)
        by, flops = 8 * n + width * e * (2 if case["bias"] else 1), 8 * elements
        if case["step"]:  # dy, the stream again, its own gradient; dx, and the residual's apart where there is a mask
            streams += 3 + (1 if case["residual"] else 0) + (1 if case["residual"] and case["p"] > 0 else 0)
            by += 8 * n + width * (e + (8 if case["bias"] else 4))
            flops += 13 * elements
        return {"bytes": elements * streams * e + by, "flops": flops + (24 if case["step"] else 12) * elements * (case["p"] > 0)}
    if case["op"] == "drop":  # ten rounds of a generator for eight elements
        return {"bytes": elements * e * (5 if case["residual"] else 4), "flops": 24 * elements}
    v = case["vocab"]
    by, flops = (elements + v * width) * e + 12 * n, 2 * n * v * width + 4 * n * v
    if case["step"]:  # the two products of the gradients; without the logits the projection's is done again besides
        by += (elements + v * width) * e
        flops += 4 * n * v * width + 4 * n * v
    return {"bytes": by, "flops": flops}
