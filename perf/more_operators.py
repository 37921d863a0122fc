"""Cases of products with a model's weights that leave nothing large in
memory between them and what stands before or after them: products grouped by
expert over ragged rows with their gradients, the cross entropy of a large
vocabulary from hidden states, without logits, with its gradients, and
products of few rows with weights of 4 bits and group scales.

``listed`` gives the cases, ``prepare`` what a program has in hand before a
call, ``run`` one pass (the plain form in elementary torch operations, or with
``own`` the package's kernels), ``exact`` the same in 64 bits, ``work`` the
bytes and operations that a pass cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token through 8 of 64 small experts: a row each, where latency counts
        {"name": "grouped-1-token", "op": "grouped", "tokens": 1, "experts": 64, "top_k": 8, "cols": 2048, "rows": 1024,
         "dtype": "bf16", "padded": False},
        # a serving batch on few wide experts, in half precision: the weights are read once
        {"name": "grouped-batch", "op": "grouped", "tokens": 61, "experts": 8, "top_k": 2, "cols": 4096, "rows": 14336,
         "dtype": "fp16", "padded": False},
        # prompts on the 256 experts of 7168 x 2048 that the benchmark compresses; a buffer of fixed size, not filled
        {"name": "grouped-prompts", "op": "grouped", "tokens": 4096, "experts": 256, "top_k": 8, "cols": 7168, "rows": 2048,
         "dtype": "bf16", "padded": True},
        # a short fine-tuning step on small experts
        {"name": "grouped-gradient-short", "op": "grouped_gradient", "tokens": 301, "experts": 16, "top_k": 2, "cols": 768,
         "rows": 2304, "dtype": "fp16", "padded": True},
        # a fine-tuning batch on wide experts
        {"name": "grouped-gradient-batch", "op": "grouped_gradient", "tokens": 8192, "experts": 8, "top_k": 2, "cols": 4096,
         "rows": 14336, "dtype": "bf16", "padded": False},
        # the loss of one answer's token, small model
        {"name": "loss-1-token", "op": "loss", "m": 1, "vocab": 50257, "cols": 768, "dtype": "bf16"},
        # scoring a batch of single tokens
        {"name": "loss-batch", "op": "loss", "m": 61, "vocab": 128256, "cols": 4096, "dtype": "bf16"},
        # scoring whole prompts
        {"name": "loss-prompts", "op": "loss", "m": 4096, "vocab": 128256, "cols": 4096, "dtype": "bf16"},
        # a short fine-tuning step of a small model, in half precision with a scaled loss
        {"name": "loss-gradient-short", "op": "loss_gradient", "m": 100, "vocab": 50257, "cols": 768, "dtype": "fp16",
         "penalty": False},
        # a whole fine-tuning batch, with a penalty on the size of the logits (a gradient of lse)
        {"name": "loss-gradient-batch", "op": "loss_gradient", "m": 4096, "vocab": 128256, "cols": 4096, "dtype": "bf16",
         "penalty": True},
        # one new token through a projection of 4096 x 4096 held in 4 bits, where latency counts
        {"name": "4bit-1-token", "op": "4bit", "m": 1, "rows": 4096, "cols": 4096, "group": 64, "dtype": "bf16", "zeros": False},
        # a serving batch through a wide projection, with zero points
        {"name": "4bit-batch", "op": "4bit", "m": 61, "rows": 14336, "cols": 4096, "group": 128, "dtype": "fp16", "zeros": True},
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high + 1)))
    return max(low, min(high, int(v / step) * step))


def draw(rng):
    op = rng.choice(["grouped", "grouped_gradient", "loss", "loss_gradient", "4bit"])
    if op == "4bit":
        group = rng.choice([32, 64, 128])
        return {"op": op, "m": _spread(rng, 1, 64), "rows": _spread(rng, 256, 14336), "cols": _spread(rng, 256, 14336, group),
                "group": group, "dtype": rng.choice(["bf16", "fp16"]), "zeros": rng.random() < 0.5}
    if op.startswith("grouped"):
        cols, rows, top_k = _spread(rng, 256, 7168, 8), _spread(rng, 256, 14336, 8), _spread(rng, 1, 8)
        experts = _spread(rng, top_k, max(top_k, min(256, (7 << 29) // (cols * rows))))
        most = 16384 * 4096 * 14336 // (cols * rows * top_k)  # products of the largest listed case
        return {"op": op, "tokens": _spread(rng, 1, max(1, min(65536 // top_k, most))), "experts": experts, "top_k": top_k,
                "cols": cols, "rows": rows, "dtype": rng.choice(["bf16", "fp16"]), "padded": rng.random() < 0.5}
    vocab, cols = _spread(rng, 1000, 128256), _spread(rng, 256, 7168, 8)
    most = 4096 * 128256 * 4096 // (vocab * cols)
    case = {"op": op, "m": _spread(rng, 1, min(16384, most)), "vocab": vocab, "cols": cols,
            "dtype": rng.choice(["bf16", "fp16"])}
    if op == "loss_gradient":
        case["penalty"] = rng.random() < 0.5
    return case


# ------------------------------------------------- what a program has in hand

def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=TYPES[dtype], device="cuda").normal_(0.0, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"g": _prepare_grouped, "l": _prepare_loss, "4": _prepare_4bit}[case["op"][0]]
    return {"case": case, **make(case, g)}


def _rows(case):
    used = case["tokens"] * case["top_k"]
    return used, used + (used // 16 + 1 if case["padded"] else 0)


def _prepare_grouped(case, g):
    t, e, k, cols, rows, dtype = (case[f] for f in ("tokens", "experts", "top_k", "cols", "rows", "dtype"))
    # each token's experts, some experts liked better than others; the rows sorted by expert, so that only their numbers are left
    like = 0.5 * torch.randn(e, generator=g, device="cuda")
    chance = torch.rand((t, e), generator=g, device="cuda").clamp_(min=1e-9)
    chosen = torch.topk(like - (-chance.log()).log(), k, dim=1).indices
    count = torch.bincount(chosen.flatten(), minlength=e)
    m = _rows(case)[1]
    s = {"x": _normal(g, (m, cols), 1.0, dtype), "w": _normal(g, (e, rows, cols), 1 / math.sqrt(cols), dtype),
         "ends": count.cumsum(0), "most": int(count.max())}
    if case["op"] == "grouped_gradient":
        s["grad"] = _normal(g, (m, rows), 1.0, dtype)
    return s


def _prepare_loss(case, g):
    m, v, cols, dtype = (case[f] for f in ("m", "vocab", "cols", "dtype"))
    w = _normal(g, (v, cols), 1.5 / math.sqrt(cols), dtype)
    tokens = torch.randint(0, v, (m,), generator=g, device="cuda")
    # half of the tokens are well predicted
    near = 4.0 * (torch.rand(m, generator=g, device="cuda") < 0.5)
    h = torch.randn((m, cols), generator=g, device="cuda") + near[:, None] * w[tokens].float()
    h = h.to(TYPES[dtype])
    tokens[7::8] = -1  # a prompt's tokens have no loss
    s = {"hidden": h, "weight": w, "tokens": tokens}
    if case["op"] == "loss_gradient":
        # what the forward pass left behind
        s["lse"] = _lse64(h, w).float()
        mean = (tokens >= 0) * (1.0 / max(1, m - m // 8))
        scale = 65536.0 if dtype == "fp16" else 1.0
        s["grad_loss"] = scale * mean.float()
        s["grad_lse"] = (scale * 2e-4 / m) * s["lse"] if case["penalty"] else None
    return s


def _prepare_4bit(case, g):
    m, rows, cols, group, dtype = (case[f] for f in ("m", "rows", "cols", "group", "dtype"))
    groups = cols // group
    # normal weights in 16 steps of a third of their deviation, which differs from group to group
    steps = torch.empty((rows, cols), device="cuda").normal_(0.0, 3.0, generator=g).round_()
    zeros = torch.full((rows, groups), 8.0, device="cuda")
    if case["zeros"]:
        zeros += torch.randint(-2, 3, (rows, groups), generator=g, device="cuda")
    q = (steps.view(rows, groups, group) + zeros[..., None]).clamp_(0, 15).to(torch.uint8).view(rows, cols)
    scales = (0.5 + torch.rand((rows, groups), generator=g, device="cuda")) / (3 * math.sqrt(cols))
    return {"x": _normal(g, (m, cols), 1.0, dtype), "q": q[:, ::2] | (q[:, 1::2] << 4), "scales": scales.to(TYPES[dtype]),
            "zeros": zeros.to(TYPES[dtype]) if case["zeros"] else None}


def _lse64(h, w):
    step, w = max(1, (1 << 27) // w.shape[0]), w.double()
    return torch.cat([torch.logsumexp(part.double() @ w.T, 1) for part in h.split(step)])


# ------------------------------------------------------------------- one pass

def run(state):
    return {"grouped": _run_grouped, "grouped_gradient": _run_grouped_gradient, "loss": _run_loss,
            "loss_gradient": _run_loss_gradient, "4bit": _run_4bit}[state["case"]["op"]](state)


def _padded(s, t):
    """The rows of t in a place of their own among `most` for each expert, and these places (the last one for rows behind)."""
    e, most = s["w"].shape[0], s["most"]
    r = torch.arange(t.shape[0], device=t.device)
    at = torch.searchsorted(s["ends"], r, right=True)
    first = torch.cat([s["ends"].new_zeros(1), s["ends"]])
    place = torch.where(at < e, at * most + r - first[at], e * most)
    wide = torch.zeros((e * most + 1, t.shape[1]), device=t.device)
    wide[place] = t.float()
    return wide[:-1].view(e, most, -1), place


def _back(wide, place, dtype):
    flat = wide.reshape(-1, wide.shape[2])
    return torch.cat([flat, flat.new_zeros((1, flat.shape[1]))])[place].to(dtype)


def _run_grouped(s):
    if own:
        from lossless_weight_compression_bf16_amd import grouped
        return grouped.grouped_linear(s["x"], s["w"], s["ends"], check=False)
    x, place = _padded(s, s["x"])
    return _back(x @ s["w"].float().transpose(1, 2), place, s["x"].dtype)


def _run_grouped_gradient(s):
    if own:
        from lossless_weight_compression_bf16_amd import grouped
        return grouped.grouped_linear_backward(s["x"], s["w"], s["ends"], s["grad"], check=False)
    x, place = _padded(s, s["x"])
    dy, _ = _padded(s, s["grad"])
    dtype = s["x"].dtype
    return _back(dy @ s["w"].float(), place, dtype), (dy.transpose(1, 2) @ x).to(dtype)


def _run_loss(s):
    if own:
        from lossless_weight_compression_bf16_amd import loss
        r = loss.linear_cross_entropy(s["hidden"], s["weight"], s["tokens"], check=False)
        return {"loss": r.loss, "lse": r.lse}
    z = s["hidden"].float() @ s["weight"].float().T
    most = z.amax(1, keepdim=True)
    lse = (most + (z - most).exp().sum(1, keepdim=True).log())[:, 0]
    t = s["tokens"]
    given = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return {"loss": (lse - given).masked_fill(t < 0, 0.0), "lse": lse}


def _run_loss_gradient(s):
    if own:
        from lossless_weight_compression_bf16_amd import loss
        return loss.linear_cross_entropy_backward(s["hidden"], s["weight"], s["tokens"], s["lse"], s["grad_loss"],
                                                  s["grad_lse"], check=False)
    h, w, t = s["hidden"].float(), s["weight"].float(), s["tokens"]
    of_token = s["grad_loss"].masked_fill(t < 0, 0.0)
    of_lse = of_token if s["grad_lse"] is None else of_token + s["grad_lse"]
    g = (h @ w.T - s["lse"][:, None]).exp() * of_lse[:, None]
    g.scatter_add_(1, t.clamp(min=0)[:, None], -of_token[:, None])
    return (g @ w).to(s["hidden"].dtype), (g.T @ h).to(s["weight"].dtype)


def _run_4bit(s):
    group = s["case"]["group"]
    if own:
        from lossless_weight_compression_bf16_amd import fourbit
        return fourbit.linear4(s["x"], fourbit.Weights4(s["q"], s["scales"], s["zeros"], group))
    rows, groups = s["scales"].shape
    q = torch.stack([s["q"] & 15, s["q"] >> 4], 2).view(rows, groups, group).float()
    zeros = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = ((q - zeros) * s["scales"].float()[..., None]).view(rows, -1)
    return (s["x"].float() @ w.T).to(s["x"].dtype)


# ------------------------------------------------------- what it cannot do without

def work(case):
    if case["op"].startswith("grouped"):
        e, cols, rows, (used, m) = case["experts"], case["cols"], case["rows"], _rows(case)
        hit = e * (1.0 - (1.0 - case["top_k"] / e) ** case["tokens"])  # experts with rows, on average
        if case["op"] == "grouped":
            return {"bytes": 2.0 * (used * cols + m * rows + hit * rows * cols) + 8 * e, "flops": 2.0 * used * rows * cols}
        return {"bytes": 2.0 * (used * (cols + rows) + m * cols + (hit + e) * rows * cols) + 8 * e,
                "flops": 4.0 * used * rows * cols}
    if case["op"] == "4bit":
        m, rows, cols = case["m"], case["rows"], case["cols"]
        per_group = 4.0 if case["zeros"] else 2.0
        return {"bytes": rows * cols * (0.5 + per_group / case["group"]) + 2.0 * m * (rows + cols), "flops": 2.0 * m * rows * cols}
    m, v, cols = case["m"], case["vocab"], case["cols"]
    if case["op"] == "loss":
        return {"bytes": 2.0 * cols * (m + v) + 16 * m, "flops": 2.0 * m * v * cols}
    return {"bytes": 4.0 * cols * (m + v) + 20 * m, "flops": 6.0 * m * v * cols}


# ------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"grouped": _exact_grouped, "grouped_gradient": _exact_grouped_gradient, "loss": _exact_loss,
            "loss_gradient": _exact_loss_gradient, "4bit": _exact_4bit}[case["op"]](s)


def _experts(s):
    """Each expert's number, its weights in 64 bits and its rows."""
    lo = 0
    for e, hi in enumerate(s["ends"].tolist()):
        yield e, s["w"][e].double(), slice(lo, hi)
        lo = hi


def _exact_grouped(s):
    y = torch.zeros((s["x"].shape[0], s["w"].shape[1]), dtype=torch.float64, device="cuda")
    for _, w, at in _experts(s):
        y[at] = s["x"][at].double() @ w.T
    return y


def _exact_grouped_gradient(s):
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    for e, w, at in _experts(s):
        dy = s["grad"][at].double()
        dx[at] = dy @ w
        dw[e] = dy.T @ s["x"][at].double()
    return dx, dw


def _exact_loss(s):
    lse = _lse64(s["hidden"], s["weight"])
    t = s["tokens"]
    given = (s["hidden"].double() * s["weight"][t.clamp(min=0)].double()).sum(1)
    return {"loss": torch.where(t < 0, 0.0, lse - given), "lse": lse}


def _exact_loss_gradient(s):
    h, w = s["hidden"], s["weight"].double()
    dh, dw = torch.zeros(h.shape, dtype=torch.float64, device="cuda"), torch.zeros_like(w)
    step = max(1, (1 << 27) // w.shape[0])
    for lo in range(0, h.shape[0], step):
        at = slice(lo, lo + step)
        part, t = h[at].double(), s["tokens"][at]
        weight = torch.where(t < 0, 0.0, s["grad_loss"][at].double())
        p = torch.exp(part @ w.T - s["lse"][at, None].double())
        given = torch.zeros_like(p)
        given[torch.nonzero(t >= 0)[:, 0], t[t >= 0]] = 1.0
        g = weight[:, None] * (p - given)
        if s["grad_lse"] is not None:
            g += s["grad_lse"][at, None].double() * p
        dh[at] = g @ w
        dw += g.T @ part
    return dh, dw


def _exact_4bit(s):
    group, x = s["case"]["group"], s["x"].double()
    y = torch.zeros((x.shape[0], s["q"].shape[0]), dtype=torch.float64, device="cuda")
    for i in range(s["scales"].shape[1]):  # a group of columns at a time
        at = slice(i * group // 2, (i + 1) * group // 2)
        zero = 8.0 if s["zeros"] is None else s["zeros"][:, i].double()
        part = x[:, i * group:(i + 1) * group]
        low, high = (s["q"][:, at] % 16).double(), (s["q"][:, at] // 16).double()
        y += s["scales"][:, i].double() * (part[:, ::2] @ low.T + part[:, 1::2] @ high.T - zero * part.sum(1, keepdim=True))
    return y
