"""The operators that fit the drafter's head to its target, as measured: the residual addition with the
root-mean-square norm and its gradient, the LM head's cross entropy and its gradient, and the global norm
and clipping of gradients.

Each case is one call.  ``run`` computes it in plain float32 torch operations, or (``own``) with the
framework's kernels; ``exact`` computes it from the definition in float64.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
TOP = 448.0  # the largest e4m3 code
TINY = 1e-30  # a row whose largest magnitude is below this is held as zeros


def listed():
    return [
        # one draft block of eight positions entering an 8-bit projection: latency
        {"name": "norm block e4m3", "op": "norm", "rows": 8, "dim": 4096, "out": "e4m3", "residual": True},
        # a training batch's hidden states before the head
        {"name": "norm batch", "op": "norm", "rows": 16384, "dim": 4096, "out": "bf16", "residual": True},
        # the gradient through that norm, odd row count, the gradient of the residual stream added
        {"name": "norm gradient", "op": "norm_grad", "rows": 8195, "dim": 5120, "residual": True},
        # the log-probabilities of one draft block under the 8B-class head: the weights are read once
        {"name": "loss block", "op": "loss", "rows": 16, "dim": 4096, "vocab": 151936, "ignored": False},
        # an odd batch over an odd vocabulary, a hidden size that no power of two divides far
        {"name": "loss odd", "op": "loss", "rows": 1003, "dim": 1032, "vocab": 50021, "ignored": True},
        # 1024 rows of the 262k-vocabulary head
        {"name": "loss large vocabulary", "op": "loss", "rows": 1024, "dim": 5376, "vocab": 262144, "ignored": True},
        # the smallest head: latency
        {"name": "loss gradient tiny", "op": "loss_grad", "rows": 8, "dim": 256, "vocab": 4096, "ignored": False},
        # a micro-batch of 64 rows of the 27B-class head: weights read, their gradient written
        {"name": "loss gradient few rows", "op": "loss_grad", "rows": 64, "dim": 5120, "vocab": 152064,
         "ignored": True},
        # a training batch of the 8B-class head
        {"name": "loss gradient batch", "op": "loss_grad", "rows": 2048, "dim": 4096, "vocab": 151936, "ignored": True},
        # the selector's and the norms' gradients alone: latency
        {"name": "clip small", "op": "clip", "tensors": 7, "total": 1500000, "type": "fp32", "kind": "l2", "write": True},
        # gradients of a head and a few layers: one huge tensor and many that are not, some of odd length
        {"name": "clip head and layers", "op": "clip", "tensors": 61, "total": 900000000, "type": "bf16", "kind": "l2",
         "write": True},
        # the norm alone of a deep drafter's many tensors, for the log
        {"name": "norm of many", "op": "clip", "tensors": 777, "total": 150000000, "type": "mixed", "kind": "l2",
         "write": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "loss", "loss", "loss_grad", "loss_grad", "clip"])
    if op in ("norm", "norm_grad"):
        dim = 8 * _log(rng, 8, 1024)
        rows = _log(rng, 1, min(65536, 16384 * 4096 // dim))
        case = {"op": op, "rows": rows, "dim": dim, "residual": rng.random() < 0.7}
        if op == "norm":
            case["out"] = rng.choice(["bf16", "e4m3", "both"])
        return case
    if op == "clip":
        tensors = _log(rng, 1, 800)
        return {"op": op, "tensors": tensors, "total": _log(rng, max(1000, 4 * tensors), 600000000),
                "type": rng.choice(["bf16", "fp16", "fp32", "mixed"]), "kind": rng.choice(["l2", "l2", "max"]),
                "write": rng.random() < 0.7}
    dim = 8 * _log(rng, 8, 672)
    vocab = _log(rng, 500, 262144)
    rows = _log(rng, 1, 4096)
    most = 2048 * 4096 * 151936 if op == "loss_grad" else 1024 * 5376 * 262144
    return {"op": op, "rows": max(1, min(rows, most // (dim * vocab))), "dim": dim, "vocab": vocab,
            "ignored": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------ inputs


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _uniform(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _sizes(case):
    """Lengths and types of a clip case's tensors, from the case alone: one holds about half of the elements
    (the head's), the others share the rest unevenly, down to a norm's few."""
    n, total = case["tensors"], case["total"]
    if n == 1:
        lengths = [total]
    else:
        weight = [(((i * 7919 + 13) % 97) / 97.0) ** 3 + 1e-3 for i in range(n - 1)]
        scale = (total - total // 2) / sum(weight)
        lengths = [max(1, int(w * scale)) for w in weight]
        lengths.insert(n // 2, total // 2)
    kinds = ["bf16", "fp32", "fp16"] if case["type"] == "mixed" else [case["type"]]
    return [(length, kinds[i % len(kinds)]) for i, length in enumerate(lengths)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        N, C = case["rows"], case["dim"]
        s["gamma"] = (1 + 0.2 * _randn(g, C)).to(BF16)
        # a residual stream: channels of different size, rows of different size
        stream = _randn(g, N, C) * (0.5 + 2 * _uniform(g, C)) * (0.5 + _uniform(g, N, 1))
        if op == "norm":
            s["x"] = _randn(g, N, C).to(BF16)
            s["residual"] = stream.to(BF16) if case["residual"] else None
        else:
            s["sum"] = stream.to(BF16)
            s["dy"] = (_randn(g, N, C) * 1e-3).to(BF16)
            s["d_sum"] = (_randn(g, N, C) * 1e-3).to(BF16) if case["residual"] else None
    elif op in ("loss", "loss_grad"):
        N, H, V = case["rows"], case["dim"], case["vocab"]
        s["W"] = torch.empty(V, H, dtype=BF16, device="cuda")
        for at in range(0, V, 65536):
            s["W"][at:at + 65536] = _randn(g, min(65536, V - at), H) * (2.5 / math.sqrt(H))
        labels = torch.randint(0, V, (N,), device="cuda", generator=g)
        # hidden states that point to their label, from not at all to nearly surely
        s["hidden"] = (_randn(g, N, H) + _uniform(g, N, 1) * 2.4 * s["W"][labels].float()).to(BF16)
        if case["ignored"]:  # one row in eight is a prompt's or padding
            labels = torch.where(_uniform(g, N) < 0.125, torch.full_like(labels, -1), labels)
        s["labels"] = labels.to(torch.int32)
        if op == "loss_grad":
            # what the forward pass left, and a weight for each row: later draft positions count less
            s["lse"] = torch.cat([torch.logsumexp(_plain_logits(s["hidden"][at:at + 512], s["W"]), 1)
                                  for at in range(0, N, 512)])
            s["grad"] = torch.exp(-(torch.arange(N, device="cuda") % 16) / 7.0) / N
    else:
        s["tensors"] = [(_randn(g, n) * 10 ** (-3 + 2 * i / case["tensors"])).to(TYPES[kind])
                        for i, (n, kind) in enumerate(_sizes(case))]
        s["max_norm"] = 1.0 if case["kind"] == "l2" else 0.01
        s["out"] = [torch.empty_like(t) for t in s["tensors"]] if case["write"] else None
    if own:
        s["plan"] = _plan(s)
    return s


def _plan(s):
    """The framework's handle: buffers bound once, as a training loop keeps it."""
    from speculative_decoding_drafter_gb300 import training as tr

    case = s["case"]
    if case["op"] == "norm":
        return tr.ResidualNormPlan(s["x"], s["gamma"], residual=s["residual"], eps=EPS, y=case["out"] != "e4m3",
                                   codes=torch.float8_e4m3fn if case["out"] != "bf16" else None)
    if case["op"] == "norm_grad":
        return tr.ResidualNormGradPlan(s["sum"], s["gamma"], s["dy"], d_sum=s["d_sum"], eps=EPS)
    if case["op"] == "loss":
        return tr.LossPlan(s["hidden"], s["W"], s["labels"])
    if case["op"] == "loss_grad":
        return tr.LossGradPlan(s["hidden"], s["W"], s["labels"], s["lse"], s["grad"])
    return tr.GradClipPlan(s["tensors"], max_norm=s["max_norm"] if case["write"] else None, kind=case["kind"],
                           out=s["out"])


# -------------------------------------------------------------------------------------- plain forms


def _plain_norm(s):
    case = s["case"]
    z = s["x"].float()
    out = {}
    if case["residual"]:
        z = z + s["residual"].float()
        out["sum"] = z.to(BF16)
    y = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    if case["out"] != "e4m3":
        out["y"] = y.to(BF16)
    if case["out"] != "bf16":
        m = y.abs().amax(-1, keepdim=True)
        top = torch.full_like(m, TOP)
        held = m >= TINY
        out["codes"] = (y * torch.where(held, top / m, torch.zeros_like(m))).to(torch.float8_e4m3fn)
        out["scale"] = torch.where(held, m / top, torch.zeros_like(m)).squeeze(-1)
    return out


def _plain_norm_grad(s):
    z, dy, gamma = s["sum"].float(), s["dy"].float(), s["gamma"].float()
    r = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
    u = dy * gamma
    dx = r * (u - z * (r * r * (u * z).mean(-1, keepdim=True)))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
    return {"dx": dx.to(BF16), "dgamma": (dy * z * r).sum(0)}


def _plain_logits(hidden, W):
    return hidden.float() @ W.float().T


def _plain_loss(s):
    logits = _plain_logits(s["hidden"], s["W"])
    top = logits.amax(1)
    lse = top + logits.sub_(top[:, None]).exp_().sum(1).log()
    labels = s["labels"].long()
    seen = (labels >= 0) & (labels < s["case"]["vocab"])
    own_row = s["W"][labels.clamp(0, s["case"]["vocab"] - 1)].float()
    loss = torch.where(seen, lse - (s["hidden"].float() * own_row).sum(1), torch.zeros_like(lse))
    return {"loss": loss, "lse": lse}


def _plain_loss_grad(s):
    hidden, W = s["hidden"].float(), s["W"].float()
    labels = s["labels"].long()
    seen = (labels >= 0) & (labels < s["case"]["vocab"])
    d = (hidden @ W.T).sub_(s["lse"][:, None]).exp_()
    rows = seen.nonzero()[:, 0]
    d[rows, labels[rows]] -= 1
    d *= torch.where(seen, s["grad"], torch.zeros_like(s["grad"]))[:, None]
    return {"d_hidden": (d @ W).to(BF16), "d_W": (d.T @ hidden).to(BF16)}


def _plain_clip(s):
    if s["case"]["kind"] == "l2":
        parts = [t.float().square().sum(dtype=torch.float64) for t in s["tensors"]]
        norm = torch.stack(parts).sum().sqrt()
    else:
        norm = torch.stack([t.abs().amax().double() for t in s["tensors"]]).amax()
    out = {"norm": norm.float()}
    if s["case"]["write"]:
        factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float()
        for t, o in zip(s["tensors"], s["out"]):
            o.copy_(t.float() * factor)
        out["tensors"] = s["out"]
    return out


def run(s):
    if own:
        return s["plan"]()
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "loss": _plain_loss, "loss_grad": _plain_loss_grad,
            "clip": _plain_clip}[s["case"]["op"]](s)


# --------------------------------------------------------------------------------------- accounting


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["dim"]
        written = (2 if case["residual"] else 0) + {"bf16": 2, "e4m3": 1, "both": 3}[case["out"]]
        scales = 4 * case["rows"] if case["out"] != "bf16" else 0
        return {"bytes": n * ((4 if case["residual"] else 2) + written) + 2 * case["dim"] + scales, "flops": 6 * n}
    if op == "norm_grad":
        n = case["rows"] * case["dim"]
        return {"bytes": n * (8 if case["residual"] else 6) + 6 * case["dim"], "flops": 12 * n}
    if op == "clip":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}
        each = _sizes(case)
        held = sum(n * size[kind] for n, kind in each)
        return {"bytes": held * (2 if case["write"] else 1) + 4, "flops": sum(n for n, _ in each) * (3 if case["write"] else 2)}
    N, H, V = case["rows"], case["dim"], case["vocab"]
    if op == "loss":
        return {"bytes": 2 * V * H + 2 * N * H + 12 * N, "flops": 2 * N * H * V}
    return {"bytes": 4 * V * H + 4 * N * H + 12 * N, "flops": 6 * N * H * V}


# -------------------------------------------------------------------------------------- definitions


def _exact_norm(s):
    case = s["case"]
    x = s["x"].double()
    if case["residual"]:
        x = x + s["residual"].double()
    y = s["gamma"].double() * x / torch.sqrt(torch.linalg.vecdot(x, x)[:, None] / case["dim"] + EPS)
    out = {"sum": x} if case["residual"] else {}
    if case["out"] != "e4m3":
        out["y"] = y
    if case["out"] != "bf16":
        out["codes"] = None  # a code is a rounding, which has no value in 64 bits
        out["scale"] = torch.linalg.vector_norm(y, math.inf, dim=1) / TOP
    return out


def _exact_norm_grad(s):
    """The vector-Jacobian product, row block by row block: y = gamma * x / n, n = sqrt(x.x / C + eps)."""
    x, C = s["sum"].double(), s["case"]["dim"]
    w = s["dy"].double() * s["gamma"].double()
    n2 = torch.linalg.vecdot(x, x)[:, None] / C + EPS
    n = n2.sqrt()
    dx = w / n - x * torch.linalg.vecdot(w, x)[:, None] / (C * n * n2)
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].double()
    return {"dx": dx, "dgamma": torch.einsum("nc,nc->c", s["dy"].double(), x / n)}


def _exact_loss(s):
    h, V = s["hidden"].double(), s["case"]["vocab"]
    lse = torch.full((h.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
    label = torch.zeros_like(lse)
    for at in range(0, V, 32768):
        z = h @ s["W"][at:at + 32768].double().T
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        here = (s["labels"] >= at) & (s["labels"] < at + z.shape[1])
        rows = here.nonzero()[:, 0]
        label[rows] = z[rows, s["labels"][rows].long() - at]
    return {"loss": torch.where((s["labels"] >= 0) & (s["labels"] < V), lse - label, 0.0), "lse": lse}


def _exact_loss_grad(s):
    h, V = s["hidden"].double(), s["case"]["vocab"]
    lse = s["lse"].double()  # an input, as the forward pass left it
    keep = ((s["labels"] >= 0) & (s["labels"] < V)).double() * s["grad"].double()
    d_hidden = torch.zeros_like(h)
    d_W = torch.empty(V, h.shape[1], dtype=torch.float64, device="cuda")
    for at in range(0, V, 32768):
        w = s["W"][at:at + 32768].double()
        token = torch.arange(at, at + w.shape[0], device="cuda")
        d = torch.exp(h @ w.T - lse[:, None]) - (s["labels"][:, None] == token).double()
        d *= keep[:, None]
        d_hidden += d @ w
        d_W[at:at + 32768] = d.T @ h
    return {"d_hidden": d_hidden, "d_W": d_W}


def _exact_clip(s):
    if s["case"]["kind"] == "l2":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["tensors"]))
    else:
        norm = max(float(t.double().abs().max()) for t in s["tensors"])
    out = {"norm": torch.tensor(norm, dtype=torch.float64)}
    if s["case"]["write"]:
        out["tensors"] = [t.double() * min(1.0, s["max_norm"] / norm) for t in s["tensors"]]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "loss": _exact_loss, "loss_grad": _exact_loss_grad,
            "clip": _exact_clip}[case["op"]](s)
