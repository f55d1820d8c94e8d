"""The attention-side operators of a draft step, as measured: rotary positions, the paged cache's
quantising write and read-back, and attention of a block of new tokens over the paged cache.

Each case is one call.  ``run`` computes it in plain float32 torch operations, or (``own``) with the
framework's kernels; ``exact`` computes it from the definition in float64.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
CACHE_TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}  # the largest code
TINY = 1e-30  # a row whose largest magnitude is below this is held as zeros


def listed():
    return [
        # one draft block of eight positions, queries and keys of a 32-query / 8-key-head layer: latency
        {"name": "rope block", "op": "rope", "tokens": 8, "heads": 40, "dim": 128, "rot": 128, "interleaved": False,
         "inverse": False, "max_pos": 8192},
        # gradient of a training batch's queries, three quarters of the head rotated, odd token count
        {"name": "rope gradient", "op": "rope", "tokens": 8195, "heads": 32, "dim": 128, "rot": 96,
         "interleaved": True, "inverse": True, "max_pos": 65536},
        # one new token for each of sixteen sequences
        {"name": "append step int8", "op": "append", "seqs": 16, "new": 1, "ctx": 2048, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "interleaved": False, "page": 16, "type": "int8", "ragged": True},
        # a prompt's chunk: four sequences of up to 4096 tokens
        {"name": "append prompt e4m3", "op": "append", "seqs": 4, "new": 4096, "ctx": 8192, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "page": 64, "type": "e4m3", "ragged": False},
        # odd everything: page size that divides nothing, narrow heads, a ragged batch, part of the head rotated
        {"name": "append odd bf16", "op": "append", "seqs": 37, "new": 61, "ctx": 700, "q_heads": 15, "kv_heads": 5,
         "dim": 80, "rot": 40, "interleaved": True, "page": 24, "type": "bf16", "ragged": True},
        # a cache taken out of its pages (to hand a sequence on, or to train on it)
        {"name": "read back e4m3", "op": "read", "seqs": 8, "new": 8192, "ctx": 8192, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "e4m3", "ragged": False},
        {"name": "read back odd int8", "op": "read", "seqs": 19, "new": 333, "ctx": 501, "kv_heads": 3, "dim": 96,
         "page": 40, "type": "int8", "ragged": True},
        # one token of one short sequence: latency
        {"name": "decode one token", "op": "attend", "seqs": 1, "new": 1, "ctx": 777, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "type": "bf16", "ragged": False, "causal": True, "window": 0},
        # the verification of 16-token draft blocks of 32 sequences
        {"name": "verify bf16", "op": "attend", "seqs": 32, "new": 16, "ctx": 8192, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "type": "bf16", "ragged": True, "causal": True, "window": 0},
        # the same with 8-token blocks, twice the context and an 8-bit cache
        {"name": "verify e4m3", "op": "attend", "seqs": 32, "new": 8, "ctx": 16384, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "type": "e4m3", "ragged": True, "causal": True, "window": 0},
        # a draft block that sees all of itself, sliding window, odd group, odd head, odd pages
        {"name": "draft odd int8", "op": "attend", "seqs": 7, "new": 16, "ctx": 3001, "q_heads": 20, "kv_heads": 4,
         "dim": 96, "page": 24, "type": "int8", "ragged": True, "causal": False, "window": 1000},
        # a prompt's chunk over what came before it
        {"name": "prompt chunk", "op": "attend", "seqs": 1, "new": 2048, "ctx": 18432, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "type": "bf16", "ragged": False, "causal": True, "window": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend", "attend"])
    dim = rng.choice([48, 64, 80, 96, 112, 128, 128, 128])
    page = rng.choice([8, 16, 24, 32, 40, 64, 96, 128, 256])
    kind = rng.choice(["bf16", "e4m3", "int8"])
    if op == "rope":
        heads = rng.randint(1, 48)
        return {"op": op, "tokens": _log(rng, 1, 8195 * 32 // max(32, heads)), "heads": heads, "dim": dim,
                "rot": 2 * rng.randint(4, dim // 2), "interleaved": rng.random() < 0.5,
                "inverse": rng.random() < 0.5, "max_pos": 65536}
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if op in ("append", "read"):
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, (16384 if op == "append" else 32768) // seqs))
        case = {"op": op, "seqs": seqs, "new": new, "ctx": new + _log(rng, 1, 2000), "kv_heads": kv_heads, "dim": dim,
                "page": page, "type": kind, "ragged": rng.random() < 0.7}
        if op == "append":
            case.update(q_heads=min(32, kv_heads * group), rot=2 * rng.randint(4, dim // 2),
                        interleaved=rng.random() < 0.5)
            case["q_heads"] -= case["q_heads"] % kv_heads
        return case
    case = {"op": op, "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page, "type": kind,
            "ragged": rng.random() < 0.7, "causal": rng.random() < 0.7,
            "window": rng.choice([0, 0, _log(rng, 1, 4096)])}
    if rng.random() < 0.7:  # tokens of many sequences: one each, or a draft block
        case["seqs"] = _log(rng, 1, 64)
        case["new"] = rng.choice([1, _log(rng, 1, 32)])
        case["ctx"] = case["new"] + _log(rng, 1, min(32768, 262144 // case["seqs"]))
    else:  # a prompt's chunk
        case["seqs"] = rng.randint(1, 3)
        case["new"] = _log(rng, 33, 2048 // case["seqs"])
        case["ctx"] = case["new"] + _log(rng, 1, 16384)
    return case


# ------------------------------------------------------------------------------------------ inputs


def _lengths(case):
    """Whole lengths and new tokens of each sequence, from the case alone."""
    B, T, ctx = case["seqs"], case["new"], case["ctx"]
    lens, news = [], []
    for b in range(B):
        f = ((b * 7919 + 13) % 97) / 97.0  # spread over [0, 1), the same for every seed
        n = max(1, T - int(f * 0.4 * T)) if case["ragged"] else T
        if case["op"] == "attend" and case["ragged"] and T <= 32:
            n = T  # draft blocks have one length
        lens.append(max(n, ctx - int(f * 0.6 * ctx)) if case["ragged"] else max(n, ctx))
        news.append(n)
    return lens, news


def _batch(case, g):
    lens, news = _lengths(case)
    B, page = case["seqs"], case["page"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    width = max(need)
    place = torch.arange(width).repeat(B, 1) + torch.tensor([0] + need[:-1]).cumsum(0)[:, None]
    table = ids[place.clamp_(max=pages - 1).cuda()]  # what lies past a sequence's last page is another's
    start = torch.tensor([0] + news).cumsum(0).to(torch.int32).cuda()
    return {"token_start": start, "kv_len": torch.tensor(lens, dtype=torch.int32).cuda(), "page_table": table.contiguous(),
            "tokens": sum(news), "max_new": max(news), "max_len": max(lens), "pages": pages}


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _quantised(x, kind):
    """Codes and scales of float32 rows: m = max |row|, scale = m / M, code = round(row * (M / m))."""
    m = x.abs().amax(-1, keepdim=True)
    top = torch.full_like(m, TOP[kind])  # a tensor, so that both divisions are the correctly rounded ones
    held = m >= TINY
    scale = torch.where(held, m / top, torch.zeros_like(m))
    y = x * torch.where(held, top / m, torch.zeros_like(m))
    y = y.round().clamp(-127, 127).to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)
    finite = torch.isfinite(m)
    if kind == "int8":
        y = torch.where(finite, y, torch.zeros_like(y))
    else:
        y = torch.where(finite, y.view(torch.uint8), torch.zeros_like(y, dtype=torch.uint8)).view(torch.float8_e4m3fn)
    return y, torch.where(finite, scale, torch.full_like(scale, math.nan)).squeeze(-1)


def _cache(case, batch, g, filled):
    shape = (batch["pages"], case["kv_heads"], case["page"], case["dim"])
    kind = case["type"]
    out = {}
    for name in ("k", "v"):
        if filled:
            # keys with channels of different size, values about one
            x = _randn(g, *shape)
            if name == "k":
                x *= 0.5 + torch.rand(case["dim"], device="cuda", generator=g)
            if kind == "bf16":
                out[name], out[name + "_scale"] = x.to(BF16), None
            else:
                out[name], out[name + "_scale"] = _quantised(x, kind)
        else:
            out[name] = torch.zeros(shape, dtype=torch.uint8, device="cuda").view(CACHE_TYPES[kind]) if kind != "bf16" \
                else torch.zeros(shape, dtype=BF16, device="cuda")
            out[name + "_scale"] = torch.zeros(shape[:3], device="cuda") if kind != "bf16" else None
    return out


def _table(max_pos, rot):
    """cos and sin of position * frequency, [max_pos, 2, rot / 2], made in float64: the table a program keeps."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], 1).to(torch.float32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "rope":
        N, heads, dim = case["tokens"], case["heads"], case["dim"]
        s["x"] = _randn(g, N, heads, dim).to(BF16)
        s["positions"] = torch.randint(0, case["max_pos"], (N,), device="cuda", generator=g, dtype=torch.int32)
        s["table"] = _table(case["max_pos"], case["rot"])
    else:
        s["batch"] = _batch(case, g)
        s["cache"] = _cache(case, s["batch"], g, case["op"] != "append")
        N, kv_heads, dim = s["batch"]["tokens"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        # the views that a fused projection leaves: q | k | v of each token side by side
        qkv = _randn(g, N, case["q_heads"] + 2 * kv_heads, dim).to(BF16)
        s["q"], s["k"], s["v"] = qkv.split([case["q_heads"], kv_heads, kv_heads], 1)
        s["table"] = _table(s["batch"]["max_len"], case["rot"])
    elif case["op"] == "attend":
        s["q"] = _randn(g, N, case["q_heads"], dim).to(BF16)
    if own:
        s["plan"] = _plan(s)
    return s


def _plan(s):
    """The framework's handle: buffers bound once, as a loop of steps keeps it."""
    from speculative_decoding_drafter_gb300 import attention as at

    case = s["case"]
    if case["op"] == "rope":
        return at.RopePlan(s["x"], s["positions"], s["table"], interleaved=case["interleaved"],
                           inverse=case["inverse"])
    b, c = s["batch"], s["cache"]
    cache = at.PagedCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
    batch = at.TokenBatch(b["token_start"], b["kv_len"], b["page_table"], tokens=b["tokens"], max_new=b["max_new"])
    if case["op"] == "append":
        return at.CacheAppendPlan(cache, batch, s["k"], s["v"], q=s["q"], table=s["table"],
                                  interleaved=case["interleaved"])
    if case["op"] == "read":
        return at.CacheReadPlan(cache, batch)
    return at.PagedAttentionPlan(s["q"], cache, batch, causal=case["causal"], window=case["window"])


# -------------------------------------------------------------------------------------- plain forms


def _rotate(x, cos, sin, interleaved, inverse=False):
    """x float32 [N, heads, dim]; cos, sin [N, rot / 2]."""
    half = cos.shape[1]
    cos, sin = cos[:, None], (-sin if inverse else sin)[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    else:
        a, b = x[..., :half], x[..., half:2 * half]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _places(b, page):
    """Sequence, order within it, position, page and slot of each new token."""
    start, lens = b["token_start"].long(), b["kv_len"].long()
    n = torch.arange(b["tokens"], device="cuda")
    seq = torch.searchsorted(start, n, right=True) - 1
    order = n - start[seq]
    pos = lens[seq] - (start[seq + 1] - start[seq]) + order
    return seq, order, pos, b["page_table"][seq, pos // page].long(), pos % page


def _held(cache, name, at):
    """float32 values of the cache's rows `at` (pages, slots): [..., kv_heads, dim]."""
    x = cache[name][at[0], :, at[1]].float()
    return x if cache[name + "_scale"] is None else x * cache[name + "_scale"][at[0], :, at[1]][..., None]


def _plain_attend(s):
    case, b, cache = s["case"], s["batch"], s["cache"]
    seq, order, _, _, _ = _places(b, case["page"])
    B, T, L = case["seqs"], b["max_new"], b["max_len"]
    kv_heads, group, dim = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["dim"]
    lens, news = b["kv_len"].long(), (b["token_start"][1:] - b["token_start"][:-1]).long()
    j = torch.arange(L, device="cuda")
    at = (b["page_table"][:, j // case["page"]].long(), (j % case["page"]).expand(B, L))
    inside = (j < lens[:, None])[:, :, None, None]
    k = _held(cache, "k", at).permute(0, 2, 3, 1)  # [B, kv_heads, dim, L]
    v = torch.where(inside, _held(cache, "v", at), torch.zeros((), device="cuda")).permute(0, 2, 1, 3)
    q = torch.zeros(B, T, kv_heads, group, dim, device="cuda")
    q[seq, order] = s["q"].float().view(-1, kv_heads, group, dim)
    pos = (lens - news)[:, None] + torch.arange(T, device="cuda")  # [B, T]
    last = pos if case["causal"] else (lens - 1)[:, None].expand(B, T)
    seen = (j <= last[..., None]) & (j < lens[:, None, None])
    if case["window"]:
        seen &= j > pos[..., None] - case["window"]
    score = (q.permute(0, 2, 3, 1, 4).reshape(B, kv_heads, group * T, dim) @ k).view(B, kv_heads, group, T, L)
    score = (score * dim ** -0.5).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = (score - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, kv_heads, group * T, L) @ v).view(B, kv_heads, group, T, dim)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1)
    out = o.permute(0, 3, 1, 2, 4)[seq, order].reshape(-1, case["q_heads"], dim)
    return {"out": out.to(BF16), "lse": lse.permute(0, 3, 1, 2)[seq, order].reshape(-1, case["q_heads"])}


def run(s):
    if own:
        return s["plan"]()
    case = s["case"]
    if case["op"] == "rope":
        t = s["table"][s["positions"].long()]
        return _rotate(s["x"].float(), t[:, 0], t[:, 1], case["interleaved"], case["inverse"]).to(BF16)
    if case["op"] == "attend":
        return _plain_attend(s)
    _, _, pos, page, slot = _places(s["batch"], case["page"])
    cache = s["cache"]
    if case["op"] == "read":
        return {"k": _held(cache, "k", (page, slot)).to(BF16), "v": _held(cache, "v", (page, slot)).to(BF16)}
    t = s["table"][pos]
    out = {"q": _rotate(s["q"].float(), t[:, 0], t[:, 1], case["interleaved"]).to(BF16)}
    for name, x in (("k", _rotate(s["k"].float(), t[:, 0], t[:, 1], case["interleaved"])), ("v", s["v"].float())):
        if case["type"] == "bf16":
            cache[name][page, :, slot] = x.to(BF16)
        else:
            codes, scale = _quantised(x, case["type"])
            # bytes, which every indexing kernel takes
            cache[name].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            cache[name + "_scale"][page, :, slot] = scale
            out[name + "_scale"] = cache[name + "_scale"]
        out[name + "_cache"] = cache[name]
    return out


# --------------------------------------------------------------------------------------- accounting


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + case["tokens"] * (4 * case["rot"] + 4), "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    lens, news = _lengths(case)
    N, dim, hkv = sum(news), case["dim"], case["kv_heads"]
    row = 2 * dim if case["type"] == "bf16" else dim + 4  # bytes of one cached row
    if case["op"] == "append":
        q = N * case["q_heads"] * dim
        return {"bytes": 4 * q + 4 * N * hkv * dim + 2 * N * hkv * row + 4 * N * case["rot"],
                "flops": 3 * N * (case["q_heads"] + hkv) * case["rot"]}
    if case["op"] == "read":
        return {"bytes": 2 * N * hkv * (row + 2 * dim), "flops": 2 * N * hkv * dim}
    seen = keys = 0
    for n, m in zip(lens, news):
        first = 0 if not case["window"] else max(0, n - m - case["window"] + 1)
        keys += n - first
        for p in range(n - m, n):
            seen += (p + 1 if case["causal"] else n) - (max(0, p - case["window"] + 1) if case["window"] else 0)
    return {"bytes": 2 * keys * hkv * row + N * case["q_heads"] * (4 * dim + 4),
            "flops": 4 * seen * case["q_heads"] * dim}


# -------------------------------------------------------------------------------------- definitions


def _turn64(x, angle_table, positions, rot, interleaved, inverse):
    """The rotation as a product of complex numbers, in 64 bits."""
    z = torch.complex(angle_table[positions.long(), 0].double(), angle_table[positions.long(), 1].double())[:, None]
    if inverse:
        z = z.conj()
    head, rest = x[..., :rot].double(), x[..., rot:].double()
    pair = head.unflatten(-1, (rot // 2, 2)) if interleaved else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    w = w if interleaved else w.transpose(-1, -2)
    return torch.cat([w.flatten(-2), rest], -1)


def _rows64(cache, name, pages, slots):
    x = cache[name].view(torch.uint8)[pages, :, slots].view(torch.uint8) if cache[name].dtype != BF16 else \
        cache[name][pages, :, slots]
    if cache[name].dtype == BF16:
        return x.double()
    x = x.view(cache[name].dtype).double()
    return x * cache[name + "_scale"][pages, :, slots].double().unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turn64(s["x"], s["table"], s["positions"], case["rot"], case["interleaved"], case["inverse"])
    b, cache, page = s["batch"], s["cache"], case["page"]
    lens, news = _lengths(case)
    if case["op"] == "read":
        got = {"k": [], "v": []}
        for i, (n, m) in enumerate(zip(lens, news)):
            p = torch.arange(n - m, n, device="cuda")
            for name in got:
                got[name].append(_rows64(cache, name, b["page_table"][i, p // page].long(), p % page))
        return {name: torch.cat(x) for name, x in got.items()}
    if case["op"] == "append":
        pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, news)])
        of = torch.cat([torch.full((m,), i, device="cuda") for i, m in enumerate(news)])
        pages, slots = b["page_table"][of, pos // page].long(), pos % page
        out = {"q": _turn64(s["q"], s["table"], pos, case["rot"], case["interleaved"], False)}
        for name in ("k", "v"):
            x = _turn64(s["k"], s["table"], pos, case["rot"], case["interleaved"], False) if name == "k" else s["v"].double()
            held = torch.zeros(cache[name].shape, dtype=torch.float64, device="cuda")
            if case["type"] == "bf16":
                held[pages, :, slots] = x
                out[name + "_cache"] = held
                continue
            # the scale has a value in 64 bits; a code is a rounding of it, which has none
            scales = torch.zeros(cache[name].shape[:3], dtype=torch.float64, device="cuda")
            scales[pages, :, slots] = x.abs().amax(-1) / TOP[case["type"]]
            out[name + "_scale"] = scales
            out[name + "_cache"] = None
        return out
    outs, lses, at = [], [], 0
    group = case["q_heads"] // case["kv_heads"]
    for i, (n, m) in enumerate(zip(lens, news)):
        p = torch.arange(n, device="cuda")
        pages, slots = b["page_table"][i, p // page].long(), p % page
        k, v = (_rows64(cache, name, pages, slots) for name in ("k", "v"))
        q = s["q"][at:at + m].double()
        at += m
        t = torch.arange(n - m, n, device="cuda")[:, None]
        hide = (p > t) if case["causal"] else torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if case["window"]:
            hide = hide | (p <= t - case["window"])
        o, e = torch.zeros_like(q), torch.zeros(m, case["q_heads"], dtype=torch.float64, device="cuda")
        for h in range(case["q_heads"]):
            z = (q[:, h] @ k[:, h // group].T / math.sqrt(case["dim"])).masked_fill(hide, -math.inf)
            e[:, h] = torch.logsumexp(z, -1)
            o[:, h] = torch.softmax(z, -1).nan_to_num(0.0) @ v[:, h // group]
        outs.append(o)
        lses.append(e)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
